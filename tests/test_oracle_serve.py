"""The serving oracle against hand-worked cases, identities and torch."""

import math

import numpy as np
import torch

from oracle import serve


def test_plan_by_hand():
    # page 4; request 0 grows from 3 to 6 (one page), 1 has ended (two pages back), 2 starts with 4 (one page)
    table = np.array([[9, -1], [7, 8], [-1, -1]])
    r = serve.plan([3, 5, 0], [3, -1, 4], table, 4, 9, np.array([1, 2, -1, -1, -1, -1, -1, -1, -1, -1]), 2)
    assert r["free_pages"][:4].tolist() == [1, 2, 7, 8]     # returned pages on top
    assert r["block_table"].tolist() == [[9, 8], [7, 8], [7, -1]]
    assert r["free_count"] == 2
    assert r["cu_q"].tolist() == [0, 3, 3, 7] and r["kv_len"].tolist() == [6, 0, 4]
    assert r["positions"].tolist() == [3, 4, 5, 0, 1, 2, 3, -1, -1]
    assert r["slots"].tolist() == [39, 32, 33, 28, 29, 30, 31, -1, -1]


def test_plan_leaves_out_entries_that_are_no_page():
    # request 0 has ended; its second entry was given away, its third is no page of the ten
    table = np.array([[9, -1, 10, 4], [-1, -1, -1, -1]])
    r = serve.plan([16, 0], [-1, 9], table, 4, 9, np.array([1, 2, -1, -1, -1, -1, -1, -1, -1, -1]), 2)
    assert r["free_pages"][:4].tolist() == [1, 2, 9, 4] and r["free_count"] == 1
    assert r["block_table"].tolist() == [[9, -1, 10, 4], [4, 9, 2, -1]]
    assert r["slots"].tolist() == [16, 17, 18, 19, 36, 37, 38, 39, 8]


def test_plan_refuses_in_order():
    # two pages serve requests 0 and 1, one page request 0 only; request 2 needs none and is served either way
    args = [0, 0, 1], [4, 4, 1], np.array([[-1, -1], [-1, -1], [5, -1]]), 4, 20, np.array([3, 4, 0, 0, 0, 0])
    r = serve.plan(*args, 2)
    assert r["kv_len"].tolist() == [4, 4, 2] and r["free_count"] == 0
    r = serve.plan(*args, 1)
    assert r["kv_len"].tolist() == [4, 0, 2] and r["free_count"] == 0
    assert r["slots"][:9].tolist() == [12, 13, 14, 15, -1, -1, -1, -1, 21]


def test_rotation_is_an_isometry_and_adds():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 32))
    p = np.array([0, 1, 7, 100, 99999])
    y = serve.rotate(x, p, 10000.0)
    assert np.allclose(y[0], x[0]) and np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(serve.rotate(y, -p, 10000.0), x)
    # scores depend on the distance of positions alone
    z = serve.rotate(x, p + 11, 10000.0)
    assert np.allclose((y[0] * y[1]).sum(), (z[0] * z[1]).sum())


def test_attention_against_torch_and_identities():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4, 16)), rng.standard_normal((9, 2, 16)), rng.standard_normal((9, 2, 16))
    out, lse, _ = serve.attention(q, k, v, 6, 0.25)
    t = lambda a: torch.tensor(a).transpose(0, 1)[None]   # noqa: E731
    bias = torch.zeros(3, 9, dtype=torch.float64)
    for i in range(3):
        bias[i, 7 + i:] = -math.inf
    want = torch.nn.functional.scaled_dot_product_attention(
        t(q), t(k).repeat_interleave(2, 1), t(v).repeat_interleave(2, 1), attn_mask=bias, scale=0.25)
    assert np.allclose(out, want[0].transpose(0, 1).numpy())
    # a window of one sees its own value; a window that covers all changes nothing
    one, _, _ = serve.attention(q, k, v, 6, 0.25, window=1)
    assert np.allclose(one[1, 0], v[7, 0])
    assert np.allclose(serve.attention(q, k, v, 6, 0.25, window=9, sinks=2)[0], out)
    # no key: zeros and an empty sum
    none, l0, _ = serve.attention(q, k, v, -3, 0.25)
    assert not none.any() and np.all(np.isneginf(l0))
    # equal keys: the mean of what is seen, and log of how many
    m, l1, _ = serve.attention(q, np.zeros_like(k), v, 0, 0.25)
    assert np.allclose(m[2, 3], v[:3, 1].mean(0)) and np.allclose(l1[2], math.log(3))
