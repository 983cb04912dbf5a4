"""Paged attention and the plan where numbers or tables leave the ordinary range.

Tolerances are those of tests/test_gpu_serve.py; what a test adds to them stands
at the test.
"""

import math

import numpy as np
import pytest
import torch

from oracle import serve
from tests.test_gpu_serve import EPS, Case, i32, np64, q  # noqa: F401  (q: the fixture)

pytestmark = pytest.mark.gpu


def put(c, b, k=None, v=None):
    """Other keys or values for request b of a case: in its cache and for the oracle."""
    for new, pages, dense in ((k, c.cache.k, c.kd), (v, c.cache.v, c.vd)):
        if new is None:
            continue
        dense[b] = new.to(c.dtype)
        for i in range(-(-new.shape[0] // c.page)):
            part = dense[b][i * c.page:(i + 1) * c.page]
            pages[int(c.table[b, i]), :, :part.shape[0]] = part.transpose(0, 1)


FAR = [  # kv_len, q_len, heads, kv_heads, D: clusters, split items with their join, chunks whole and split
    ([300], [1], 4, 4, 128), ([5000, 40, 900], [1, 1, 2], 8, 2, 64), ([300, 700], [40, 129], 4, 2, 64),
    ([9000], [30], 2, 1, 128)]


@pytest.mark.parametrize("kv_len,q_len,heads,kv_heads,D", FAR)
@pytest.mark.parametrize("dtype,size", [(torch.float16, 8000.0), (torch.bfloat16, 1e6), (torch.bfloat16, 1e9)])
def test_scores_of_any_size(q, kv_len, q_len, heads, kv_heads, D, dtype, size):  # noqa: F811
    """Scores of 2^28 and more, whose steps in fp32 are larger than any exponent: the largest
    takes all the weight.  With q and k of `size`, the fp32 products of a score are off by at most
    D 2^-24 sum_i |q_i k_i|; where the largest leads by more than twice that and 64, every other weight
    is below 2^-64, so the output is that key's value, rounded at most once."""
    c = Case(q, kv_len, q_len, heads, kv_heads, D, 16, dtype, seed=60, std=size)
    for b in range(len(kv_len)):
        put(c, b, k=c.kd[b].float() * size)
    c.run(scale=1.0)
    out, lse, qn, group, sure = np64(c.out), np64(c.lse), np64(c.qt), heads // kv_heads, 0
    for b, n in enumerate(q_len):
        k, v = np64(c.kd[b]), np64(c.vd[b])
        for i in range(n):
            x = kv_len[b] - n + i
            for h in range(heads):
                row, g = qn[int(c.cu[b]) + i, h], h // group
                s = k[:x + 1, g] @ row
                off = D * 2.0 ** -24 * (np.abs(k[:x + 1, g]) @ np.abs(row)).max()
                got = out[int(c.cu[b]) + i, h]
                assert np.isfinite(got).all(), (b, i, h)
                first = int(s.argmax())
                if (np.delete(s, first) < s[first] - 2 * off - 64).all():
                    sure += 1
                    want = v[first, g]
                    assert (np.abs(got - want) <= EPS[dtype] / 2 * np.abs(want)).all(), (b, i, h)
                    assert abs(lse[int(c.cu[b]) + i, h] - s[first]) <= off + 2.0 ** -20 * abs(s[first]) + 64, (b, i, h)
    assert sure * 2 > sum(q_len) * heads      # most rows have such a key


@pytest.mark.parametrize("above", [12.0, 14.0, 17.0])
@pytest.mark.parametrize("kv_len,q_len", [([4000], [1]), ([4000, 900, 2500], [1, 2, 1]), ([2000, 1500], [1, 1]),
                                          ([4000, 900], [40, 130])])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_key_far_above_the_others_with_a_small_value(q, above, kv_len, q_len, dtype):  # noqa: F811
    """A first token that takes nearly all weight and has no value: the output is the sum of thousands of
    small weights.  Beside the bounds of Case.check, fp16 weights of less than 2^-14 lie on a grid of 2^-24:
    off by 2^-25 where the largest is at least 2^8 (many rows) or 2^15 (few), so by 2^-33 or 2^-40 of the largest
    weight, which is at most 1.  bf16 has no such bound."""
    D, H, Hkv = 64, 4, 2
    c = Case(q, kv_len, q_len, H, Hkv, D, 32, dtype, seed=61, std=0.3)
    c.qt[..., 0] = 8.0
    for b, n in enumerate(kv_len):
        k, v = c.kd[b].float(), c.vd[b].float() * 1000.0
        k[:, :, 0] = 0.0
        k[0] = 0.0
        k[0, :, 0] = above
        v[0] = 0.0
        put(c, b, k, v)
    c.run()
    grid = 0.0 if dtype is torch.bfloat16 else 2.0 ** -40 if max(q_len) * (H // Hkv) <= 16 else 2.0 ** -33
    eps = EPS[dtype]
    p16 = eps / 2 if max(q_len) * (H // Hkv) > 16 else 2.0 ** -16
    out, lse, qn = np64(c.out), np64(c.lse), np64(c.qt)
    for b, n in enumerate(q_len):
        k, v = np64(c.kd[b]), np64(c.vd[b])
        for i in {0, n // 2, n - 1}:
            at = slice(int(c.cu[b]) + i, int(c.cu[b]) + i + 1)
            x = kv_len[b] - n + i
            want, wl, mag = serve.attention(qn[at], k, v, x, D ** -0.5)
            top = max((np.abs(qn[at][0, h]) * np.abs(k[:, h // (H // Hkv)])).sum(-1).max() for h in range(H))
            d = D ** -0.5 * D * 2.0 ** -24 * top + 2.0 ** -18
            small = grid * np.repeat(np.abs(v[:x + 1]).sum(0), H // Hkv, 0)[None]
            err = np.abs(out[at] - want)
            tol = eps / 2 * np.abs(want) * (1 + eps) + (2 * d + p16) * mag + small
            assert (err <= tol).all(), (b, i, float((err / tol).max()))
            assert (np.abs(lse[at] - wl) <= d + 2.0 ** -20 * np.abs(wl)).all(), (b, i)


@pytest.mark.parametrize("kv_len,q_len,heads", [([700], [1], 8), ([700, 500], [1, 1], 8), ([9000, 20, 300], [1, 1, 1], 8),
                                                ([700, 500], [40, 40], 8), ([9000], [40], 4)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", ["nan row", "inf row", "inf in a row", "nan key"])
def test_lse_of_a_row_that_is_not_finite(q, kv_len, q_len, heads, D, what):  # noqa: F811
    """-inf is kept for rows that see nothing: a row without a finite result has none in lse either."""
    c = Case(q, kv_len, q_len, heads, 2, D, 16, seed=62).run()
    first = c.lse.clone()
    hit = torch.zeros(c.T, heads, dtype=torch.bool, device="cuda")
    hit[0, 3] = True
    if what == "nan row":
        c.qt[0, 3] = math.nan
    elif what == "inf row":
        c.qt[0, 3] = math.inf
    elif what == "inf in a row":
        c.qt[0, 3, 1] = math.inf
    else:       # position 3 of the first request, key/value head 1: seen by all its rows
        c.cache.k[int(c.table[0, 0]), 1, 3] = math.nan
        hit[0, 3] = False
        hit[:q_len[0], heads // 2:] = True
    c.run()
    assert not torch.isfinite(c.out[hit].float()).any()
    assert not (torch.isfinite(c.lse[hit]) | torch.isneginf(c.lse[hit])).any()
    # the others up to the bound of each call: the same products, maybe against another reference
    others = ~hit
    assert ((c.lse - first).abs() <= 2.0 ** -10 + 2.0 ** -19 * first.abs())[others].all()


@pytest.mark.parametrize("seed", range(5))
def test_plan_returns_only_entries_that_are_pages(q, seed):  # noqa: F811
    """Requests under a window whose pages before it went to others: those entries hold -1 (or no page at all)
    when the request ends, and only the rest goes back to the pool."""
    rng = np.random.default_rng(100 + seed)
    B, page = [3, 50, 400, 2000, 4096][seed], 16
    width = [70, 30, 200, 12, 5][seed]
    ctx = rng.integers(0, width * page + 1, B)
    new = np.where(rng.random(B) < 0.4, -1, rng.integers(0, 2 * page, B))
    new[rng.random(B) < 0.1] = -2 ** 31
    pages = -(-ctx // page)
    ids = rng.permutation(int(pages.sum()) + 50)
    P, at = len(ids), 0
    table = np.full((B, width), -1)
    for b in range(B):
        table[b, :pages[b]] = ids[at:at + pages[b]]
        at += pages[b]
        sinks, window = int(rng.integers(0, 3)), int(rng.integers(0, width))
        if rng.random() < 0.7:      # given away: page ids below `given` are taken to be the pool's again
            table[b, sinks:max(sinks, pages[b] - window)] = rng.choice([-1, P, 2 ** 31 - 1, -2 ** 31])
    held = table[(table >= 0) & (table < P)]
    free = np.full(P, -1)
    rest = np.setdiff1d(np.arange(P), held)
    free[:len(rest)] = rest
    tokens = int(np.maximum(new, 0).sum()) + 5
    want = serve.plan(ctx, new, table, page, tokens, free, len(rest))
    kv = q.KVBatch(B, width, tokens, block_table=i32(table))
    fp, fc = i32(free), i32([len(rest)])
    q.qlora_kv_plan(kv, page, P, i32(ctx), i32(new), fp, fc)
    q.qlora_check_device_error()
    for name in ("block_table", "cu_q", "kv_len", "positions", "slots"):
        assert np.array_equal(getattr(kv, name).cpu().numpy(), want[name]), name
    assert int(fc) == want["free_count"] and np.array_equal(fp.cpu().numpy(), want["free_pages"])
    # every page is in the pool or in one live row, once
    live = want["block_table"][(new >= 0)]
    mine = np.concatenate([want["free_pages"][:want["free_count"]], live[(live >= 0) & (live < P)]])
    assert len(np.unique(mine)) == len(mine)
    assert (want["free_pages"][:want["free_count"]] >= 0).all()


def test_what_a_descriptor_holds_cannot_be_replaced(q):  # noqa: F811
    """The calls read addresses and sizes from the descriptor: a tensor set in its place would be
    ignored, and the old one's memory, free by then, used."""
    cache, kv = q.KVCache.empty(4, 16, 2, 64), q.KVBatch(2, 3, 10, max_q_len=1)
    for thing, names in ((cache, ("k", "v", "desc", "device", "num_pages", "page_size", "dtype")),
                         (kv, ("block_table", "cu_q", "kv_len", "positions", "slots", "batch", "max_pages", "tokens",
                               "desc"))):
        for name in names:
            before = getattr(thing, name)
            with pytest.raises(AttributeError):
                setattr(thing, name, before.clone() if isinstance(before, torch.Tensor) else before)
            assert getattr(thing, name) is before


def test_max_q_len_set_again_reaches_the_calls(q):  # noqa: F811
    """It chooses the kernel, and with it the workspace."""
    few, many = [Case(q, [300, 40], [1, 1], 8, 4, 128, 16, seed=63, pad=30, max_q_len=n) for n in (1, 31)]
    size = lambda c: q.qlora_paged_attn_workspace_bytes(c.cache, c.kv, 8)   # noqa: E731
    assert size(few) != size(many)
    few.run()
    many.kv.max_q_len = 1
    assert many.kv.max_q_len == 1 and size(few) == size(many)
    assert torch.equal(many.run().out, few.out)


@pytest.mark.parametrize("n", [1, 40])
def test_one_head_of_an_odd_stride(q, n):  # noqa: F811
    """The stride of a dimension of one is never used."""
    c = Case(q, [200, 50], [n, 2], 4, 1, 64, 16, seed=64)
    odd = lambda t: t.as_strided(t.shape, (t.stride(0), 3, t.stride(2), 1))   # noqa: E731
    c.cache = q.KVCache(odd(c.cache.k), odd(c.cache.v))
    assert c.cache.desc.stride_head == 3
    c.run().check()
    x = torch.randn(c.T, 1, 64, device="cuda").to(torch.bfloat16)
    q.qlora_kv_append(c.cache, q.KVBatch(1, 1, c.T, slots=torch.arange(c.T, dtype=torch.int32, device="cuda")), None,
                      c.qt, x, -x)
    flat = c.cache.k.transpose(1, 2).reshape(-1, 1, 64)
    assert torch.equal(flat[:c.T], x)


@pytest.mark.parametrize("kv_heads,lengths,window,sinks,launches", [
    (16, [0, 1, 16, 65, 300, 700, 1000, 1200], 0, 0, 1),        # two CTAs a head: 128 heads, a table of 1200 positions
    (16, [0, 1, 16, 65, 300, 2000, 4000, 5000], 900, 20, 1),    # ... or a window
    (25, [0, 1, 16, 65, 300, 500, 620, 640], 0, 0, 1),          # one: 200 heads, a table of 640
    (25, [0, 1, 16, 65, 300, 2000, 4000, 5000], 1000, 4, 1),
    (25, [0, 1, 16, 65, 300, 700, 1000, 1200], 0, 0, 2),        # a longer table: the schedule and its join
    (38, [0, 1, 16, 65, 300, 500, 620, 640], 0, 0, 2)])         # 304 heads
def test_forms_of_few_requests(q, kv_heads, lengths, window, sinks, launches):  # noqa: F811
    """Requests without rows, without keys, and (promised to be short) with several tiles of rows."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 148:
        pytest.skip("the counts are those of 148 SMs")
    for new in ([1, 0, 1, 1, 2, 1, 1, 1], [1, 1, 9, 20, 0, 30, 1, 3]):
        c = Case(q, lengths, new, 2 * kv_heads, kv_heads, 64, 16, seed=65, max_q_len=2)
        n = q.qlora_launch_count()
        c.run(window, sinks)
        assert q.qlora_launch_count() - n == launches
        c.check(window, sinks)


@pytest.mark.parametrize("kv", [1, 70, 900])
def test_one_request_of_more_heads_than_places(q, kv):  # noqa: F811
    Case(q, [kv], [1], 320, 320, 16, 16, seed=66).run().check()


@pytest.mark.parametrize("kv_len,n", [([1] * 12, 497), ([1, 0, 0] * 5, 497), ([300, 0, 0, 0, 0] * 3, 290), ([2, 0] * 8, 400)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (448, 300)])
def test_many_items_without_a_key_between_others(q, kv_len, n, window, sinks):  # noqa: F811
    """Long prompts that were refused (no positions), or rows before position 0: a CTA gets four and
    more items without a tile after one that has one."""
    c = Case(q, kv_len, [n] * len(kv_len), 68, 17, 16, 16, seed=67, max_q_len=n)
    c.run(window, sinks).check(window, sinks, rows=[0, n // 2, n - 2, n - 1])
