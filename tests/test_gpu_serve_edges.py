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
