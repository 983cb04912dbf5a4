"""GPU parity of the serving operators (plan, append, paged attention) with
the float64 oracle.

Tolerances, from the arithmetic.  Attention: with weights p_j, values v_j and
A = sum p_j |v_j|, an output is off by at most
  eps/2 |out|       its own rounding (eps of the 16-bit type),
  2 d A             from weights off by a relative d in numerator and sum:
                    d <= scale D 2^-24 max sum_i |q_i k_i| (fp32 products, any
                    order) + 2^-18 (exp2 of an argument of at most 2^5, two
                    units each; sums of nonnegative terms, split and joined),
  eps/2 A           where the weights enter the second product in 16 bits
                    (more than 16 rows per item); 2^-16 A where they enter as
                    two 16-bit parts.
log-sum-exp: d + 2^-20 |lse|.  Append: eps/2 |x| for the rounding plus 2^-19
(|a| + |b|) for sine and cosine (absolute error 2^-21 each, and an angle in
[-pi, pi] rounded at 2^-23).  Integers are equal.
"""

import math

import numpy as np
import pytest
import torch

from oracle import serve

pytestmark = pytest.mark.gpu

EPS = {torch.bfloat16: 2.0 ** -7, torch.float16: 2.0 ** -10}


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_16_b200 as q
    assert torch.cuda.is_available()
    return q


def np64(t):
    return t.double().cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A planned batch over a cache whose unused positions hold NaN."""

    def __init__(self, q, kv_len, q_len, heads, kv_heads, D, page, dtype=torch.bfloat16, order="heads first", seed=0,
                 pad=3, width=None, max_q_len=None, std=2.0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.kv_len, self.q_len, self.H, self.Hkv, self.D, self.page, self.dtype = kv_len, q_len, heads, kv_heads, D, page, dtype
        B = len(kv_len)
        need = [-(-k // page) for k in kv_len]
        self.width = width = max(need + [1]) if width is None else width
        P = sum(need) + 2
        shape = (P, kv_heads, page, D) if order == "heads first" else (P, page, kv_heads, D)
        def cache():
            t = torch.full(shape, math.nan, dtype=dtype, device="cuda")
            return t if order == "heads first" else t.transpose(1, 2)
        k, v = cache(), cache()
        ids = torch.randperm(P, generator=g, device="cuda").tolist()
        table = np.full((B, width), -1)
        self.kd, self.vd = [], []
        for b in range(B):
            mine = [ids.pop() for _ in range(need[b])]
            table[b, :len(mine)] = mine[:width]
            L = kv_len[b]
            kk = torch.randn(L, kv_heads, D, generator=g, device="cuda").to(dtype)
            vv = torch.randn(L, kv_heads, D, generator=g, device="cuda").to(dtype)
            for i, pg in enumerate(mine):
                n = min(page, L - i * page)
                k[pg, :, :n] = kk[i * page:i * page + n].transpose(0, 1)
                v[pg, :, :n] = vv[i * page:i * page + n].transpose(0, 1)
            self.kd.append(kk)
            self.vd.append(vv)
        self.cache = q.KVCache(k, v)
        self.table = i32(table)
        cu = np.concatenate([[0], np.cumsum(q_len)])
        self.T = int(cu[-1]) + pad
        self.cu = cu
        self.kv = q.KVBatch(B, width, self.T, max_q_len=max(q_len) if max_q_len is None else max_q_len,
                            block_table=self.table, cu_q=i32(cu), kv_len=i32(kv_len))
        self.qt = (torch.randn(self.T, heads, D, generator=g, device="cuda") * std).to(dtype)
        self.q = q

    def run(self, window=0, sinks=0, scale=None, stream=None, ws=None):
        scale = self.D ** -0.5 if scale is None else scale
        self.out = torch.full_like(self.qt, 7.0)
        self.lse = torch.full((self.T, self.H), 7.0, dtype=torch.float32, device="cuda")
        if ws is None:
            n = self.q.qlora_paged_attn_workspace_bytes(self.cache, self.kv, self.H)
            ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")    # NaNs as floats
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        self.q.qlora_paged_attn_fwd(self.cache, self.kv, self.qt, self.out, scale, ws, window=window, sinks=sinks,
                                    lse=self.lse, stream=stream)
        if stream is not None:
            stream.synchronize()
        self.q.qlora_check_device_error(stream)
        return self

    def check(self, window=0, sinks=0, scale=None, present=None, rows=None):
        """rows: of each request, compare only these (the oracle is slow on whole prompts)."""
        scale = self.D ** -0.5 if scale is None else scale
        eps = EPS[self.dtype]
        out, lse, qn = np64(self.out), np64(self.lse), np64(self.qt)
        p16 = eps / 2 if max(self.q_len) * (self.H // self.Hkv) > 16 else 2.0 ** -16
        for b, n in enumerate(self.q_len):
            if n == 0:
                continue
            a, L = int(self.cu[b]), self.kv_len[b]
            k, v = np64(self.kd[b]), np64(self.vd[b])
            for i in range(n) if rows is None else [r for r in rows if r < n]:
                s = slice(a + i, a + i + 1)
                want, wl, mag = serve.attention(qn[s], k, v, L - n + i, scale, window, sinks,
                                                None if present is None else present[b])
                top = 0.0
                if L:
                    top = max((np.abs(qn[a + i, h]) * np.abs(k[:, h // (self.H // self.Hkv)])).sum(-1).max()
                              for h in range(self.H))
                d = scale * self.D * 2.0 ** -24 * top + 2.0 ** -18
                err = np.abs(out[s] - want)
                tol = eps / 2 * np.abs(want) * (1 + eps) + (2 * d + p16) * mag + 1e-30
                assert np.all(err <= tol), (b, i, float((err / tol).max()))
                if np.isneginf(wl).all():
                    assert np.all(np.isneginf(lse[s])) and not out[s].any()
                else:
                    assert np.all(np.abs(lse[s] - wl) <= d + 2.0 ** -20 * np.abs(wl)), (b, i)
        end = int(self.cu[-1])
        assert np.all(out[end:] == 7.0) and np.all(lse[end:] == 7.0)     # rows behind the last request
        return self


LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 130, 300, 1000]


@pytest.mark.parametrize("D", [16, 48, 64, 80, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_decode_lengths(q, D, dtype):
    Case(q, LENGTHS, [1] * 12, 4, 2, D, 16, dtype).run().check()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (8, 1), (14, 2), (16, 1), (32, 2), (40, 2)])
@pytest.mark.parametrize("page,order", [(16, "tokens first"), (64, "heads first"), (256, "tokens first")])
def test_decode_heads_pages_and_orders(q, heads, kv_heads, page, order):
    Case(q, [700, 5, 0, 257], [1, 1, 1, 1], heads, kv_heads, 128, page, order=order, seed=1).run().check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 1), (100, 4), (100, 70), (64, 128), (5000, 4), (2 ** 30, 0)])
def test_decode_window(q, window, sinks):
    Case(q, LENGTHS + [3000], [1] * 13, 8, 2, 64, 32, seed=2).run(window, sinks).check(window, sinks)


@pytest.mark.parametrize("n", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_several_tokens_and_none(q, n, window, sinks):
    Case(q, [200, 3, 17, 1000], [n, 1, 0, 3], 8, 4, 128, 16, torch.float16, seed=3).run(window, sinks).check(window, sinks)


def test_rows_without_a_key(q):
    """More new tokens than positions: the first rows lie before position 0."""
    Case(q, [3, 0, 1], [6, 2, 1], 2, 2, 64, 16, seed=4).run().check()


@pytest.mark.parametrize("heads,kv_heads,n", [(1, 1, 1), (16, 1, 1), (8, 8, 2)])
def test_one_long_request_is_split(q, heads, kv_heads, n):
    c = Case(q, [30001], [n], heads, kv_heads, 128, 64, seed=5).run()
    c.check()
    first = c.out.clone()
    assert torch.equal(c.run().out, first)      # the same bits again


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (16, 1), (5, 5), (32, 32), (64, 64), (100, 100), (200, 200)])
@pytest.mark.parametrize("kv,n,window,sinks", [(1000, 1, 0, 0), (1, 1, 0, 0), (70, 1, 0, 0), (4000, 1, 500, 3)])
def test_one_request_alone(q, heads, kv_heads, kv, n, window, sinks):
    """Clusters of CTAs per key/value head, down to none for many heads."""
    Case(q, [kv], [n], heads, kv_heads, 64, 16, seed=50).run(window, sinks).check(window, sinks)


@pytest.mark.parametrize("D", [16, 48, 128])
@pytest.mark.parametrize("kv,n", [(0, 1), (0, 0), (3, 8), (90, 8), (2000, 3)])
def test_one_request_alone_lengths(q, D, kv, n):
    c = Case(q, [kv], [n], 4, 2, D, 32, torch.float16, seed=51, pad=9 - n)
    first = c.run().check().out.clone()
    assert torch.equal(c.run().out, first)


@pytest.mark.parametrize("kv_heads,window,sinks", [(1, 0, 0), (4, 0, 0), (9, 100, 5), (25, 0, 0)])
def test_few_requests(q, kv_heads, window, sinks):
    """Clusters of eight, four, two and one CTAs per key/value head of eight requests."""
    Case(q, [0, 1, 16, 65, 300, 700, 1000, 1200], [1, 0, 1, 1, 2, 1, 1, 1], 2 * kv_heads, kv_heads, 64, 16,
         seed=54).run(window, sinks).check(window, sinks)


def test_one_request_with_more_rows_than_promised(q):
    """max_q_len only steers the choice of kernel."""
    Case(q, [150], [30], 4, 2, 64, 16, seed=52, max_q_len=1).run().check()
    Case(q, [150, 40], [30, 9], 4, 2, 64, 16, seed=53, max_q_len=1).run().check()


def test_many_requests(q):
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 200, 1300).tolist()
    new = [min(int(x), 1) for x in rng.integers(0, 3, 1300)]
    Case(q, lens, new, 2, 1, 64, 16, seed=6).run().check()


def test_most_requests(q):
    lens = [1 + i % 3 for i in range(4096)]
    Case(q, lens, [1] * 4096, 1, 1, 16, 16, seed=7).run().check()


@pytest.mark.parametrize("D", [16, 64, 80, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_chunk_types_and_dims(q, D, dtype):
    Case(q, [300, 17, 0, 129], [60, 17, 2, 1], 4, 2, D, 16, dtype, seed=30).run().check()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (8, 1), (14, 2), (12, 4)])
@pytest.mark.parametrize("page,order", [(16, "heads first"), (32, "tokens first"), (128, "heads first"), (256, "tokens first")])
def test_chunk_heads_pages_and_orders(q, heads, kv_heads, page, order):
    Case(q, [400, 5, 130, 700], [150, 5, 128, 33], heads, kv_heads, 128, page, order=order, seed=31).run().check()


@pytest.mark.parametrize("n", [17, 31, 127, 128, 129, 255, 256, 257, 300])
def test_chunk_rows(q, n):
    Case(q, [n + 77, n], [n, n], 1, 1, 64, 16, seed=32).run().check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 1), (100, 4), (130, 200), (256, 128), (5000, 4)])
def test_chunk_window(q, window, sinks):
    Case(q, [900, 300, 40], [200, 300, 1], 4, 2, 64, 32, seed=33).run(window, sinks).check(window, sinks)


def test_chunk_rows_without_a_key(q):
    """Rows before position 0, requests without any position, and many of them in a row."""
    Case(q, [3, 0, 0, 0, 0, 0, 0, 40, 0], [60, 20, 1, 300, 2, 2, 5, 20, 9], 4, 4, 64, 16, seed=34).run().check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_chunk_whole_prompt(q, dtype):
    c = Case(q, [2048], [2048], 4, 4, 128, 16, dtype, seed=35).run()
    c.check(rows=[0, 1, 2, 127, 128, 129, 255, 256, 1000, 1023, 1024, 2047])
    first = c.out.clone()
    assert torch.equal(c.run().out, first)


@pytest.mark.parametrize("window,sinks", [(0, 0), (3000, 20)])
def test_chunk_over_a_long_context_is_split(q, window, sinks):
    c = Case(q, [20011, 64], [40, 64], 4, 2, 128, 64, seed=36).run(window, sinks)
    c.check(window, sinks, rows=[0, 1, 20, 39, 40, 63])


def test_chunk_many_requests(q):
    rng = np.random.default_rng(37)
    lens = rng.integers(0, 150, 700).tolist()
    Case(q, lens, [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 30, 700))], 2, 1, 64, 16, seed=37).run().check(
        rows=[0, 7, 15, 29])


def test_chunk_growing_scores(q):
    """Keys that grow along the context: the running maximum is passed again and again."""
    c = Case(q, [700], [64], 2, 1, 64, 16, torch.float16, seed=38)
    ramp = torch.linspace(0.05, 6.0, 700, device="cuda")[:, None, None]
    c.kd[0] = (c.kd[0].abs() * ramp).to(torch.float16)
    c.qt = c.qt.abs()
    for i in range(44):
        n = min(16, 700 - 16 * i)
        c.cache.k[int(c.table[0, i]), :, :n] = c.kd[0][16 * i:16 * i + n].transpose(0, 1)
    c.run().check()


def test_kernels_agree(q):
    """The bound on q_len chooses the kernel, not the result: both stay within
    their bounds of the oracle, so within the sum of them of each other."""
    a = Case(q, [300, 40, 1000], [2, 1, 3], 8, 4, 128, 16, seed=39).run()
    b = Case(q, [300, 40, 1000], [2, 1, 3], 8, 4, 128, 16, seed=39, max_q_len=0).run()
    assert not torch.equal(a.out, b.out)
    diff, size = (a.out.float() - b.out.float()).abs()[:6], a.out.float().abs()[:6]
    # half a step each, and half a step of a weight on values of at most 4 deviations
    assert (diff <= 2.0 ** -7 * size + 2.0 ** -8 * 4).all()


def test_chunk_bad_pages_are_left_out(q):
    c = Case(q, [200, 90, 64], [100, 2, 30], 4, 2, 64, 16, seed=40)
    present = [np.ones(200, bool), np.ones(90, bool), np.zeros(64, bool)]
    for b, i, v in [(0, 0, -1), (0, 3, c.cache.num_pages), (0, 12, 2 ** 31 - 1), (1, 5, -2 ** 31), (1, 0, -7)]:
        c.table[b, i] = v
        present[b][16 * i:16 * i + 16] = False
    c.table[2] = c.cache.num_pages
    c.run().check(present=present)


def test_chunk_positions_beyond_the_table_are_left_out(q):
    c = Case(q, [200, 90], [70, 20], 4, 2, 64, 16, seed=41, width=6)
    c.run().check(present=[np.arange(200) < 96, np.arange(90) < 96])


@pytest.mark.parametrize("n,D,page", [(1, 64, 16), (1, 128, 128), (40, 64, 16), (40, 128, 64), (300, 128, 32)])
@pytest.mark.parametrize("sinks", [0, 5, 140])
def test_pages_that_no_row_sees_may_hold_anything(q, n, D, page, sinks):
    """Pages between the sinks and the first row's window went back to the pool and hold NaN."""
    window, lengths = 100, [1000, 700, 430]
    c = Case(q, lengths, [n] * 3, 4, 2, D, page, seed=43)
    for b, L in enumerate(lengths):
        for i in range(-(-sinks // page), max(0, L - n - window + 1) // page):
            page_id = int(c.table[b, i])
            c.cache.k[page_id], c.cache.v[page_id] = math.nan, math.nan
    c.run(window, sinks).check(window, sinks, rows=None if n < 100 else [0, 1, 99, 127, 128, 200, 299])


def test_bad_pages_are_left_out(q):
    c = Case(q, [200, 90, 64], [1, 2, 1], 4, 2, 64, 16, seed=8)
    present = [np.ones(200, bool), np.ones(90, bool), np.zeros(64, bool)]
    for b, i, v in [(0, 0, -1), (0, 3, c.cache.num_pages), (0, 12, 2 ** 31 - 1), (1, 5, -2 ** 31), (1, 0, -7)]:
        c.table[b, i] = v
        present[b][16 * i:16 * i + 16] = False
    c.table[2] = c.cache.num_pages
    c.run().check(present=present)


def test_positions_beyond_the_table_are_left_out(q):
    c = Case(q, [200, 90], [1, 1], 4, 2, 64, 16, seed=9, width=6)
    present = [np.arange(200) < 96, np.arange(90) < 96]
    c.run().check(present=present)


def test_offsets_past_32_bits(q):
    """Pages more than 2^32 elements apart."""
    far = 2 ** 32 + 4096
    store = [torch.empty(far + 2 * 16 * 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = [s.as_strided((2, 2, 16, 64), (far, 1024, 64, 1)) for s in store]
    g = torch.Generator("cuda").manual_seed(10)
    k.copy_(torch.randn(2, 2, 16, 64, generator=g, device="cuda"))
    v.copy_(torch.randn(2, 2, 16, 64, generator=g, device="cuda"))
    c = Case(q, [29], [1], 4, 2, 64, 16, seed=10)
    c.cache = q.KVCache(k, v)
    c.table[0] = i32([1, 0])
    c.kd = [torch.cat([k[1], k[0]], 1).transpose(0, 1)[:29]]
    c.vd = [torch.cat([v[1], v[0]], 1).transpose(0, 1)[:29]]
    c.run().check()
    # the append reaches the same places
    kv = q.KVBatch(1, 2, 2, slots=i32([17, 5]), positions=i32([0, 0]))
    x = torch.randn(2, 2, 64, generator=g, device="cuda").to(torch.bfloat16)
    q.qlora_kv_append(c.cache, kv, None, x, x, -x)
    assert torch.equal(k[1, :, 1], x[0]) and torch.equal(k[0, :, 5], x[1]) and torch.equal(v[1, :, 1], -x[0])


def test_large_scores(q):
    """One key far above the others, and scores of hundreds: no overflow, the weight goes to the largest."""
    c = Case(q, [500], [1], 2, 1, 128, 16, torch.float16, seed=11, std=60.0)
    c.run(scale=1.0)
    assert torch.isfinite(c.out.float()).all()
    c.check(scale=1.0)


def test_another_stream(q):
    Case(q, [300, 40], [1, 1], 4, 2, 128, 16, seed=12).run(stream=torch.cuda.Stream()).check()


@pytest.mark.parametrize("n,D", [(1, 64), (1, 128), (40, 64), (300, 128)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_row_that_is_not_finite_stays_alone(q, n, D, value):
    """One head of one token: every other row keeps its value, up to half a step of
    itself and of the weights (on values of at most max |v|) in each of the two calls."""
    c = Case(q, [700, 500], [n, n], 8, 2, D, 16, seed=44).run()
    clean = c.out.float()
    c.qt[n // 2, 5] = value
    c.run()
    others = torch.ones(c.T, 8, dtype=torch.bool, device="cuda")
    others[n // 2, 5] = False
    assert not torch.isfinite(c.out[n // 2, 5].float()).any()
    top = max(float(v.float().abs().max()) for v in c.vd)
    diff = (c.out.float() - clean).abs()
    assert (diff <= 2.0 ** -7 * clean.abs() * (1 + 2.0 ** -7) + (2.0 ** -7 + 2.0 ** -16) * top)[others].all()


def test_calls_at_once(q):
    """Four calls on four streams, each with its workspace, over and over."""
    cases = [Case(q, [900, 33], [1, 1], 8, 2, 128, 16, seed=45), Case(q, [900, 330], [70, 300], 8, 2, 128, 16, seed=46),
             Case(q, [2000], [1], 32, 32, 64, 16, seed=47), Case(q, [600, 20], [200, 20], 8, 8, 64, 32, seed=48)]
    calls = []
    for c in cases:
        c.run()
        n = q.qlora_paged_attn_workspace_bytes(c.cache, c.kv, c.H)
        calls.append((c, torch.cuda.Stream(), torch.full((n,), 0xff, dtype=torch.uint8, device="cuda"),
                      torch.full_like(c.out, 7.0), torch.full_like(c.lse, 7.0)))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, stream, ws, out, lse in calls:
            q.qlora_paged_attn_fwd(c.cache, c.kv, c.qt, out, c.D ** -0.5, ws, lse=lse, stream=stream)
    torch.cuda.synchronize()
    q.qlora_check_device_error()
    for c, _, _, out, lse in calls:     # the same call gives the same bits
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse)


def test_captured_and_replayed_with_other_lengths(q):
    a = Case(q, [300, 40, 77], [1, 1, 1], 4, 2, 128, 16, seed=13, width=30)
    b = Case(q, [5, 470, 0], [1, 1, 1], 4, 2, 128, 16, seed=14, width=30)
    ws = torch.empty(q.qlora_paged_attn_workspace_bytes(a.cache, a.kv, 4), dtype=torch.uint8, device="cuda")
    cache = q.KVCache.empty(max(a.cache.num_pages, b.cache.num_pages), 16, 2, 128)
    kv = q.KVBatch(3, 30, a.T, max_q_len=1)
    qt, out, lse = torch.empty_like(a.qt), torch.full_like(a.qt, 7.0), torch.full_like(a.qt[..., 0].float(), 7.0)
    call = lambda: q.qlora_paged_attn_fwd(cache, kv, qt, out, 128 ** -0.5, ws, lse=lse)   # noqa: E731
    call()      # first use sets the kernels up
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]     # two graphs on one workspace
    for g in graphs:
        with torch.cuda.graph(g):
            call()
    for c, g in ((a, graphs[0]), (b, graphs[1]), (a, graphs[1])):
        cache.k[:c.cache.num_pages], cache.v[:c.cache.num_pages] = c.cache.k, c.cache.v
        for name in ("block_table", "cu_q", "kv_len"):
            getattr(kv, name).copy_(getattr(c.kv, name))
        qt.copy_(c.qt)
        out.fill_(7.0)
        g.replay()
        c.out, c.lse = out.clone(), lse.clone()
        c.check()


@pytest.mark.parametrize("seed", range(6))
def test_plan(q, seed):
    rng = np.random.default_rng(seed)
    B = [1, 7, 40, 513, 1200, 4096][seed]
    page = [16, 32, 16, 64, 16, 256][seed]
    width = 12
    ctx = rng.integers(0, width * page + 1, B)
    new = rng.integers(0, 3 * page, B)
    new[rng.random(B) < 0.3] = 1
    new[rng.random(B) < 0.1] = -1
    if B > 7:
        ctx[rng.integers(0, B, 3)] = -5
        new[rng.integers(0, B, 3)] = 0
    pages = -(-np.maximum(ctx, 0) // page)
    P = int(pages.sum()) + [40, 5, 30, 200, 900, 9000][seed]
    ids = rng.permutation(P)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = ids[at:at + pages[b]]
        at += pages[b]
    free = np.full(P, -1)
    free[:P - at] = ids[at:]
    tokens = int(np.maximum(new, 0).sum() * [1.0, 1.0, 0.6, 1.1, 0.9, 1.0][seed]) + 1
    want = serve.plan(ctx, new, table, page, tokens, free, P - at)
    kv = q.KVBatch(B, width, tokens, block_table=i32(table))
    fp, fc = i32(free), i32([P - at])
    for where in (torch.zeros_like(fc), None):     # elsewhere, then in place
        kv.block_table.copy_(i32(table))
        fp.copy_(i32(free))
        q.qlora_kv_plan(kv, page, P, i32(ctx), i32(new), fp, fc, where)
        q.qlora_check_device_error()
        for name in ("block_table", "cu_q", "kv_len", "positions", "slots"):
            assert np.array_equal(getattr(kv, name).cpu().numpy(), want[name]), name
        assert np.array_equal(fp.cpu().numpy(), want["free_pages"])
        assert int(fc if where is None else where) == want["free_count"]


def test_plan_with_an_overdrawn_pool_and_odd_values(q):
    """More than the pool has, rows past the step, a count beyond the pool and a negative one."""
    B, page, width = 4096, 16, 2 ** 14
    P = 64
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    kv = q.KVBatch(B, width, 2 ** 24, block_table=table)
    new = torch.full((B,), 2 ** 18, dtype=torch.int32, device="cuda")
    free = torch.arange(P, dtype=torch.int32, device="cuda")
    for count in (P, P + 1000, -3):
        fc = i32([count])
        q.qlora_kv_plan(kv, page, P, torch.zeros_like(new), new, free, fc)
        assert not kv.kv_len.any() and (kv.slots == -1).all() and int(fc) == min(max(count, 0), P)
    assert (table == -1).all()


@pytest.mark.parametrize("D", [16, 64, 80, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,heads,kv_heads,order", [(1, 1, 1, 0), (5, 6, 2, 1), (700, 4, 4, 0), (3001, 3, 1, 1)])
def test_append(q, D, dtype, T, heads, kv_heads, order):
    g = torch.Generator("cuda").manual_seed(T + D)
    rng = np.random.default_rng(T)
    page, P = 32, T // 32 + 5
    def empty():
        t = torch.full((P, page, kv_heads, D) if order else (P, kv_heads, page, D), 3.0, dtype=dtype, device="cuda")
        return t.transpose(1, 2) if order else t
    cache = q.KVCache(empty(), empty())
    slots = rng.permutation(P * page)[:T]
    pos = rng.integers(0, 2 ** 20, T)
    pos[0] = 2 ** 30 - 1
    if T > 4:
        slots[1], slots[2], slots[3], pos[1] = -1, P * page, 2 ** 31 - 1, -1
    x = {n: torch.randn(T, h, D, generator=g, device="cuda").to(dtype) for n, h in
         (("q", heads), ("k", kv_heads), ("v", kv_heads))}
    kv = q.KVBatch(1, 1, T, positions=i32(pos), slots=i32(slots))
    out = torch.full_like(x["q"], 5.0)
    q.qlora_kv_append(cache, kv, q.qlora_build_rope(D, 10000.0), x["q"], x["k"], x["v"], out)
    kept = (slots >= 0) & (slots < P * page)
    eps = EPS[dtype]
    def close(got, x, what):
        x = np64(x)[kept]
        want = serve.rotate(x, pos[kept], 10000.0)
        pair = np.abs(x) + np.abs(np.roll(x, D // 2, -1))
        err = np.abs(got - want)
        assert np.all(err <= eps / 2 * np.abs(want) * (1 + eps) + 2.0 ** -19 * pair + 2.0 ** -25), what
    close(np64(out)[kept], x["q"], "q")
    assert np.all(np64(out)[~kept] == 5.0)
    flat = lambda t: t.transpose(1, 2).reshape(P * page, kv_heads, D)   # noqa: E731
    where = torch.tensor(slots[kept], device="cuda")
    close(np64(flat(cache.k)[where]), x["k"], "k")
    assert torch.equal(flat(cache.v)[where], x["v"][torch.tensor(kept, device="cuda")])
    others = torch.ones(P * page, dtype=torch.bool, device="cuda")
    others[where] = False
    assert (flat(cache.k)[others] == 3.0).all() and (flat(cache.v)[others] == 3.0).all()
    # in place, and without a rotation
    inp = x["q"].clone()
    q.qlora_kv_append(cache, kv, q.qlora_build_rope(D, 10000.0), inp, x["k"], x["v"])
    assert torch.equal(inp[torch.tensor(kept, device="cuda")], out[torch.tensor(kept, device="cuda")])
    q.qlora_kv_append(cache, kv, None, x["q"], x["k"], x["v"], out)
    assert torch.equal(flat(cache.k)[where], x["k"][torch.tensor(kept, device="cuda")])


def test_a_run_of_steps(q):
    """Prompts in chunks, then single tokens; requests end, others take their
    pages: plan, append and attention together, against attention over the
    requests' own keys."""
    H, Hkv, D, page, P, width, B, T = 8, 2, 64, 16, 26, 10, 4, 160
    g = torch.Generator("cuda").manual_seed(20)
    cache, rope = q.KVCache.empty(P, page, Hkv, D), q.qlora_build_rope(D, 10000.0)
    kv = q.KVBatch(B, width, T)
    free, count = torch.arange(P, dtype=torch.int32, device="cuda"), i32([P])
    ws = torch.empty(q.qlora_paged_attn_workspace_bytes(cache, kv, H), dtype=torch.uint8, device="cuda")
    ctx = [0] * B
    hist = [([], []) for _ in range(B)]
    steps = [[100, 37, 1, 0], [30, 1, 1, 50], [1, 1, 40, 1], [-1, 1, 1, 1], [90, 1, -1, 100], [1, 1, 33, 1], [1, 1, 1, 1]]
    for n, new in enumerate(steps):
        x = {m: torch.randn(T, h, D, generator=g, device="cuda").to(torch.bfloat16) for m, h in
             (("q", H), ("k", Hkv), ("v", Hkv))}
        out = torch.full_like(x["q"], 7.0)
        qr = torch.empty_like(x["q"])
        q.qlora_kv_plan(kv, page, P, i32(ctx), i32(new), free, count)
        q.qlora_kv_append(cache, kv, rope, x["q"], x["k"], x["v"], qr)
        q.qlora_paged_attn_fwd(cache, kv, qr, out, D ** -0.5, ws)
        q.qlora_check_device_error()
        got_len, at = kv.kv_len.tolist(), 0
        for b in range(B):
            if new[b] < 0:
                ctx[b], hist[b] = 0, ([], [])
                continue
            rows = slice(at, at + new[b])
            at += new[b]
            if new[b] and not got_len[b]:
                assert not out[rows].any()       # refused: tried again later
                continue
            pos = np.arange(ctx[b], ctx[b] + new[b])
            # the cache holds 16-bit keys: the oracle takes the library's rounded ones
            if new[b]:
                flat = cache.k.transpose(1, 2).reshape(P * page, Hkv, D)
                hist[b][0].append(np64(flat[kv.slots[rows].long()]))
                hist[b][1].append(np64(x["v"][rows]))
                k, v = np.concatenate(hist[b][0]), np.concatenate(hist[b][1])
                assert np.abs(hist[b][0][-1] - serve.rotate(np64(x["k"][rows]), pos, 10000.0)).max() < 2.0 ** -5
                want, _, mag = serve.attention(np64(qr[rows]), k, v, ctx[b], D ** -0.5)
                err = np.abs(np64(out[rows]) - want)
                assert np.all(err <= 2.0 ** -8 * np.abs(want) * 1.01 + (2.0 ** -8 + 2.0 ** -11) * mag), (n, b)
            ctx[b] += new[b]
        assert (out[at:] == 7.0).all()
    held = sum(-(-c // page) for c in ctx)
    assert int(count) == P - held
    ids = free[:P - held].tolist() + [kv.block_table[b, i].item() for b in range(B) for i in range(-(-ctx[b] // page))]
    assert sorted(ids) == list(range(P))         # no page lost, none given twice


def test_refusals(q):
    c = Case(q, [20], [1], 4, 2, 64, 16)
    n = q.qlora_paged_attn_workspace_bytes(c.cache, c.kv, 4)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.qt)
    f = lambda **k: q.qlora_paged_attn_fwd(**{**dict(cache=c.cache, kv=c.kv, q=c.qt, out=out, scale=0.1,   # noqa: E731
                                                     workspace=ws), **k})
    def status(**k):
        with pytest.raises(q.QLoraError) as e:
            f(**k)
        return e.value.status
    assert status(scale=0.0) == 1 and status(scale=-1.0) == 1 and status(scale=math.nan) == 1 and status(scale=math.inf) == 1
    assert status(window=-1) == 1 and status(sinks=-1) == 1
    assert status(workspace=ws[:-256]) == 4
    for bad in (dict(out=c.qt), dict(out=out.float()), dict(out=out[:, :2]), dict(q=c.qt.transpose(0, 1)),
                dict(lse=torch.empty(1, device="cuda")), dict(out=out.cpu()), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            f(**bad)
    three = torch.empty(c.T, 3, 64, dtype=torch.bfloat16, device="cuda")
    assert status(q=three, out=torch.empty_like(three)) == 2
    for shape in ((2, 2, 24, 64), (2, 2, 8, 64), (2, 2, 512, 64), (2, 2, 16, 8), (2, 2, 16, 144), (2, 2, 16, 72)):
        k = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(ValueError):
            q.qlora_paged_attn_workspace_bytes(q.KVCache(k, k.clone()), c.kv, 4)
    with pytest.raises(ValueError):
        q.KVCache(c.cache.k, c.cache.v.float())
    with pytest.raises(ValueError):
        q.KVBatch(1, 2, 3, cu_q=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(q.QLoraError):
        q.qlora_build_rope(24)
    with pytest.raises(q.QLoraError):
        q.qlora_build_rope(64, 1.0)
