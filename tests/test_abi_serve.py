"""The serving entry points check their arguments on the host before any CUDA
call, and the rotary frequencies are those of the definition."""

import ctypes
import math

import pytest

from tests.test_abi import _no_gpu, lib  # noqa: F401  (the built library)

FAKE = 0x10000     # aligned, never dereferenced: every call below fails first
P, I32, I64, F, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class Cache(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("num_pages", I32), ("page_size", I32), ("kv_heads", I32), ("head_dim", I32),
                ("stride_page", I64), ("stride_head", I64), ("stride_token", I64), ("dtype", ctypes.c_int)]


class Batch(ctypes.Structure):
    _fields_ = [("batch", I32), ("max_pages", I32), ("tokens", I32), ("max_q_len", I32), ("block_table", P),
                ("cu_q", P), ("kv_len", P), ("positions", P), ("slots", P)]


class Rope(ctypes.Structure):
    _fields_ = [("head_dim", I32), ("turns", ctypes.c_double * 64)]


def cache(**kw):
    c = Cache(FAKE, FAKE, 10, 16, 2, 64, 2048, 1024, 64, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def batch(**kw):
    b = Batch(3, 8, 40, 0, FAKE, FAKE, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def test_rope_frequencies(lib):  # noqa: F811
    f = lib.qlora_build_rope
    f.argtypes = [I32, ctypes.c_double, P]
    r = Rope()
    for D in (16, 48, 128):
        assert f(D, 10000.0, ctypes.byref(r)) == 0 and r.head_dim == D
        for i in range(64):
            want = 10000.0 ** (-2 * i / D) / (2 * math.pi) if i < D // 2 else 0.0
            assert abs(r.turns[i] - want) <= 4e-16 * want
    assert f(128, 10000.0, None) == 1
    assert f(8, 10000.0, ctypes.byref(r)) == 2 and f(24, 10000.0, ctypes.byref(r)) == 2 and f(144, 1e4, ctypes.byref(r)) == 2
    for base in (1.0, -3.0, math.nan, math.inf):
        assert f(64, base, ctypes.byref(r)) == 1


needs_no_gpu = pytest.mark.skipif(not _no_gpu(), reason="host-only validation test with placeholder pointers")


@needs_no_gpu
def test_plan_arguments(lib):  # noqa: F811
    f = lib.qlora_kv_plan
    f.argtypes = [P, I32, I32, P, P, P, P, P, P]

    def call(kv=None, page=16, pages=10, args=None):
        kv = batch() if kv is None else kv
        return f(ctypes.byref(kv), page, pages, *(args or [FAKE] * 5), None)

    assert f(None, 16, 10, *[FAKE] * 5, None) == 1
    for kw in (dict(batch=0), dict(batch=4097), dict(max_pages=0), dict(tokens=0), dict(tokens=-5), dict(max_q_len=-1),
               dict(max_pages=2 ** 27)):
        assert call(batch(**kw)) == 2, kw
    for page in (0, -16, 8, 24, 512):
        assert call(page=page) == 2
    assert call(pages=0) == 2 and call(pages=2 ** 30) == 2
    for i in range(5):
        a = [FAKE] * 5
        a[i] = None
        assert call(args=a) == 1
        a[i] = FAKE + 4
        assert call(args=a) == 3
    for name in ("block_table", "cu_q", "kv_len", "positions", "slots"):
        assert call(batch(**{name: None})) == 1
        assert call(batch(**{name: FAKE + 8})) == 3


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(dtype=1), 1), (dict(dtype=7), 1), (dict(page_size=24), 2),
              (dict(page_size=8), 2), (dict(num_pages=0), 2), (dict(num_pages=2 ** 28), 2), (dict(kv_heads=0), 2),
              (dict(head_dim=8), 2), (dict(head_dim=72), 2), (dict(head_dim=144), 2), (dict(stride_token=60), 2),
              (dict(stride_token=32), 2), (dict(stride_head=512), 2), (dict(stride_page=1024), 2),
              (dict(stride_page=-2048), 2), (dict(stride_page=2 ** 40), 2), (dict(k=FAKE + 2), 3), (dict(v=FAKE + 8), 3)]


@needs_no_gpu
def test_append_arguments(lib):  # noqa: F811
    f = lib.qlora_kv_append
    f.argtypes = [P, P, P, P, P, P, I32, P, P]
    rope = Rope()
    rope.head_dim = 64

    def call(c=None, kv=None, r=rope, heads=4, q=FAKE, k=FAKE, v=FAKE, out=FAKE):
        c, kv = cache() if c is None else c, batch() if kv is None else kv
        return f(ctypes.byref(c), ctypes.byref(kv), None if r is None else ctypes.byref(r), q, k, v, heads, out, None)

    for kw, want in BAD_CACHES:
        assert call(cache(**kw)) == want, kw
    assert call(heads=0) == 2 and call(heads=3) == 2 and call(heads=2048) == 2
    other = Rope()
    other.head_dim = 128
    assert call(r=other) == 2
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None)):
        assert call(**kw) == 1
    assert call(kv=batch(slots=None)) == 1 and call(kv=batch(positions=None)) == 1
    assert call(q=FAKE + 2) == 3 and call(kv=batch(slots=FAKE + 4)) == 3
    # both orders of heads and positions are strides of a valid cache: only the device is missing
    assert call(cache(stride_head=64, stride_token=128)) in (5, 6)
    assert call(r=None, kv=batch(positions=None)) in (5, 6)


@needs_no_gpu
def test_attention_arguments(lib):  # noqa: F811
    f = lib.qlora_paged_attn_fwd
    f.argtypes = [P, P, P, I32, F, I32, I32, P, P, P, S, P]

    def call(c=None, kv=None, q=FAKE, heads=4, scale=0.125, window=0, sinks=0, out=FAKE, lse=None, ws=FAKE):
        c, kv = cache() if c is None else c, batch() if kv is None else kv
        return f(ctypes.byref(c), ctypes.byref(kv), q, heads, scale, window, sinks, out, lse, ws, 1 << 40, None)

    for kw, want in BAD_CACHES:
        assert call(cache(**kw)) == want, kw
    assert call(heads=3) == 2 and call(heads=0) == 2
    assert call(kv=batch(tokens=2 ** 29), heads=4) == 2 and call(kv=batch(max_pages=2 ** 27)) == 2
    for kw in (dict(q=None), dict(out=None), dict(ws=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
               dict(scale=math.inf), dict(window=-1), dict(sinks=-1)):
        assert call(**kw) == 1, kw
    for name in ("block_table", "cu_q", "kv_len"):
        assert call(kv=batch(**{name: None})) == 1
        assert call(kv=batch(**{name: FAKE + 4})) == 3
    assert call(q=FAKE + 2) == 3 and call(out=FAKE + 8) == 3 and call(lse=FAKE + 4) == 3 and call(ws=FAKE + 8) == 3
    assert call(kv=batch(positions=None, slots=None)) in (5, 6)
    n = lib.qlora_paged_attn_workspace_bytes
    n.restype, n.argtypes = S, [P, P, I32]
    assert n(ctypes.byref(cache(page_size=8)), ctypes.byref(batch()), 4) == 0


@needs_no_gpu
def test_a_dimension_of_one_has_any_stride(lib):  # noqa: F811
    """The stride of one head or one page is never used, and tensors of one carry all kinds: only
    the device is missing."""
    f = lib.qlora_kv_append
    f.argtypes = [P, P, P, P, P, P, I32, P, P]
    for kw in (dict(kv_heads=1, stride_head=1), dict(kv_heads=1, stride_head=-4), dict(num_pages=1, stride_page=3),
               dict(num_pages=1, stride_page=2 ** 50), dict(kv_heads=1, stride_head=0, stride_page=1024)):
        assert f(ctypes.byref(cache(**kw)), ctypes.byref(batch()), None, FAKE, FAKE, FAKE, 4, FAKE, None) in (5, 6), kw
    # the others count as they did
    assert f(ctypes.byref(cache(kv_heads=1, stride_head=1, stride_page=1000)), ctypes.byref(batch()), None, FAKE, FAKE,
             FAKE, 4, FAKE, None) == 2
