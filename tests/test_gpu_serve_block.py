"""The serving form of the QLoRA block against the float64 oracle: prompts in
chunks and single tokens, over a paged cache, give the rows of the whole
sequence.

The bar is that of the block itself (tests/test_gpu_block.py): the same bf16
stores on the longest path, with the rotated q and k and the attention's
output rounded once each as there, and weights of the softmax that are
rounded no coarser; relative Frobenius error <= 3e-2 and every element within
3e-2 of the largest reference magnitude.
"""

import numpy as np
import pytest
import torch

import synthetic
from oracle import block as oblk
from tests.test_gpu_block import build, close, np64, oracle_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_16_b200 as q
    assert torch.cuda.is_available()
    return q


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def oracle_rows(case, x):
    cfg, W, A, B, g1, g2 = oracle_inputs(case)
    return oblk.forward(np64(x), dict(cfg, batch=1, seq=x.shape[0]), W, A, B, g1, g2)


def serve(q, case, xs, steps, T, page=16, width=16, pages=40, graph=False):
    """xs: the requests' sequences; steps: how many tokens of each per step.  Returns their rows."""
    blk = build(q, case)
    heads, D = case["heads"], case["hidden"] // case["heads"]
    cache, kv = q.KVCache.empty(pages, page, heads, D), q.KVBatch(len(xs), width, T)
    rope = q.qlora_build_rope(D, 10000.0)
    ws = torch.empty(q.qlora_block_cached_workspace_bytes(blk, cache, kv), dtype=torch.uint8, device="cuda")
    free, count = torch.arange(pages, dtype=torch.int32, device="cuda"), i32([pages])
    ctx_t, new_t = i32([0] * len(xs)), i32([0] * len(xs))
    x = torch.zeros(T, case["hidden"], dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)

    def step():
        q.qlora_kv_plan(kv, page, pages, ctx_t, new_t, free, count)
        q.qlora_block_fwd_cached(blk, cache, kv, rope, x, y, ws)

    g = None
    if graph:
        step()      # no request has tokens: the pool stays as it is
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    done, rows = [0] * len(xs), [[] for _ in xs]
    for new in steps:
        ctx_t.copy_(i32(done))
        new_t.copy_(i32(new))
        at = 0
        for b, n in enumerate(new):
            x[at:at + n] = xs[b][done[b]:done[b] + n].cuda()
            at += n
        if g is not None:
            g.replay()
        else:
            step()
        q.qlora_check_device_error()
        at = 0
        for b, n in enumerate(new):
            rows[b].append(y[at:at + n].clone())
            at += n
            done[b] += n
    return [torch.cat(r) for r in rows]


@pytest.mark.parametrize("graph", [False, True])
def test_chunks_and_single_tokens_give_the_whole_sequence(q, graph):
    """Two sequences of 40 and 29 tokens; hidden 256 in two heads of 128."""
    case = synthetic.block_case(1, 48, 256, 2, 512, 16, alpha=16.0, seed=2400)
    xs = [case["x"][:40], case["dy"][:29]]
    steps = [[24, 8], [14, 1], [1, 0], [1, 20]]
    for got, x in zip(serve(q, case, xs, steps, 33, graph=graph), xs):
        close(got, oracle_rows(case, x), "y")


def test_decode_of_many_requests(q):
    """Nine requests, their prompts in one step, then one token each (the decode form of the linears)."""
    case = synthetic.block_case(2, 80, 512, 8, 1024, 32, alpha=16.0, seed=2500)
    xs = [case["x"][17 * b:17 * b + 5 + b] for b in range(9)]
    steps = [[x.shape[0] - 2 for x in xs], [1] * 9, [1] * 9]
    for got, x in zip(serve(q, case, xs, steps, 64), xs):
        close(got, oracle_rows(case, x), "y")


def test_agrees_with_the_training_form(q):
    """One sequence of 128 tokens: both forms stay within the bar of the oracle, so within twice it of each other."""
    case = synthetic.block_case(1, 128, 256, 2, 512, 16, alpha=16.0, seed=2600)
    blk = build(q, case)
    ws = torch.empty(q.qlora_block_workspace_bytes(blk), dtype=torch.uint8, device="cuda")
    x = case["x"].cuda()
    y = torch.empty_like(x)
    q.qlora_block_fwd(blk, x, y, ws)
    got = serve(q, case, [case["x"]], [[128]], 128)[0]
    ref = np64(y)
    assert np.linalg.norm(np64(got) - ref) <= 6e-2 * np.linalg.norm(ref)


def test_refusals(q):
    case = synthetic.block_case(1, 16, 256, 2, 512, 16, alpha=16.0, seed=2700)
    blk = build(q, case)
    cache, kv, rope = q.KVCache.empty(4, 16, 2, 128), q.KVBatch(1, 4, 16), q.qlora_build_rope(128)
    n = q.qlora_block_cached_workspace_bytes(blk, cache, kv)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    x = case["x"].cuda()
    y = torch.empty_like(x)
    def status(*a, **k):
        with pytest.raises(q.QLoraError) as e:
            q.qlora_block_fwd_cached(*a, **k)
        return e.value.status
    assert status(blk, cache, kv, rope, x, y, ws[:-256]) == 4
    assert status(blk, cache, kv, q.qlora_build_rope(64), x, y, ws) == 2
    assert status(blk, cache, kv, rope, x, y, ws, window=-1) == 1
    assert status(blk, q.KVCache.empty(4, 16, 1, 128), kv, rope, x, y, ws) == 2
    assert status(blk, q.KVCache.empty(4, 16, 2, 128, torch.float16), kv, rope, x, y, ws) == 1
    assert status(blk, q.KVCache.empty(4, 24, 2, 128), kv, rope, x, y, ws) == 2
    for bad in (dict(x=x[:8]), dict(y=x), dict(y=y.float())):
        with pytest.raises(ValueError):
            q.qlora_block_fwd_cached(blk, cache, kv, rope, bad.get("x", x), bad.get("y", y), ws)


def test_a_missing_adapter_is_refused_before_anything_is_written(q):
    case = synthetic.block_case(1, 16, 256, 2, 512, 16, alpha=16.0, seed=2800)
    blk = build(q, case)
    cache, kv, rope = q.KVCache.empty(4, 16, 2, 128), q.KVBatch(1, 4, 16), q.qlora_build_rope(128)
    ws = torch.empty(q.qlora_block_cached_workspace_bytes(blk, cache, kv), dtype=torch.uint8, device="cuda")
    for t in (cache.k, cache.v):
        t.zero_()
    kv.slots.copy_(torch.arange(16, dtype=torch.int32))
    kv.positions.copy_(torch.arange(16, dtype=torch.int32))
    x = case["x"].cuda()
    y = torch.full_like(x, 7.0)
    blk.desc.B[6] = None      # the last linear's
    with pytest.raises(q.QLoraError) as e:
        q.qlora_block_fwd_cached(blk, cache, kv, rope, x, y, ws)
    assert e.value.status == 1
    torch.cuda.synchronize()
    assert not cache.k.any() and not cache.v.any() and (y == 7.0).all()


def test_no_rope_is_refused(q):
    case = synthetic.block_case(1, 16, 256, 2, 512, 16, alpha=16.0, seed=2900)
    blk = build(q, case)
    cache, kv = q.KVCache.empty(4, 16, 2, 128), q.KVBatch(1, 4, 16)
    ws = torch.empty(q.qlora_block_cached_workspace_bytes(blk, cache, kv), dtype=torch.uint8, device="cuda")
    x = case["x"].cuda()
    with pytest.raises(q.QLoraError) as e:
        q.qlora_block_fwd_cached(blk, cache, kv, None, x, torch.empty_like(x), ws)
    assert e.value.status == 1


@pytest.mark.parametrize("which", ["A", "B"])
def test_a_misaligned_adapter_is_refused_before_anything_is_written(q, which):
    """The last linear's: the first six would have run, and the cache been written."""
    case = synthetic.block_case(1, 16, 256, 2, 512, 16, alpha=16.0, seed=3000)
    blk = build(q, case)
    cache, kv, rope = q.KVCache.empty(4, 16, 2, 128), q.KVBatch(1, 4, 16), q.qlora_build_rope(128)
    ws = torch.empty(q.qlora_block_cached_workspace_bytes(blk, cache, kv), dtype=torch.uint8, device="cuda")
    for t in (cache.k, cache.v):
        t.zero_()
    kv.slots.copy_(torch.arange(16, dtype=torch.int32))
    kv.positions.copy_(torch.arange(16, dtype=torch.int32))
    x = case["x"].cuda()
    y = torch.full_like(x, 7.0)
    getattr(blk.desc, which)[6] += 8
    with pytest.raises(q.QLoraError) as e:
        q.qlora_block_fwd_cached(blk, cache, kv, rope, x, y, ws)
    assert e.value.status == 3
    torch.cuda.synchronize()
    assert not cache.k.any() and not cache.v.any() and (y == 7.0).all()
