// Paged attention for many query rows (chunks and whole prompts): bound by the
// tensor cores, and at head_dim 64 by the exponentials.
//
// One CTA per SM, persistent over its items of 256 rows x tiles of 128
// positions.  The rows form two halves of 128, A and B, whose softmax alternates
// with the other half's products:
//   warps 0-3, 4-7  softmax of half A, B: one thread per row
//   warp 8          the schedule (it hands the items to the other warps through
//                   a ring in shared memory), and keys and values: a ring of
//                   tiles filled by TMA page by page
//   warp 9          issues the products
//   warps 10, 11    query rows of half A, B
// Scores S = Q K^T (tcgen05, both operands in shared memory) land in tensor
// memory; a softmax thread reads its row, and writes the weights as 16-bit
// values over the scores, where the second product O += P V takes them as its
// left operand: they never pass through shared memory.  The 512 columns of
// tensor memory hold S/P and O of both halves.  The order of issue is
//   S_A(0) S_B(0) | PV_A(0) S_A(1) PV_B(0) S_B(1) | PV_A(1) ...
// and runs on across items, so that one half's epilogue overlaps the other's
// products.  Products of one CTA complete in order: the completion of S(j + 1)
// tells the softmax that PV(j) is done too.
//
// Softmax: one pass, with weights against a reference m that is the row's maximum
// over its first tile and moves only when it has to.  Any reference gives the same
// quotient as long as no weight leaves the 16-bit type's range, and the sum
// of a tile's weights, which is needed anyway, tells: up to kMost none has at the upper end (for
// the lower one see kRaiseMany).  So the
// maximum of a tile is not looked for at all, unless that sum is larger or the row
// has had no reference yet; then the weights are formed again against the new
// maximum, and the output is rescaled by the softmax threads before they are
// handed over.  The weights are rounded to the operands' 16-bit type (half a step
// each, averaged over the keys: the output's own rounding is as large; fp16 weights below 2^-22 of the
// row's largest, 2^-33 of that); sums are
// taken of the unrounded fp32 weights.
//
// Measured (B200, by box: clocks under this kernel were 1.66 to 1.97 GHz).  2048 tokens over 16000 positions,
// 32 heads of 128, at the highest clock: 530 to 550 us, 1030 to 1090 TFLOP/s (0.61 to 0.65 of the measured
// GEMM rate).  A whole prompt of 4096 tokens, 32 heads of 128: 152 to 176 us, 780 TFLOP/s at the last (0.46).
// Four chunks of 1500 to 2048 tokens, window 1024: 219 to 254 us (0.28 to 0.32 of that rate: whole tiles are
// computed at the window's ends).  Seven ragged chunks, heads of 64: 61 us (0.21; 9 tiles an item).
// The prompt's 57 tiles an SM take 258,000 cycles, 4500 each.  By the counters the tensor pipe is
// busy for 2050 of them (64 for each of the 32 products) and the exponentials' for 2050 (16 a
// cycle and SM).  A half needs 1020 cycles of products and 1500 of softmax (measured alone), in turn;
// the other 1900 are hand-overs and waiting between the warps, not told apart further.
// The references and the raised fp16 weights (see attn_common.cuh) cost, on one box: prompt 166 to 168 us
// (fp16 168 to 172), windowed chunks 227 to 231 (fp16 229 to 254: the few sinks that a first tile holds
// make a low reference, and the second tile is mostly formed twice).
// Tried, and no faster: two threads per row (194 us for a prompt that took 159
// at that time, and 169 for 157 later); S in steps of 64 columns with two buffers (184 for
// 182, 221 with a group of warps for each buffer); a quarter of the exponentials by a
// polynomial (215 for 182); signalling the first 64 weights early (174 for 170);
// a transposing epilogue (163 for 157).  At heads of 64, which leave room: the weights in
// columns of their own, so that the next S is formed during the softmax (ragged chunks
// 62 to 69, by where the softmax waits, for 61); two buffers of query rows (60.5 for 61.1).
#pragma once
#include "attn_common.cuh"

namespace qlora {
namespace attn {

template <int DP>
struct ChunkCfg {
    // kOv: what an item costs beside its tiles.  1 to 4 measured on prompts, ragged and windowed chunks: 2 is
    // best or within noise (ragged chunks 61.6 us, 63.2 with 1, 67.8 with 4).
    static constexpr int kThreads = 384, kRows = 256, kTile = 128, kOv = 2;
    static constexpr uint32_t kQBytes = 128 * DP * 2;      // one half
    static constexpr uint32_t kTileBytes = 128 * DP * 2;   // keys or values of one tile
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr uint32_t kRingOff = 2 * kQBytes;
    static constexpr uint32_t kBarOff = kRingOff + kStages * kTileBytes;
    static constexpr uint32_t kBytes = kBarOff + 1024 + 1024;   // + alignment slack
    static constexpr int kSlotFloats = kRows * DP + 2 * kRows;
    static constexpr uint32_t kOCol = 256;                 // O_A, O_B at 256 + DP * half; S at 128 * half
    // From this size of a reference (in powers of two) on, scores lose their reference before they are scaled; below it
    // the rounding of reference * scale, which is the same for all of a row's weights, moves them by 2^-9 at most.
    static constexpr float kFar = 65536.0f;
    static constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;   // 2 * 200 + 104 = 3 * 168, the launch's share
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats in one 64-bit register, for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t r)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The products of this kernel.  Descriptors of one operand differ in the low
// word only (the start address), so a step costs one addition: the issuing
// thread has no time for more (64 cycles per product).
template <bool kAccumulate>
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "n"(kAccumulate ? 1 : 0)
        : "memory");
}

// D[tmem] (+)= A[tmem, K-major 16-bit] * B[smem desc]
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The CTA's tiles that a half of an item takes: from the first to the last that
// any of its rows sees, without those between its sinks and its window.
struct Range {
    int first, last;   // last < first: none
    int gap, gap_end;  // [gap, gap_end) is left out

    __device__ __forceinline__ bool has() const { return last >= first; }
    __device__ __forceinline__ bool takes(int t) const { return t >= first && t <= last && (t < gap || t >= gap_end); }
};

// One half of an item: its rows' positions, and its tiles.
struct Half {
    int rows, first, last;   // valid rows (0: none), position of the first and the last
    Range t;
};

__device__ __forceinline__ Half half_of(const BatchView &v, const Item &it, int half)
{
    Half f;
    f.rows = min(max(it.r.qn * v.group - it.rt * 256 - half * 128, 0), 128);
    f.first = f.last = -1;
    f.t = Range{it.t0, it.t0 - 1, 0, 0};
    if (f.rows == 0) return f;
    item_positions<128>(v, it.r, it.rt * 2 + half, f.first, f.last);
    auto sees = [&](int t) {
        const int a = it.tiles.at(t) * 128;
        return a <= f.last && (v.window <= 0 || a + 127 > f.first - v.window || a < v.sinks);
    };
    f.t.last = it.t1 - 1;
    while (f.t.has() && !sees(f.t.last)) f.t.last--;
    while (f.t.has() && !sees(f.t.first)) f.t.first++;
    f.t.gap = f.t.gap_end = max(f.t.first, it.tiles.sink_tiles);
    while (f.t.gap_end <= f.t.last && !sees(f.t.gap_end)) f.t.gap_end++;
    return f;
}

// What the schedule hands to the other warps.
struct ChunkItem {
    Tiles tiles;
    int t0, t1;
    int h;            // key/value head; -1: no more items
    int q0;           // first row of the request
    int row0;         // first row of the item: r / group is a token of the request
    int pos0;         // position of the request's first row
    int whole, begins;
    Half half[2];
    int parts;
};

struct ChunkBars {
    uint64_t kv_full[8], kv_empty[8];
    uint64_t s_full[2], p_ready[2], o_full[2], q_full[2], q_free[2];
    uint64_t item_full[4], item_empty[4];
    uint64_t tail, drain;
    uint32_t tmem;
    int abort;
    uint32_t bad[8];   // per tile (mod 8): bit i, positions 16 i ... + 15 are on no page of the cache
    ChunkItem item[4];
};

// True in one thread of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Bits 0 ... n - 1 of a word (n of any size).
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Bounded wait; false after the limit or when another role gave up.
__device__ __forceinline__ bool chunk_wait(uint64_t *bar, uint32_t parity, ChunkBars *b, const AttnParams &p)
{
    if (sm100::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = sm100::globaltimer_ns();
    for (uint32_t spin = 0;; spin++) {
        if (sm100::mbar_try_wait(bar, parity)) return true;
        if ((spin & 63u) == 63u) {
            if (*reinterpret_cast<volatile int *>(&b->abort)) return false;
            if (sm100::globaltimer_ns() - t0 > p.timeout_ns) {
                atomicExch(p.err, 1);
                *reinterpret_cast<volatile int *>(&b->abort) = 1;
                return false;
            }
        }
    }
}

template <int DP, bool F16>
__global__ void __launch_bounds__(384, 1) chunk_kernel(const __grid_constant__ AttnParams p)
{
    using C = ChunkCfg<DP>;
    using W = Walker<C::kThreads, C::kRows, C::kTile, C::kOv>;
    using namespace sm100;
    constexpr int ST = C::kStages;
    constexpr float kRaise = kRaiseMany<F16>;
    constexpr float kMost = F16 ? 65504.0f : 32768.0f;   // of a tile's sum: fp16's largest value, 2^15
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    ChunkBars *bars = reinterpret_cast<ChunkBars *>(smem + C::kBarOff);
    static_assert(sizeof(ChunkBars) <= 1024, "barriers and items fit their place");
    int64_t *pre = reinterpret_cast<int64_t *>(smem + C::kRingOff);   // before the ring is used
    const BatchView &v = p.v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; s++) {
            mbar_init(&bars->kv_full[s], 1);
            mbar_init(&bars->kv_empty[s], 1);
        }
        for (int h = 0; h < 2; h++) {
            mbar_init(&bars->s_full[h], 1);
            mbar_init(&bars->p_ready[h], 4);
            mbar_init(&bars->o_full[h], 1);
            mbar_init(&bars->q_full[h], 1);
            mbar_init(&bars->q_free[h], 1);
        }
        for (int i = 0; i < 4; i++) {
            mbar_init(&bars->item_full[i], 1);
            mbar_init(&bars->item_empty[i], 11);   // 8 softmax warps, the products, 2 warps of query rows
        }
        mbar_init(&bars->tail, 1);
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&p.tk);
        tma_prefetch_desc(&p.tv);
    }
    if (warp == 9) {
        tmem_alloc(&bars->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    pdl_wait();
    pdl_trigger();
    schedule_scan<C::kThreads, C::kRows, C::kTile, C::kOv>(v, pre);   // its barriers publish the above
    tc_fence_after();
    const int64_t total = pre[C::kThreads];
    const int64_t G = min((int64_t)gridDim.x, total), cta = blockIdx.x;
    if (threadIdx.x == 0) p.desc[cta].parts = 0;
    const uint32_t tmem = bars->tmem;
    W walk;
    if (warp == 8) {
        walk.init(v, pre, cta < G ? first_unit(cta, G, total) : 0, cta < G ? first_unit(cta + 1, G, total) : 0);
        fence_proxy_async_smem();
    }
    __syncthreads();   // the prefix sums have been read: the ring is free

    // The n-th item of this CTA, or null at the end or after a failure.
    auto item_at = [&](uint32_t n) -> const ChunkItem * {
        bool ok = chunk_wait(&bars->item_full[n & 3], (n >> 2) & 1, bars, p);
        if (warp != 9) ok = __all_sync(0xffffffffu, ok);   // the products' warp runs one thread
        if (!ok) return nullptr;
        const ChunkItem *it = &bars->item[n & 3];
        return it->h < 0 ? nullptr : it;
    };
    // The row of q, out and lse (times heads, plus the head) of an item's row.
    auto tensor_row = [&](const ChunkItem *it, int r) {
        const int g = it->row0 + r, t = v.token_of(g);
        return (int64_t)(it->q0 + t) * v.heads + it->h * v.group + g - t * v.group;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        if (warp == 8) {
            // ---- schedule; keys and values, in the order K(0) V(0) K(1) V(1) ... ----
            const int box = min(1 << v.page_shift, 128), pieces = 128 / box;
            uint32_t n = 0, tiles = 0, tails = 0, items = 0;   // ring entries, tiles, tail waits, items so far
            bool ok = true, more = true;
            while (more) {
                Item it;
                more = walk.next(v, it);
                ok = chunk_wait(&bars->item_empty[items & 3], ((items >> 2) & 1) ^ 1, bars, p);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    ChunkItem &o = bars->item[items & 3];
                    o.h = -1;
                    if (more) {
                        o.tiles = it.tiles;
                        o.t0 = it.t0;
                        o.t1 = it.t1;
                        o.h = it.h;
                        o.q0 = it.r.q0;
                        o.row0 = it.rt * 256;
                        o.pos0 = it.r.kv - it.r.qn;
                        o.whole = it.whole;
                        o.begins = it.begins;
                        o.half[0] = half_of(v, it, 0);
                        o.half[1] = half_of(v, it, 1);
                        o.parts = it.begins ? cta_of_last(it.end, G, total) - (int)cta + 1 : 0;
                    }
                    mbar_arrive(&bars->item_full[items & 3]);
                }
                items++;
                if (!more) break;
                // positions from the sinks to here: no row sees them
                const int before = v.window > 0 ? it.r.kv - it.r.qn + v.token_of(it.rt * C::kRows) - v.window : -1;
                for (int t = it.t0; ok && t < it.t1; t++, tiles++) {
                    const int tok0 = it.tiles.at(t) * 128, mine = tok0 + lane * box;
                    int page = v.num_pages;   // a page outside the cache: the copy fills zeros
                    bool bad = false;
                    // (a page that no row sees may be another request's by now, or hold anything)
                    if (lane < pieces && mine < it.r.kv && (mine < v.sinks || mine + box - 1 > before)) {
                        const int id = page_of(v, it.b, mine);
                        bad = id < 0;
                        if (id >= 0) page = id;
                    }
                    const uint32_t bad_mask = __ballot_sync(0xffffffffu, __shfl_sync(0xffffffffu, bad, (lane & 7) * 16 / box)) & 0xffu;
                    const int row = mine & ((1 << v.page_shift) - 1);
                    for (int kv = 0; kv < 2; kv++, n++) {
                        const int s = n % ST;
                        ok = chunk_wait(&bars->kv_empty[s], ((n / ST) & 1) ^ 1, bars, p);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        uint8_t *dst = smem + C::kRingOff + s * C::kTileBytes;
                        const bool tail = kv == 1 && tok0 + 128 > it.r.kv;
                        uint64_t *bar = tail ? &bars->tail : &bars->kv_full[s];
                        if (lane == 0) {
                            if (kv == 0) bars->bad[tiles & 7] = bad_mask;
                            mbar_arrive_expect_tx(bar, C::kTileBytes);
                        }
                        __syncwarp();
                        if (lane < pieces) {
#pragma unroll
                            for (int c = 0; c < DP / 64; c++)
                                tma_load_4d(dst + c * 16384 + lane * box * 128, kv ? &p.tv : &p.tk, bar, 64 * c, row, it.h,
                                            page);
                        }
                        if (tail) {
                            // positions at or beyond the length were never written and may hold
                            // anything; their weight is 0, but 0 times a NaN is not
                            ok = chunk_wait(&bars->tail, tails & 1, bars, p);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            tails++;
                            const int r0 = max(it.r.kv - tok0, 0), r1 = min((r0 + box - 1) / box * box, 128);
                            for (int i = lane; i < (r1 - r0) * (DP / 8); i += 32) {
                                const int r = r0 + i / (DP / 8), ch = i % (DP / 8);
                                *reinterpret_cast<uint4 *>(dst + (ch >> 3) * 16384 + r * 128 + (ch & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars->kv_full[s]);
                        }
                    }
                }
                if (!ok) break;
            }
            if (!ok) {
                // wait (bounded) for the copies in flight
                for (uint32_t j = n > (uint32_t)ST ? n - ST : 0; j < n; j++)
                    mbar_wait_bounded(&bars->kv_full[j % ST], (j / ST) & 1, p.timeout_ns / 8);
                mbar_wait_bounded(&bars->tail, tails & 1, p.timeout_ns / 8);
            }
        } else if (warp == 9) {
            // ---- products ----
            // (elect.sync, not lane == 0: the compiler then keeps the products' operands in uniform
            // registers; with a lane's branch each product took 130 cycles to issue)
            if (elect_one()) {
                const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0, F16), idesc_o = idesc_bf16_f32(128, DP, 0, 1, F16);
                const uint64_t qd = smem_desc_sw128(smem_u32(smem), 16, 1024),
                               kd = smem_desc_sw128(smem_u32(smem + C::kRingOff), 16, 1024),
                               vd = smem_desc_sw128(smem_u32(smem + C::kRingOff), 16384, 1024);
                const uint32_t q_desc = (uint32_t)qd, k_desc = (uint32_t)kd, v_desc = (uint32_t)vd, hi = (uint32_t)(qd >> 32);
                uint32_t n_p = 0, n_q = 0;   // bit h: parity of the next weights, query rows of half h
                bool ok = true;
                auto wait = [&](uint64_t *bar, uint32_t parity) {
                    if (ok) ok = chunk_wait(bar, parity, bars, p);
                    if (ok) tc_fence_after();
                };
                // S runs one tile ahead of PV, across items.  The thread keeps what it needs of
                // both tiles' items in registers: what it does between two products is
                // latency that nothing hides.
                Range sr[2] = {};
                // for each half (4 h + ...): 1 it takes the tile, 2 as its first of the item, 4 as its last
                uint32_t s_how = 0;
                bool more = true, crossed = false;   // is there a tile for S; is it of another item than PV's
                uint32_t items = 0;                  // items begun
                int st = -1, s_end = 0;
                auto next_item = [&]() {
                    if (items) mbar_arrive(&bars->item_empty[(items - 1) & 3]);
                    const ChunkItem *it = item_at(items++);
                    more = it != nullptr;
                    if (!more) return;
                    st = it->t0;
                    s_end = it->t1;
#pragma unroll
                    for (int h = 0; h < 2; h++) sr[h] = it->half[h].t;
                };
                auto next_tile = [&]() {   // one item ahead at most: it may have none
                    st++;
                    crossed = st >= s_end;
                    if (crossed) next_item();
                };
                // Past the items without a tile.  Not with a second product to issue: the schedule cannot
                // publish the fourth item from here before this item's place is free, which is
                // when its rows are written, behind that product.
                auto skip_empty = [&]() {
                    while (more && st >= s_end) next_item();
                };
                auto look = [&]() {
                    s_how = 0;
#pragma unroll
                    for (int h = 0; h < 2; h++)
                        if (sr[h].takes(st)) s_how |= (1u | (st == sr[h].first ? 2u : 0u) | (st == sr[h].last ? 4u : 0u)) << (4 * h);
                };
                auto scores = [&](int h, uint32_t slot) {
                    const uint32_t how = s_how >> (4 * h);
                    if (!(how & 1u)) return;
                    if (how & 2u) {
                        wait(&bars->q_full[h], (n_q >> h) & 1);
                        n_q ^= 1u << h;
                    }
                    if (!ok) return;
                    const uint32_t d = tmem + 128 * h, q_lo = q_desc + h * (C::kQBytes >> 4),
                                   k_lo = k_desc + slot * (C::kTileBytes >> 4);
                    tc_mma_ss<false>(d, q_lo, k_lo, hi, idesc_s);
#pragma unroll
                    for (int kk = 1; kk < DP / 16; kk++) {
                        const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                        tc_mma_ss<true>(d, q_lo + o, k_lo + o, hi, idesc_s);
                    }
                    tc_commit(&bars->s_full[h]);
                    if (how & 4u) tc_commit(&bars->q_free[h]);
                };
                auto values = [&](int h, uint32_t hows, uint32_t slot) {
                    const uint32_t how = hows >> (4 * h);
                    if (!(how & 1u)) return;
                    const uint32_t d = tmem + C::kOCol + DP * h, a = tmem + 128 * h,
                                   v_lo = v_desc + slot * (C::kTileBytes >> 4);
                    wait(&bars->p_ready[h], (n_p >> h) & 1);
                    if (!ok) return;
#pragma unroll
                    for (int kk = 0; kk < 8; kk++)
                        tc_mma_ts(d, a + 8 * kk, v_lo + (2048 >> 4) * kk, hi, idesc_o, kk > 0 || !(how & 2u));
                    n_p ^= 1u << h;
                    if (how & 4u) tc_commit(&bars->o_full[h]);
                };
                uint32_t slot = 0, phase = 0;   // of the next ring entry
                auto advance = [&]() {
                    const uint32_t s = slot;
                    wait(&bars->kv_full[s], phase);
                    if (++slot == ST) {
                        slot = 0;
                        phase ^= 1;
                    }
                    return s;
                };
                next_tile();
                skip_empty();
                if (more) {
                    look();
                    const uint32_t ks = advance();
                    scores(0, ks);
                    scores(1, ks);
                    if (ok) tc_commit(&bars->kv_empty[ks]);
                }
                while (more && ok) {
                    // PV of this tile, S of the next
                    const uint32_t p_how = s_how;
                    next_tile();
                    const uint32_t vs = advance();
                    if (!crossed) {
                        look();
                        const uint32_t ks = advance();
                        values(0, p_how, vs);
                        if (ok) scores(0, ks);
                        if (ok) values(1, p_how, vs);
                        if (!ok) break;
                        tc_commit(&bars->kv_empty[vs]);
                        scores(1, ks);
                        if (ok) tc_commit(&bars->kv_empty[ks]);
                    } else {   // the next item's query rows may still be on their way
                        if (ok) values(0, p_how, vs);
                        if (ok) values(1, p_how, vs);
                        if (!ok) break;
                        tc_commit(&bars->kv_empty[vs]);
                        skip_empty();
                        if (!more) break;
                        look();
                        const uint32_t ks = advance();
                        if (ok) scores(0, ks);
                        if (ok) scores(1, ks);
                        if (ok) tc_commit(&bars->kv_empty[ks]);
                    }
                }
                if (!ok) {
                    // wait (bounded) until the products already issued finish
                    tc_commit(&bars->drain);
                    mbar_wait_bounded(&bars->drain, 0, p.timeout_ns);
                }
            }
        } else {
            // ---- query rows of one half ----
            const int h = warp - 10;
            uint8_t *dst = smem + h * C::kQBytes;
            uint32_t n = 0, items = 0;
            bool ok = true;
            for (const ChunkItem *it; ok && (it = item_at(items)); items++) {
                const Half f = it->half[h];
                if (f.t.has()) {
                    if (n > 0) ok = chunk_wait(&bars->q_free[h], (n - 1) & 1, bars, p);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    // this lane's part of the rows 32 i + lane: where they begin, or -1
                    int64_t begin[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int r = 32 * i + lane;
                        begin[i] = r < f.rows ? tensor_row(it, h * 128 + r) * v.head_dim : -1;
                    }
                    constexpr int kPerRow = DP / 8, kRowsAtOnce = 32 / kPerRow;   // 16-byte pieces
                    const int ch = lane % kPerRow;
                    const bool in = ch * 8 < v.head_dim;
#pragma unroll
                    for (int i = 0; i < 4; i++)
#pragma unroll 8
                        for (int j = 0; j < 32; j += kRowsAtOnce) {
                            const int rr = j + lane / kPerRow, r = 32 * i + rr;
                            const int64_t o = __shfl_sync(0xffffffffu, begin[i], rr) + ch * 8;
                            const bool there = in && o >= ch * 8 && QLORA_IN(o + 7, (int64_t)v.tokens * v.heads * v.head_dim);
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                             smem_u32(dst + (ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4))),
                                         "l"(static_cast<const uint16_t *>(p.q) + (there ? o : 0)), "r"(there ? 16 : 0)
                                         : "memory");
                        }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_proxy_async_smem();
                    n++;
                }
                __syncwarp();
                if (lane == 0) {
                    if (f.t.has()) mbar_arrive(&bars->q_full[h]);
                    mbar_arrive(&bars->item_empty[items & 3]);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        // ---- softmax and epilogue of one half ----
        const int h = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t s_addr = tmem + lanes + 128 * h, o_addr = tmem + lanes + C::kOCol + DP * h;
        uint32_t n_s = 0, n_o = 0, tiles = 0;
        bool ok = true;
        const ChunkItem *it;
        for (uint32_t items = 0; ok && (it = item_at(items)); items++) {
            const Half &f = it->half[h];
            const int t_first = f.t.first, t_last = f.t.last;
            const bool valid = row < f.rows, has = f.t.has();
            const int pos = valid ? it->pos0 + v.token_of(it->row0 + h * 128 + row) : -1;
            float m = valid ? -INFINITY : 0.0f, l = 0.0f;   // m: the reference of the weights, a score; -inf: none yet
            bool far = false;                               // a row of this warp has one of kFar or more
            for (int t = t_first; t <= t_last; t++) {
                if (!f.t.takes(t)) continue;
                const int tok0 = it->tiles.at(t) * 128;
                const bool inside = tok0 + 127 <= f.first && (v.window <= 0 || tok0 > f.last - v.window || tok0 + 127 < v.sinks);
                ok = chunk_wait(&bars->s_full[h], n_s, bars, p);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                n_s ^= 1;
                tc_fence_after();
                const uint32_t bad = bars->bad[(tiles + t - it->t0) & 7];
                if (!inside || bad) {
                    // columns [0, up) are not after the row; of them [0, front) are sinks and [low, up) in
                    // the window.  Masked in tensor memory, 32 columns at a time: done on the registers
                    // below, the code (6 KB, run by one tile in three under a window) came
                    // from far caches each time and cost as much as the tile's exponentials.
                    const int up = pos - tok0 + 1, low = v.window > 0 ? pos - v.window + 1 - tok0 : 0, front = v.sinks - tok0;
#pragma unroll 1
                    for (int g = 0; g < 4; g++) {
                        uint32_t seen = bits_below(up - 32 * g) & (~bits_below(low - 32 * g) | bits_below(front - 32 * g));
                        if ((bad >> (2 * g)) & 1u) seen &= 0xffff0000u;
                        if ((bad >> (2 * g + 1)) & 1u) seen &= 0x0000ffffu;
                        if (!__any_sync(0xffffffffu, seen != ~0u)) continue;
                        uint32_t x[2][16];
                        tmem_ld_x16(s_addr + 32 * g, x[0]);
                        tmem_ld_x16(s_addr + 32 * g + 16, x[1]);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 32; c++) x[c >> 4][c & 15] = seen & (1u << c) ? x[c >> 4][c & 15] : 0xff800000u;
                        tmem_st_x16(s_addr + 32 * g, x[0]);
                        tmem_st_x16(s_addr + 32 * g + 16, x[1]);
                    }
                    tmem_st_wait();
                }
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; c++) tmem_ld_32x32b_x32(s_addr + 32 * c, s[c]);
                tmem_ld_wait();
                float sum;
                bool again = t == t_first || far;   // find a reference first
#pragma unroll 1
                for (;;) {
                    if (again) {
                        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < 128; c++) x[c & 3] = fmaxf(x[c & 3], __uint_as_float(s[c >> 5][c & 31]));
                        const float nm = fmaxf(m, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
                        if (t > t_first) {
                            // the product of the tile before is complete (this S came after it)
                            const float fac = nm == -INFINITY ? 1.0f : ex2((m - nm) * p.scale_log2);
                            l *= fac;
#pragma unroll 1
                            for (int c = 0; c < DP / 16; c++) {
                                uint32_t o[16];
                                tmem_ld_x16(o_addr + 16 * c, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * fac);
                                tmem_st_x16(o_addr + 16 * c, o);
                            }
                        }
                        m = nm;
                        far = __any_sync(0xffffffffu, m != -INFINITY && fabsf(m * p.scale_log2) >= C::kFar);
                    }
                    const float ref = m == -INFINITY ? 0.0f : m;   // against 0, all weights of a row without a key are 0
                    float shift = __fmaf_rn(-ref, p.scale_log2, kRaise);
                    if (far) {   // (only in a pass that has looked for the reference, so it is the last)
                        shift = kRaise;
#pragma unroll
                        for (int c = 0; c < 128; c++) s[c >> 5][c & 31] = __float_as_uint(__uint_as_float(s[c >> 5][c & 31]) - ref);
                    }
                    const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), shift2 = pair(shift, shift);
                    uint64_t sums[2] = {0, 0};
#pragma unroll
                    for (int g = 0; g < 4; g++) {
                        uint32_t w[16];
#pragma unroll
                        for (int c = 0; c < 16; c++) {
                            const float2 e = unpair(fma2(pair(__uint_as_float(s[g][2 * c]), __uint_as_float(s[g][2 * c + 1])), scale2, shift2));
                            const float a = ex2(e.x), b = ex2(e.y);
                            sums[c & 1] = add2(sums[c & 1], pair(a, b));
                            w[c] = pack2<F16>(a, b);
                        }
                        tmem_st_x16(s_addr + 16 * g, w);
                    }
                    const float2 total = unpair(add2(sums[0], sums[1]));
                    sum = total.x + total.y;
                    if (again) break;
                    again = __any_sync(0xffffffffu, !(sum <= kMost) || m == -INFINITY);
                    if (!again) break;
                }
                l += sum;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->p_ready[h]);
            }
            if (!ok) break;
            // ---- epilogue ----
            const bool whole = it->whole;
            const int slot = 2 * (int)cta + (items == 0 ? 0 : 1), pr = h * 128 + row;
            float *part = p.part + (int64_t)slot * C::kSlotFloats;
            const int64_t orow = valid ? tensor_row(it, pr) : 0;
            const float inv = whole ? inverse_sum(l) : 1.0f;
            if (has) {
                ok = chunk_wait(&bars->o_full[h], n_o, bars, p);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                n_o ^= 1;
                tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < DP / 32; c++) {
                uint32_t o[32];
                if (has) {
                    tmem_ld_32x32b_x32(o_addr + 32 * c, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] = 0u;
                }
                if (!valid) continue;
                if (whole) {
                    const int64_t at = orow * v.head_dim + 32 * c;
                    uint16_t *dst = static_cast<uint16_t *>(p.out) + at;
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if (32 * c + 8 * i >= v.head_dim ||
                            !QLORA_IN(at + 8 * i + 7, (int64_t)v.tokens * v.heads * v.head_dim))
                            break;
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            w[j] = pack2<F16>(__uint_as_float(o[8 * i + 2 * j]) * inv, __uint_as_float(o[8 * i + 2 * j + 1]) * inv);
                        *reinterpret_cast<uint4 *>(dst + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        *reinterpret_cast<uint4 *>(part + ((8 * c + i) * C::kRows + pr) * 4) =   // four columns of a row together
                            make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
            }
            if (valid && !whole) {
                part[C::kRows * DP + pr] = m;
                part[C::kRows * DP + C::kRows + pr] = l;
            } else if (valid && p.lse) {
                p.lse[orow] = log_sum<kRaiseMany<F16>>(m, l, p.scale_log2);
            }
            if (it->begins && threadIdx.x == 0) p.desc[cta] = Desc{it->q0, it->h, it->row0, it->half[0].rows + it->half[1].rows, slot, (int)cta, it->parts};
            tiles += it->t1 - it->t0;
            tc_fence_before();   // these reads of O come before the next item's first product, behind p_ready
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->item_empty[items & 3]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace attn
}  // namespace qlora
