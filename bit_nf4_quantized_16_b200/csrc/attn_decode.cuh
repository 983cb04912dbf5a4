// Paged attention for few query rows (one token, or a handful, per request):
// bound by the bytes of the keys and values.
//
// Tensor-core tiles of 16 rows (mma m16n8k16).  The four warps of a CTA work
// alone inside an item: warp w takes positions 64 t + 16 w ... + 15 of each
// tile t, with a ring of its own that tensor copies fill (a 16-position step
// never leaves a page: page sizes are powers of two from 16 on), its own
// barriers, and its own running maximum, sum and output in registers (one pass
// over the keys).  Nothing synchronizes the warps until the item's end, where
// they join their results through shared memory.  The copies run ahead of
// the products across items: the producer walks the schedule a second time,
// ring depth ahead of the consumer.  Two CTAs per SM keep up to 128 KB of copies
// on their way, and one streams while the other joins.
//
// The weights p of the softmax enter the second product as hi + lo 16-bit
// pairs: p - hi is exact, and lo rounds it, to 2^-18 of p in bf16, and in fp16 to 2^-22
// of p or 2^-40 of the largest weight (see kRaiseFew).  With a single
// 16-bit p the output would carry its rounding beside the output's own.  The
// products have time for it: 16 rows x 16 positions take 48 of them for 8 KB.
//
// Measured (B200, by box): 16 requests of 4100 positions, 64 heads of 128 (2.1 GB): 320 to 341 us,
// 6.3 to 6.7 TB/s (0.96 to 1.03 of the measured copy rate, which writes half of its bytes); 64 requests of 100 to
// 16000 positions, 8 heads: 115 to 121 us, 5.8 to 6.1 TB/s (0.88 to 0.93); one request of 500 positions, 32 heads: 7.4 us a call, of which
// launch, lengths, table and first copy are four dependent latencies; 32 requests under a window of
// 1024 with 4 sinks, 8 heads: 30.7 us, 4.4 TB/s (0.67: 256 whole items on 296 places, start and join around them).
#pragma once
#include <type_traits>

#include "attn_common.cuh"

namespace qlora {
namespace attn {

template <int DP>
struct DecodeCfg {
    static constexpr int kWarps = 4, kThreads = 32 * kWarps;
    static constexpr int kRows = 16, kTile = 16 * kWarps, kOv = 3;   // an item costs three tiles beside its own (64 ragged requests on one box: 149 us with 0, 121 with 2, 116 with 3)
    static constexpr int kStages = DP == 128 ? 2 : 4;
    static constexpr uint32_t kStageBytes = 2 * 16 * DP * 2;   // keys, then values, of 16 positions
    static constexpr uint32_t kRing = kWarps * kStages * kStageBytes;
    static constexpr int kLd = DP + 8;   // floats between rows of a warp's result (bank spread)
    static constexpr uint32_t kMergeOff = kRing;
    static constexpr uint32_t kStatOff = kMergeOff + kWarps * 16 * kLd * 4;
    static constexpr uint32_t kBarOff = kStatOff + kWarps * 32 * 4;
    static constexpr uint32_t kMetaOff = kBarOff + kWarps * kStages * 8;
    static constexpr uint32_t kBytes = kMetaOff + kWarps * kStages * 8 + 1024;   // + alignment slack
    static constexpr int kSlotFloats = kRows * DP + 2 * kRows;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The walk of a CTA whose cluster has one key/value head of one request: an
// equal share of the tiles of each of its row tiles (mostly there is one).
template <int ROWS, int TILE>
struct OneHead {
    int b, h, rt, n_rt, rank, ranks;
    Request r;

    __device__ __forceinline__ void init(const BatchView &v)
    {
        rank = (int)sm100::cluster_ctarank();
        ranks = (int)sm100::cluster_nctarank();
        h = blockIdx.x / ranks;
        b = h / v.kv_heads;
        h -= b * v.kv_heads;
        rt = 0;
        r = load_request(v, b);
        n_rt = row_tiles<ROWS>(v, r);
    }
    __device__ __forceinline__ bool next(const BatchView &v, Item &it)
    {
        if (rt >= n_rt) return false;
        it.b = b;
        it.h = h;
        it.rt = rt;
        it.r = r;
        it.tiles = item_tiles<ROWS, TILE>(v, r, rt);
        it.t0 = (int)((int64_t)it.tiles.n * rank / ranks);
        it.t1 = (int)((int64_t)it.tiles.n * (rank + 1) / ranks);
        it.whole = it.begins = false;
        it.end = 0;
        rt++;
        return true;
    }
};

__device__ __forceinline__ float ld_dsmem_f1(uint32_t addr)
{
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}

// CLUSTER: few items.  Every key/value head of every request has a cluster of CTAs
// (of one to eight), which divide its keys and join their results through
// distributed shared memory: no schedule to scan, no partial results in memory and
// no second kernel.
template <int DP, bool F16, bool CLUSTER>
__global__ void __launch_bounds__(DecodeCfg<DP>::kThreads, 2) decode_kernel(const __grid_constant__ AttnParams p)
{
    using C = DecodeCfg<DP>;
    using W = std::conditional_t<CLUSTER, OneHead<C::kRows, C::kTile>, Walker<C::kThreads, C::kRows, C::kTile, C::kOv>>;
    using namespace sm100;
    constexpr int ST = C::kStages;
    constexpr float kRaise = kRaiseFew<F16>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int64_t pre[C::kThreads + 1 + C::kWarps];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const BatchView &v = p.v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem + warp * ST * C::kStageBytes;
    float *merge = reinterpret_cast<float *>(smem + C::kMergeOff);
    float *stat = reinterpret_cast<float *>(smem + C::kStatOff);   // [warp][16 maxima, 16 sums]
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff) + warp * ST;
    int2 *meta = reinterpret_cast<int2 *>(smem + C::kMetaOff) + warp * ST;   // item number, first position

    if (lane == 0) {
        for (int s = 0; s < ST; s++) mbar_init(&full[s], 1);
        fence_barrier_init();
        if (warp == 0) {
            tma_prefetch_desc(&p.tk);
            tma_prefetch_desc(&p.tv);
        }
    }
    pdl_wait();
    pdl_trigger();
    const int64_t cta = blockIdx.x;
    int64_t G = 0, total = 0;
    W wp, wc;   // the producer's walk, and the consumer's
    if constexpr (CLUSTER) {
        wp.init(v);
    } else {
        schedule_scan<C::kThreads, C::kRows, C::kTile, C::kOv>(v, pre);
        total = pre[C::kThreads];
        G = min((int64_t)gridDim.x, total);
        if (threadIdx.x == 0) p.desc[cta].parts = 0;
        if (cta >= G) return;
        wp.init(v, pre, first_unit(cta, G, total), first_unit(cta + 1, G, total));
    }
    wc = wp;

    // ---- producer: one 16-position step of the next item that has any ----
    Item pi;
    bool p_more = wp.next(v, pi);
    int pt = p_more ? pi.t0 : 0, p_item = 0, produced = 0, cache_t = -64, cache_page = -1;
    bool dead = false;
    auto needed = [&](const Item &it, int tok0, int first, int last) {
        return tok0 <= last && tok0 < it.r.reach &&
               (v.window <= 0 || tok0 + 15 > first - v.window || tok0 < v.sinks);
    };
    auto produce = [&]() {
        while (p_more) {
            if (pt >= pi.t1) {
                p_more = wp.next(v, pi);
                pt = pi.t0;
                p_item++;
                cache_t = -64;
                if (p_more && warp == 0) {   // its query rows, for the consumer: two lanes a row, a line each
                    const int g = pi.rt * C::kRows + (lane >> 1), tok = v.token_of(g);
                    if (g < pi.r.qn * v.group && (lane & 1) * 64 < v.head_dim)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(
                            static_cast<const uint16_t *>(p.q) +
                            ((int64_t)(pi.r.q0 + tok) * v.heads + pi.h * v.group + g - tok * v.group) * v.head_dim + (lane & 1) * 64));
                }
                continue;
            }
            const int t = pt++;
            if (t >= cache_t + 32 || t < cache_t) {   // pages of the next 32 steps, one per lane
                cache_t = t;
                cache_page = t + lane < pi.t1 ? page_of(v, pi.b, pi.tiles.at(t + lane) * C::kTile + 16 * warp) : -1;
            }
            const int page = __shfl_sync(0xffffffffu, cache_page, t - cache_t);
            const int tok0 = pi.tiles.at(t) * C::kTile + 16 * warp;
            int first, last;
            item_positions<C::kRows>(v, pi.r, pi.rt, first, last);
            if (page < 0 || !needed(pi, tok0, first, last)) continue;
            if (lane == 0) {
                const int s = produced % ST, row = tok0 & ((1 << v.page_shift) - 1);
                meta[s] = make_int2(p_item, tok0);
                uint8_t *k = ring + s * C::kStageBytes, *vv = k + C::kStageBytes / 2;
                mbar_arrive_expect_tx(&full[s], C::kStageBytes);
#pragma unroll
                for (int c = 0; c < DP / 64; c++) {
                    tma_load_4d(k + c * 2048, &p.tk, &full[s], 64 * c, row, pi.h, page);
                    tma_load_4d(vv + c * 2048, &p.tv, &full[s], 64 * c, row, pi.h, page);
                }
            }
            produced++;
            break;
        }
        __syncwarp();
    };
    for (int s = 0; s < ST; s++) produce();

    // ---- consumer ----
    Item it;
    int consumed = 0;
    for (int item = 0; wc.next(v, it); item++) {
        const int rows = min(it.r.qn * v.group - it.rt * C::kRows, C::kRows);
        const int pos0 = it.r.kv - it.r.qn;
        const int ra = lane >> 2, rb = ra + 8, gr0 = it.rt * C::kRows;
        const int pos_a = ra < rows ? pos0 + v.token_of(gr0 + ra) : -1;
        const int pos_b = rb < rows ? pos0 + v.token_of(gr0 + rb) : -1;
        int first, last;
        item_positions<C::kRows>(v, it.r, it.rt, first, last);
        // query rows as A operands: this lane's rows ra and rb
        uint32_t qf[DP / 16][4];
        {
            const uint32_t *qa = nullptr, *qb = nullptr;
            [[maybe_unused]] const int64_t q_n = (int64_t)v.tokens * v.heads * v.head_dim;
            auto row_ptr = [&](int r) -> const uint32_t * {
                const int g = gr0 + r;
                const int64_t o = ((int64_t)(it.r.q0 + v.token_of(g)) * v.heads + it.h * v.group + g - v.token_of(g) * v.group) * v.head_dim;
                return QLORA_IN(o + v.head_dim - 1, q_n)
                           ? reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.q) + o)
                           : nullptr;
            };
            if (ra < rows) qa = row_ptr(ra);
            if (rb < rows) qb = row_ptr(rb);
#pragma unroll
            for (int kk = 0; kk < DP / 16; kk++) {
                const int c = kk * 8 + (lane & 3);   // 32-bit column
                const bool in = kk * 16 < v.head_dim;
                qf[kk][0] = in && qa ? qa[c] : 0u;
                qf[kk][1] = in && qb ? qb[c] : 0u;
                qf[kk][2] = in && qa ? qa[c + 4] : 0u;
                qf[kk][3] = in && qb ? qb[c + 4] : 0u;
            }
        }
        float o[DP / 8][4];
#pragma unroll
        for (int n = 0; n < DP / 8; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) o[n][i] = 0.0f;
        float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.0f, l_b = 0.0f;

        while (consumed < produced && meta[consumed % ST].x == item) {
            const int s = consumed % ST, tok0 = meta[s].y;
            if (!dead && !mbar_wait_bounded(&full[s], (consumed / ST) & 1, p.timeout_ns)) {
                if (lane == 0) atomicExch(p.err, 1);
                dead = true;
            }
            dead = __any_sync(0xffffffffu, dead);
            if (dead) {   // take no more copies, and wait (bounded) for those in flight
                p_more = false;
                for (int j = consumed; j < produced; j++) mbar_wait_bounded(&full[j % ST], (j / ST) & 1, p.timeout_ns);
                consumed = produced;
                break;
            }
            uint8_t *kp = ring + s * C::kStageBytes, *vp = kp + C::kStageBytes / 2;
            const uint32_t ka = smem_u32(kp), va = smem_u32(vp);
            bool wrote = false;
            if (tok0 + 16 > it.r.kv) {
                // positions that were never written may hold anything; their weight is 0,
                // but 0 times a NaN is not
                const int from_row = it.r.kv - tok0;
                for (int c = lane; c < (16 - from_row) * (DP / 8); c += 32) {
                    const int row = from_row + c / (DP / 8), ch = c % (DP / 8);
                    *reinterpret_cast<uint4 *>(vp + (ch >> 3) * 2048 + row * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                wrote = true;
                __syncwarp();
            }
            // scores: 16 rows x 16 positions
            float sc[2][4] = {};
            {
                const int mid = lane >> 3, row = (mid >> 1) * 8 + (lane & 7);
#pragma unroll
                for (int kk = 0; kk < DP / 16; kk++) {
                    uint32_t b[4];
                    ldsm4(ka + (kk >> 2) * 2048 + row * 128 + ((((kk & 3) * 2 + (mid & 1)) ^ (row & 7)) << 4), b);
                    mma<F16>(sc[0], qf[kk], b[0], b[1]);
                    mma<F16>(sc[1], qf[kk], b[2], b[3]);
                }
            }
            const bool all_seen = tok0 + 15 <= first && tok0 + 15 < it.r.reach &&
                                  (v.window <= 0 || tok0 > last - v.window || tok0 + 15 < v.sinks);
            if (!all_seen) {
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int pos = i < 2 ? pos_a : pos_b, j = tok0 + 8 * n + (lane & 3) * 2 + (i & 1);
                        const bool seen = j <= pos && j < it.r.reach && (v.window <= 0 || j > pos - v.window || j < v.sinks);
                        if (!seen) sc[n][i] = -INFINITY;
                    }
            }
            float x_a = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
            float x_b = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                x_a = fmaxf(x_a, __shfl_xor_sync(0xffffffffu, x_a, d));
                x_b = fmaxf(x_b, __shfl_xor_sync(0xffffffffu, x_b, d));
            }
            if (__any_sync(0xffffffffu, x_a > m_a || x_b > m_b)) {
                const float n_a = fmaxf(m_a, x_a), n_b = fmaxf(m_b, x_b);
                const float f_a = n_a == -INFINITY ? 1.0f : exp2f((m_a - n_a) * p.scale_log2);
                const float f_b = n_b == -INFINITY ? 1.0f : exp2f((m_b - n_b) * p.scale_log2);
                m_a = n_a;
                m_b = n_b;
                l_a *= f_a;
                l_b *= f_b;
#pragma unroll
                for (int n = 0; n < DP / 8; n++) {
                    o[n][0] *= f_a;
                    o[n][1] *= f_a;
                    o[n][2] *= f_b;
                    o[n][3] *= f_b;
                }
            }
            // a row that has seen nothing yet: every score is -inf, every weight 0
            const float u_a = m_a == -INFINITY ? 0.0f : m_a, u_b = m_b == -INFINITY ? 0.0f : m_b;
            float w[2][4];
#pragma unroll
            for (int n = 0; n < 2; n++) {
                w[n][0] = exp2f(__fmaf_rn(sc[n][0] - u_a, p.scale_log2, kRaise));
                w[n][1] = exp2f(__fmaf_rn(sc[n][1] - u_a, p.scale_log2, kRaise));
                w[n][2] = exp2f(__fmaf_rn(sc[n][2] - u_b, p.scale_log2, kRaise));
                w[n][3] = exp2f(__fmaf_rn(sc[n][3] - u_b, p.scale_log2, kRaise));
                l_a += w[n][0] + w[n][1];
                l_b += w[n][2] + w[n][3];
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float w0 = w[i >> 1][(i & 1) * 2], w1 = w[i >> 1][(i & 1) * 2 + 1];
                hi[i] = pack2<F16>(w0, w1);
                const float2 h = unpack2<F16>(hi[i]);
                lo[i] = pack2<F16>(w0 - h.x, w1 - h.y);
            }
            {
                const int mid = lane >> 3, row = (mid & 1) * 8 + (lane & 7);
#pragma unroll
                for (int j = 0; j < DP / 16; j++) {
                    uint32_t b[4];
                    ldsm4_t(va + (j >> 2) * 2048 + row * 128 + ((((j & 3) * 2 + (mid >> 1)) ^ (row & 7)) << 4), b);
                    mma<F16>(o[2 * j], hi, b[0], b[1]);
                    mma<F16>(o[2 * j + 1], hi, b[2], b[3]);
                    mma<F16>(o[2 * j], lo, b[0], b[1]);
                    mma<F16>(o[2 * j + 1], lo, b[2], b[3]);
                }
            }
            if (wrote) fence_proxy_async_smem();
            __syncwarp();
            consumed++;
            produce();
        }

        // ---- join the warps ----
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            l_a += __shfl_xor_sync(0xffffffffu, l_a, d);
            l_b += __shfl_xor_sync(0xffffffffu, l_b, d);
        }
        float *mo = merge + warp * 16 * C::kLd;
        if (ra < rows) {
#pragma unroll
            for (int n = 0; n < DP / 8; n++)
                *reinterpret_cast<float2 *>(mo + ra * C::kLd + 8 * n + 2 * (lane & 3)) = make_float2(o[n][0], o[n][1]);
        }
        if (rb < rows) {
#pragma unroll
            for (int n = 0; n < DP / 8; n++)
                *reinterpret_cast<float2 *>(mo + rb * C::kLd + 8 * n + 2 * (lane & 3)) = make_float2(o[n][2], o[n][3]);
        }
        if ((lane & 3) == 0) {
            stat[warp * 32 + ra] = m_a;
            stat[warp * 32 + rb] = m_b;
            stat[warp * 32 + 16 + ra] = l_a;
            stat[warp * 32 + 16 + rb] = l_b;
        }
        __syncthreads();
        if constexpr (CLUSTER) {
            // this CTA's joined rows over warp 0's, its maxima and sums over warp 0's
            for (int i = threadIdx.x; i < rows * (DP / 4); i += C::kThreads) {
                const int r = i / (DP / 4), c = (i % (DP / 4)) * 4;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < C::kWarps; w++) M = fmaxf(M, stat[w * 32 + r]);
                float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int w = 0; w < C::kWarps; w++) {
                    const float mw = stat[w * 32 + r], f = mw == -INFINITY ? 0.0f : exp2f((mw - M) * p.scale_log2);
                    const float4 x = *reinterpret_cast<const float4 *>(merge + (w * 16 + r) * C::kLd + c);
                    a.x += f * x.x;
                    a.y += f * x.y;
                    a.z += f * x.z;
                    a.w += f * x.w;
                }
                *reinterpret_cast<float4 *>(merge + r * C::kLd + c) = a;   // only this thread has read it
            }
            __syncthreads();
            if (threadIdx.x < 16) {
                const int r = threadIdx.x;
                float M = -INFINITY, L = 0.0f;
#pragma unroll
                for (int w = 0; w < C::kWarps; w++) M = fmaxf(M, stat[w * 32 + r]);
#pragma unroll
                for (int w = 0; w < C::kWarps; w++) {
                    const float mw = stat[w * 32 + r];
                    const float f = mw == -INFINITY ? 0.0f : exp2f((mw - M) * p.scale_log2);
                    L += f * stat[w * 32 + 16 + r];   // (a product: a sum of NaN shows in L even where no score was a number)
                }
                stat[r] = M;
                stat[16 + r] = L;
            }
            cluster_sync();
            const uint32_t merge_at = smem_u32(merge), stat_at = smem_u32(stat);
            [[maybe_unused]] const int64_t out_n = (int64_t)v.tokens * v.heads * v.head_dim;
            for (int i = wc.rank * C::kThreads + threadIdx.x; i < rows * (DP / 4); i += wc.ranks * C::kThreads) {
                const int r = i / (DP / 4), c = (i % (DP / 4)) * 4;
                float M = -INFINITY, L = 0.0f;
                for (int k = 0; k < wc.ranks; k++) M = fmaxf(M, ld_dsmem_f1(mapa_shared(stat_at + 4 * r, k)));
                float4 a = make_float4(0, 0, 0, 0);
                for (int k = 0; k < wc.ranks; k++) {
                    const float m = ld_dsmem_f1(mapa_shared(stat_at + 4 * r, k));
                    const float f = m == -INFINITY ? 0.0f : exp2f((m - M) * p.scale_log2);
                    L += f * ld_dsmem_f1(mapa_shared(stat_at + 4 * (16 + r), k));
                    const float4 x = ld_dsmem_f4(mapa_shared(merge_at + 4 * (r * C::kLd + c), k));
                    a.x += f * x.x;
                    a.y += f * x.y;
                    a.z += f * x.z;
                    a.w += f * x.w;
                }
                const float inv = inverse_sum(L);
                const int g = gr0 + r, t = v.token_of(g);
                const int64_t row = (int64_t)(it.r.q0 + t) * v.heads + it.h * v.group + g - t * v.group;
                const int64_t at = row * v.head_dim + c;
                if (c < v.head_dim && QLORA_IN(at + 3, out_n))
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
                        make_uint2(pack2<F16>(a.x * inv, a.y * inv), pack2<F16>(a.z * inv, a.w * inv));
                if (c == 0 && p.lse) p.lse[row] = log_sum<kRaiseFew<F16>>(M, L, p.scale_log2);
            }
            cluster_sync();   // the others have read this CTA's results
            continue;
        }
        const int slot = 2 * (int)cta + (item == 0 ? 0 : 1);
        float *part = p.part + (int64_t)slot * C::kSlotFloats;
        [[maybe_unused]] const int64_t out_n = (int64_t)v.tokens * v.heads * v.head_dim;
        for (int i = threadIdx.x; i < rows * (DP / 4); i += C::kThreads) {
            const int r = i / (DP / 4), c = (i % (DP / 4)) * 4;
            float mw[C::kWarps], M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int w = 0; w < C::kWarps; w++) {
                mw[w] = stat[w * 32 + r];
                M = fmaxf(M, mw[w]);
            }
            float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < C::kWarps; w++) {
                const float f = mw[w] == -INFINITY ? 0.0f : exp2f((mw[w] - M) * p.scale_log2);
                const float4 x = *reinterpret_cast<const float4 *>(merge + (w * 16 + r) * C::kLd + c);
                L += f * stat[w * 32 + 16 + r];
                a.x += f * x.x;
                a.y += f * x.y;
                a.z += f * x.z;
                a.w += f * x.w;
            }
            if (it.whole) {
                const float inv = inverse_sum(L);
                const int g = gr0 + r;
                const int64_t row = (int64_t)(it.r.q0 + v.token_of(g)) * v.heads + it.h * v.group + g - v.token_of(g) * v.group;
                const int64_t at = row * v.head_dim + c;
                if (c < v.head_dim && QLORA_IN(at + 3, out_n))
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
                        make_uint2(pack2<F16>(a.x * inv, a.y * inv), pack2<F16>(a.z * inv, a.w * inv));
                if (c == 0 && p.lse) p.lse[row] = log_sum<kRaiseFew<F16>>(M, L, p.scale_log2);
            } else {
                *reinterpret_cast<float4 *>(part + r * DP + c) = a;
                if (c == 0) {
                    part[C::kRows * DP + r] = M;
                    part[C::kRows * DP + C::kRows + r] = L;
                }
            }
        }
        if (it.begins && threadIdx.x == 0)
            p.desc[cta] = Desc{it.r.q0, it.h, it.rt * C::kRows, rows, slot, (int)cta, cta_of_last(it.end, G, total) - (int)cta + 1};
        __syncthreads();
    }
}

}  // namespace attn
}  // namespace qlora
