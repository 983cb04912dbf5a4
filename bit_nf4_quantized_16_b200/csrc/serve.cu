// The step of a served model around its attention: the plan (block tables,
// slots and positions from the requests' lengths, built on the GPU) and the
// append of rotated keys and values to the paged cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "debug.cuh"
#include "serve.cuh"
#include "sm100.cuh"

namespace qlora {
namespace {

// ---- plan ---------------------------------------------------------------------------
//
// One cluster of CTAs.  Every CTA scans all requests (three prefix sums: rows,
// pages returned, pages taken), so that any of them can answer for any page or
// token with a binary search in its shared memory; then the CTAs divide the
// outputs.  An ended request returns those of its entries that are pages (a caller
// under a window may have given others away), so they are counted before the scan, a
// warp a request.  If any are returned, the CTAs push them first and meet at the cluster's
// barrier; from there on the pool is read only.  The count may be updated in
// place: it is read before the barrier at the end and written after it.
//
// The call moves a few hundred KB at most; what bounds it is latency (a launch,
// three dependent reads, two scans), so a small batch gets one small CTA and a large
// one as many threads as a cluster has; a thread takes four neighbouring
// tokens, which mostly share the search.
// Measured (B200, replayed): 16 requests of one token 4.0 us (append_kernel, which only
// streams, takes 2.6 at its smallest); 1000 requests with 20651 tokens, 5937 returned and
// 1308 taken pages 12.4 us, 7.5 without a returned one; with 300 ended requests 22 us.  (With one load
// at a time in the count and the push: 17.6 and 31.)

struct PlanParams {
    const int32_t *ctx, *qlen;
    int32_t *free_pages;
    const int32_t *free_count;
    int32_t *free_count_out;
    int32_t *table, *cu_q, *kv_len, *positions, *slots;
    int batch, max_pages, tokens, num_pages, page_shift;
};

// Exclusive prefixes of two values per thread over the block, and their totals.
struct Two {
    int64_t a, b;
};
__device__ __forceinline__ Two block_scan(Two mine, Two *warp_sum, Two &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    Two incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ua = __shfl_up_sync(0xffffffffu, incl.a, o), ub = __shfl_up_sync(0xffffffffu, incl.b, o);
        if (lane >= o) {
            incl.a += ua;
            incl.b += ub;
        }
    }
    __syncthreads();   // the sums of the scan before have been read
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {   // (every warp adding up the sums on its own took three times as long with 32 of them)
        Two s = lane < warps ? warp_sum[lane] : Two{0, 0};
        const Two own = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t ua = __shfl_up_sync(0xffffffffu, s.a, o), ub = __shfl_up_sync(0xffffffffu, s.b, o);
            if (lane >= o) {
                s.a += ua;
                s.b += ub;
            }
        }
        if (lane == 31) warp_sum[32] = s;
        warp_sum[lane] = Two{s.a - own.a, s.b - own.b};
    }
    __syncthreads();
    total = warp_sum[32];
    return Two{warp_sum[warp].a + incl.a - mine.a, warp_sum[warp].b + incl.b - mine.b};
}

// The index i with pre[i] <= x < pre[i + 1] (pre ascending, pre[0] <= x < pre[n]).
__device__ __forceinline__ int owner_of(const int32_t *pre, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int32_t clamp31(int64_t x) { return (int32_t)min(x, (int64_t)INT32_MAX); }

__global__ void __launch_bounds__(1024) plan_kernel(const PlanParams p)
{
    extern __shared__ int32_t plan_smem[];
    __shared__ Two warp_sum[33];
    const int n = p.batch, tid = threadIdx.x, threads = blockDim.x;
    int32_t *rows_pre = plan_smem;             // [n + 1] rows before request i, at most `tokens`
    int32_t *back_pre = rows_pre + n + 1;      // pages returned before i
    int32_t *take_pre = back_pre + n + 1;      // pages asked for before i
    int32_t *ctx_of = take_pre + n + 1;        // [n] ctx_len, -1 for a request that is refused or has ended
    const int rank = (int)sm100::cluster_ctarank(), ctas = (int)sm100::cluster_nctarank();
    const int64_t step = (int64_t)ctas * threads, first = (int64_t)rank * threads + tid;
    sm100::pdl_wait();
    sm100::pdl_trigger();
    const int page = 1 << p.page_shift;
    const int count = min(max(*p.free_count, 0), p.num_pages);
    auto pages = [&](int64_t t) { return (t + page - 1) >> p.page_shift; };
    const int64_t capacity = (int64_t)p.max_pages << p.page_shift;
    auto is_page = [&](int32_t id) { return (unsigned)id < (unsigned)p.num_pages; };
    constexpr int kAtOnce = 16;   // loads of a lane that do not wait for one another
    const int lane = tid & 31;

    Two at{0, 0};            // rows and returned pages so far
    int64_t take_at = 0;
    for (int b0 = 0; b0 < n; b0 += threads) {
        const int b = b0 + tid;
        const int64_t ctx = b < n ? p.ctx[b] : 0, q = b < n ? p.qlen[b] : 0;
        const int64_t rows = max(q, (int64_t)0);
        const int held = q < 0 ? (int)min(pages(max(ctx, (int64_t)0)), (int64_t)p.max_pages) : 0;
        int64_t back = 0;
        for (unsigned left = __ballot_sync(0xffffffffu, held > 0); left; left &= left - 1) {
            const int l = __ffs(left) - 1, entries = __shfl_sync(0xffffffffu, held, l);
            const int32_t *row = p.table + (int64_t)(b - lane + l) * p.max_pages;
            int found = 0;
            for (int i0 = 0; i0 < entries; i0 += 32 * kAtOnce) {
                int32_t id[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; k++) id[k] = i0 + 32 * k + lane < entries ? row[i0 + 32 * k + lane] : -1;
#pragma unroll
                for (int k = 0; k < kAtOnce; k++) found += is_page(id[k]);
            }
            found = __reduce_add_sync(0xffffffffu, found);
            if (lane == l) back = found;
        }
        Two total;
        const Two pre = block_scan(Two{rows, back}, warp_sum, total);
        const int64_t rows0 = at.a + pre.a, back0 = at.b + pre.b;
        at.a += total.a;
        at.b += total.b;
        const bool fits = q >= 0 && ctx >= 0 && ctx + rows <= capacity && (rows == 0 || rows0 + rows <= p.tokens);
        const int64_t take = fits ? pages(ctx + rows) - pages(ctx) : 0;
        const int64_t take0 = take_at + block_scan(Two{take, 0}, warp_sum, total).a;
        take_at += total.a;
        if (b < n) {
            rows_pre[b] = (int32_t)min(rows0, (int64_t)p.tokens);
            back_pre[b] = clamp31(back0);
            take_pre[b] = clamp31(take0);
            ctx_of[b] = fits ? (int32_t)ctx : -1;
        }
    }
    if (tid == 0) {
        rows_pre[n] = (int32_t)min(at.a, (int64_t)p.tokens);
        back_pre[n] = clamp31(at.b);
        take_pre[n] = clamp31(take_at);
    }
    __syncthreads();
    // a valid call returns no more pages than are not in the pool
    const int pool = (int)min((int64_t)count + at.b, (int64_t)p.num_pages);
    const int returned = pool - count;
    // requests take pages in order, and none after the first that the pool cannot serve
    int lo = 0, hi = n + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (take_pre[mid] <= pool) lo = mid; else hi = mid;
    }
    const int used = take_pre[lo];
    if (returned > 0) {   // the same in every CTA
        const int warps = (int)(step >> 5);
        for (int b = (int)(first >> 5); b < n; b += warps) {   // a warp a request, its pages in their order
            int to = back_pre[b];
            const int end = min(back_pre[b + 1], returned);
            const int32_t *row = p.table + (int64_t)b * p.max_pages;
            for (int i0 = 0; to < end && i0 < p.max_pages; i0 += 32 * kAtOnce) {
                int32_t id[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; k++) id[k] = i0 + 32 * k + lane < p.max_pages ? row[i0 + 32 * k + lane] : -1;
#pragma unroll
                for (int k = 0; k < kAtOnce; k++) {
                    const unsigned found = __ballot_sync(0xffffffffu, is_page(id[k]));
                    const int at = to + __popc(found & ((1u << lane) - 1));
                    if (is_page(id[k]) && at < end && QLORA_IN(count + at, p.num_pages)) p.free_pages[count + at] = id[k];
                    to += __popc(found);
                }
            }
        }
        if (ctas > 1) sm100::cluster_sync(); else __syncthreads();
    }
    // Whether request b, which fits, gets its pages.  (The prefix counts what refused requests
    // asked for too; that is at most tokens / 16 + batch pages, so it stays in 32 bits.)
    auto granted = [&](int b) { return take_pre[b + 1] == take_pre[b] || take_pre[b + 1] <= pool; };

    for (int64_t b = first; b <= n; b += step) {
        p.cu_q[b] = rows_pre[b];
        if (b == n) break;
        const bool ok = ctx_of[b] >= 0 && granted((int)b);
        p.kv_len[b] = ok ? ctx_of[b] + max(p.qlen[b], 0) : 0;
    }
    for (int64_t u = step - 1 - first; u < used; u += step) {   // (the last threads have the least to do below)
        const int b = owner_of(take_pre, n, (int)u);
        const int64_t i = (int64_t)b * p.max_pages + pages(ctx_of[b]) + u - take_pre[b];
        if (QLORA_IN(i, (int64_t)n * p.max_pages)) p.table[i] = p.free_pages[pool - 1 - u];
    }
    const int all_rows = rows_pre[n];
    for (int64_t t4 = 4 * first; t4 < p.tokens; t4 += 4 * step) {
        int32_t pos[4], slot[4];
        const int32_t *id_at[4];   // four loads that do not wait for one another
        int b = t4 < all_rows ? owner_of(rows_pre, n, (int)t4) : n;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int t = (int)t4 + k;
            pos[k] = -1;
            id_at[k] = nullptr;
            if (t >= all_rows) continue;
            while (rows_pre[b + 1] <= t) b++;
            if (ctx_of[b] < 0 || !granted(b)) continue;
            pos[k] = ctx_of[b] + t - rows_pre[b];
            const int held = (int)pages(ctx_of[b]), i = pos[k] >> p.page_shift;
            id_at[k] = i < held ? p.table + (int64_t)b * p.max_pages + i
                                : p.free_pages + (pool - 1 - (take_pre[b] + i - held));
        }
#pragma unroll
        for (int k = 0; k < 4; k++) slot[k] = id_at[k] ? *id_at[k] : -1;
#pragma unroll
        for (int k = 0; k < 4; k++)
            slot[k] = (unsigned)slot[k] < (unsigned)p.num_pages ? (slot[k] << p.page_shift) + (pos[k] & (page - 1)) : -1;
        if (t4 + 4 <= p.tokens) {
            *reinterpret_cast<int4 *>(p.positions + t4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4 *>(p.slots + t4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
            for (int k = 0; k < (int)(p.tokens - t4); k++) {
                p.positions[t4 + k] = pos[k];
                p.slots[t4 + k] = slot[k];
            }
        }
    }
    // every CTA has read the count
    if (ctas > 1) sm100::cluster_sync(); else __syncthreads();
    if (rank == 0 && tid == 0) *p.free_count_out = pool - used;
}

// ---- append -------------------------------------------------------------------------
//
// Pairs (i, i + D/2) of each head rotate by position * base^(-2i/D).  The angle
// is formed in turns: position times turns per position in binary64, of
// which the whole part is dropped before anything is rounded to binary32, so
// that far positions lose nothing (in binary32 the angle of position 130000 is
// off by up to 2^-7 radians).  The sine and cosine of the rest come from the
// fast intrinsics on an argument in [-pi, pi], whose absolute error (2^-21) is
// far below half a step of the 16-bit results.
//
// A block takes kTok tokens: it forms their angles once in shared memory, then
// its threads move 16-byte pieces (a low and a high one that rotate together)
// of q, k and v.  Bound by memory: every value is read and written once.  The
// angles lie so in shared memory that the threads of a warp read neighbours.
// Measured (B200): 7983 tokens, 32 + 8 + 8 heads of 128 (196 MB): 37.5 us, 5.2 TB/s (0.80 of
// the measured copy rate); 16 tokens of 3 x 64 heads: 2.6 us, latency.

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;   // at most, per block

struct AppendParams {
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *kc, *vc;
    const int32_t *positions, *slots;
    int64_t stride_page, stride_head, stride_token;
    int tokens, heads, kv_heads, head_dim, page_shift, num_pages;
    int block_tokens;
    int rotate;
    double turns[64];
};

template <bool F16>
__device__ __forceinline__ float2 up2(uint32_t w)
{
    if (F16) return __half22float2(*reinterpret_cast<__half2 *>(&w));
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&w));
}

template <bool F16>
__device__ __forceinline__ uint32_t down2(float a, float b)
{
    if (F16) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

template <bool F16>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ float2 cs[kAppendTokens * 64];
    __shared__ int32_t slot_of[kAppendTokens];
    sm100::pdl_wait();
    sm100::pdl_trigger();
    const int half = p.head_dim / 2, groups = half / 8;
    const int64_t t0 = (int64_t)blockIdx.x * p.block_tokens;
    const int toks = (int)min((int64_t)p.block_tokens, p.tokens - t0);
    if (threadIdx.x < toks) slot_of[threadIdx.x] = p.slots[t0 + threadIdx.x];
    if (p.rotate) {
        for (int e = threadIdx.x; e < toks * half; e += kAppendThreads) {
            const double turn = (double)p.positions[t0 + e / half] * p.turns[e % half];
            const float rest = (float)(turn - rint(turn));
            float s, c;
            __sincosf(rest * 6.28318530718f, &s, &c);
            // pair 8 g + j at j * groups + g: the threads of a warp, one piece g each, read neighbours
            const int i = e % half;
            cs[e - i + (i & 7) * groups + (i >> 3)] = make_float2(c, s);
        }
    }
    __syncthreads();
    // thread: piece i0 of every stride-th head, counted over the block's tokens; two at a time, so
    // that four loads are on their way
    const int per_token = p.heads + 2 * p.kv_heads, lanes = kAppendThreads / groups;
    const int i0 = ((int)threadIdx.x % groups) * 8, stride = lanes * (int)gridDim.y;
    if ((int)threadIdx.x >= lanes * groups) return;
    const int64_t slots = (int64_t)p.num_pages << p.page_shift;
    int head = blockIdx.y * lanes + (int)threadIdx.x / groups, tk = 0;
    while (tk < toks) {
        uint4 lo[2], hi[2];
        uint16_t *dst[2];
        const float2 *tab[2];   // null: no rotation
#pragma unroll
        for (int n = 0; n < 2; n++, head += stride) {
            while (head >= per_token) {
                head -= per_token;
                tk++;
            }
            dst[n] = nullptr;
            if (tk >= toks) continue;
            const int64_t slot = slot_of[tk], t = t0 + tk;
            if (slot < 0 || slot >= slots) continue;   // padding, a refused request, or not a place of the cache
            const uint16_t *src;
            tab[n] = p.rotate ? cs + tk * half + (i0 >> 3) : nullptr;
            if (head < p.heads) {
                const int64_t o = (t * p.heads + head) * p.head_dim;
                src = p.q + o;
                dst[n] = p.q_out + o;
            } else {
                const bool is_v = head >= p.heads + p.kv_heads;
                const int h = head - p.heads - (is_v ? p.kv_heads : 0);
                src = (is_v ? p.v : p.k) + (t * p.kv_heads + h) * p.head_dim;
                dst[n] = (is_v ? p.vc : p.kc) + (slot >> p.page_shift) * p.stride_page + h * p.stride_head +
                         (slot & ((1 << p.page_shift) - 1)) * p.stride_token;
                if (is_v) tab[n] = nullptr;
            }
            lo[n] = *reinterpret_cast<const uint4 *>(src + i0);
            hi[n] = *reinterpret_cast<const uint4 *>(src + i0 + half);
        }
#pragma unroll
        for (int n = 0; n < 2; n++) {
            if (!dst[n]) continue;
            uint4 a = lo[n], b = hi[n];
            if (tab[n]) {
                uint32_t *pa = reinterpret_cast<uint32_t *>(&a), *pb = reinterpret_cast<uint32_t *>(&b);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float2 x = up2<F16>(pa[j]), y = up2<F16>(pb[j]);
                    const float2 c0 = tab[n][2 * j * groups], c1 = tab[n][(2 * j + 1) * groups];
                    pa[j] = down2<F16>(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
                    pb[j] = down2<F16>(x.x * c0.y + y.x * c0.x, x.y * c1.y + y.y * c1.x);
                }
            }
            *reinterpret_cast<uint4 *>(dst[n] + i0) = a;
            *reinterpret_cast<uint4 *>(dst[n] + i0 + half) = b;
        }
    }
}

}  // namespace

qlora_status check_pages(int32_t page_size, int32_t num_pages)
{
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return QLORA_ERR_SHAPE;
    if (num_pages < 1 || (int64_t)num_pages * page_size > INT32_MAX) return QLORA_ERR_SHAPE;
    return QLORA_OK;
}

qlora_status check_cache(const qlora_kv_cache *c)
{
    if (!c || !c->k || !c->v) return QLORA_ERR_INVALID_ARG;
    if (c->dtype != QLORA_BF16 && c->dtype != QLORA_FP16) return QLORA_ERR_INVALID_ARG;
    QLORA_TRY(check_pages(c->page_size, c->num_pages));
    if (c->kv_heads < 1 || c->kv_heads > kMaxHeads) return QLORA_ERR_SHAPE;
    if (c->head_dim < 16 || c->head_dim > 128 || c->head_dim % 16) return QLORA_ERR_SHAPE;
    // rows of head_dim values that do not overlap, each on a 16-byte boundary
    const int64_t st[3] = {c->stride_token, c->stride_head, c->stride_page};
    const int64_t n[3] = {c->page_size, c->kv_heads, c->num_pages};
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return st[a] < st[b]; });
    int64_t reach = c->head_dim;
    for (int i : order) {
        if (n[i] == 1) continue;   // its stride is never used
        if (st[i] % 8 || st[i] < 0 || st[i] >= ((int64_t)1 << 39) / 2) return QLORA_ERR_SHAPE;
        if (st[i] < reach) return QLORA_ERR_SHAPE;
        reach = st[i] * (n[i] - 1) + reach;
    }
    if (!aligned16(c->k) || !aligned16(c->v)) return QLORA_ERR_ALIGNMENT;
    return QLORA_OK;
}

qlora_status check_batch(const qlora_kv_batch *kv)
{
    if (!kv) return QLORA_ERR_INVALID_ARG;
    if (kv->batch < 1 || kv->batch > kMaxRequests || kv->max_pages < 1 || kv->tokens < 1 ||
        kv->tokens > kMaxPositions || kv->max_q_len < 0)
        return QLORA_ERR_SHAPE;
    return QLORA_OK;
}

qlora_status make_cache_map(CUtensorMap *m, const qlora_kv_cache *c, const void *base, uint32_t rows)
{
    const uint64_t dims[4] = {(uint64_t)c->head_dim, (uint64_t)c->page_size, (uint64_t)c->kv_heads,
                              (uint64_t)c->num_pages};
    // a dimension of one element may have any stride; the encoder wants a multiple of 16 bytes above 0
    auto bytes = [](int64_t stride, int64_t n) { return n == 1 ? (uint64_t)256 : (uint64_t)stride * 2; };
    const uint64_t strides[3] = {bytes(c->stride_token, c->page_size), bytes(c->stride_head, c->kv_heads),
                                 bytes(c->stride_page, c->num_pages)};
    const uint32_t box[4] = {64, rows, 1, 1};
    return make_map_4d(m, c->dtype == QLORA_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace qlora

using namespace qlora;

extern "C" qlora_status qlora_build_rope(int32_t head_dim, double base, qlora_rope *out)
{
    if (!out) return QLORA_ERR_INVALID_ARG;
    if (head_dim < 16 || head_dim > 128 || head_dim % 16) return QLORA_ERR_SHAPE;
    if (!(base > 1.0) || !isfinite(base)) return QLORA_ERR_INVALID_ARG;
    out->head_dim = head_dim;
    for (int i = 0; i < 64; i++)
        out->turns[i] = i < head_dim / 2 ? pow(base, -2.0 * i / head_dim) / 6.283185307179586476925 : 0.0;
    return QLORA_OK;
}

extern "C" qlora_status qlora_kv_plan(const qlora_kv_batch *kv, int32_t page_size, int32_t num_pages,
                                      const int32_t *ctx_len, const int32_t *q_len, int32_t *free_pages,
                                      const int32_t *free_count, int32_t *free_count_out, void *stream)
{
    QLORA_TRY(check_batch(kv));
    QLORA_TRY(check_pages(page_size, num_pages));
    if (!ctx_len || !q_len || !free_pages || !free_count || !free_count_out || !kv->block_table || !kv->cu_q ||
        !kv->kv_len || !kv->positions || !kv->slots)
        return QLORA_ERR_INVALID_ARG;
    if ((int64_t)kv->max_pages * page_size > kMaxPositions) return QLORA_ERR_SHAPE;
    const void *all[] = {ctx_len, q_len, free_pages, free_count, free_count_out, kv->block_table, kv->cu_q, kv->kv_len,
                         kv->positions, kv->slots};
    for (const void *a : all)
        if (!aligned16(a)) return QLORA_ERR_ALIGNMENT;
    DeviceInfo dev;
    QLORA_TRY(device_info(&dev));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    PlanParams p{ctx_len, q_len, free_pages, free_count, free_count_out, kv->block_table, kv->cu_q, kv->kv_len,
                 kv->positions, kv->slots, kv->batch, kv->max_pages, kv->tokens, num_pages, page_shift(page_size)};
    const size_t smem = 4 * ((size_t)kv->batch + 1) * 4;   // at most 65,552 bytes
    static PerDeviceOnce once;
    QLORA_TRY(once.run(dev.device, [] {
        QLORA_CUDA_TRY(cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            4 * (kMaxRequests + 1) * 4));
        return QLORA_OK;
    }));
    cudaLaunchConfig_t cfg{};
    const bool small = kv->tokens <= 512 && kv->batch <= 128;
    const int ctas = small ? 1 : 8;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(small ? 128 : 1024);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    {
        LaunchScope ls(QLORA_KERNEL_BLOCK, s);
        QLORA_CUDA_TRY(cudaLaunchKernelEx(&cfg, plan_kernel, p));
    }
    return launch_status();
}

extern "C" qlora_status qlora_kv_append(const qlora_kv_cache *cache, const qlora_kv_batch *kv, const qlora_rope *rope,
                                        const void *q, const void *k, const void *v, int32_t heads, void *q_out,
                                        void *stream)
{
    QLORA_TRY(check_cache(cache));
    QLORA_TRY(check_batch(kv));
    if (heads < 1 || heads > kMaxHeads || heads % cache->kv_heads) return QLORA_ERR_SHAPE;
    if (rope && rope->head_dim != cache->head_dim) return QLORA_ERR_SHAPE;
    if (!q || !k || !v || !q_out || !kv->slots || (rope && !kv->positions)) return QLORA_ERR_INVALID_ARG;
    const void *all[] = {q, k, v, q_out, kv->slots, kv->positions};
    for (const void *a : all)
        if (!aligned16(a)) return QLORA_ERR_ALIGNMENT;
    DeviceInfo dev;
    QLORA_TRY(device_info(&dev));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AppendParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.kc = static_cast<uint16_t *>(cache->k);
    p.vc = static_cast<uint16_t *>(cache->v);
    p.positions = kv->positions;
    p.slots = kv->slots;
    p.stride_page = cache->stride_page;
    p.stride_head = cache->stride_head;
    p.stride_token = cache->stride_token;
    p.tokens = kv->tokens;
    p.heads = heads;
    p.kv_heads = cache->kv_heads;
    p.head_dim = cache->head_dim;
    p.page_shift = page_shift(cache->page_size);
    p.num_pages = cache->num_pages;
    p.rotate = rope ? 1 : 0;
    if (rope)
        for (int i = 0; i < 64; i++) p.turns[i] = rope->turns[i];
    // as many tokens per block as leave two blocks for every SM; with few tokens, several blocks per token
    const int per_block = kAppendThreads / (cache->head_dim / 16);   // heads at once
    p.block_tokens = std::max(1, std::min(kAppendTokens, kv->tokens / (2 * dev.sms)));
    const int blocks = (kv->tokens + p.block_tokens - 1) / p.block_tokens;
    int split = std::max(1, 2 * dev.sms / blocks);
    split = std::min(split, (p.block_tokens * (heads + 2 * cache->kv_heads) + per_block - 1) / per_block);
    {
        LaunchScope ls(QLORA_KERNEL_BLOCK, s);
        const dim3 grid((unsigned)blocks, (unsigned)split);
        if (cache->dtype == QLORA_FP16)
            QLORA_CUDA_TRY(launch_pdl(append_kernel<true>, grid, dim3(kAppendThreads), 0, s, p));
        else
            QLORA_CUDA_TRY(launch_pdl(append_kernel<false>, grid, dim3(kAppendThreads), 0, s, p));
    }
    return launch_status();
}
