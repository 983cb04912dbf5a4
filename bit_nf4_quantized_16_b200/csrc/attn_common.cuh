// What the paged attention kernels share: the view of a planned batch, the
// schedule that every CTA derives from the requests' lengths on its own, and
// the layout of partial results.
//
// Work is cut into items: (request, key/value head, tile of ROWS query rows).
// The rows of an item are the new tokens of the request times the heads that
// share the key/value head, token-major: row r is token r / group, head
// kv_head * group + r % group.  An item's keys are walked in tiles of TILE
// positions; tiles that no row of the item can see are not part of it (after
// the causal diagonal; between the sinks and the window).
//
// Schedule: item i costs max(tiles_i, 1) + OV units, items are laid end to end in
// the order (request, head, row tile), and CTA c of G takes the units from
// floor(c W / G) to floor((c + 1) W / G).  Lengths are read on the device, so a
// call needs no copy to the host, can be captured in a graph, and balances
// requests of any mix of lengths.  A CTA whose part of an item is not the whole
// item writes a partial result (unnormalized output, running maximum, sum);
// a second kernel joins the parts in the order of their CTAs.  The cut depends
// on the lengths and the device alone, so results are bitwise reproducible.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "debug.cuh"
#include "sm100.cuh"

namespace qlora {
namespace attn {

struct BatchView {
    const int32_t *cu_q, *kv_len, *table;
    int batch, max_pages, tokens, num_pages, page_shift;
    int heads, kv_heads, group, head_dim;
    int window, sinks;   // window 0: every earlier position is visible
    int group_shift;     // group = 1 << group_shift, or -1

    __device__ __forceinline__ int token_of(int row) const { return group_shift >= 0 ? row >> group_shift : row / group; }
};

// A CTA's partial results: at most two, of its first item (slot 2c) and of its
// last (slot 2c + 1).  A slot holds ROWS x DP outputs (in the kernel of many rows
// four columns of all rows together, so that a warp of rows writes whole lines),
// ROWS references and ROWS sums, all fp32.
//
// References are scores: a weight is 2^((s - reference) * scale * log2 e).  The difference is
// formed first, and with the largest score as reference it is 0 for that one, exactly.  (A product
// rounded before the subtraction is off by up to half its step, which is 16 at 2^28: weights of 2^16 or
// 2^-16 where the largest has to be 1.)
//
// In fp16 all weights of a call carry a power of two more, 2^kRaise, which cancels in the quotient.
// Below 2^-14 fp16 has a fixed step of 2^-24, so that with weights of at most 1 the many small ones beside a
// key that takes nearly all weight would lose their bits (a key 2^20 above the others: 3 of 11
// left, none at 2^25); above 1 the type has room that costs nothing.  With few rows the reference is the
// largest score so far: 2^15.  With many rows it is the largest of the first tile, of whose 128
// keys the sum has to stay in range: 2^8.  A weight is then off by half a step or by
// 2^-40 (few rows) or 2^-33 (many) of the row's largest.  bf16 has the exponents of fp32.
struct Desc {
    int32_t q0, h;        // of the item: the request's first row, the key/value head,
    int32_t row0, rows;   // its first row in the request and how many it has
    int32_t first_slot;   // of the item's first part; the next ones are 2 (c + 1), 2 (c + 2), ...
    int32_t cta, parts;   // parts = 0: this CTA begins no split item
};

struct AttnParams {
    CUtensorMap tk, tv;   // caches as (dim, token in page, head, page), 128-byte swizzle
    BatchView v;
    const void *q;
    void *out;
    float *lse;           // [tokens][heads] or null
    float *part;
    Desc *desc;
    float scale_log2;     // softmax scale * log2 e
    int *err;
    uint64_t timeout_ns;
};

template <bool F16> constexpr int kRaiseFew = F16 ? 15 : 0;
template <bool F16> constexpr int kRaiseMany = F16 ? 8 : 0;

// log sum exp of a row from its reference and the sum of its weights.  A sum of 0 is that of a row that sees
// nothing: with a key of finite score the largest weight alone is at least 1.  NaN stays NaN.
template <int RAISE>
__device__ __forceinline__ float log_sum(float ref, float sum, float scale_log2)
{
    constexpr float kLower = 1.0f / (float)(1 << RAISE);
    return sum == 0.0f ? -INFINITY : __fmaf_rn(ref, scale_log2, log2f(sum * kLower)) * 0.69314718056f;
}

// What a row's output is multiplied with in the end.
__device__ __forceinline__ float inverse_sum(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }

struct Request {
    int q0, qn;   // rows of the batch's tensors [q0, q0 + qn)
    int kv;       // positions after this step
    int reach;    // positions that the block table can hold, at most kv
};

__device__ __forceinline__ Request load_request(const BatchView &v, int b)
{
    Request r;
    const int a = v.cu_q[b], e = v.cu_q[b + 1];
    r.q0 = min(max(a, 0), v.tokens);
    r.qn = min(max(e, r.q0), v.tokens) - r.q0;
    r.kv = min(max(v.kv_len[b], 0), 1 << 30);
    const int64_t cap = (int64_t)v.max_pages << v.page_shift;
    r.reach = (int)min((int64_t)r.kv, cap);
    return r;
}

// The tiles of one item: `sink_tiles` from the front, then [lo_tile, ...).
struct Tiles {
    int n, sink_tiles, lo_tile;
    __device__ __forceinline__ int at(int t) const { return t < sink_tiles ? t : lo_tile + t - sink_tiles; }
};

// Positions of the item's first and last row.
template <int ROWS>
__device__ __forceinline__ void item_positions(const BatchView &v, const Request &r, int rt, int &first, int &last)
{
    const int r0 = rt * ROWS, r1 = min(r.qn * v.group, r0 + ROWS) - 1;
    first = r.kv - r.qn + v.token_of(r0);
    last = r.kv - r.qn + v.token_of(r1);
}

template <int ROWS, int TILE>
__device__ __forceinline__ Tiles item_tiles(const BatchView &v, const Request &r, int rt)
{
    int first, last;
    item_positions<ROWS>(v, r, rt, first, last);
    Tiles t{0, 0, 0};
    const int hi = min(last + 1, r.reach);
    if (hi <= 0) return t;
    const int hi_tile = (hi + TILE - 1) / TILE;
    if (v.window > 0) {
        t.lo_tile = min(max(first - v.window + 1, 0) / TILE, hi_tile);
        t.sink_tiles = min((min(v.sinks, hi) + TILE - 1) / TILE, t.lo_tile);
    }
    t.n = t.sink_tiles + hi_tile - t.lo_tile;
    return t;
}

template <int ROWS>
__device__ __forceinline__ int row_tiles(const BatchView &v, const Request &r)
{
    return (int)(((int64_t)r.qn * v.group + ROWS - 1) / ROWS);
}

// Units of one key/value head of a request.
template <int ROWS, int TILE, int OV>
__device__ __forceinline__ int64_t head_units(const BatchView &v, const Request &r)
{
    int64_t u = 0;
    const int n = row_tiles<ROWS>(v, r);
    for (int rt = 0; rt < n; rt++) u += max(item_tiles<ROWS, TILE>(v, r, rt).n, 1) + OV;
    return u;
}

struct Item {
    int b, h, rt;
    Request r;
    Tiles tiles;
    int t0, t1;   // this CTA's tiles
    bool whole;   // all of the item
    bool begins;  // the item's first tile, but not its last, is here
    int64_t end;  // unit after the item's last
};

// Exclusive prefix of the units of NT runs of consecutive requests, in shared
// memory (pre[NT] = total; NT / 32 values more are scratch).  Called by all NT threads.
template <int NT, int ROWS, int TILE, int OV>
__device__ __forceinline__ void schedule_scan(const BatchView &v, int64_t *pre)
{
    int64_t *warp_sum = pre + NT + 1;
    const int tid = threadIdx.x, lane = tid & 31, run = (v.batch + NT - 1) / NT;
    int64_t mine = 0;
    if (ROWS > 16 && v.batch <= NT / 8) {   // few requests, maybe of many row tiles: a warp for each, its lanes take the tiles
        for (int b = tid >> 5; b < v.batch; b += NT / 32) {
            const Request r = load_request(v, b);
            const int n = row_tiles<ROWS>(v, r);
            int64_t u = 0;
            for (int rt = lane; rt < n; rt += 32) u += max(item_tiles<ROWS, TILE>(v, r, rt).n, 1) + OV;
#pragma unroll
            for (int o = 16; o; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
            if (lane == 0) pre[b] = v.kv_heads * u;
        }
        __syncthreads();
        if (tid < v.batch) mine = pre[tid];
        __syncthreads();
    } else {
        for (int b = tid * run; b < min((tid + 1) * run, v.batch); b++)
            mine += v.kv_heads * head_units<ROWS, TILE, OV>(v, load_request(v, b));
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) warp_sum[tid >> 5] = incl;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; w++) {
        if (w < (tid >> 5)) before += warp_sum[w];
        total += warp_sum[w];
    }
    pre[tid] = before + incl - mine;
    if (tid == 0) pre[NT] = total;
    __syncthreads();
}

// a / b of nonnegative numbers; 32-bit whenever they are (a 64-bit division takes some 250 cycles, and several of
// them stand before a CTA's first copy).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// The CTA that takes unit e - 1, of G that share W units; a CTA's first unit.
__device__ __forceinline__ int cta_of_last(int64_t e, int64_t G, int64_t W) { return (int)quotient(e * G - 1, W); }
__device__ __forceinline__ int64_t first_unit(int64_t cta, int64_t G, int64_t W) { return quotient(cta * W, G); }

// Walks a CTA's items.  Every lane of a warp runs it with the same values.
template <int NT, int ROWS, int TILE, int OV>
struct Walker {
    int64_t u, u1;        // units still to take
    int64_t start;        // first unit of the current item
    int b, h, rt, n_rt;
    Request r;

    __device__ __forceinline__ void init(const BatchView &v, const int64_t *pre, int64_t from, int64_t to)
    {
        u = from;
        u1 = to;
        if (u >= u1) return;
        int lo = 0, hi = NT;   // the last run that begins at or before `from`
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= from) lo = mid; else hi = mid;
        }
        const int lane = threadIdx.x & 31, run = (v.batch + NT - 1) / NT;
        int64_t per_head = 0;
        if (run == 1) {
            b = lo;
            start = pre[lo];
            per_head = quotient(pre[lo + 1] - start, v.kv_heads);
        } else {   // the request inside the run: 32 at a time, one per lane
            const int b_end = min((lo + 1) * run, v.batch);
            int64_t base = pre[lo];
            for (int b0 = lo * run; b0 < b_end; b0 += 32) {
                int64_t mine = 0;
                if (b0 + lane < b_end) mine = head_units<ROWS, TILE, OV>(v, load_request(v, b0 + lane));
                int64_t incl = v.kv_heads * mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += up;
                }
                const unsigned past = __ballot_sync(0xffffffffu, base + incl > from);
                if (past) {
                    const int l = __ffs(past) - 1;
                    b = b0 + l;
                    per_head = __shfl_sync(0xffffffffu, mine, l);
                    start = base + __shfl_sync(0xffffffffu, incl, l) - v.kv_heads * per_head;
                    break;
                }
                base += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        r = load_request(v, b);
        n_rt = row_tiles<ROWS>(v, r);
        h = (int)quotient(from - start, per_head);
        start += h * per_head;
        for (rt = 0;; rt += 32) {   // the row tile: 32 at a time (past the last one: cost 0)
            int incl = rt + lane < n_rt ? max(item_tiles<ROWS, TILE>(v, r, rt + lane).n, 1) + OV : 0;
            const int mine = incl;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            const unsigned past = __ballot_sync(0xffffffffu, start + incl > from);
            if (past) {
                const int l = __ffs(past) - 1;
                rt += l;
                start += __shfl_sync(0xffffffffu, incl - mine, l);
                break;
            }
            start += __shfl_sync(0xffffffffu, incl, 31);
            if (rt + 32 >= n_rt) break;   // not reached: `from` lies inside the head
        }
    }

    __device__ __forceinline__ void step(const BatchView &v, int64_t cost)
    {
        start += cost;
        if (++rt < n_rt) return;
        rt = 0;
        if (++h < v.kv_heads) return;
        h = 0;
        do {
            if (++b >= v.batch) {
                u = u1;
                start = u1;
                return;
            }
            r = load_request(v, b);
            n_rt = row_tiles<ROWS>(v, r);
        } while (n_rt == 0);
    }

    __device__ __forceinline__ bool next(const BatchView &v, Item &it)
    {
        while (u < u1 && start < u1) {
            const Tiles tl = item_tiles<ROWS, TILE>(v, r, rt);
            const int64_t cost = max(tl.n, 1) + OV, end = start + cost;
            const int64_t lo = max(u, start), hi = min(u1, end);
            it.b = b;
            it.h = h;
            it.rt = rt;
            it.r = r;
            it.tiles = tl;
            it.t0 = (int)min((int64_t)tl.n, max((int64_t)0, lo - start - OV));
            it.t1 = (int)min((int64_t)tl.n, max((int64_t)0, hi - start - OV));
            it.whole = it.t0 == 0 && hi == end;
            it.begins = it.t0 == 0 && it.t1 > 0 && !it.whole;
            it.end = end;
            u = hi;
            if (hi == end) step(v, cost);
            if (it.whole || it.t1 > it.t0) return true;
        }
        return false;
    }
};

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2, int c3)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
        "%6}], [%2];" ::"r"(sm100::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(sm100::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// The page that holds position `pos`, or -1: beyond the table, or not a page of the cache.
__device__ __forceinline__ int page_of(const BatchView &v, int b, int pos)
{
    const int i = pos >> v.page_shift;
    if (i >= v.max_pages || !QLORA_IN((int64_t)b * v.max_pages + i, (int64_t)v.batch * v.max_pages)) return -1;
    const int id = v.table[(int64_t)b * v.max_pages + i];
    return (unsigned)id < (unsigned)v.num_pages ? id : -1;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if (F16) {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if (F16) return __half22float2(*reinterpret_cast<__half2 *>(&w));
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&w));
}

}  // namespace attn
}  // namespace qlora
