// Attention of new tokens over a paged key/value cache: the entry point, the
// choice of kernel and the kernel that joins split items.  See attn_common.cuh
// for the schedule, attn_decode.cuh for the kernel of few rows.
#include <math.h>

#include <algorithm>

#include "attn_chunk.cuh"
#include "attn_decode.cuh"
#include "common.cuh"
#include "serve.cuh"

namespace qlora {
namespace attn {

// Joins the parts of one split item (block x: the CTA that begins it; block y:
// eight of its rows).  One to eight warps share a row, each taking every
// n-th part; parts are weighted by 2^((m_i - M) scale log2 e) and summed in a fixed order.
template <int ROWS, int DP, bool F16>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int V = DP / 32;   // columns per lane
    __shared__ float acc[8][DP];
    __shared__ float sum[8];
    sm100::pdl_wait();
    sm100::pdl_trigger();
    const BatchView &v = p.v;
    const Desc d = p.desc[blockIdx.x];
    if (d.parts == 0) return;
    const int row0 = blockIdx.y * 8, rows = min(d.rows - row0, 8);
    if (rows <= 0) return;
    const int rp = rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : 8, share = 8 / rp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = warp % rp, sp = warp / rp;
    constexpr int64_t kSlot = (int64_t)ROWS * DP + 2 * ROWS;
    auto slot = [&](int i) { return p.part + (i == 0 ? d.first_slot : 2 * (d.cta + i)) * kSlot; };
    float M = -INFINITY, L = 0.0f;
    float a[V];
#pragma unroll
    for (int k = 0; k < V; k++) a[k] = 0.0f;
    if (row < rows) {
        for (int i = lane; i < d.parts; i += 32) M = fmaxf(M, slot(i)[ROWS * DP + row0 + row]);
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll 4
        for (int i = sp; i < d.parts; i += share) {
            const float *s = slot(i);
            const float m = s[ROWS * DP + row0 + row];
            const float f = m == -INFINITY ? 0.0f : exp2f((m - M) * p.scale_log2);
            L += f * s[ROWS * DP + ROWS + row0 + row];
            const float *x = s + (row0 + row) * DP + lane * V;
#pragma unroll
            for (int k = 0; k < V; k++) a[k] += f * x[k];
        }
    }
    if (share > 1) {
#pragma unroll
        for (int k = 0; k < V; k++) acc[warp][lane * V + k] = a[k];
        if (lane == 0) sum[warp] = L;
        __syncthreads();
        if (sp > 0) return;
        for (int w = warp + rp; w < 8; w += rp) {
            L += sum[w];
#pragma unroll
            for (int k = 0; k < V; k++) a[k] += acc[w][lane * V + k];
        }
    }
    if (row >= rows) return;
    const float inv = inverse_sum(L);
    const int g = d.row0 + row0 + row, tok = v.token_of(g);
    const int64_t orow = (int64_t)(d.q0 + tok) * v.heads + d.h * v.group + g - tok * v.group;
    const int64_t at = orow * v.head_dim + lane * V;
    if (lane * V < v.head_dim && QLORA_IN(at + V - 1, (int64_t)v.tokens * v.heads * v.head_dim)) {
        uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + at);
#pragma unroll
        for (int k = 0; k < V / 2; k++) o[k] = pack2<F16>(a[2 * k] * inv, a[2 * k + 1] * inv);
    }
    if (lane == 0 && p.lse) p.lse[orow] = log_sum<kRaiseFew<F16>>(M, L, p.scale_log2);
}

// The same for the items of the kernel of many rows: block y takes 32 rows, one
// per lane; its warps divide the columns, which the parts hold four by four for
// all rows.  The joined rows pass through shared memory, so that they leave
// as whole lines.
template <int DP, bool F16>
__global__ void __launch_bounds__(256) combine_rows_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int ROWS = ChunkCfg<DP>::kRows;
    __shared__ uint2 rows_out[32][DP / 4 + 1];
    sm100::pdl_wait();
    sm100::pdl_trigger();
    const BatchView &v = p.v;
    const Desc d = p.desc[blockIdx.x];
    if (d.parts == 0) return;
    const int row0 = blockIdx.y * 32, rows = min(d.rows - row0, 32);
    if (rows <= 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int64_t kSlot = ChunkCfg<DP>::kSlotFloats;
    auto slot = [&](int i) { return p.part + (i == 0 ? d.first_slot : 2 * (d.cta + i)) * kSlot; };
    auto tensor_row = [&](int row) {
        const int g = d.row0 + row0 + row, t = v.token_of(g);
        return (int64_t)(d.q0 + t) * v.heads + d.h * v.group + g - t * v.group;
    };
    if (lane < rows) {
        float M = -INFINITY, L = 0.0f;
        for (int i = 0; i < d.parts; i++) M = fmaxf(M, slot(i)[ROWS * DP + row0 + lane]);
        float4 a[DP / 32];
#pragma unroll
        for (int k = 0; k < DP / 32; k++) a[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
        for (int i = 0; i < d.parts; i++) {
            const float *s = slot(i) + row0 + lane;
            const float m = s[ROWS * DP], f = m == -INFINITY ? 0.0f : exp2f((m - M) * p.scale_log2);
            L += f * s[ROWS * DP + ROWS];
#pragma unroll
            for (int k = 0; k < DP / 32; k++) {
                const float4 x = *reinterpret_cast<const float4 *>(slot(i) + ((8 * k + warp) * ROWS + row0 + lane) * 4);
                a[k].x += f * x.x;
                a[k].y += f * x.y;
                a[k].z += f * x.z;
                a[k].w += f * x.w;
            }
        }
        const float inv = inverse_sum(L);
#pragma unroll
        for (int k = 0; k < DP / 32; k++)
            rows_out[lane][8 * k + warp] = make_uint2(pack2<F16>(a[k].x * inv, a[k].y * inv), pack2<F16>(a[k].z * inv, a[k].w * inv));
        if (warp == 0 && p.lse) p.lse[tensor_row(lane)] = log_sum<kRaiseMany<F16>>(M, L, p.scale_log2);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (DP / 4); i += 256) {
        const int row = i / (DP / 4), c = i % (DP / 4);
        const int64_t at = tensor_row(row) * v.head_dim + 4 * c;
        if (4 * c < v.head_dim && QLORA_IN(at + 3, (int64_t)v.tokens * v.heads * v.head_dim))
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) = rows_out[row][c];
    }
}

namespace {

int log2_of(int32_t n)   // -1 if n is no power of two
{
    return n & (n - 1) ? -1 : page_shift(n);
}

constexpr uint64_t kTimeoutNs = 2000000000ull;

// CTAs of the kernel for few rows: two per SM.
int decode_grid(const DeviceInfo &d) { return 2 * d.sms; }

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

// CTAs per key/value head of the cluster form, or 0: not used.  The form gives
// every head of every request the same number of CTAs, whatever the lengths are (the
// host does not know them).  It saves 4 to 6 us a call where the requests are alike (500
// positions of one request with 32 heads: 6.8 us for 11.2; 30000: 77 for 83) and loses
// where one is much longer than the others.  So it is taken for one request alone that
// fills the device, and otherwise where a CTA reads few positions: at most kOpen, or
// under a window kWindowed.  Its time over that of the schedule, by positions a CTA at most,
// measured with 32, 16, 8 and 4 requests of 8 heads of 128 (256 of 296 places taken):
//   positions                          320         640         960         1280        2560
//   no window, all alike            .71 to .77  .77 to .82  .84 to .86  .86 to .89  .89 to .93
//   no window, spread evenly        .73 to .82  .83 to .91  .91 to 1.1  .97 to 1.1  1.1 to 1.2
//   no window, one long, others 5%  .72 to .83  .89 to 1.1  1.0 to 1.4  1.1 to 1.7  1.5 to 2.4
//   positions of the window            256         512        1024        1280        2048        4096
//   all contexts beyond it          .73 to .80  .79 to .83  .86 to .88  .85 to .90  .92 to .94  .93 to .95
// With half the places taken (2 requests) the last line is .76, .89, .98, 1.04 and 1.13 up to 2048.  A
// window evens lengths out only where contexts exceed it: with one long request and short
// others the third line holds for it too.
constexpr int64_t kWindowed = 1280, kOpen = 640;
int cluster_ctas(const AttnParams &p, const DeviceInfo &dev)
{
    const int64_t items = (int64_t)p.v.batch * p.v.kv_heads;
    int n = 8;
    while (n && n * items > decode_grid(dev)) n /= 2;
    if (!n) return 0;
    if (p.v.batch == 1 && n * items >= decode_grid(dev) / 2) return n;
    const int64_t table = (int64_t)p.v.max_pages << p.v.page_shift;   // positions of a request, at most
    const bool few = table <= kOpen * n || (p.v.window > 0 && (int64_t)p.v.window + p.v.sinks <= kWindowed * n);
    return few ? n : 0;
}

template <int DP, bool F16>
qlora_status launch_decode(AttnParams &p, const DeviceInfo &dev, cudaStream_t s)
{
    using C = DecodeCfg<DP>;
    static PerDeviceOnce once;
    QLORA_TRY(once.run(dev.device, [] {
        QLORA_CUDA_TRY(cudaFuncSetAttribute(decode_kernel<DP, F16, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            C::kBytes));
        QLORA_CUDA_TRY(cudaFuncSetAttribute(decode_kernel<DP, F16, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            C::kBytes));
        return QLORA_OK;
    }));
    if (const int n = cluster_ctas(p, dev)) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(n * p.v.batch * p.v.kv_heads);
        cfg.blockDim = dim3(C::kThreads);
        cfg.dynamicSmemBytes = C::kBytes;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {(unsigned)n, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        LaunchScope ls(QLORA_KERNEL_ATTENTION, s);
        QLORA_CUDA_TRY(cudaLaunchKernelEx(&cfg, decode_kernel<DP, F16, true>, p));
        return launch_status();
    }
    const int grid = decode_grid(dev);
    {
        LaunchScope ls(QLORA_KERNEL_ATTENTION, s);
        QLORA_CUDA_TRY(launch_pdl(decode_kernel<DP, F16, false>, dim3(grid), dim3(C::kThreads), C::kBytes, s, p));
    }
    {
        LaunchScope ls(QLORA_KERNEL_ATTENTION, s);
        QLORA_CUDA_TRY(launch_pdl(combine_kernel<C::kRows, DP, F16>, dim3(grid, C::kRows / 8), dim3(256), 0, s, p));
    }
    return launch_status();
}

template <int DP, bool F16>
qlora_status launch_chunk(AttnParams &p, const DeviceInfo &dev, cudaStream_t s)
{
    using C = ChunkCfg<DP>;
    static PerDeviceOnce once;
    QLORA_TRY(once.run(dev.device, [] {
        QLORA_CUDA_TRY(cudaFuncSetAttribute(chunk_kernel<DP, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            C::kBytes));
        return QLORA_OK;
    }));
    {
        LaunchScope ls(QLORA_KERNEL_ATTENTION, s);
        QLORA_CUDA_TRY(launch_pdl(chunk_kernel<DP, F16>, dim3(dev.sms), dim3(C::kThreads), C::kBytes, s, p));
    }
    {
        LaunchScope ls(QLORA_KERNEL_ATTENTION, s);
        QLORA_CUDA_TRY(launch_pdl(combine_rows_kernel<DP, F16>, dim3(dev.sms, C::kRows / 32), dim3(256), 0, s, p));
    }
    return launch_status();
}

// More than one tile of 16 rows per key/value head: the kernel of many rows.
bool many_rows(const qlora_kv_batch *kv, int group)
{
    const int64_t q = kv->max_q_len ? std::min(kv->max_q_len, kv->tokens) : kv->tokens;
    return q * group > 16;
}

qlora_status check_attn(const qlora_kv_cache *c, const qlora_kv_batch *kv, int32_t heads)
{
    QLORA_TRY(check_cache(c));
    QLORA_TRY(check_batch(kv));
    if (heads < 1 || heads > kMaxHeads || heads % c->kv_heads) return QLORA_ERR_SHAPE;
    if ((int64_t)kv->max_pages * c->page_size > kMaxPositions || (int64_t)kv->tokens * heads > kMaxPositions)
        return QLORA_ERR_SHAPE;
    return QLORA_OK;
}

size_t workspace_bytes_for(const qlora_kv_cache *c, const qlora_kv_batch *kv, int32_t heads, const DeviceInfo &dev)
{
    const bool wide = c->head_dim > 64, many = many_rows(kv, heads / c->kv_heads);
    const int grid = many ? dev.sms : decode_grid(dev);
    const size_t slot = 4 * (size_t)(many ? (wide ? ChunkCfg<128>::kSlotFloats : ChunkCfg<64>::kSlotFloats)
                                          : (wide ? DecodeCfg<128>::kSlotFloats : DecodeCfg<64>::kSlotFloats));
    return round_up(decode_grid(dev) * sizeof(Desc)) + round_up(2 * grid * slot);
}

}  // namespace
}  // namespace attn
}  // namespace qlora

using namespace qlora;
using namespace qlora::attn;

extern "C" size_t qlora_paged_attn_workspace_bytes(const qlora_kv_cache *cache, const qlora_kv_batch *kv, int32_t heads)
{
    DeviceInfo dev;
    if (check_attn(cache, kv, heads) != QLORA_OK || device_info(&dev) != QLORA_OK) return 0;
    return workspace_bytes_for(cache, kv, heads, dev);
}

extern "C" qlora_status qlora_paged_attn_fwd(const qlora_kv_cache *cache, const qlora_kv_batch *kv, const void *q,
                                             int32_t heads, float scale, int32_t window, int32_t sinks, void *out,
                                             float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    QLORA_TRY(check_attn(cache, kv, heads));
    if (!q || !out || !workspace || !kv->block_table || !kv->cu_q || !kv->kv_len) return QLORA_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !isfinite(scale) || window < 0 || sinks < 0) return QLORA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || (lse && !aligned16(lse)) || !aligned16(workspace) ||
        !aligned16(kv->block_table) || !aligned16(kv->cu_q) || !aligned16(kv->kv_len))
        return QLORA_ERR_ALIGNMENT;
    DeviceInfo dev;
    QLORA_TRY(device_info(&dev));
    if (workspace_bytes < workspace_bytes_for(cache, kv, heads, dev)) return QLORA_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AttnParams p{};
    const bool many = many_rows(kv, heads / cache->kv_heads);
    const uint32_t box = many ? std::min(cache->page_size, 128) : 16;
    QLORA_TRY(make_cache_map(&p.tk, cache, cache->k, box));
    QLORA_TRY(make_cache_map(&p.tv, cache, cache->v, box));
    p.v = BatchView{kv->cu_q, kv->kv_len, kv->block_table, kv->batch, kv->max_pages, kv->tokens, cache->num_pages,
                    log2_of(cache->page_size), heads, cache->kv_heads, heads / cache->kv_heads, cache->head_dim,
                    window >= kMaxPositions ? 0 : window, std::min(sinks, (int32_t)kMaxPositions),
                    log2_of(heads / cache->kv_heads)};
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.desc = static_cast<Desc *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + round_up(decode_grid(dev) * sizeof(Desc)));
    p.scale_log2 = scale * 1.44269504089f;
    p.err = device_error_word();
    if (!p.err) return QLORA_ERR_CUDA;
    p.timeout_ns = kTimeoutNs;
    const bool f16 = cache->dtype == QLORA_FP16;
    if (many) {
        if (cache->head_dim <= 64)
            return f16 ? launch_chunk<64, true>(p, dev, s) : launch_chunk<64, false>(p, dev, s);
        return f16 ? launch_chunk<128, true>(p, dev, s) : launch_chunk<128, false>(p, dev, s);
    }
    if (cache->head_dim <= 64)
        return f16 ? launch_decode<64, true>(p, dev, s) : launch_decode<64, false>(p, dev, s);
    return f16 ? launch_decode<128, true>(p, dev, s) : launch_decode<128, false>(p, dev, s);
}
