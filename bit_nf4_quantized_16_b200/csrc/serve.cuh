// Host-side checks and tensor maps that the serving entry points share.
#pragma once
#include "common.cuh"

namespace qlora {

constexpr int kMaxRequests = 4096;
constexpr int kMaxHeads = 1024;
constexpr int64_t kMaxPositions = 1 << 30;   // positions of a request, rows of a step: sums of two stay in 32 bits

// Checks of the plain fields; each entry point checks the arrays that it uses.
qlora_status check_cache(const qlora_kv_cache *c);
qlora_status check_batch(const qlora_kv_batch *kv);
qlora_status check_pages(int32_t page_size, int32_t num_pages);

inline int page_shift(int32_t page_size)
{
    int s = 0;
    while ((1 << s) < page_size) s++;
    return s;
}

// Tensor map of a cache as (dim, token in page, head, page); box 64 x `rows` x 1 x 1,
// 128-byte swizzle.  Coordinates past head_dim read zeros.
qlora_status make_cache_map(CUtensorMap *m, const qlora_kv_cache *c, const void *base, uint32_t rows);

// Common 4-D tensor map encoder (api.cu): strides in bytes of dimensions 1..3.
qlora_status make_map_4d(CUtensorMap *m, CUtensorMapDataType dt, const void *base, const uint64_t dims[4],
                         const uint64_t strides[3], const uint32_t box[4], CUtensorMapSwizzle sw);

}  // namespace qlora
