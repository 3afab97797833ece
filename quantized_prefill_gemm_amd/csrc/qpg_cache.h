// Internal definitions shared by the kernels over a paged cache of keys and values (not part of the C ABI).
#pragma once

#include "qpg_mx.h"

namespace qpg {

typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The index arrays of a batch. They are read on the device: offsets are clamped to [0, T], lengths to
// [0, width * page], so a wrong array gives wrong rows, never an access outside the buffers.
struct CacheBatch {
    const int32_t* table;         // [B][width]: pages of a sequence
    const int32_t* lens;          // [B]: length with the new tokens
    const int32_t* offsets;       // [B + 1]: rows of the new tokens
    int B, width, T;

    __device__ __forceinline__ int offset(int b) const { return min(max(offsets[b], 0), T); }
};

// The largest i of [0, n) with f(i) <= u, for f that does not fall; 0 if there is none. The 64 lanes
// probe together: n <= 64 takes one round of loads, n <= 4096 two.
template <typename F>
__device__ __forceinline__ int last_not_above(int n, int64_t u, F f)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, end = n;
    while (end - lo > 1) {
        const int step = (end - lo + 63) >> 6;
        const int64_t at = lo + (int64_t)lane * step;
        const uint64_t hit = __ballot(at < end && f((int)at) <= u);
        const int last = hit ? 63 - __builtin_clzll(hit) : 0;
        lo = __builtin_amdgcn_readfirstlane(lo + last * step);
        end = min(end, lo + step);
    }
    return lo;
}

}  // namespace qpg

// Kernel launchers (arguments validated by the C ABI layer).
hipError_t qpg_launch_cache_append(const qpg_cache& cache, const qpg_batch& batch, const void* q, const void* k,
                                   const void* v, int type, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                   int64_t heads, const int32_t* positions, const float* freqs, int64_t rot, int adjacent,
                                   const float* q_norm, const float* k_norm, float eps, void* y, hipStream_t s);
// Number of pieces that the keys of a tile are split into (1: no workspace).
int qpg_cache_attention_splits(int64_t T, int64_t B, int64_t heads, int64_t kv, int64_t dim, int64_t length);
// Workgroups of the launch (less than 2^24), and its threads (less than 2^32).
int64_t qpg_cache_attention_grid(int64_t T, int64_t B, int64_t heads, int64_t kv, int64_t dim, int64_t length, int64_t* threads);
hipError_t qpg_launch_cache_attention(const qpg_cache& cache, const qpg_batch& batch, const qpg_scores& scores,
                                      const void* q, int64_t heads, const int64_t* tree, int64_t words,
                                      const int32_t* positions, void* y, int y_type, void* ws, hipStream_t s);
