// New tokens' queries, keys and values: norm of each head, rotation by position, the rows of the
// paged cache (include/qpg.h, cache_append).
//
//   x' = x * rsqrt(mean(x^2) + eps) * w;   (a, b) -> (a cos - b sin, a sin + b cos), angle = position * freq
//
// One pass: every value is read once and written once, where it belongs. A head is taken by a group
// of lanes, eight values a lane: both halves of four pairs (values 4u .. 4u + 3 and their partners half a
// rotation further), or four adjacent pairs, or eight values that are not rotated. The place in the
// head is the lane's for all heads, so a lane has its four angles, and its eight weights, for the whole
// token. Angles reach 1e6 and more, where f32 has no fraction left: the product with the
// frequency is made in 64 bits, in turns, and its fraction goes to f32's sine and cosine.
//
// Bound by memory: 7622 tokens of 32 + 2 * 8 heads of 128, bf16, normed 39.9 us, 4.7 TB/s; 1024 tokens of 96 heads f32 to
// f16 14.7 us, 5.1 TB/s. A few tokens are bound by the loads that find their place, one round behind the
// other: one token 3.5 us. Weights read one by one instead of by four cost 49 us there, adjacent pairs 72.
#include "qpg_cache.h"

namespace qpg {

struct AppendArgs {
    CacheBatch batch;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    void *y, *kc, *vc;
    int64_t k_page, v_page;       // elements from page to page
    int pages, page_bits, dim, heads, kv, rot, lane_bits, per;
    const int32_t* positions;
    const float *freqs, *q_norm, *k_norm;
    float eps;
};

// Four values at p, as f32. VEC: p is aligned to all four.
template <bool VEC, typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[8], int at)
{
    if constexpr (VEC) {
        const Pack<T, 4> x = *reinterpret_cast<const Pack<T, 4>*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[at + i] = (float)x.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[at + i] = (float)p[i];
    }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&f)[8], int at)
{
    Pack<T, 4> x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = (T)f[at + i];            // the one rounding, to nearest even
    *reinterpret_cast<Pack<T, 4>*>(p) = x;
}

constexpr int HEADS_AT_ONCE = 3;   // a lane's loads of so many heads are under way together

// The sum over aligned groups of 2^bits lanes, in all of them. A step's partner holds the other half's sum whichever of
// its lanes it is, so mirrors do for exchanges.
__device__ __forceinline__ float group_sum(float x, int bits)
{
    auto with = [](float v, auto how) {
        return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(how)::value, 0xF, 0xF, false));
    };
    if (bits > 0) x = with(x, std::integral_constant<int, 0xB1>());        // lane ^ 1
    if (bits > 1) x = with(x, std::integral_constant<int, 0x4E>());        // lane ^ 2
    if (bits > 2) x = with(x, std::integral_constant<int, 0x141>());       // mirrored in eight lanes
    if (bits > 3) x = with(x, std::integral_constant<int, 0x140>());       // mirrored in sixteen
    if (bits > 4) x += __shfl_xor(x, 16);
    return x;
}

// 1 / sqrt(x), to a step; x is scaled to where the instruction takes it (it has no subnormal numbers).
__device__ __forceinline__ float inverse_root(float x)
{
    const bool tiny = x < 0x1p-100f;
    return __builtin_amdgcn_rsqf(tiny ? x * 0x1p80f : x) * (tiny ? 0x1p40f : 1.0f);
}

template <typename TI, typename TC, bool VEC, bool ADJACENT, bool NORM>
__global__ void __launch_bounds__(256) cache_append_kernel(AppendArgs a)
{
    const int t = blockIdx.x, lanes = 1 << a.lane_bits;
    const int u = threadIdx.x & (lanes - 1), group = threadIdx.x >> a.lane_bits, groups = 256 >> a.lane_bits;
    const int first = blockIdx.y * a.per, all = a.heads + 2 * a.kv, end = min(first + a.per, all);
    const bool on = 8 * u < a.dim;

    // where the lane's two fours are in a head, and whether they are rotated
    const bool turn = 8 * u < a.rot, split = turn && !ADJACENT;
    const int o0 = split ? 4 * u : 8 * u, o1 = split ? 4 * u + a.rot / 2 : 8 * u + 4;
    const TI* q = static_cast<const TI*>(a.q) + t * a.q_stride;
    const TI* k = static_cast<const TI*>(a.k) + t * a.k_stride;
    const TI* v = static_cast<const TI*>(a.v) + t * a.v_stride;

    float x[HEADS_AT_ONCE][8];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < HEADS_AT_ONCE; ++i) {
            const int h = h0 + i * groups;
            const TI* p = h < a.heads ? q + (int64_t)h * a.dim
                        : h < a.heads + a.kv ? k + (int64_t)(h - a.heads) * a.dim : v + (int64_t)(h - a.heads - a.kv) * a.dim;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = 0.0f;
            if (on && h < end) {
                load4<VEC>(p + o0, x[i], 0);
                load4<VEC>(p + o1, x[i], 4);
            }
        }
    };
    load(first + group);           // under way while the place is looked up

    // The token's sequence, its numbers with those it is found by where there are few.
    int b = 0, row0, row1, length;
    if (a.batch.B < 64) {
        const int lane = threadIdx.x & 63;
        const int at = min(max(a.batch.offsets[min(lane, a.batch.B)], 0), a.batch.T), long_ = a.batch.lens[min(lane, a.batch.B - 1)];
        const uint64_t hit = __ballot(lane < a.batch.B && at <= t);
        b = hit ? 63 - __builtin_clzll(hit) : 0;
        row0 = __builtin_amdgcn_readlane(at, b);
        row1 = __builtin_amdgcn_readlane(at, b + 1);
        length = __builtin_amdgcn_readlane(long_, b);
    } else {
        b = last_not_above(a.batch.B, t, [&](int i) { return a.batch.offset(i); });
        row0 = a.batch.offset(b);
        row1 = a.batch.offset(b + 1);
        length = a.batch.lens[b];
    }
    if (t < row0 || t >= row1) return;                 // of no sequence
    const int64_t most = (int64_t)a.batch.width << a.page_bits;
    const int64_t place = min((int64_t)max(length, 0), most) - (row1 - t);
    int page = -1;
    if (place >= 0 && place < most) page = a.batch.table[(int64_t)b * a.batch.width + (place >> a.page_bits)];
    const bool kept = page >= 0 && page < a.pages;
    const int64_t in_page = place & ((1 << a.page_bits) - 1);
    TC* kc = static_cast<TC*>(a.kc) + page * a.k_page + in_page * a.dim;
    TC* vc = static_cast<TC*>(a.vc) + page * a.v_page + in_page * a.dim;

    float c[4], s[4], wq[8], wk[8];
    if (turn) {
        const double position = a.positions ? (double)a.positions[t] : (double)place;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            double turns = position * (double)a.freqs[4 * u + i] * 0.15915494309189533577;      // 1 / (2 pi)
            turns -= rint(turns);
            sincospif((float)(2.0 * turns), &s[i], &c[i]);
        }
    }
    if (NORM) {
#pragma unroll
        for (int i = 0; i < 8; ++i) wq[i] = wk[i] = 1.0f;
        if (on && a.q_norm) {
            load4<VEC>(a.q_norm + o0, wq, 0);
            load4<VEC>(a.q_norm + o1, wq, 4);
        }
        if (on && a.k_norm) {
            load4<VEC>(a.k_norm + o0, wk, 0);
            load4<VEC>(a.k_norm + o1, wk, 4);
        }
    }
    const float share = 1.0f / (float)a.dim;

    for (int h0 = first + group; h0 < end; h0 += HEADS_AT_ONCE * groups) {
#pragma unroll
        for (int i = 0; i < HEADS_AT_ONCE; ++i) {
            const int h = h0 + i * groups;
            const bool is_q = h < a.heads, is_k = !is_q && h < a.heads + a.kv;
            float (&f)[8] = x[i];
            if (NORM) {                                // by all lanes: the sum's exchanges are of whole groups
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += f[j] * f[j];
                const float r = inverse_root(group_sum(sum, a.lane_bits) * share + a.eps);
                if ((is_q && a.q_norm) || (is_k && a.k_norm)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] *= r * (is_q ? wq[j] : wk[j]);
                }
            }
            if (turn && (is_q || is_k)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float &p = f[ADJACENT ? 2 * j : j], &q2 = f[ADJACENT ? 2 * j + 1 : j + 4];
                    const float p1 = p * c[j] - q2 * s[j], q1 = p * s[j] + q2 * c[j];
                    p = p1;
                    q2 = q1;
                }
            }
            if (!on || h >= end || (!is_q && !kept)) continue;
            TC* to = is_q ? static_cast<TC*>(a.y) + ((int64_t)t * a.heads + h) * a.dim
                   : is_k ? kc + ((int64_t)(h - a.heads) << a.page_bits) * a.dim
                          : vc + ((int64_t)(h - a.heads - a.kv) << a.page_bits) * a.dim;
            store4(to + o0, f, 0);
            store4(to + o1, f, 4);
        }
        load(h0 + HEADS_AT_ONCE * groups);
    }
}

}  // namespace qpg

hipError_t qpg_launch_cache_append(const qpg_cache& cache, const qpg_batch& batch, const void* q, const void* k,
                                   const void* v, int type, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                   int64_t heads, const int32_t* positions, const float* freqs, int64_t rot, int adjacent,
                                   const float* q_norm, const float* k_norm, float eps, void* y, hipStream_t s)
{
    using namespace qpg;
    int lane_bits = 0, page_bits = 0;
    while ((8 << lane_bits) < cache.dim) ++lane_bits;
    while ((1 << page_bits) < cache.page) ++page_bits;
    const int64_t all = heads + 2 * cache.heads, groups = 256 >> lane_bits;
    // A workgroup takes all heads of a token where there are tokens enough to fill the card, and
    // as few as its lanes hold at once where there are few.
    int64_t parts = (all + groups - 1) / groups;
    if (batch.T * parts > 2048) parts = batch.T >= 2048 ? 1 : (2048 + batch.T - 1) / batch.T;
    const int64_t per = ((all + parts - 1) / parts + groups - 1) / groups * groups;
    const size_t unit = 4 * type_bytes(type);
    auto fits = [&](const void* p, int64_t stride) {
        return (uintptr_t)p % unit == 0 && (size_t)stride * type_bytes(type) % unit == 0;
    };
    // accesses of four values, the weights' among them: else one by one
    const bool vec = (!heads || fits(q, q_stride)) && fits(k, k_stride) && fits(v, v_stride) && (uintptr_t)q_norm % 16 == 0 &&
                     (uintptr_t)k_norm % 16 == 0;
    const AppendArgs a = {{batch.table, batch.lens, batch.offsets, (int)batch.B, (int)batch.width, (int)batch.T},
                          q, k, v, q_stride, k_stride, v_stride, y, cache.k, cache.v, cache.k_stride, cache.v_stride,
                          (int)cache.pages, page_bits, (int)cache.dim, (int)heads, (int)cache.heads, (int)rot,
                          lane_bits, (int)per, positions, freqs, q_norm, k_norm, eps};
    const dim3 grid((unsigned)batch.T, (unsigned)((all + per - 1) / per));
    return qpg_by_type(type, [&](auto ti) {
        typedef typename Store<decltype(ti)::value>::type TI;
        auto run = [&](auto tc) {
            typedef typename Store<decltype(tc)::value>::type TC;
            auto go = [&](auto adj, auto norm) {
                constexpr bool A = decltype(adj)::value, N = decltype(norm)::value;
                if (vec)
                    hipLaunchKernelGGL((cache_append_kernel<TI, TC, true, A, N>), grid, dim3(256), 0, s, a);
                else
                    hipLaunchKernelGGL((cache_append_kernel<TI, TC, false, A, N>), grid, dim3(256), 0, s, a);
                return hipGetLastError();
            };
            const bool norm = q_norm || k_norm;
            if (adjacent) return norm ? go(std::true_type(), std::true_type()) : go(std::true_type(), std::false_type());
            return norm ? go(std::false_type(), std::true_type()) : go(std::false_type(), std::false_type());
        };
        return cache.type == QPG_F16 ? run(std::integral_constant<int, QPG_F16>()) : run(std::integral_constant<int, QPG_BF16>());
    });
}
