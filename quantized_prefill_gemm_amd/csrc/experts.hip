// Tokens to experts and back, for gfx950: a stable counting sort of T * top_k expert ids, the
// copy of token rows into sorted order and its gradient, the weighted sum back and its
// gradients. All of it is memory-bound; every sum runs in a fixed order, so results do not
// depend on scheduling.
//
// A slot is t * top_k + j, the j-th choice of token t. slots[slot] is its row in sorted order
// or -1 (its id is no expert of this call); order[row] is the slot back. Rows from
// offsets[E] on belong to no slot.
#include "qpg_mx.h"

namespace qpg {

// ---------------------------------------------------------------------------- sort

constexpr int SORT_WAVES = 16;
constexpr int SORT_THREADS = 64 * SORT_WAVES;
constexpr int SORT_MAX_E = 1024;          // one thread per expert in the scans

template <typename ID>
__device__ __forceinline__ int sort_key(const ID* ids, int64_t i, int64_t end, int E)
{
    if (i >= end) return E;
    const ID v = ids[i];
    return v >= 0 && v < (ID)E ? (int)v : E;
}

// counts[block][e]: ids equal to e in the block's part.
template <typename ID>
__global__ void __launch_bounds__(SORT_THREADS) sort_count_kernel(const ID* __restrict__ ids, int64_t S, int64_t part,
                                                                  int E, int32_t* __restrict__ counts)
{
    __shared__ int32_t n[SORT_MAX_E];
    const int tid = threadIdx.x;
    if (tid < E) n[tid] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * part, end = begin + part < S ? begin + part : S;
    for (int64_t i = begin + tid; i < end; i += SORT_THREADS) {
        const int key = sort_key(ids, i, end, E);
        if (key < E) atomicAdd(&n[key], 1);       // a count: the same in any order
    }
    __syncthreads();
    if (tid < E) counts[(int64_t)blockIdx.x * E + tid] = n[tid];
}

// Each block places its part of the slots, [begin, end), stably: wave v of the block takes the
// v-th piece of the part. A slot's row is (rows of smaller experts) + (rows of its expert in
// earlier blocks) + (in earlier waves of this block) + (earlier in its wave). The first two
// come from counts (with one block, from the block's own), the third from per-wave counts in
// LDS, the last from a ballot per bit of the id, which gives each lane the lanes that share it.
template <typename ID, int MAX_E>
__global__ void __launch_bounds__(SORT_THREADS) sort_place_kernel(const ID* __restrict__ ids, int64_t S, int64_t part,
                                                                  int E, int bits, const int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ order,
                                                                  int32_t* __restrict__ slots)
{
    __shared__ int32_t at[SORT_WAVES * MAX_E];    // [SORT_WAVES][E]: counts, then next rows
    __shared__ int32_t wave_sum[SORT_WAVES];
    __shared__ int32_t total_rows;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t begin = blockIdx.x * part, end = begin + part < S ? begin + part : S;
    const int64_t piece = (part + SORT_WAVES * 64 - 1) / (SORT_WAVES * 64) * 64;
    const int64_t wbegin = begin + wave * piece, wend = wbegin + piece < end ? wbegin + piece : end;

    for (int i = tid; i < SORT_WAVES * E; i += SORT_THREADS) at[i] = 0;
    __syncthreads();
    for (int64_t i = wbegin + lane; i < wend; i += 64) {
        const int key = sort_key(ids, i, wend, E);
        if (key < E) atomicAdd(&at[wave * E + key], 1);
    }
    __syncthreads();

    // thread e: rows of expert e in earlier blocks and in all blocks
    int before = 0, all = 0;
    if (tid < E) {
        if (gridDim.x == 1) {
            for (int v = 0; v < SORT_WAVES; ++v) all += at[v * E + tid];
        } else {
            for (unsigned b = 0; b < gridDim.x; ++b) {
                const int c = counts[(int64_t)b * E + tid];
                all += c;
                before += b < blockIdx.x ? c : 0;
            }
        }
    }
    int incl = all;                               // inclusive scan over the experts
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    for (int v = 0; v < wave; ++v) incl += wave_sum[v];
    if (tid == SORT_THREADS - 1) total_rows = incl;
    if (tid < E) {
        int row = incl - all;
        if (blockIdx.x == 0) {
            offsets[tid] = row;
            if (tid == E - 1) offsets[E] = incl;
        }
        row += before;
        for (int v = 0; v < SORT_WAVES; ++v) {
            const int c = at[v * E + tid];
            at[v * E + tid] = row;
            row += c;
        }
    }
    __syncthreads();

    for (int64_t i0 = wbegin; i0 < wend; i0 += 64) {
        const int64_t i = i0 + lane;
        const int key = sort_key(ids, i, wend, E);
        unsigned long long same = ~0ull;
        for (int b = 0; b < bits; ++b) {
            const unsigned long long m = __ballot((key >> b) & 1);
            same &= (key >> b) & 1 ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const int leader = __ffsll(same) - 1;
        int row = 0;
        if (key < E && lane == leader) row = atomicAdd(&at[wave * E + key], (int)__popcll(same));
        row = __shfl(row, leader) + rank;
        if (i < wend) {
            slots[i] = key < E ? row : -1;
            if (key < E) order[row] = (int32_t)i;
        }
    }
    const int64_t rows = total_rows;
    for (int64_t i = rows + (int64_t)blockIdx.x * SORT_THREADS + tid; i < S; i += (int64_t)gridDim.x * SORT_THREADS)
        order[i] = -1;
}

template <typename ID>
hipError_t launch_sort(const ID* ids, int64_t S, int E, int32_t* offsets, int32_t* order, int32_t* slots, int32_t* ws,
                       hipStream_t s)
{
    const int blocks = qpg_experts_sort_blocks(S);
    const int64_t part = (S + blocks - 1) / blocks;
    int bits = 1;
    while ((1 << bits) <= E) ++bits;              // the value E itself stands for "no expert"
    if (blocks > 1) {
        hipLaunchKernelGGL(sort_count_kernel<ID>, dim3(blocks), dim3(SORT_THREADS), 0, s, ids, S, part, E, ws);
        const hipError_t rc = hipGetLastError();
        if (rc != hipSuccess) return rc;
    }
    auto place = E <= 128 ? sort_place_kernel<ID, 128> : sort_place_kernel<ID, SORT_MAX_E>;
    hipLaunchKernelGGL(place, dim3(blocks), dim3(SORT_THREADS), 0, s, ids, S, part, E, bits, ws, offsets, order, slots);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------- rows

// A row of H values is cut into segments of 64 lanes * VEC * UNROLL values, one wave each: VEC
// values per access (16 bytes of the wider type where H and the pointers allow, else 1).
template <typename T, int VEC>
__device__ __forceinline__ void load_row(float (&f)[VEC], const T* p)
{
    const Pack<T, VEC> v = *reinterpret_cast<const Pack<T, VEC>*>(p);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = (float)v.v[i];
}
template <typename T, int VEC>
__device__ __forceinline__ void store_row(T* p, const float (&f)[VEC])
{
    Pack<T, VEC> v;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v.v[i] = (T)f[i];
    *reinterpret_cast<Pack<T, VEC>*>(p) = v;
}

// A slot's row, or -1 where it has none: a value outside [0, S) is treated as -1, so a wrong
// array never takes a kernel out of its buffers.
__device__ __forceinline__ int64_t slot_row(const int32_t* slots, int64_t slot, int64_t S)
{
    const int32_t r = slots[slot];
    return r >= 0 && r < S ? r : -1;
}

constexpr int ROW_UNROLL = 4;

// xs[slots[t][j]] = x[t]: a wave reads its segment of a token once and writes it top_k times.
// T here is only a width: the values are moved, not read.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) gather_kernel(const T* __restrict__ x, const int32_t* __restrict__ slots,
                                                     T* __restrict__ xs, int64_t tokens, int top_k, int64_t H,
                                                     int segs)
{
    typedef Pack<T, VEC> P;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t t = item / segs;
    if (t >= tokens) return;
    const int64_t h0 = (item - t * segs) * (64 * VEC * ROW_UNROLL) + (threadIdx.x & 63) * VEC;
    P v[ROW_UNROLL];
#pragma unroll
    for (int u = 0; u < ROW_UNROLL; ++u)
        if (h0 + u * 64 * VEC < H) v[u] = *reinterpret_cast<const P*>(x + t * H + h0 + u * 64 * VEC);
    for (int j = 0; j < top_k; ++j) {
        const int64_t row = slot_row(slots, t * top_k + j, tokens * top_k);
        if (row < 0) continue;
#pragma unroll
        for (int u = 0; u < ROW_UNROLL; ++u)
            if (h0 + u * 64 * VEC < H) *reinterpret_cast<P*>(xs + row * H + h0 + u * 64 * VEC) = v[u];
    }
}

// y[t] = sum over j of weights[t][j] * ys[slots[t][j]], in f32, j upwards; weights null: ones
// (the gradient of the gather).
template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(256) combine_kernel(const TI* __restrict__ ys, const int32_t* __restrict__ slots,
                                                      const float* __restrict__ weights, TO* __restrict__ y,
                                                      int64_t tokens, int top_k, int64_t H, int segs)
{
    constexpr int U = 2;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t t = item / segs;
    if (t >= tokens) return;
    const int64_t h0 = (item - t * segs) * (64 * VEC * U) + (threadIdx.x & 63) * VEC;
    float acc[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[u][i] = 0.f;
    for (int j = 0; j < top_k; ++j) {
        const int64_t row = slot_row(slots, t * top_k + j, tokens * top_k);
        if (row < 0) continue;
        const float w = weights ? weights[t * top_k + j] : 1.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (h0 + u * 64 * VEC >= H) continue;
            float f[VEC];
            load_row<TI, VEC>(f, ys + row * H + h0 + u * 64 * VEC);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[u][i] += w * f[i];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (h0 + u * 64 * VEC < H) store_row<TO, VEC>(y + t * H + h0 + u * 64 * VEC, acc[u]);
}

__device__ __forceinline__ float wave_sum64(float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Gradients of the weighted sum, one workgroup per token: dys[slots[t][j]] = weights[t][j] * dy[t],
// dweights[t][j] = <dy[t], ys[slots[t][j]]> (0 where the slot has no row). GRAD_SLOTS choices
// are taken together, so dy is read once per GRAD_SLOTS of them.
constexpr int GRAD_SLOTS = 8;

template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(256) combine_grad_kernel(const TO* __restrict__ dy, const TI* __restrict__ ys,
                                                           const int32_t* __restrict__ slots,
                                                           const float* __restrict__ weights, TI* __restrict__ dys,
                                                           float* __restrict__ dweights, int64_t tokens, int top_k,
                                                           int64_t H)
{
    __shared__ float part[4][GRAD_SLOTS];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j0 = 0; j0 < top_k; j0 += GRAD_SLOTS) {
        int64_t row[GRAD_SLOTS];
        float w[GRAD_SLOTS], dot[GRAD_SLOTS];
#pragma unroll
        for (int j = 0; j < GRAD_SLOTS; ++j) {
            row[j] = j0 + j < top_k ? slot_row(slots, t * top_k + j0 + j, tokens * top_k) : -1;
            w[j] = j0 + j < top_k ? weights[t * top_k + j0 + j] : 0.f;
            dot[j] = 0.f;
        }
        for (int64_t h = threadIdx.x * VEC; h < H; h += 256 * VEC) {
            float g[VEC];
            load_row<TO, VEC>(g, dy + t * H + h);
#pragma unroll
            for (int j = 0; j < GRAD_SLOTS; ++j) {
                if (row[j] < 0) continue;
                float f[VEC], o[VEC];
                load_row<TI, VEC>(f, ys + row[j] * H + h);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    dot[j] += g[i] * f[i];
                    o[i] = w[j] * g[i];
                }
                store_row<TI, VEC>(dys + row[j] * H + h, o);
            }
        }
#pragma unroll
        for (int j = 0; j < GRAD_SLOTS; ++j) {
            const float v = wave_sum64(dot[j]);
            if (lane == 0) part[wave][j] = v;
        }
        __syncthreads();
        if (threadIdx.x < GRAD_SLOTS && j0 + (int)threadIdx.x < top_k) {
            const int j = threadIdx.x;
            dweights[t * top_k + j0 + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
        }
        __syncthreads();
    }
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename F>
hipError_t by_types(int a, int b, F f)
{
    return qpg_by_type(a, [&](auto ta) { return qpg_by_type(b, [&](auto tb) { return f(ta, tb); }); });
}

}  // namespace qpg

// Blocks of the sort: one up to 8192 slots (a single launch), then one per 4096, at most 64.
int qpg_experts_sort_blocks(int64_t S)
{
    if (S <= 8192) return 1;
    const int64_t b = (S + 4095) / 4096;
    return (int)(b < 64 ? b : 64);
}

hipError_t qpg_launch_experts_sort(const void* ids, int id_bytes, int64_t S, int64_t E, int32_t* offsets,
                                   int32_t* order, int32_t* slots, void* ws, hipStream_t s)
{
    int32_t* counts = static_cast<int32_t*>(ws);
    if (id_bytes == 8)
        return qpg::launch_sort(static_cast<const int64_t*>(ids), S, (int)E, offsets, order, slots, counts, s);
    return qpg::launch_sort(static_cast<const int32_t*>(ids), S, (int)E, offsets, order, slots, counts, s);
}

hipError_t qpg_launch_experts_gather(const void* x, int type, const int32_t* slots, void* xs, int64_t T, int64_t top_k,
                                     int64_t H, hipStream_t s)
{
    auto go = [&](auto unit, auto vec) {
        typedef decltype(unit) U;
        constexpr int VEC = decltype(vec)::value;
        const int64_t n = H * (int64_t)qpg::type_bytes(type) / (int64_t)sizeof(U);
        const int segs = (int)((n + 64 * VEC * qpg::ROW_UNROLL - 1) / (64 * VEC * qpg::ROW_UNROLL));
        hipLaunchKernelGGL((qpg::gather_kernel<U, VEC>), dim3((unsigned)((T * segs + 3) / 4)), dim3(256), 0, s,
                           static_cast<const U*>(x), slots, static_cast<U*>(xs), T, (int)top_k, n, segs);
        return hipGetLastError();
    };
    const int64_t row = H * (int64_t)qpg::type_bytes(type);
    if (row % 16 == 0 && qpg::aligned16(x) && qpg::aligned16(xs)) return go(uint32_t(), std::integral_constant<int, 4>());
    if (type == QPG_F32) return go(uint32_t(), std::integral_constant<int, 1>());
    return go(uint16_t(), std::integral_constant<int, 1>());
}

hipError_t qpg_launch_experts_combine(const void* ys, int ys_type, const int32_t* slots, const float* weights, void* y,
                                      int y_type, int64_t T, int64_t top_k, int64_t H, hipStream_t s)
{
    return qpg::by_types(ys_type, y_type, [&](auto ti, auto to) {
        typedef typename qpg::Store<decltype(ti)::value>::type TI;
        typedef typename qpg::Store<decltype(to)::value>::type TO;
        auto go = [&](auto vec) {
            constexpr int VEC = decltype(vec)::value;
            const int segs = (int)((H + 64 * VEC * 2 - 1) / (64 * VEC * 2));
            hipLaunchKernelGGL((qpg::combine_kernel<TI, TO, VEC>), dim3((unsigned)((T * segs + 3) / 4)), dim3(256), 0,
                               s, static_cast<const TI*>(ys), slots, weights, static_cast<TO*>(y), T, (int)top_k, H,
                               segs);
            return hipGetLastError();
        };
        constexpr int V = 16 / (sizeof(TI) > sizeof(TO) ? sizeof(TI) : sizeof(TO));
        if (H % V == 0 && qpg::aligned16(ys) && qpg::aligned16(y)) return go(std::integral_constant<int, V>());
        return go(std::integral_constant<int, 1>());
    });
}

hipError_t qpg_launch_experts_combine_grad(const void* dy, int dy_type, const void* ys, int ys_type,
                                           const int32_t* slots, const float* weights, void* dys, float* dweights,
                                           int64_t T, int64_t top_k, int64_t H, hipStream_t s)
{
    return qpg::by_types(ys_type, dy_type, [&](auto ti, auto to) {
        typedef typename qpg::Store<decltype(ti)::value>::type TI;
        typedef typename qpg::Store<decltype(to)::value>::type TO;
        auto go = [&](auto vec) {
            constexpr int VEC = decltype(vec)::value;
            hipLaunchKernelGGL((qpg::combine_grad_kernel<TI, TO, VEC>), dim3((unsigned)T), dim3(256), 0, s,
                               static_cast<const TO*>(dy), static_cast<const TI*>(ys), slots, weights,
                               static_cast<TI*>(dys), dweights, T, (int)top_k, H);
            return hipGetLastError();
        };
        constexpr int V = 16 / (sizeof(TI) > sizeof(TO) ? sizeof(TI) : sizeof(TO));
        if (H % V == 0 && qpg::aligned16(ys) && qpg::aligned16(dys) && qpg::aligned16(dy))
            return go(std::integral_constant<int, V>());
        return go(std::integral_constant<int, 1>());
    });
}
