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
#pragma unroll
            for (int v = 0; v < SORT_WAVES; ++v) all += at[v * E + tid];
        } else {
#pragma unroll 16
            for (unsigned b = 0; b < gridDim.x; ++b) {       // 16 loads under way
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

// Rows are read and written through buffer descriptors that end with the row: a lane past its
// end reads zeros and writes nothing, and a slot without a row has an empty one. So there is
// no branch around an access, and all loads of a wave are under way together (with branches the
// compiler waits for each: the weighted sum of 268 MB took 84 us). VEC values per access: 16
// bytes of the wider type where H and the pointers allow, else 1 (4096 x 4 rows in us, gather /
// weighted sum / its gradients: of 8192 bytes f16 27 / 27 / 49, of 8196 67 / 48 / 91; of 16384 bytes f32 54 / 51 /
// 116, of 16388 93 / 51 / 174).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* p, int64_t row, int64_t H, int bytes)
{
    const char* at = static_cast<const char*>(p) + (row < 0 ? 0 : row * H * bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), 0, row < 0 ? 0 : (int)(H * bytes), 0x00020000);
}

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_row(__amdgpu_buffer_rsrc_t r, unsigned h)
{
    constexpr int BYTES = sizeof(T) * VEC;
    const int off = (int)(h * (unsigned)sizeof(T));
    if constexpr (BYTES == 16)
        return __builtin_bit_cast(Pack<T, VEC>, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
    else if constexpr (BYTES == 8)
        return __builtin_bit_cast(Pack<T, VEC>, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
    else if constexpr (BYTES == 4)
        return __builtin_bit_cast(Pack<T, VEC>, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
    else
        return __builtin_bit_cast(Pack<T, VEC>, __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
}
// Stores are non-temporal: the rows are not read again here, and ordinary ones push the rows
// being read out of the caches (gather and gradient, 8192 x 4 rows of 8 KB: 158 -> 138 us; weighted
// sum and gradients, 4096 x 8: 177 -> 149 us. Non-temporal loads as well: 135 and 161 us).
template <typename T, int VEC>
__device__ __forceinline__ void store_row(__amdgpu_buffer_rsrc_t r, unsigned h, const Pack<T, VEC>& v)
{
    constexpr int BYTES = sizeof(T) * VEC;
    const int off = (int)(h * (unsigned)sizeof(T));
    if constexpr (BYTES == 16)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uint32x4, v), r, off, 0, NONTEMPORAL);
    else if constexpr (BYTES == 8)
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(uint32x2, v), r, off, 0, NONTEMPORAL);
    else if constexpr (BYTES == 4)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, off, 0, NONTEMPORAL);
    else
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), r, off, 0, NONTEMPORAL);
}

// A slot's row, or -1 where it has none: a value outside [0, S) is treated as -1, so a wrong
// array never takes a kernel out of its buffers.
__device__ __forceinline__ int64_t slot_row(int32_t r, int64_t S)
{
    r = __builtin_amdgcn_readfirstlane(r);             // the same for the wave
    return r >= 0 && r < S ? r : -1;
}

// Work of one wave: a segment of a token's row, 64 lanes * VEC * UNROLL values. A workgroup's
// four waves take neighbouring segments of a token, or where a row has fewer the segments of
// several tokens (per_block: segments a workgroup takes of a token, 1, 2 or 4).
struct Item {
    int64_t t;
    int64_t seg;
};
__device__ __forceinline__ Item wave_item(unsigned block, int per_block)
{
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int shift = per_block >> 1;                 // log2 of 1, 2, 4
    return {(int64_t)block * (4 >> shift) + (wave >> shift), (int64_t)blockIdx.y * per_block + (wave & (per_block - 1))};
}

struct Grid {
    dim3 blocks;
    int per_block;
};
inline Grid grid_of(int64_t tokens, int64_t H, int segment)
{
    const int64_t segs = (H + segment - 1) / segment;
    const int per = segs >= 3 ? 4 : (int)segs;
    const int64_t y = (segs + per - 1) / per;
    return {dim3((unsigned)((tokens * per + 3) / 4), (unsigned)(y < 65535 ? y : 65535)), per};
}

// Rows that no slot names become zeros where the caller asks for it: the launch then starts with
// zero_blocks(S) workgroups that take ZERO_ROWS of the S rows each, mark in LDS those that any
// slot names and zero the others, beside the workgroups that write the named ones. Each reads all
// slots, S^2 / ZERO_ROWS reads, where zeroing all rows in a launch of its own writes S rows; so the
// one or the other by slots to bytes of a row, and up to 2^14 slots, which are read faster than
// a launch is made, always the first. Gather in us, zeroed beside / by itself / not at all: 2^14
// slots of 32 bytes 8.8 / 11.9 / 7.2, 2^17 of 256 bytes 33 / 26 / 20, of 2 KB 54 / 87 / 54, 2^18 of 256 bytes
// 82 / 44 / 34, of 2 KB 111 / 191 / 106, of 8 KB 418 / 840 / 423, 2^19 of 2 KB 323 / 403 / 208 (and the
// gradients of the weighted sum there 673 / 653 / 460).
constexpr int ZERO_ROWS = 256, ZERO_UNROLL = 16;

inline bool zero_beside(int64_t S, int64_t row_bytes)
{
    return S <= 1 << 14 || (S <= 128 * row_bytes && S <= (int64_t)1 << 22);      // S / 256 more workgroups: launchable
}

inline unsigned zero_blocks(int64_t S) { return (unsigned)((S + ZERO_ROWS - 1) / ZERO_ROWS); }

template <typename T, int VEC>
__device__ __forceinline__ void zero_unnamed(unsigned block, const int32_t* __restrict__ slots, int S, T* __restrict__ rows,
                                             int64_t H)
{
    __shared__ uint32_t named[ZERO_ROWS / 32];
    const int tid = threadIdx.x, first = (int)block * ZERO_ROWS;
    if (tid < ZERO_ROWS / 32) named[tid] = 0;
    __syncthreads();
    for (int i0 = tid; i0 < S; i0 += 256 * ZERO_UNROLL) {
        int32_t r[ZERO_UNROLL];
#pragma unroll
        for (int u = 0; u < ZERO_UNROLL; ++u) r[u] = slots[min(i0 + 256 * u, S - 1)];      // past the last: the last again
#pragma unroll
        for (int u = 0; u < ZERO_UNROLL; ++u) {
            const unsigned d = (unsigned)r[u] - (unsigned)first;
            if (d < ZERO_ROWS) atomicOr(&named[d >> 5], 1u << (d & 31));
        }
    }
    __syncthreads();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int q = wave; q < ZERO_ROWS / 32; q += 4) {
        const int row0 = first + 32 * q;
        uint32_t left = ~(uint32_t)__builtin_amdgcn_readfirstlane((int)named[q]);
        if (S - row0 < 32) left &= S > row0 ? (1u << (S - row0)) - 1 : 0u;
        for (; left; left &= left - 1) {
            const __amdgpu_buffer_rsrc_t to = row_of(rows, row0 + __builtin_ctz(left), H, sizeof(T));
            for (int64_t h0 = (int64_t)blockIdx.y * 64 * VEC; h0 < H; h0 += (int64_t)gridDim.y * 64 * VEC)
                store_row<T, VEC>(to, (unsigned)h0 + (tid & 63) * VEC, Pack<T, VEC>{});
        }
    }
}

constexpr int ZERO_STORES = 4;

template <typename V>
__global__ void __launch_bounds__(256) zero_kernel(V* __restrict__ p, int64_t n)
{
    constexpr int PART = 256 * ZERO_STORES;
    for (int64_t at = (int64_t)blockIdx.x * PART; at < n; at += (int64_t)gridDim.x * PART) {
#pragma unroll
        for (int u = 0; u < ZERO_STORES; ++u) {
            const int64_t i = at + 256 * u + threadIdx.x;
            if (i < n) p[i] = V{};
        }
    }
}

constexpr int GATHER_UNROLL = 4;

// xs[slots[t][j]] = x[t]: a wave reads its segment of a token once and writes it top_k times
// (8192 tokens of 8 KB to 4 rows each: 336 MB in 64 us, 5.3 TB/s, what a large copy reaches).
// T here is only a width: the values are moved, not read.
template <typename T, int VEC, bool ZERO>
__global__ void __launch_bounds__(256) gather_kernel(const T* __restrict__ x, const int32_t* __restrict__ slots,
                                                     T* __restrict__ xs, int64_t tokens, int top_k, int64_t H,
                                                     int per_block, unsigned zeroing)
{
    constexpr int SEG = 64 * VEC * GATHER_UNROLL;
    unsigned block = blockIdx.x;
    if constexpr (ZERO) {
        if (block < zeroing) return zero_unnamed<T, VEC>(block, slots, (int)(tokens * top_k), xs, H);
        block -= zeroing;
    }
    const Item it = wave_item(block, per_block);
    if (it.t >= tokens) return;
    const __amdgpu_buffer_rsrc_t from = row_of(x, it.t, H, sizeof(T));
    for (int64_t s0 = it.seg * SEG; s0 < H; s0 += (int64_t)gridDim.y * per_block * SEG) {
        const unsigned h0 = (unsigned)s0 + (threadIdx.x & 63) * VEC;
        Pack<T, VEC> v[GATHER_UNROLL];
#pragma unroll
        for (int u = 0; u < GATHER_UNROLL; ++u) v[u] = load_row<T, VEC>(from, h0 + u * 64 * VEC);
        for (int j = 0; j < top_k; ++j) {
            const int64_t row = slot_row(slots[it.t * top_k + j], tokens * top_k);
            const __amdgpu_buffer_rsrc_t to = row_of(xs, row, H, sizeof(T));
#pragma unroll
            for (int u = 0; u < GATHER_UNROLL; ++u) store_row<T, VEC>(to, h0 + u * 64 * VEC, v[u]);
        }
    }
}

// y[t] = sum over j of weights[t][j] * ys[slots[t][j]], in f32, j upwards; weights null: ones
// (the gradient of the gather). The rows of four choices are loaded before the first is added.
// Bound by memory: 8192 x 4 rows of 8 KB 336 MB in 59 us (5.6 TB/s), 4096 x 8 weighted 302 MB in 56 us.
constexpr int COMBINE_UNROLL = 2, COMBINE_SLOTS = 4;

template <typename TI, typename TO, int VEC, bool WEIGHTED>
__global__ void __launch_bounds__(256) combine_kernel(const TI* __restrict__ ys, const int32_t* __restrict__ slots,
                                                      const float* __restrict__ weights, TO* __restrict__ y,
                                                      int64_t tokens, int top_k, int64_t H, int per_block)
{
    constexpr int U = COMBINE_UNROLL, J = COMBINE_SLOTS, SEG = 64 * VEC * U;
    const Item it = wave_item(blockIdx.x, per_block);
    if (it.t >= tokens) return;
    const __amdgpu_buffer_rsrc_t to = row_of(y, it.t, H, sizeof(TO));
    for (int64_t s0 = it.seg * SEG; s0 < H; s0 += (int64_t)gridDim.y * per_block * SEG) {
        const unsigned h0 = (unsigned)s0 + (threadIdx.x & 63) * VEC;
        float acc[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[u][i] = 0.f;
        for (int j0 = 0; j0 < top_k; j0 += J) {
            int32_t r[J];
            float w[J];
            Pack<TI, VEC> v[J][U];
#pragma unroll
            for (int j = 0; j < J; ++j) {                  // a choice past the last: the last again
                const int64_t slot = it.t * top_k + min(j0 + j, top_k - 1);
                r[j] = slots[slot];
                w[j] = WEIGHTED ? weights[slot] : 1.f;
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int64_t row = j0 + j < top_k ? slot_row(r[j], tokens * top_k) : -1;
                w[j] = row < 0 ? 0.f : w[j];
                const __amdgpu_buffer_rsrc_t from = row_of(ys, row, H, sizeof(TI));
#pragma unroll
                for (int u = 0; u < U; ++u) v[j][u] = load_row<TI, VEC>(from, h0 + u * 64 * VEC);
            }
            __builtin_amdgcn_sched_barrier(0);             // all loads before the first use
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[u][i] += w[j] * (float)v[j][u].v[i];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Pack<TO, VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i) o.v[i] = (TO)acc[u][i];
            store_row<TO, VEC>(to, h0 + u * 64 * VEC, o);
        }
    }
}

__device__ __forceinline__ float wave_sum64(float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Gradients of the weighted sum, one workgroup per token: dys[slots[t][j]] = weights[t][j] * dy[t],
// dweights[t][j] = <dy[t], ys[slots[t][j]]> (0 where the slot has no row). GRAD_SLOTS choices
// are taken together, so dy is read once per GRAD_SLOTS of them. Bound by memory: 4096 x 8 rows of
// 8 KB, 570 MB in 94 us (6.1 TB/s).
constexpr int GRAD_SLOTS = 8;

template <typename TI, typename TO, int VEC, bool ZERO>
__global__ void __launch_bounds__(256) combine_grad_kernel(const TO* __restrict__ dy, const TI* __restrict__ ys,
                                                           const int32_t* __restrict__ slots,
                                                           const float* __restrict__ weights, TI* __restrict__ dys,
                                                           float* __restrict__ dweights, int64_t tokens, int top_k,
                                                           int64_t H, unsigned zeroing)
{
    __shared__ float part[4][GRAD_SLOTS];
    unsigned block = blockIdx.x;
    if constexpr (ZERO) {
        if (block < zeroing) return zero_unnamed<TI, VEC>(block, slots, (int)(tokens * top_k), dys, H);
        block -= zeroing;
    }
    const int64_t t = block;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const __amdgpu_buffer_rsrc_t dy_row = row_of(dy, t, H, sizeof(TO));
    for (int j0 = 0; j0 < top_k; j0 += GRAD_SLOTS) {
        __amdgpu_buffer_rsrc_t from[GRAD_SLOTS], to[GRAD_SLOTS];
        int32_t r[GRAD_SLOTS];
        float w[GRAD_SLOTS], dot[GRAD_SLOTS];
#pragma unroll
        for (int j = 0; j < GRAD_SLOTS; ++j) {
            const int64_t slot = t * top_k + min(j0 + j, top_k - 1);      // past the last: the last again
            r[j] = slots[slot];
            w[j] = weights[slot];
            dot[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < GRAD_SLOTS; ++j) {
            const int64_t row = j0 + j < top_k ? slot_row(r[j], tokens * top_k) : -1;
            from[j] = row_of(ys, row, H, sizeof(TI));
            to[j] = row_of(dys, row, H, sizeof(TI));
        }
        for (int64_t s0 = 0; s0 < H; s0 += 256 * VEC) {
            const unsigned h = (unsigned)s0 + threadIdx.x * VEC;
            const Pack<TO, VEC> g = load_row<TO, VEC>(dy_row, h);
            Pack<TI, VEC> v[GRAD_SLOTS];
#pragma unroll
            for (int j = 0; j < GRAD_SLOTS; ++j) v[j] = load_row<TI, VEC>(from[j], h);
            __builtin_amdgcn_sched_barrier(0);             // all loads before the first use
#pragma unroll
            for (int j = 0; j < GRAD_SLOTS; ++j) {
                Pack<TI, VEC> o;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    // past the row's end g is 0 too, and a slot without a row is not written out
                    dot[j] += (float)g.v[i] * (float)v[j].v[i];
                    o.v[i] = (TI)(w[j] * (float)g.v[i]);
                }
                store_row<TI, VEC>(to[j], h, o);
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
            const int32_t row = slots[t * top_k + j0 + j];
            dweights[t * top_k + j0 + j] = row >= 0 && row < tokens * top_k ? (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]) : 0.f;
        }
        __syncthreads();
    }
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// All rows zeroed, ahead of a launch whose workgroups would have too many slots to read.
template <typename V>
hipError_t launch_zero_as(void* p, int64_t bytes, hipStream_t s)
{
    const int64_t n = bytes / (int64_t)sizeof(V), blocks = (n + 256 * ZERO_STORES - 1) / (256 * ZERO_STORES);
    hipLaunchKernelGGL(zero_kernel<V>, dim3((unsigned)(blocks < 1 << 22 ? blocks : 1 << 22)), dim3(256), 0, s,
                       static_cast<V*>(p), n);
    return hipGetLastError();
}

inline hipError_t launch_zero(void* p, int64_t bytes, hipStream_t s)
{
    if (aligned16(p) && bytes % 16 == 0) return launch_zero_as<uint32x4>(p, bytes, s);
    return launch_zero_as<uint16_t>(p, bytes, s);
}

template <typename F>
hipError_t by_types(int a, int b, F f)
{
    return qpg_by_type(a, [&](auto ta) { return qpg_by_type(b, [&](auto tb) { return f(ta, tb); }); });
}

}  // namespace qpg

// Blocks of the sort: one up to 4096 slots, a single launch, which is worth more to a call from the
// host (4096 slots, 128 experts 7.3 us, 16 blocks 9.9) than it costs at the upper end of a graph
// (7.1 against 6.0; 2048 slots, 8 experts 4.3 against 5.3). Beyond 16, doubled while a block has
// more than 1024 slots, at most 128 (each reads all blocks' counts). With 128 experts, a call among
// others in a graph: 8192 slots 6.3 us (one block 11.5), 32768 7.1 us (8 blocks 11.9), 2^20 19.8
// us (a trace gives each of the two kernels its own start: 32768 slots 4.7 and 5.0 us).
int qpg_experts_sort_blocks(int64_t S)
{
    if (S <= 4096) return 1;
    int b = 16;
    while (b < 128 && S > 1024 * (int64_t)b) b *= 2;
    return b;
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
                                     int64_t H, bool zero, hipStream_t s)
{
    const int64_t row = H * (int64_t)qpg::type_bytes(type);
    if (zero && !qpg::zero_beside(T * top_k, row)) {
        const hipError_t rc = qpg::launch_zero(xs, T * top_k * row, s);
        if (rc != hipSuccess) return rc;
        zero = false;
    }
    auto go = [&](auto unit, auto vec) {
        typedef decltype(unit) U;
        constexpr int VEC = decltype(vec)::value;
        const int64_t n = row / (int64_t)sizeof(U);
        qpg::Grid g = qpg::grid_of(T, n, 64 * VEC * qpg::GATHER_UNROLL);
        const unsigned zeroing = zero ? qpg::zero_blocks(T * top_k) : 0;
        g.blocks.x += zeroing;
        auto kernel = zero ? qpg::gather_kernel<U, VEC, true> : qpg::gather_kernel<U, VEC, false>;
        hipLaunchKernelGGL(kernel, g.blocks, dim3(256), 0, s, static_cast<const U*>(x), slots, static_cast<U*>(xs), T,
                           (int)top_k, n, g.per_block, zeroing);
        return hipGetLastError();
    };
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
            const qpg::Grid g = qpg::grid_of(T, H, 64 * VEC * qpg::COMBINE_UNROLL);
            auto kernel = weights ? qpg::combine_kernel<TI, TO, VEC, true> : qpg::combine_kernel<TI, TO, VEC, false>;
            hipLaunchKernelGGL(kernel, g.blocks, dim3(256), 0, s, static_cast<const TI*>(ys), slots, weights,
                               static_cast<TO*>(y), T, (int)top_k, H, g.per_block);
            return hipGetLastError();
        };
        constexpr int V = 16 / (sizeof(TI) > sizeof(TO) ? sizeof(TI) : sizeof(TO));
        if (H % V == 0 && qpg::aligned16(ys) && qpg::aligned16(y)) return go(std::integral_constant<int, V>());
        return go(std::integral_constant<int, 1>());
    });
}

hipError_t qpg_launch_experts_combine_grad(const void* dy, int dy_type, const void* ys, int ys_type,
                                           const int32_t* slots, const float* weights, void* dys, float* dweights,
                                           int64_t T, int64_t top_k, int64_t H, bool zero, hipStream_t s)
{
    const int64_t row = H * (int64_t)qpg::type_bytes(ys_type);
    if (zero && !qpg::zero_beside(T * top_k, row)) {
        const hipError_t rc = qpg::launch_zero(dys, T * top_k * row, s);
        if (rc != hipSuccess) return rc;
        zero = false;
    }
    const unsigned zeroing = zero ? qpg::zero_blocks(T * top_k) : 0;
    return qpg::by_types(ys_type, dy_type, [&](auto ti, auto to) {
        typedef typename qpg::Store<decltype(ti)::value>::type TI;
        typedef typename qpg::Store<decltype(to)::value>::type TO;
        auto go = [&](auto vec) {
            constexpr int VEC = decltype(vec)::value;
            auto kernel = zero ? qpg::combine_grad_kernel<TI, TO, VEC, true> : qpg::combine_grad_kernel<TI, TO, VEC, false>;
            hipLaunchKernelGGL(kernel, dim3((unsigned)T + zeroing), dim3(256), 0, s, static_cast<const TO*>(dy),
                               static_cast<const TI*>(ys), slots, weights, static_cast<TI*>(dys), dweights, T, (int)top_k, H,
                               zeroing);
            return hipGetLastError();
        };
        constexpr int V = 16 / (sizeof(TI) > sizeof(TO) ? sizeof(TI) : sizeof(TO));
        if (H % V == 0 && qpg::aligned16(ys) && qpg::aligned16(dys) && qpg::aligned16(dy))
            return go(std::integral_constant<int, V>());
        return go(std::integral_constant<int, 1>());
    });
}
