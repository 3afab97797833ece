// Attention of new tokens over a paged cache of keys and values (include/qpg.h, cache_attention and
// cache_attention_tree).
//
//   y = sum over seen keys of exp(s_j - m) v_j / sum of exp(s_j - m),  s = cap(scale <q, k>) - slope |i - j|
//
// One pass over the keys with the running maximum m and sum. The query rows of one key head -- its
// new tokens times its G query heads, token by token -- are the columns of the matrix products, so prompts,
// single tokens and trees are one kernel, and a key is read once for all that share it. A tile is BC = 32 * WC columns
// of one sequence and key head. Products are taken transposed, with 32 x 32 x 16 matrix instructions:
//   S^T [keys][columns] = K Q^T,   O^T [dim][columns] = V^T P^T.
// A column is then a lane (and its partner 32 away) in both results: the softmax needs one exchange a stage,
// the scaling of O no exchange, and P^T goes from the first result to the second operand in its own lane, since the
// order of the keys in a product is free: register r of a lane in half h is key 8 (r >> 2) + 4h + (r & 3), and V^T
// is read as the same keys, four at a time, by the transposing LDS read.
//
// Keys and values go from memory straight to LDS, a stage ahead; 16-byte slot c of row r holds
// piece c ^ swizzle(r), which spreads both kinds of reads over all banks, and is made by the loads'
// source offsets. Rows behind the sequence's end and pieces behind dim come from behind the descriptor's
// end: zeros. A 16-row block lies in one page, and has its own descriptor: 64-bit page addresses.
//
// Long prompts are bound by the vector arithmetic and the matrix instructions together, which hardly overlap in a wave:
// 8192 tokens of 32 query over 8 heads of 128 in bf16 530 to 545 us by machine, 1.01 to 1.04 PFLOP/s, the matrix units busy 54 % of the time and
// the vector units 48 % (powers are a quarter of a step's vector cycles), no LDS conflicts. (A pipeline of 32-key steps, one's K Q^T
// among the powers of the one before, came to 557 to 619.) Decoding is bound by memory: 64 tokens over 130 to
// 8100 of 8 heads 190 us, 5.5 TB/s. Few tiles are bound by the time of a tile's rounds, about 1.1 us each and 2.6
// where eight waves share a CU, and of 7 us around them: finding the tile, the first loads, the join. What that time
// was before: a table read by vector loads, whose wait was one for the prefetch as well, made the decode batch 251.
#include "qpg_cache.h"

namespace qpg {

typedef __attribute__((address_space(3))) void lds_void;
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) shortx4 lds_shortx4;

struct AttentionArgs {
    CacheBatch batch;
    const void *q, *k, *v;
    void* y;
    float* part_o;                // [splits][T * heads][dim]
    floatx2* part_ml;             // [splits][T * heads]: maximum (of scores in powers of two), sum
    int64_t k_page, v_page;       // elements from page to page
    int pages, page_bits, dim, heads, kv, group, slots, splits, least, y_type;
    float scale, cap;             // scale * log2(e); cap * log2(e) with cap_scale = 2 scale / cap * log2(e)
    float cap_scale;
    const float* slopes;
    int window;                   // NO_WINDOW and more: none
    const int32_t* prefix;
    const int64_t* tree;
    const int32_t* positions;
    int words;
};

template <typename T> struct Matrix;
template <> struct Matrix<_Float16> {
    typedef halfx8 x8;
    static constexpr unsigned INF = 0x7C00;
    static constexpr int LIFT = 6;            // shares are 2^6 times their value: small ones stay normal numbers
    static constexpr int PIECES = 2;
    static __device__ __forceinline__ floatx16 mul(x8 a, x8 b, floatx16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float sum2(x8 a, int i, float c)
    {
        typedef _Float16 x2 __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2(x2{a[2 * i], a[2 * i + 1]}, x2{(_Float16)1.0f, (_Float16)1.0f}, c, false);
    }
};
template <> struct Matrix<__bf16> {
    typedef bf16x8 x8;
    static constexpr unsigned INF = 0x7F80;
    static constexpr int LIFT = 0;
    static constexpr int PIECES = 3;
    static __device__ __forceinline__ floatx16 mul(x8 a, x8 b, floatx16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ float sum2(x8 a, int i, float c)
    {
        typedef __bf16 x2 __attribute__((ext_vector_type(2)));
        return __builtin_amdgcn_fdot2_f32_bf16(x2{a[2 * i], a[2 * i + 1]}, x2{(__bf16)1.0f, (__bf16)1.0f}, c, false);
    }
};

// Each lane's 16 bytes at voff go to LDS byte lds_wave_base + 16 * lane. Inline asm, so that the
// compiler's own waits leave the prefetch alone; the kernel waits before a stage is read. m0
// carries the wave-uniform LDS address. The compiler does not look into the asm: five wait states, since
// its scalar operands may come straight from a lane (v_readlane, v_readfirstlane).
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, unsigned lds_wave_base, unsigned voff, bool fresh)
{
    if (!fresh)
        asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(voff), "s"(r), "{m0}"(lds_wave_base) : "memory");
    else
        asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(voff), "s"(r), "{m0}"(lds_wave_base) : "memory");
}

// A descriptor of `bytes` bytes from p, both the same for the wave.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int bytes)
{
    const uint64_t a = (uint64_t)p;
    const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)a), hi = __builtin_amdgcn_readfirstlane((unsigned)(a >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

constexpr unsigned NOWHERE = 0xFFFFFFF0u;      // past the end of every descriptor here

// Both halves' maximum, in both.
__device__ __forceinline__ float half_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// x * s of an s that is 0 or more, where an infinite x stays.
__device__ __forceinline__ float scaled(float x, float s) { return fabsf(x) == INFINITY ? x : x * s; }

// n / d for 0 <= n < 2^24, 1 <= d: f32's quotient is off by one at most.
__device__ __forceinline__ int divide(int n, int d)
{
    const int q = (int)((float)n * __builtin_amdgcn_rcpf((float)d)), r = n - q * d;
    return r < 0 ? q - 1 : r >= d ? q + 1 : q;
}

constexpr int NO_WINDOW = 1 << 30;
constexpr float LOG2E = 1.4426950408889634f;

// cap tanh(x) = cap - 2 cap / (exp(2x) + 1), with `cap` in powers of two and exp(2x) = 2^(s * cap_scale). Next to 0, where
// that cancels, `fine` takes the series to x^9 (the next term is below 2^-24 of x up to |x| = 0.2); without it the
// error is a few steps of 1 times the cap: up to COARSE_CAP far below a share's rounding to 16 bits.
constexpr float COARSE_CAP = 128.0f * LOG2E;
__device__ __forceinline__ float capped(float s, float cap, float cap_scale, bool fine)
{
    const float t = s * cap_scale;
    const float big = cap - 2.0f * cap * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(t) + 1.0f);
    if (!fine) return big;
    const float z = t * 0.34657359027997264f, z2 = z * z;               // ln(2) / 2
    const float small = cap * (z + z * z2 * (-0.33333333333f + z2 * (0.13333333333f + z2 * (-0.053968253968f + z2 * 0.021869488536f))));
    return fabsf(z) < 0.2f ? small : big;
}

// The slot of a row's 16-byte piece: piece ^ swizzle(row). Rows of 64 values (two to a bank cycle of
// 256 bytes), or of 128 and 256.
template <int DP>
__device__ __forceinline__ int swizzle(int row)
{
    return DP == 64 ? (((row >> 1) & 1) << 2) | ((row >> 2) & 3) : ((row & 3) << 2) | ((row >> 2) & 3);
}

template <int DP, int KT, int WK>
struct AttentionLds {
    static constexpr int STAGE = KT * DP * 2;          // bytes of a stage's keys, or values
    uint8_t k[WK][2][STAGE];
    uint8_t v[WK][2][STAGE];
};

constexpr float DONE = -1.0f;                  // in place of a row's sum where its tile had no second piece
constexpr float FAR = -3.402823466e38f;        // in place of a maximum of nothing: finite, so differences are numbers

// T: cache type; DP: dim rounded up to 64, 128, 256; WC waves of 32 columns each share a stage of KT
// keys, WK such groups take every WK-th stage of the tile's keys and are joined at the end; NP: pieces of a share.
template <typename T, int DP, int WC, int WK, int KT, int NP>
__global__ void __launch_bounds__(64 * WC * WK, DP == 256 || WK > 1 ? 1 : 2) cache_attention_kernel(AttentionArgs a)
{
    typedef typename Matrix<T>::x8 x8;
    constexpr int BC = 32 * WC, NS = KT / 32, ND = DP / 32, NK = DP / 16, NB = KT / WC < 16 ? 1 : KT / WC / 16;
    constexpr int ROWS = KT / WC;                      // rows of a stage that a wave loads
    constexpr int RPI = 512 / DP, LOADS = ROWS / RPI;  // rows of one load, loads of a wave
    constexpr int STAGE = AttentionLds<DP, KT, WK>::STAGE;
    constexpr size_t JOIN = WK > 1 ? (size_t)WC * WK * 32 * (DP * 4 + 8) : 0;      // groups joined: o, maxima and sums
    __shared__ __align__(1024) uint8_t lds_raw[sizeof(AttentionLds<DP, KT, WK>) > JOIN ? sizeof(AttentionLds<DP, KT, WK>) : JOIN];
    __shared__ int lds_again;
    AttentionLds<DP, KT, WK>& lds = *reinterpret_cast<AttentionLds<DP, KT, WK>*>(lds_raw);

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l31 = lane & 31, half = lane >> 5, wc = wave % WC, wk = wave / WC;

    // Head, slot, split of this workgroup: where the heads are a multiple of the eight dies, a
    // head's tiles run on one of them and share its cache; tiles with the most keys first.
    int unit = blockIdx.x, h;
    if (a.kv % 8 == 0) {
        const int per_head = a.slots * a.splits, q = divide(unit >> 3, per_head);
        h = (unit & 7) + 8 * q;
        unit = (unit >> 3) - q * per_head;
    } else {
        const int q = divide(unit, a.kv);
        h = unit - q * a.kv;
        unit = q;
    }
    const int slot = a.slots - 1 - divide(unit, a.splits), split = unit - (a.slots - 1 - slot) * a.splits;

    // Sequence b has slots first(b) .. first(b + 1): enough for its tiles wherever its rows begin. Its numbers come
    // with those it is found by where there are few sequences, since each round of loads is time in which nothing
    // else happens.
    typedef __attribute__((address_space(4))) const int32_t uniform_int;
    auto clamped = [&](int at) { return min(max(at, 0), a.batch.T); };
    auto first = [&](int at, int i) { return (int64_t)at * a.group / BC + i; };
    int b = 0, row0, row1, n;
    if (a.batch.B > 1 && a.batch.B < 64) {
        const int at = clamped(a.batch.offsets[min(lane, a.batch.B)]), length = a.batch.lens[min(lane, a.batch.B - 1)];
        const uint64_t hit = __ballot(lane < a.batch.B && first(at, lane) <= slot);
        b = hit ? 63 - __builtin_clzll(hit) : 0;
        row0 = __builtin_amdgcn_readlane(at, b);
        row1 = __builtin_amdgcn_readlane(at, b + 1);
        n = __builtin_amdgcn_readlane(length, b);
    } else {
        if (a.batch.B > 1) b = last_not_above(a.batch.B, slot, [&](int i) { return first(a.batch.offset(i), i); });
        const uniform_int* offsets = (const uniform_int*)a.batch.offsets;
        row0 = clamped(offsets[b]);
        row1 = clamped(offsets[b + 1]);
        n = ((const uniform_int*)a.batch.lens)[b];
    }
    const int news = row1 - row0;
    const int64_t tile0 = (slot - first(row0, b)) * BC;
    if (tile0 < 0 || tile0 >= (int64_t)news * a.group) return;      // the same for the whole workgroup
    const int c0 = (int)tile0, columns = min(BC, news * a.group - c0);
    n = min(max(n, 0), a.batch.width << a.page_bits);
    const int ctx = n - news;                          // below 0: the first rows have no place
    const int prefix = a.prefix ? min(max(((const uniform_int*)a.prefix)[b], 0), n) : 0;

    // This lane's column. Columns behind the last do as the last does, and are not written.
    const int token0 = c0 / a.group, spare = c0 - token0 * a.group;         // columns are token * group + head in group
    auto token_of = [&](int i) __attribute__((always_inline)) { return token0 + divide(spare + i, a.group); };
    const int col = 32 * wc + l31, own = min(col, columns - 1);
    const int token = token_of(own), head = h * a.group + spare + own - (token - token0) * a.group;
    auto position_of = [&](int t) __attribute__((always_inline)) {
        return a.tree ? min(max(a.positions[row0 + t], 0), 1 << 30) : ctx + t;
    };
    const int position = position_of(token);
    // The range of the positions of the tile's columns, and of this wave's.
    int low, high, wave_low, wave_high;
    if (a.tree) {
        low = 1 << 30, high = 0;
        if (a.window < NO_WINDOW)
            for (int t = token0 + lane; t <= token_of(columns - 1); t += 64) {
                low = min(low, position_of(t));
                high = max(high, position_of(t));
            }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            low = min(low, __shfl_xor(low, m));
            high = max(high, __shfl_xor(high, m));
        }
        low = wave_low = __builtin_amdgcn_readfirstlane(low);
        high = wave_high = __builtin_amdgcn_readfirstlane(high);
    } else {
        low = ctx + token0;
        high = ctx + __builtin_amdgcn_readfirstlane(token_of(columns - 1));
        wave_low = ctx + __builtin_amdgcn_readfirstlane(token_of(min(32 * wc, columns - 1)));
        wave_high = ctx + __builtin_amdgcn_readfirstlane(token_of(min(32 * wc + 31, columns - 1)));
    }
    // Positions are at most 2^30 and windows are clamped to it: no difference here overflows.
    // The window bounds the places of earlier tokens alone, whose positions they are: a node may lie before its ancestors.
    int begin = a.window < NO_WINDOW ? max(low - a.window + 1, 0) : 0;
    if (a.tree) begin = min(begin, max(ctx, 0));
    const int end = a.tree ? n : min(n, max(high + 1, prefix));
    // Stages: those of the prefix, then those from the window on.
    const int head_stages = (min(prefix, end) + KT - 1) / KT;
    const int begin_stage = max(begin / KT, head_stages), end_stage = (end + KT - 1) / KT;
    const int stages = head_stages + max(end_stage - begin_stage, 0);
    auto key_of = [&](int i) __attribute__((always_inline)) { return (i < head_stages ? i : i - head_stages + begin_stage) * KT; };
    const int share = max(((stages + a.splits - 1) / a.splits + WK - 1) / WK * WK, WK * a.least);
    const int i0 = min(split * share, stages), i1 = min(i0 + share, stages);
    const bool parts = stages > share;                 // else the first piece is all, and writes y
    if (!parts && split > 0) return;
    const int rounds = (i1 - i0 + WK - 1) / WK;

    // Columns of Q^T: 8 values of 16-byte piece 2t + half.
    x8 qt[NK];
    {
        const T* q = static_cast<const T*>(a.q) + ((int64_t)(row0 + token) * a.heads + head) * a.dim;
#pragma unroll
        for (int t = 0; t < NK; ++t) {
            const int d = 8 * (2 * t + half);
#pragma unroll
            for (int i = 0; i < 8; ++i) qt[t][i] = (T)0.0f;
            if (d < a.dim) qt[t] = *reinterpret_cast<const x8*>(q + d);
        }
    }

    // Loads of a stage: block j of 16 rows of this wave, by its page.
    const T* kc = static_cast<const T*>(a.k) + ((int64_t)h << a.page_bits) * a.dim;
    const T* vc = static_cast<const T*>(a.v) + ((int64_t)h << a.page_bits) * a.dim;
    // Scalar loads: a vector load's wait would be one for the stage under way as well.
    const uniform_int* table = (const uniform_int*)(a.batch.table + (int64_t)b * a.batch.width);
    const int row_bytes = a.dim * 2;
    unsigned voff[LOADS];                              // from the first row of its block
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
        const int r = wc * ROWS + j * RPI + lane / (DP / 8), piece = (lane % (DP / 8)) ^ swizzle<DP>(r);
        voff[j] = 8 * piece < a.dim ? (unsigned)((r & 15) * row_bytes + 16 * piece) : NOWHERE;
    }
    int pages[NB];
    auto look_up = [&](int i) __attribute__((always_inline)) {
        const int key = i < i1 ? key_of(i) : 0;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int at = (key + wc * ROWS + 16 * j) >> a.page_bits;
            pages[j] = min(max(table[min(at, a.batch.width - 1)], 0), a.pages - 1);
        }
    };
    const unsigned lds_k = (unsigned)(uintptr_t)(lds_void*)&lds.k[wk][0][0], lds_v = (unsigned)(uintptr_t)(lds_void*)&lds.v[wk][0][0];
    auto load_stage = [&](int i, int buffer) __attribute__((always_inline)) {
        const int key = i < i1 ? key_of(i) : 1 << 30;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int row = wc * ROWS + j * RPI, block = row & ~15;          // row of the stage
            const int first_key = key + block, in_page = first_key & ((1 << a.page_bits) - 1);
            const int there = min(max(n - first_key, 0), 16) * row_bytes;
            const int page = pages[NB == 1 ? 0 : (j * RPI) / 16];
            const int64_t in_block = (int64_t)in_page * a.dim;
            load_to_lds(buffer_of(kc + page * a.k_page + in_block, there), lds_k + buffer * STAGE + row * DP * 2, voff[j],
                        j * RPI % 16 == 0);
            load_to_lds(buffer_of(vc + page * a.v_page + in_block, there), lds_v + buffer * STAGE + row * DP * 2, voff[j],
                        j * RPI % 16 == 0);
        }
    };

    floatx16 o[ND];
    float m, sum;                                      // m: in powers of two

    // The first seen key position of this column, the position of a key, and the seen ones of keys j .. j + 63 as bits
    // (of nodes without the window).
    const int from = a.window < NO_WINDOW ? position - a.window + 1 : -1;
    const float slope = a.slopes ? a.slopes[head] * LOG2E : 0.0f;
    auto key_position = [&](int j) __attribute__((always_inline)) {
        return a.tree && j >= ctx ? position_of(min(j - ctx, news - 1)) : j;
    };
    auto seen_from = [&](int j) __attribute__((always_inline)) {
        auto range = [&](int lo, int hi) -> uint64_t {
            const int x = max(lo - j, 0), z = min(hi - j, 63);
            return z < x ? 0 : (~(uint64_t)0 << x) & (~(uint64_t)0 >> (63 - z));
        };
        if (!a.tree) return range(from, min(position, n - 1)) | range(0, prefix - 1);
        uint64_t seen = range(from, min(ctx, n) - 1);
        if (j + 63 >= ctx) {
            const int64_t* row = a.tree + (int64_t)(row0 + token) * a.words;
            auto word = [&](int i) { return i >= 0 && i < a.words ? (uint64_t)row[i] : 0; };
            const int node = j - ctx, shift = node & 63;
            uint64_t bits = word(node >> 6) >> shift;
            if (shift) bits |= word((node >> 6) + 1) << (64 - shift);
            seen |= bits & range(max(ctx, 0), n - 1);
        }
        return seen;
    };

    // LDS places of this lane's operands in a stage.
    const int k_place = l31 * DP * 2 + ((half ^ swizzle<DP>(l31)) << 4);       // piece 2t + half: ^ (t << 5)
    const int i16 = lane & 15, v_row = 4 * half + (i16 >> 2);
    int v_place[2];                                    // rows v_row and v_row + 8; columns of d tile 0: ^ (tile << 6)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int piece = ((lane >> 4) & 1) * 2 + ((i16 & 3) >> 1);
        v_place[e] = (v_row + 8 * e) * DP * 2 + ((piece ^ swizzle<DP>(v_row + 8 * e)) << 4) + (i16 & 1) * 8;
    }

    // Values that are no numbers. Times a share of 0, a key's that is not seen, or times a piece of a share, they make NaN in
    // the products. So a wave whose results hold a NaN in a row whose sum is a number walks its stages a second time, with care:
    // of each stage that has landed such values are added to the rows that see them, whatever their shares, and
    // then are 0 in LDS. One of them costs a tile a second walk (8192 tokens, one call: 580 us, with a NaN in the last token 890,
    // NaN throughout 25.8 ms); tiles whose results are numbers pay one multiplication a value at their end.
    auto careful = [&](int i, int buffer) __attribute__((always_inline)) {
        uint8_t* vb = lds.v[wk][buffer];
        auto bad = [](uint32_t x) {                    // of two values: all bits of one that is no number
            const uint32_t lo = (x & Matrix<T>::INF) == Matrix<T>::INF ? 0xFFFFu : 0;
            const uint32_t hi = ((x >> 16) & Matrix<T>::INF) == Matrix<T>::INF ? 0xFFFF0000u : 0;
            return lo | hi;
        };
        auto landed = [] {                             // what the waves of the stage read and wrote of it
            if (WC > 1)
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        };
        bool any = false;
        if (i < i1) {
#pragma unroll 1
            for (int at = lane * 16; at < STAGE; at += 1024) {
                const uint32x4 x = *reinterpret_cast<const uint32x4*>(vb + at);
                any |= (bad(x[0]) | bad(x[1]) | bad(x[2]) | bad(x[3])) != 0;
            }
            any = __ballot(any) != 0;
        }
        if (any) {
            const int key = key_of(i);
            const uint64_t seen = seen_from(key);
#pragma unroll 1
            for (int j = 0; j < KT && key + j < n; ++j) {
                const bool on = ((seen >> j) & 1) && (!a.tree || key_position(key + j) >= from);
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const Pack<T, 4> x = *reinterpret_cast<const Pack<T, 4>*>(
                            vb + j * DP * 2 + (((4 * d + r) ^ swizzle<DP>(j)) << 4) + 8 * half);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float f = (float)x.v[e];
                            if (on && !(fabsf(f) < INFINITY)) o[d][4 * r + e] += f;
                        }
                    }
            }
        }
        landed();
        if (any) {
#pragma unroll 1
            for (int at = wc * (STAGE / WC) + lane * 16; at < (wc + 1) * (STAGE / WC); at += 1024) {
                uint32x4 x = *reinterpret_cast<const uint32x4*>(vb + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] &= ~bad(x[e]);
                *reinterpret_cast<uint32x4*>(vb + at) = x;
            }
        }
        landed();
    };

    if (WC > 1 && threadIdx.x == 0) lds_again = 0;     // (before the first barrier of a walk)
    // Stages whose keys every column of the wave sees, and whose scores are the products, take a short way.
    int plain_low = a.window < NO_WINDOW ? wave_high - a.window + 1 : 0, plain_high = min(wave_low, n - 1);
    if (a.tree) plain_low = a.window < NO_WINDOW ? high - a.window + 1 : 0, plain_high = min(ctx, n) - 1;
    if (a.slopes || a.cap > 0.0f) plain_high = -1;
    auto walk = [&](auto care) __attribute__((always_inline)) {
        constexpr bool CARE = decltype(care)::value;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
        m = FAR, sum = 0.0f;
        // The careful walk, which is rare, asks for its first stage in a round of its own: one place for its loads.
        int round = CARE ? -1 : 0;
        if constexpr (CARE) asm volatile("" : "+s"(round));
        if (rounds > 0) {
            look_up(i0 + wk);
            if (!CARE) {
                load_stage(i0 + wk, 0);
                look_up(i0 + wk + WK);
            }
        }
        // The compiler's own loads end here, so that none of its waits in the loop is one for the stage under way.
#pragma unroll
        for (int t = 0; t < NK; ++t) {
            if (DP == 256)                                 // kept in accumulation registers, which products read as well
                asm volatile("" : "+a"(qt[t]));
            else
                asm volatile("" : "+v"(qt[t]));
        }
        for (; round < rounds; ++round) {
            const int i = i0 + wk + round * WK, buffer = round & 1;
            // this stage has landed, and every wave is done with the other buffer
            if (WC > 1)
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            if (CARE && round >= 0) careful(i, buffer);
            if (round + 1 < rounds) {
                load_stage(i + WK, buffer ^ 1);
                look_up(i + 2 * WK);
            }
            if (i >= i1 || (CARE && round < 0)) continue;
            const int key = key_of(i), last = key + KT - 1;
            // a stage that none of the wave's columns sees
            if (!a.tree && key >= prefix && (key > wave_high || last < wave_low - a.window + 1)) continue;

            const uint8_t* kb = lds.k[wk][buffer];
            const uint8_t* vb = lds.v[wk][buffer];
            floatx16 s[NS];
#pragma unroll
            for (int e = 0; e < NS; ++e)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[e][r] = 0.0f;
            // A block's operands are read while the block before it is multiplied.
            auto keys = [&](int e, int t) { return *reinterpret_cast<const x8*>(kb + e * 32 * DP * 2 + (k_place ^ (t << 5))); };
            x8 kf[NK];
#pragma unroll
            for (int t = 0; t < NK; ++t) kf[t] = keys(0, t);
#pragma unroll
            for (int e = 0; e < NS; ++e)
#pragma unroll
                for (int t = 0; t < NK; ++t) {
                    s[e] = Matrix<T>::mul(kf[t], qt[t], s[e]);
                    if (e + 1 < NS) kf[t] = keys(e + 1, t);
                }
            __builtin_amdgcn_sched_group_barrier(0x100, NK, 0);             // LDS reads
#pragma unroll
            for (int t = 0; t < (NS - 1) * NK; ++t) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // matrix
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, NK, 0);

            float c = a.scale;                             // c * s are scores in powers of two
            if (key < plain_low || last > plain_high) {
                if (a.cap > 0.0f) {
                    c = 1.0f;
                    if (NP > 1 || a.cap > COARSE_CAP) {
#pragma unroll
                        for (int e = 0; e < NS; ++e)
#pragma unroll
                            for (int r = 0; r < 16; ++r) s[e][r] = capped(s[e][r], a.cap, a.cap_scale, true);
                    } else {
#pragma unroll
                        for (int e = 0; e < NS; ++e)
#pragma unroll
                            for (int r = 0; r < 16; ++r) s[e][r] = capped(s[e][r], a.cap, a.cap_scale, false);
                    }
                }
                const bool whole = a.tree ? last < ctx && (a.window >= NO_WINDOW || high - key < a.window)
                                          : last < n && (last < prefix || (last <= wave_low && wave_high - key < a.window));
                // Node positions, where they matter, are fetched by the lanes together.
                const bool placed = a.tree && last >= ctx && (a.slopes || a.window < NO_WINDOW);
                int at_lane = 0;
                if (placed) {
                    at_lane = key_position(key + lane);
                    asm volatile("" : "+v"(at_lane));          // its load ends here
                }
                if (a.slopes) {
                    const float gap = (float)(position - key - 4 * half);
#pragma unroll
                    for (int e = 0; e < NS; ++e)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const int i = 32 * e + 8 * (r >> 2) + (r & 3);
                            float far = gap - (float)i;
                            if (placed) far = (float)(position - __shfl(at_lane, i + 4 * half));
                            s[e][r] = __builtin_fmaf(-slope, fabsf(far), s[e][r] * c);
                        }
                    c = 1.0f;
                }
                if (!whole) {
                    const uint64_t seen = seen_from(key) >> (4 * half);        // bit i: key + 4 half + i is seen
#pragma unroll
                    for (int e = 0; e < NS; ++e) {
                        const uint32_t bits = (uint32_t)(seen >> (32 * e));
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const int i = 8 * (r >> 2) + (r & 3);
                            bool on = (bits >> i) & 1;
                            if (placed) {
                                const int at = __shfl(at_lane, 32 * e + i + 4 * half);         // by all lanes
                                on = on && at >= from;
                            }
                            s[e][r] = on ? s[e][r] : -INFINITY;
                        }
                    }
                }
            }

            // Running maximum. It is moved only when it has grown by 2^8 (8 bits of f32's, and f16's, range are spare).
            float top = s[0][0];
#pragma unroll
            for (int e = 0; e < NS; ++e)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, s[e][r]);
            top = half_max(top) * c;
            if (__ballot(top > m + 8.0f)) {
                const float next = fmaxf(m, top), shrink = __builtin_amdgcn_exp2f(m - next);
                m = next;
                sum *= shrink;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[d][r] = CARE ? scaled(o[d][r], shrink) : o[d][r] * shrink;
            }
            // V^T rows 32d .. 32d + 31, keys 16f + 4 half + 0..3 and + 8
            auto values = [&](int f, int d) {
                union { shortx4 s[2]; x8 v; } u;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    u.s[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4*)(vb + f * 16 * DP * 2 + (v_place[e] ^ (d << 6))));
                return u.v;
            };
            x8 vf[ND];
#pragma unroll
            for (int d = 0; d < ND; ++d) vf[d] = values(0, d);
            const float base = (float)Matrix<T>::LIFT - m;
            float part = 0.0f;
#pragma unroll
            for (int f = 0; f < 2 * NS; ++f) {
                x8 p[NP];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float rest = __builtin_amdgcn_exp2f(__builtin_fmaf(s[f >> 1][8 * (f & 1) + i], c, base));
                    if (NP > 1) part += rest;
#pragma unroll
                    for (int g = 0; g < NP; ++g) {
                        // To nearest even; the next piece is what it left. One piece where y has no more bits than the cache:
                        // half a step of each share, where y's own rounding is half a step of their sum. Every further
                        // piece is one more product over V (1024 tokens MHA: f16 one 27.4 us, two 33.9; bf16 one
                        // 26.7, three 36.9; 8192 GQA bf16 531 and 925).
                        const T piece = (T)rest;
                        p[g][i] = piece;
                        rest -= (float)piece;
                    }
                }
                if (NP == 1)                               // the sum of the shares as they are multiplied, two at a time
#pragma unroll
                    for (int i = 0; i < 4; ++i) part = Matrix<T>::sum2(p[0], i, part);
#pragma unroll
                for (int d = 0; d < ND; ++d) {
#pragma unroll
                    for (int g = 0; g < NP; ++g) o[d] = Matrix<T>::mul(vf[d], p[g], o[d]);
                    if (f + 1 < 2 * NS) vf[d] = values(f + 1, d);
                }
            }
            sum += part;
        }
    };
    walk(std::false_type());
    bool strange = false;                              // a result of the wave is no number
    if (rounds > 0) {
        float zero = 0.0f;                             // NaN where one is
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) zero = __builtin_fmaf(o[d][r], 0.0f, zero);
        strange = __ballot(zero != zero) != 0;
        bool care = false;
        if (__builtin_expect(strange, false)) {
            bool none = false;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) none |= o[d][r] != o[d][r];
            const float total = half_sum(sum);
            care = __ballot(none && total == total) != 0;
        }
        if constexpr (WC > 1) {                        // waves that share stages do them again together
            if (care && lane == 0) lds_again = 1;
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            care = __builtin_amdgcn_readfirstlane(lds_again) != 0;
        }
        if (__builtin_expect(care, false)) walk(std::true_type());
    }
    m -= (float)Matrix<T>::LIFT;                       // sum and o are of powers relative to this
    sum = half_sum(sum);

    // Groups of one column joined: all to the largest maximum, then added in their order.
    if constexpr (WK > 1) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        constexpr int WAVES = WC * WK;
        float* join = reinterpret_cast<float*>(lds_raw);          // [waves][ND][4][64] x 4, then maxima and sums
        floatx2* ml = reinterpret_cast<floatx2*>(lds_raw + (size_t)WAVES * DP * 32 * 4);
        if (half == 0) ml[wave * 32 + l31] = floatx2{m, sum};
        __syncthreads();
        float top = m;
#pragma unroll
        for (int g = 0; g < WK; ++g) top = fmaxf(top, ml[(g * WC + wc) * 32 + l31][0]);
        float shrink = __builtin_amdgcn_exp2f(m - top);
        sum = 0.0f;
#pragma unroll
        for (int g = 0; g < WK; ++g) {
            const floatx2 x = ml[(g * WC + wc) * 32 + l31];
            sum += x[1] * __builtin_amdgcn_exp2f(x[0] - top);
        }
        m = top;
        if (__builtin_expect(strange, false) && shrink == 0.0f) {        // an infinite value stays
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[d][r] = scaled(o[d][r], 0.0f);
            shrink = 1.0f;
        }
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                floatx4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = o[d][4 * r + e] * shrink;
                *reinterpret_cast<floatx4*>(join + (((size_t)wave * ND + d) * 4 + r) * 256 + lane * 4) = x;
            }
        __syncthreads();
        // wave wk of the columns adds up the quarters d * 4 + r with that number
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if ((d * 4 + r) % WK != wk) continue;
                floatx4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int g = 0; g < WK; ++g) {
                    const floatx4 z = *reinterpret_cast<const floatx4*>(join + (((size_t)(g * WC + wc) * ND + d) * 4 + r) * 256 + lane * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] += z[e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) o[d][4 * r + e] = x[e];
            }
    }

    if (col >= columns) return;
    const int64_t row = (int64_t)(row0 + token) * a.heads + head;
    const int64_t part_row = (int64_t)split * a.batch.T * a.heads + row;
    if (a.splits > 1 && half == 0 && wk == 0) a.part_ml[part_row] = floatx2{m, parts ? sum : DONE};
    if (parts && rounds == 0) return;
    const float inv = parts ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (WK > 1 && (d * 4 + r) % WK != wk) continue;
            const int at = 32 * d + 8 * r + 4 * half;
            if (at >= a.dim) continue;
            floatx4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = o[d][4 * r + e] * inv;
            if (parts) {
                *reinterpret_cast<floatx4*>(a.part_o + part_row * a.dim + at) = x;
            } else if (a.y_type == QPG_F32) {
                *reinterpret_cast<floatx4*>(static_cast<float*>(a.y) + row * a.dim + at) = x;
            } else if (a.y_type == QPG_F16) {
                *reinterpret_cast<Pack<_Float16, 4>*>(static_cast<_Float16*>(a.y) + row * a.dim + at) =
                    Pack<_Float16, 4>{(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
            } else {
                *reinterpret_cast<Pack<__bf16, 4>*>(static_cast<__bf16*>(a.y) + row * a.dim + at) =
                    Pack<__bf16, 4>{(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]};
            }
        }
}

// The pieces of a row's keys: y = sum of 2^(m_s - m) o_s / sum of 2^(m_s - m) sum_s, s upwards. A thread has four
// values. Bound by the time of its loads one behind the other: 4 us, of 11 in all for one token over 1024, MHA.
template <typename TY>
__global__ void __launch_bounds__(256) cache_attention_join_kernel(const float* __restrict__ part_o,
                                                                   const floatx2* __restrict__ part_ml, TY* __restrict__ y,
                                                                   CacheBatch batch, int64_t rows, int heads, int dim,
                                                                   int splits)
{
    const int fours = dim / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / fours;
    if (row >= rows) return;
    const int t = (int)(row / heads), at = (int)(i % fours) * 4;
    if (t < batch.offset(0) || t >= batch.offset(batch.B)) return;
    // Four pieces' loads at a time are under way together; the maximum runs along.
    float m = FAR, sum = 0.0f;
    floatx4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < splits; s0 += 4) {
        floatx2 ml[4];
        floatx4 z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at_row = min(s0 + i, splits - 1) * rows + row;
            ml[i] = part_ml[at_row];
            z[i] = *reinterpret_cast<const floatx4*>(part_o + at_row * dim + at);
        }
        if (ml[0][1] == DONE) return;                  // (of the first piece)
        float next = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (s0 + i >= splits) ml[i][1] = 0.0f;
            if (ml[i][1] != 0.0f) next = fmaxf(next, ml[i][0]);
        }
        const float shrink = __builtin_amdgcn_exp2f(m - next);
        m = next;
        sum *= shrink;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = scaled(o[e], shrink);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (ml[i][1] == 0.0f) continue;            // an empty piece: o is not written
            const float w = __builtin_amdgcn_exp2f(ml[i][0] - m);
            sum += w * ml[i][1];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fabsf(z[i][e]) == INFINITY ? o[e] + z[i][e] : __builtin_fmaf(w, z[i][e], o[e]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    Pack<TY, 4> x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x.v[e] = (TY)(o[e] * inv);
    *reinterpret_cast<Pack<TY, 4>*>(y + row * dim + at) = x;
}

}  // namespace qpg

namespace {

// How a call is laid over the card: WC * 32 columns to a tile, WK groups of waves, keys in `splits` pieces.
struct AttentionForm {
    int wc, wk, splits;
    int64_t slots;
};

// Chosen by what the host knows: the mean number of columns and the longest length that the table holds. Both sides
// measured (us, heads of 128 unless said; MHA: 32 of 32 heads, GQA: 32 of 8):
//   tiles of 128 where they are 256 and more, shared by two groups of waves up to 1024 of them: prompts of 1024, 2048,
//     4096 tokens MHA 34, 69, 176 against 41, 71, 175 by one group; of 8192 GQA, 2048 tiles, 570 against 523
//   else tiles of 64 where they are 192 and more (512 tokens MHA 15.9; tiles of 128 19.6, of 32 22.6), and of 32 below
//     (256 tokens 11.1; of 64 12.9; 26 drafts over 2048 tokens GQA 16.6; of 64 19.2, of 128 20.1)
//   but not over long caches, where larger tiles in pieces read less: 512 tokens over 8000 GQA 87 against 98 of 64
//     and 152 of 32; 128 tokens over 8000 37.8 (64, four pieces) against 48.3 (32)
//   heads of up to 256: tiles of 128 from 512 of them (4096 tokens, 16 of 8 heads: 204, of 64 250; 1024 tokens: of
//     64 38.8, of 128 48.9)
//   pieces until there are about 128 workgroups, since joining them costs 3 us and more (one token over 4096, MHA: one
//     piece 41, two 28.6, four 21.4, eight 22.2), and four where long caches would leave CUs without work at the end
//     (64 tokens over up to 8100 GQA: one piece 203, two 196, four 190, eight 219). A piece has at least 256 keys. One
//     piece against four, 200 to 8000 tokens: 64 GQA 213, 203; 128 GQA 388, 381; 16 MHA 208, 182; 100 of 16 over 4 heads of 64
//     106, 88; 64 of 16 over 8 of 256 425, 382. They cost where lengths are alike (64 over 4100 184, 203; 16 47, 52), and
//     where the table is far longer than they are (64 over 200 to 1000 34, 67; 32 over 2000 48, 60).
AttentionForm form_of(int64_t T, int64_t B, int64_t heads, int64_t kv, int64_t dim, int64_t length)
{
    const int64_t group = heads / kv, busy = B < T ? B : T, mean = (T * group + busy - 1) / busy;
    auto tiles = [&](int64_t columns) { return busy * ((mean + columns - 1) / columns) * kv; };
    const bool wide = dim > 128, far = length >= 4096;
    AttentionForm f;
    if (mean > 64 && tiles(128) >= (wide ? 512 : 256)) {
        f.wc = 4;
        f.wk = !wide && tiles(128) <= 1024 ? 2 : 1;
    } else if (mean > 64 && !wide && far && tiles(128) * length >= 512 * 1024) {
        f.wc = 4;
        f.wk = 2;
    } else if (mean > 32 && (tiles(64) >= (wide ? 128 : 192) || (mean > 64 && far))) {
        f.wc = 2;
        f.wk = wide ? 2 : 4;
    } else {
        f.wc = 1;
        f.wk = wide ? 2 : 4;
    }
    const int64_t count = tiles(32 * f.wc), goal = f.wc == 1 ? 128 : 256;
    int64_t splits = (goal + count - 1) / count;
    if (splits < 4 && far && f.wc == 1 && count <= 1024) splits = 4;
    if (f.wc > 1 && !far) splits = 1;
    if (splits > length / 256) splits = length / 256;
    if (splits > 64) splits = 64;
    f.splits = splits < 1 ? 1 : (int)splits;
    f.slots = T * group / (32 * f.wc) + B;
    return f;
}

constexpr int LEAST_STAGES = 2;    // of a group of waves, in a piece

}  // namespace

int qpg_cache_attention_splits(int64_t T, int64_t B, int64_t heads, int64_t kv, int64_t dim, int64_t length)
{
    return form_of(T, B, heads, kv, dim, length).splits;
}

int64_t qpg_cache_attention_grid(int64_t T, int64_t B, int64_t heads, int64_t kv, int64_t dim, int64_t length, int64_t* threads)
{
    const AttentionForm f = form_of(T, B, heads, kv, dim, length);
    const int64_t grid = f.slots * kv * f.splits;
    *threads = grid * 64 * f.wc * f.wk;
    return grid;
}

hipError_t qpg_launch_cache_attention(const qpg_cache& cache, const qpg_batch& batch, const qpg_scores& scores,
                                      const void* q, int64_t heads, const int64_t* tree, int64_t words,
                                      const int32_t* positions, void* y, int y_type, void* ws, hipStream_t s)
{
    using namespace qpg;
    const int64_t group = heads / cache.heads, rows = batch.T * heads;
    int page_bits = 0;
    while ((1 << page_bits) < cache.page) ++page_bits;
    const AttentionForm form = form_of(batch.T, batch.B, heads, cache.heads, cache.dim, batch.width * cache.page);
    const int64_t slots = form.slots;
    const int splits = form.splits;
    const bool cap = scores.cap > 0.0f;
    AttentionArgs a = {{batch.table, batch.lens, batch.offsets, (int)batch.B, (int)batch.width, (int)batch.T},
                       q, cache.k, cache.v, y, static_cast<float*>(ws),
                       reinterpret_cast<floatx2*>(static_cast<float*>(ws) + (splits > 1 ? splits * rows * cache.dim : 0)),
                       cache.k_stride, cache.v_stride, (int)cache.pages, page_bits, (int)cache.dim, (int)heads,
                       (int)cache.heads, (int)group, (int)slots, splits, LEAST_STAGES, y_type,
                       scores.scale * LOG2E, cap ? scores.cap * LOG2E : 0.0f,
                       cap ? 2.0f * scores.scale / scores.cap * LOG2E : 0.0f, scores.slopes,
                       scores.window > 0 && scores.window < NO_WINDOW ? (int)scores.window : NO_WINDOW, scores.prefix, tree,
                       positions, (int)words};
    const bool fine = y_type == QPG_F32 || (y_type == QPG_F16 && cache.type == QPG_BF16);
    const dim3 grid((unsigned)(slots * cache.heads * splits));
    auto launch = [&](auto t, auto dp, auto wc, auto wk, auto kt) {
        typedef typename Store<decltype(t)::value>::type T;
        constexpr int DP = decltype(dp)::value, WC = decltype(wc)::value, WK = decltype(wk)::value, KT = decltype(kt)::value;
        if (fine)
            hipLaunchKernelGGL((cache_attention_kernel<T, DP, WC, WK, KT, Matrix<T>::PIECES>), grid, dim3(64 * WC * WK), 0, s, a);
        else
            hipLaunchKernelGGL((cache_attention_kernel<T, DP, WC, WK, KT, 1>), grid, dim3(64 * WC * WK), 0, s, a);
        return hipGetLastError();
    };
    using std::integral_constant;
    auto by_columns = [&](auto t, auto dp) {
        const integral_constant<int, 1> one;
        const integral_constant<int, 2> two;
        const integral_constant<int, 4> four;
        const integral_constant<int, 32> half_stage;
        const integral_constant<int, 64> stage;
        if constexpr (decltype(dp)::value == 256) {
            if (form.wc == 4) return launch(t, dp, four, one, half_stage);
            if (form.wc == 2) return launch(t, dp, two, two, half_stage);
            return launch(t, dp, one, two, half_stage);
        } else {
            if (form.wc == 4 && form.wk == 1) return launch(t, dp, four, one, stage);
            if (form.wc == 4) return launch(t, dp, four, two, stage);
            if (form.wc == 2) return launch(t, dp, two, four, half_stage);
            return launch(t, dp, one, four, half_stage);
        }
    };
    auto by_dim = [&](auto t) {
        if (cache.dim <= 64) return by_columns(t, integral_constant<int, 64>());
        if (cache.dim <= 128) return by_columns(t, integral_constant<int, 128>());
        return by_columns(t, integral_constant<int, 256>());
    };
    const hipError_t e = cache.type == QPG_F16 ? by_dim(integral_constant<int, QPG_F16>())
                                               : by_dim(integral_constant<int, QPG_BF16>());
    if (e != hipSuccess || splits == 1) return e;
    return qpg_by_type(y_type, [&](auto t) {
        typedef typename Store<decltype(t)::value>::type TY;
        const int64_t threads = rows * (cache.dim / 4);
        hipLaunchKernelGGL(cache_attention_join_kernel<TY>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s,
                           a.part_o, a.part_ml, static_cast<TY*>(y), a.batch, rows, (int)heads, (int)cache.dim, splits);
        return hipGetLastError();
    });
}
