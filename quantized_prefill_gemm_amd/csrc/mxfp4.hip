// MXFP4 quantiser and its inverse for gfx950.
//
// Per 32 values of a row: with E = floor(log2(max|x|)) the shared scale is 2^(E - 2) (2 is the
// exponent of the largest 4-bit value, 6 = 1.5 * 2^2), kept as a byte e = E - 2 + 127, not
// below 0; each value is x / 2^(e - 127) rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6,
// ties to the even code, magnitudes above 6 to 6, the sign kept. For a finite f32 the exponent
// field of max|x| is E + 127 (0 for a subnormal, where the bound e >= 0 holds anyway), so
// e = max(field - 2, 0) with no logarithm. The division is by a power of two: the conversion
// instruction divides and rounds in one step, exactly (checked over every exponent, the
// halfway points and their neighbours). A block with a NaN or an infinity has no scale that
// keeps it: it gets the NaN scale 255 and zero codes, so all 32 values come back as NaN.
//
// Memory-bound: 4 (2) bytes read and 17/32 written per value (2048 x 11008 f32: 102 MB in 17.8 us,
// 5.7 TB/s; back to f32 18.2 us). A lane takes eight consecutive
// values (32 or 16 bytes, one dword of codes), four lanes share a block and find its maximum
// by two lane exchanges. Blocks are indexed flat over (row, block), which is contiguous in x
// and in both planes, so K % 32 == 0 is enough and rows have no tails.
#include "qpg_mx.h"

namespace qpg {

constexpr int MX_SLICES = 2;      // 8-value groups per lane, 256 groups apart: more bytes in flight

template <int TYPE>
__global__ void __launch_bounds__(256) quantize_mxfp4_kernel(const typename Store<TYPE>::type* __restrict__ x,
                                                             uint32_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales, int64_t groups)
{
    typedef typename Store<TYPE>::type T;
    constexpr int V = 16 / sizeof(T);
    Pack<T, V> in[MX_SLICES][8 / V];
    const int64_t base = (int64_t)blockIdx.x * (256 * MX_SLICES) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < MX_SLICES; ++u) {
        const int64_t g = base + 256 * u;
#pragma unroll
        for (int i = 0; i < 8 / V; ++i) {
            if (g < groups)
                in[u][i] = reinterpret_cast<const Pack<T, V>*>(x)[g * (8 / V) + i];
            else
                in[u][i] = Pack<T, V>{};
        }
    }
#pragma unroll
    for (int u = 0; u < MX_SLICES; ++u) {
        const int64_t g = base + 256 * u;       // the four lanes of a block pass the test together
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)in[u][i / V].v[i % V];
        int e;
        const uint32_t c = mx_encode8(f, e);
        if (g < groups) {
            codes[g] = c;
            if ((threadIdx.x & 3) == 0) scales[g >> 2] = (uint8_t)e;
        }
    }
}

template <int TYPE>
__global__ void __launch_bounds__(256) dequantize_mxfp4_kernel(const uint32_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales,
                                                               typename Store<TYPE>::type* __restrict__ y,
                                                               int64_t groups)
{
    typedef typename Store<TYPE>::type T;
    constexpr int V = 16 / sizeof(T);
    const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (g >= groups) return;
    const uint32_t c = codes[g];
    const float s = mx_scale(scales[g >> 2]);
    float f[8];
    floatx2 p;
    // the conversion with scale 1, then one multiplication: exact in f32 for every code and
    // scale (6 * 2^127 overflows to infinity, as the value itself does)
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0); f[0] = p[0]; f[1] = p[1];
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1); f[2] = p[0]; f[3] = p[1];
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2); f[4] = p[0]; f[5] = p[1];
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3); f[6] = p[0]; f[7] = p[1];
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) {
        Pack<T, V> out;
#pragma unroll
        for (int j = 0; j < V; ++j) out.v[j] = (T)(f[i * V + j] * s);
        reinterpret_cast<Pack<T, V>*>(y)[g * (8 / V) + i] = out;
    }
}

}  // namespace qpg

hipError_t qpg_launch_quantize_mxfp4(const void* x, int x_type, void* xm, int64_t M, int64_t K, hipStream_t s)
{
    const int64_t groups = M * (K / 8);
    uint32_t* codes = static_cast<uint32_t*>(xm);
    uint8_t* scales = static_cast<uint8_t*>(xm) + M * (K / 2);
    const unsigned blocks = (unsigned)((groups + 256 * qpg::MX_SLICES - 1) / (256 * qpg::MX_SLICES));
    return qpg_by_type(x_type, [&](auto t) {
        typedef typename qpg::Store<decltype(t)::value>::type T;
        hipLaunchKernelGGL(qpg::quantize_mxfp4_kernel<decltype(t)::value>, dim3(blocks), dim3(256), 0, s,
                           static_cast<const T*>(x), codes, scales, groups);
        return hipGetLastError();
    });
}

hipError_t qpg_launch_dequantize_mxfp4(const void* xm, void* y, int y_type, int64_t M, int64_t K, hipStream_t s)
{
    const int64_t groups = M * (K / 8);
    const uint32_t* codes = static_cast<const uint32_t*>(xm);
    const uint8_t* scales = static_cast<const uint8_t*>(xm) + M * (K / 2);
    const unsigned blocks = (unsigned)((groups + 255) / 256);
    return qpg_by_type(y_type, [&](auto t) {
        typedef typename qpg::Store<decltype(t)::value>::type T;
        hipLaunchKernelGGL(qpg::dequantize_mxfp4_kernel<decltype(t)::value>, dim3(blocks), dim3(256), 0, s, codes,
                           scales, static_cast<T*>(y), groups);
        return hipGetLastError();
    });
}
