// Internal definitions shared by the MXFP4 and expert kernels of libqpg (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qpg.h"

namespace qpg {

typedef unsigned uint32x2 __attribute__((ext_vector_type(2)));
typedef unsigned uint32x4 __attribute__((ext_vector_type(4)));
typedef int int32x4 __attribute__((ext_vector_type(4)));
typedef int int32x8 __attribute__((ext_vector_type(8)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int NONTEMPORAL = 2;        // a buffer store's bit for memory that is not read again soon

// Storage type of a QPG_F32 / QPG_F16 / QPG_BF16 argument; conversions from f32 round to
// nearest even (half a step of the stored type, once, at the end of each operator).
template <int TYPE> struct Store;
template <> struct Store<QPG_F32> { typedef float type; };
template <> struct Store<QPG_F16> { typedef _Float16 type; };
template <> struct Store<QPG_BF16> { typedef __bf16 type; };

// N values of T moved as one access (16 bytes or less) and widened to f32.
template <typename T, int N> struct alignas(sizeof(T) * N) Pack { T v[N]; };

// f32 value of a scale byte: 2^(e - 127), NaN for 255. 2^-127 is a subnormal f32.
__device__ __forceinline__ float mx_scale(int e)
{
    return __int_as_float(e == 255 ? 0x7FC00000 : e == 0 ? 0x00400000 : e << 23);
}

// The quantiser of mxfp4.hip, whose head has the rule.
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);   // lane ^ 1
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);            // lane ^ 2
    return v > o ? v : o;
}

// Eight values of one lane (four lanes a block) to eight codes; e: the block's scale byte.
__device__ __forceinline__ uint32_t mx_encode8(const float (&f)[8], int& e)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = __float_as_uint(f[i]) & 0x7FFFFFFFu;     // NaN > infinity > finite
        m = m > a ? m : a;
    }
    m = quad_max(m);
    const bool finite = m < 0x7F800000u;
    const int field = (int)(m >> 23) - 2;
    e = finite ? (field > 0 ? field : 0) : 255;
    const float scale = mx_scale(finite ? e : 127);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], scale, 3);
    return finite ? c : 0u;
}

inline size_t type_bytes(int type) { return type == QPG_F32 ? 4 : 2; }

}  // namespace qpg

// QPG_OK on a gfx950 device that is current, else QPG_EDEVICE (api.hip).
int qpg_check_device();

// Calls F.operator()<TYPE>() for a validated QPG_F32 / QPG_F16 / QPG_BF16 value.
template <typename F>
hipError_t qpg_by_type(int type, F f)
{
    switch (type) {
    case QPG_F32: return f(std::integral_constant<int, QPG_F32>());
    case QPG_F16: return f(std::integral_constant<int, QPG_F16>());
    case QPG_BF16: return f(std::integral_constant<int, QPG_BF16>());
    default: return hipErrorInvalidValue;
    }
}

// Kernel launchers (arguments validated by the C ABI layer); they return hipGetLastError().
hipError_t qpg_launch_quantize_mxfp4(const void* x, int x_type, void* xm, int64_t M, int64_t K, hipStream_t s);
hipError_t qpg_launch_dequantize_mxfp4(const void* xm, void* y, int y_type, int64_t M, int64_t K, hipStream_t s);
hipError_t qpg_launch_mmq_mxfp4(const void* w, const void* xm, void* y, int y_type, int64_t M, int64_t N, int64_t K,
                                hipStream_t s);
// Quantisation and product of few tokens in one launch, xm as quantize_mxfp4 would leave it;
// qpg_mmq_mxfp4_fuses says for which shapes.
bool qpg_mmq_mxfp4_fuses(int64_t M, int64_t N, int64_t K);
hipError_t qpg_launch_mmq_mxfp4_fused(const void* w, const void* x, int x_type, void* xm, void* y, int y_type,
                                      int64_t M, int64_t N, int64_t K, hipStream_t s);
hipError_t qpg_launch_mmq_mxfp4_experts(const void* w, const void* xm, int64_t rows, const int32_t* offsets,
                                        const int32_t* order, int64_t top_k, void* y, int y_type, int64_t S, int64_t E,
                                        int64_t N, int64_t K, hipStream_t s);
int qpg_experts_sort_blocks(int64_t S);
hipError_t qpg_launch_experts_sort(const void* ids, int id_bytes, int64_t S, int64_t E, int32_t* offsets,
                                   int32_t* order, int32_t* slots, void* ws, hipStream_t s);
hipError_t qpg_launch_experts_gather(const void* x, int type, const int32_t* slots, void* xs, int64_t T, int64_t top_k,
                                     int64_t H, bool zero, hipStream_t s);
hipError_t qpg_launch_experts_combine(const void* ys, int ys_type, const int32_t* slots, const float* weights, void* y,
                                      int y_type, int64_t T, int64_t top_k, int64_t H, hipStream_t s);
hipError_t qpg_launch_experts_combine_grad(const void* dy, int dy_type, const void* ys, int ys_type,
                                           const int32_t* slots, const float* weights, void* dys, float* dweights,
                                           int64_t T, int64_t top_k, int64_t H, bool zero, hipStream_t s);
