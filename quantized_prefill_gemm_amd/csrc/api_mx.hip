// C ABI of the MXFP4 and expert operators (declared in include/qpg.h): argument validation,
// device check, then the kernel launches. Nothing here allocates, frees, prints or synchronises.
#include "qpg_mx.h"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxK = (int64_t)1 << 24;
// A thread takes 8 values, a launch holds < 2^32 threads in whole workgroups of 256.
constexpr int64_t kMaxValues = ((int64_t)1 << 35) - (1 << 11);
constexpr int64_t kMaxTokens = (int64_t)1 << 24;     // likewise, 256 threads to a token
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxSlots = (int64_t)1 << 30;      // a row plus a tile's height is an int
constexpr int64_t kMaxRow = (int64_t)1 << 28;        // a row's bytes stay below 2^31

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool type_ok(int t) { return t == QPG_F32 || t == QPG_F16 || t == QPG_BF16; }
int status_of(hipError_t e) { return e == hipSuccess ? QPG_OK : QPG_EHIP; }

bool mx_shape_ok(int64_t rows, int64_t K)
{
    return rows >= 1 && rows < kMaxDim && K >= 32 && K % 32 == 0 && K <= kMaxK && rows <= kMaxValues / K;
}

bool product_shape_ok(int64_t M, int64_t N, int64_t K)
{
    return mx_shape_ok(M, K) && mx_shape_ok(N, K) && ((M + 15) / 16) * ((N + 15) / 16) < kMaxDim;
}

bool slots_ok(int64_t T, int64_t top_k, int64_t H)
{
    if (T < 1 || top_k < 1 || H < 1 || T >= kMaxTokens || top_k >= kMaxDim || H >= kMaxRow) return false;
    // the vector lanes of all rows, and a row's segments at one value to a lane
    return T <= kMaxSlots / top_k && T <= kMaxValues / H;
}

int quantize(const void* x, int x_type, void* xm, int64_t M, int64_t K, hipStream_t s)
{
    if (!x || !xm || !type_ok(x_type) || !mx_shape_ok(M, K)) return QPG_EINVAL;
    if (!aligned(x, 16) || !aligned(xm, 16)) return QPG_EALIGN;
    const int rc = qpg_check_device();
    if (rc != QPG_OK) return rc;
    return status_of(qpg_launch_quantize_mxfp4(x, x_type, xm, M, K, s));
}

int product(const void* w, const void* xm, void* y, int y_type, int64_t M, int64_t N, int64_t K, hipStream_t s)
{
    if (!w || !xm || !y || !type_ok(y_type) || !product_shape_ok(M, N, K)) return QPG_EINVAL;
    if (!aligned(w, 16) || !aligned(xm, 16) || !aligned(y, qpg::type_bytes(y_type))) return QPG_EALIGN;
    const int rc = qpg_check_device();
    if (rc != QPG_OK) return rc;
    return status_of(qpg_launch_mmq_mxfp4(w, xm, y, y_type, M, N, K, s));
}

// zero: rows that no slot names become zeros, else they are left as they were.
int gather(const void* x, int type, const int32_t* slots, void* xs, int64_t T, int64_t top_k, int64_t H, bool zero,
           hipStream_t s)
{
    if (!x || !slots || !xs || !type_ok(type) || !slots_ok(T, top_k, H)) return QPG_EINVAL;
    const uintptr_t a = qpg::type_bytes(type);
    if (!aligned(x, a) || !aligned(xs, a) || !aligned(slots, 4)) return QPG_EALIGN;
    const int rc = qpg_check_device();
    if (rc != QPG_OK) return rc;
    return status_of(qpg_launch_experts_gather(x, type, slots, xs, T, top_k, H, zero, s));
}

int combine_grad(const void* dy, int dy_type, const void* ys, int ys_type, const int32_t* slots, const float* weights,
                 void* dys, float* dweights, int64_t T, int64_t top_k, int64_t H, bool zero, hipStream_t s)
{
    if (!dy || !ys || !slots || !weights || !dys || !dweights) return QPG_EINVAL;
    if (!type_ok(dy_type) || !type_ok(ys_type) || !slots_ok(T, top_k, H)) return QPG_EINVAL;
    if (!aligned(dy, qpg::type_bytes(dy_type)) || !aligned(ys, qpg::type_bytes(ys_type)) ||
        !aligned(dys, qpg::type_bytes(ys_type)) || !aligned(slots, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
        return QPG_EALIGN;
    const int rc = qpg_check_device();
    if (rc != QPG_OK) return rc;
    return status_of(qpg_launch_experts_combine_grad(dy, dy_type, ys, ys_type, slots, weights, dys, dweights, T, top_k,
                                                     H, zero, s));
}

}  // namespace

extern "C" {

size_t qpg_mxfp4_bytes(int64_t rows, int64_t K)
{
    return mx_shape_ok(rows, K) ? (size_t)(rows * (K / 2) + rows * (K / 32)) : 0;
}

int quantize_mxfp4(const void* x, int x_type, void* xm, int64_t M, int64_t K, qpg_stream_t stream)
{
    return quantize(x, x_type, xm, M, K, reinterpret_cast<hipStream_t>(stream));
}

int dequantize_mxfp4(const void* xm, void* y, int y_type, int64_t M, int64_t K, qpg_stream_t stream)
{
    if (!xm || !y || !type_ok(y_type) || !mx_shape_ok(M, K)) return QPG_EINVAL;
    if (!aligned(xm, 16) || !aligned(y, 16)) return QPG_EALIGN;
    const int rc = qpg_check_device();
    if (rc != QPG_OK) return rc;
    return status_of(qpg_launch_dequantize_mxfp4(xm, y, y_type, M, K, reinterpret_cast<hipStream_t>(stream)));
}

int mmq_mxfp4_mx(const void* w, const void* xm, void* y, int y_type, int64_t M, int64_t N, int64_t K,
                 qpg_stream_t stream)
{
    return product(w, xm, y, y_type, M, N, K, reinterpret_cast<hipStream_t>(stream));
}

int mmq_mxfp4(const void* w, const void* x, int x_type, void* y, int y_type, int64_t M, int64_t N, int64_t K,
              void* xm_ws, qpg_stream_t stream)
{
    if (!w || !x || !y || !xm_ws || !type_ok(x_type) || !type_ok(y_type) || !product_shape_ok(M, N, K))
        return QPG_EINVAL;
    if (!aligned(w, 16) || !aligned(x, 16) || !aligned(xm_ws, 16) || !aligned(y, qpg::type_bytes(y_type)))
        return QPG_EALIGN;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (qpg_mmq_mxfp4_fuses(M, N, K)) {
        const int dv = qpg_check_device();
        if (dv != QPG_OK) return dv;
        return status_of(qpg_launch_mmq_mxfp4_fused(w, x, x_type, xm_ws, y, y_type, M, N, K, s));
    }
    const int rc = quantize(x, x_type, xm_ws, M, K, s);
    if (rc != QPG_OK) return rc;
    return product(w, xm_ws, y, y_type, M, N, K, s);
}

size_t qpg_experts_sort_bytes(int64_t S, int64_t E)
{
    if (S < 1 || S > kMaxSlots || E < 1 || E > kMaxExperts) return 0;
    const int blocks = qpg_experts_sort_blocks(S);
    return blocks > 1 ? (size_t)blocks * (size_t)E * sizeof(int32_t) : 0;
}

int experts_sort(const void* ids, int id_bytes, int64_t S, int64_t E, int32_t* offsets, int32_t* order, int32_t* slots,
                 void* ws, qpg_stream_t stream)
{
    if (!ids || !offsets || !order || !slots || (id_bytes != 4 && id_bytes != 8)) return QPG_EINVAL;
    if (S < 1 || S > kMaxSlots || E < 1 || E > kMaxExperts) return QPG_EINVAL;
    if (!ws && qpg_experts_sort_bytes(S, E)) return QPG_EINVAL;
    if (!aligned(ids, id_bytes) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(slots, 4) || !aligned(ws, 4))
        return QPG_EALIGN;
    const int rc = qpg_check_device();
    if (rc != QPG_OK) return rc;
    return status_of(qpg_launch_experts_sort(ids, id_bytes, S, E, offsets, order, slots, ws,
                                             reinterpret_cast<hipStream_t>(stream)));
}

int mmq_mxfp4_experts(const void* w, const void* xm, int64_t rows, const int32_t* offsets, const int32_t* order,
                      int64_t top_k, void* y, int y_type, int64_t S, int64_t E, int64_t N, int64_t K,
                      qpg_stream_t stream)
{
    if (!w || !xm || !offsets || !y || !type_ok(y_type)) return QPG_EINVAL;
    if (S < 1 || S > kMaxSlots || E < 1 || E > kMaxExperts || top_k < 1 || top_k >= kMaxDim) return QPG_EINVAL;
    // the row tiles that any offsets can stand for: every expert all S rows
    if (E * ((S + 15) / 16) >= kMaxDim) return QPG_EINVAL;
    if (!order && rows != S) return QPG_EINVAL;
    if (!mx_shape_ok(rows, K) || N < 1 || N >= kMaxDim || !mx_shape_ok(E * N, K)) return QPG_EINVAL;
    if (((S + 15) / 16 + E) * ((N + 15) / 16) >= kMaxDim) return QPG_EINVAL;
    if (!aligned(w, 16) || !aligned(xm, 16) || !aligned(offsets, 4) || !aligned(order, 4) ||
        !aligned(y, qpg::type_bytes(y_type)))
        return QPG_EALIGN;
    const int rc = qpg_check_device();
    if (rc != QPG_OK) return rc;
    return status_of(qpg_launch_mmq_mxfp4_experts(w, xm, rows, offsets, order, top_k, y, y_type, S, E, N, K,
                                                  reinterpret_cast<hipStream_t>(stream)));
}

int experts_gather(const void* x, int type, const int32_t* slots, void* xs, int64_t T, int64_t top_k, int64_t H,
                   qpg_stream_t stream)
{
    return gather(x, type, slots, xs, T, top_k, H, false, reinterpret_cast<hipStream_t>(stream));
}

int experts_gather_zero(const void* x, int type, const int32_t* slots, void* xs, int64_t T, int64_t top_k, int64_t H,
                        qpg_stream_t stream)
{
    return gather(x, type, slots, xs, T, top_k, H, true, reinterpret_cast<hipStream_t>(stream));
}

int experts_combine(const void* ys, int ys_type, const int32_t* slots, const float* weights, void* y, int y_type,
                    int64_t T, int64_t top_k, int64_t H, qpg_stream_t stream)
{
    if (!ys || !slots || !y || !type_ok(ys_type) || !type_ok(y_type) || !slots_ok(T, top_k, H)) return QPG_EINVAL;
    if (!aligned(ys, qpg::type_bytes(ys_type)) || !aligned(y, qpg::type_bytes(y_type)) || !aligned(slots, 4) ||
        !aligned(weights, 4))
        return QPG_EALIGN;
    const int rc = qpg_check_device();
    if (rc != QPG_OK) return rc;
    return status_of(qpg_launch_experts_combine(ys, ys_type, slots, weights, y, y_type, T, top_k, H,
                                                reinterpret_cast<hipStream_t>(stream)));
}

int experts_combine_grad(const void* dy, int dy_type, const void* ys, int ys_type, const int32_t* slots,
                         const float* weights, void* dys, float* dweights, int64_t T, int64_t top_k, int64_t H,
                         qpg_stream_t stream)
{
    return combine_grad(dy, dy_type, ys, ys_type, slots, weights, dys, dweights, T, top_k, H, false,
                        reinterpret_cast<hipStream_t>(stream));
}

int experts_combine_grad_zero(const void* dy, int dy_type, const void* ys, int ys_type, const int32_t* slots,
                              const float* weights, void* dys, float* dweights, int64_t T, int64_t top_k, int64_t H,
                              qpg_stream_t stream)
{
    return combine_grad(dy, dy_type, ys, ys_type, slots, weights, dys, dweights, T, top_k, H, true,
                        reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
