// mxq_ragged_api.cu -- extern "C" entry points of the ragged grouped products
// (bf16, int8) and of dropout declared in include/mxq.h: host-side checks, then
// one launch on the caller's stream. Nothing here synchronizes or allocates.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/mxq.h"
#include "mxq_internal.h"
#include "mxq_ragged.h"

using mxq::aligned16;
using mxq::arch_ok;
using mxq::device_pointer;
using mxq::fail_cuda;

namespace {

// At most 2^28 rows: a wgrad tile that sums over all of them takes 1.5 s, less than the kernels' bounded waits.
constexpr int64_t kMaxRows = (int64_t)1 << 28, kMaxWidth = (int64_t)1 << 20;

// Shapes shared by the ragged products: every width a multiple of `step`.
int check_ragged(int64_t M, int64_t N, int64_t K, int step_n, int step_k, int E, const int64_t* m_splits) {
    if (!arch_ok()) return MXQ_ERR_ARCH;
    if (M < 0 || M > kMaxRows || N <= 0 || K <= 0 || N > kMaxWidth || K > kMaxWidth || N % step_n || K % step_k)
        return MXQ_ERR_SHAPE;
    if (E < 1 || E > MXQ_MAX_EXPERTS) return MXQ_ERR_SHAPE;
    if (!m_splits) return MXQ_ERR_NULL;
    return device_pointer(m_splits) ? MXQ_OK : MXQ_ERR_HOST_POINTER;
}
// per-row and per-channel scales are read and written one float at a time
bool aligned4(const float* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
bool bad_stride(int64_t ld, int64_t width) { return ld < width || ld % 8 || ld > ((int64_t)1 << 36); }

int run(const mxq::ragged::GemmCall& c, mxq_stream_t stream) {
    const cudaError_t e = mxq::ragged::run_gemm(c, (cudaStream_t)stream);
    return e == cudaSuccess ? MXQ_OK : fail_cuda(e);
}

// p -> elements dropped of 65536, or -1 if p is outside [0, 1]
int64_t dropped(double p) { return p >= 0.0 && p <= 1.0 ? (int64_t)std::nearbyint(p * 65536.0) : -1; }

int check_dropout(int64_t M, int64_t F, const int64_t* d_rng, double p) {
    if (!arch_ok()) return MXQ_ERR_ARCH;
    if (M < 0 || F < 0 || (F > 0 && M > ((int64_t)1 << 60) / F)) return MXQ_ERR_SHAPE;
    if (!d_rng) return MXQ_ERR_NULL;
    if (!device_pointer(d_rng)) return MXQ_ERR_HOST_POINTER;
    return dropped(p) < 0 ? MXQ_ERR_VALUE : MXQ_OK;
}

}  // namespace

extern "C" {

int mxq_ragged_gemm_fprop(const void* x_bf16, int64_t ldx, const void* w_bf16, const void* bias_bf16, int64_t M,
                          int64_t N, int64_t K, int E, const int64_t* d_m_splits, int flags, void* y,
                          int32_t* d_status, mxq_stream_t stream) {
    if (flags & ~MXQ_OUT_F32) return MXQ_ERR_FLAGS;
    if (!w_bf16 || (M != 0 && (!x_bf16 || !y))) return MXQ_ERR_NULL;
    if (int r = check_ragged(M, N, K, 8, 8, E, d_m_splits)) return r;
    if (bad_stride(ldx, K)) return MXQ_ERR_SHAPE;
    if (!aligned16(x_bf16) || !aligned16(w_bf16) || !aligned16(bias_bf16) || !aligned16(y)) return MXQ_ERR_ALIGN;
    if (M == 0) return MXQ_OK;
    return run({mxq::ragged::kFprop, x_bf16, ldx, w_bf16, 0, bias_bf16, M, N, K, E, d_m_splits, y,
                (flags & MXQ_OUT_F32) != 0, 0, d_status},
               stream);
}

int mxq_ragged_gemm_dgrad(const void* dy_bf16, int64_t lddy, const void* w_bf16, int64_t M, int64_t N, int64_t K,
                          int E, const int64_t* d_m_splits, int flags, void* dx, int32_t* d_status,
                          mxq_stream_t stream) {
    if (flags & ~MXQ_OUT_F32) return MXQ_ERR_FLAGS;
    if (!w_bf16 || (M != 0 && (!dy_bf16 || !dx))) return MXQ_ERR_NULL;
    if (int r = check_ragged(M, N, K, 8, 8, E, d_m_splits)) return r;
    if (bad_stride(lddy, N)) return MXQ_ERR_SHAPE;
    if (!aligned16(dy_bf16) || !aligned16(w_bf16) || !aligned16(dx)) return MXQ_ERR_ALIGN;
    if (M == 0) return MXQ_OK;
    return run({mxq::ragged::kDgrad, dy_bf16, lddy, w_bf16, 0, nullptr, M, N, K, E, d_m_splits, dx,
                (flags & MXQ_OUT_F32) != 0, 0, d_status},
               stream);
}

int mxq_ragged_gemm_wgrad(const void* dy_bf16, int64_t lddy, const void* x_bf16, int64_t ldx, int64_t M, int64_t N,
                          int64_t K, int E, const int64_t* d_m_splits, int flags, void* dw, int32_t* d_status,
                          mxq_stream_t stream) {
    if (flags & ~(MXQ_ACCUMULATE | MXQ_OUT_BF16)) return MXQ_ERR_FLAGS;
    if (!dw || (M != 0 && (!dy_bf16 || !x_bf16))) return MXQ_ERR_NULL;
    if (int r = check_ragged(M, N, K, 8, 8, E, d_m_splits)) return r;
    if (bad_stride(lddy, N) || bad_stride(ldx, K)) return MXQ_ERR_SHAPE;
    if (!aligned16(dy_bf16) || !aligned16(x_bf16) || !aligned16(dw)) return MXQ_ERR_ALIGN;
    return run({mxq::ragged::kWgrad, x_bf16, ldx, dy_bf16, lddy, nullptr, M, N, K, E, d_m_splits, dw,
                (flags & MXQ_OUT_BF16) == 0, (flags & MXQ_ACCUMULATE) != 0, d_status},
               stream);
}

int mxq_int8_quantize_rows(const void* x_bf16, int64_t ldx, int64_t M, int64_t K, void* q, float* scale,
                           mxq_stream_t stream) {
    if (M != 0 && (!x_bf16 || !q || !scale)) return MXQ_ERR_NULL;
    if (!arch_ok()) return MXQ_ERR_ARCH;
    if (M < 0 || M > kMaxRows || K <= 0 || K > kMaxWidth || K % 16 || bad_stride(ldx, K)) return MXQ_ERR_SHAPE;
    if (!aligned16(x_bf16) || !aligned16(q) || !aligned4(scale)) return MXQ_ERR_ALIGN;
    const cudaError_t e = mxq::ragged::run_int8_quantize(x_bf16, M, K, ldx, q, scale, (cudaStream_t)stream);
    return e == cudaSuccess ? MXQ_OK : fail_cuda(e);
}

int mxq_int8_gemm_fprop(const void* xq, const float* x_scale, const void* wq, const float* w_scale,
                        const void* bias_bf16, int64_t M, int64_t N, int64_t K, int E, const int64_t* d_m_splits,
                        int flags, void* y, int32_t* d_status, mxq_stream_t stream) {
    if (flags & ~MXQ_OUT_F32) return MXQ_ERR_FLAGS;
    if (!wq || !w_scale || (M != 0 && (!xq || !x_scale || !y))) return MXQ_ERR_NULL;
    if (int r = check_ragged(M, N, K, 8, 16, E, d_m_splits)) return r;
    if (!aligned16(xq) || !aligned4(x_scale) || !aligned16(wq) || !aligned4(w_scale) || !aligned16(bias_bf16) ||
        !aligned16(y))
        return MXQ_ERR_ALIGN;
    if (M == 0) return MXQ_OK;
    const cudaError_t e = mxq::ragged::run_int8(
        {xq, x_scale, wq, w_scale, bias_bf16, M, N, K, E, d_m_splits, y, (flags & MXQ_OUT_F32) != 0, d_status},
        (cudaStream_t)stream);
    return e == cudaSuccess ? MXQ_OK : fail_cuda(e);
}

int mxq_swiglu_dropout_fwd(const void* y_bf16, int64_t M, int64_t F, const int64_t* d_rng, double p, void* h_bf16,
                           mxq_stream_t stream) {
    if (M != 0 && (!y_bf16 || !h_bf16)) return MXQ_ERR_NULL;
    if (int r = check_dropout(M, F, d_rng, p)) return r;
    if (F <= 0 || F % 8 || F > ((int64_t)1 << 31)) return MXQ_ERR_SHAPE;
    if (!aligned16(y_bf16) || !aligned16(h_bf16)) return MXQ_ERR_ALIGN;
    const cudaError_t e = mxq::ragged::run_swiglu_dropout_fwd(y_bf16, M, F, d_rng, (uint32_t)dropped(p), h_bf16,
                                                              (cudaStream_t)stream);
    return e == cudaSuccess ? MXQ_OK : fail_cuda(e);
}

int mxq_swiglu_dropout_bwd(const void* dh_bf16, const void* y_bf16, int64_t M, int64_t F, const int64_t* d_rng,
                           double p, void* dy_bf16, mxq_stream_t stream) {
    if (M != 0 && (!dh_bf16 || !y_bf16 || !dy_bf16)) return MXQ_ERR_NULL;
    if (int r = check_dropout(M, F, d_rng, p)) return r;
    if (F <= 0 || F % 8 || F > ((int64_t)1 << 31)) return MXQ_ERR_SHAPE;
    if (!aligned16(dh_bf16) || !aligned16(y_bf16) || !aligned16(dy_bf16)) return MXQ_ERR_ALIGN;
    const cudaError_t e = mxq::ragged::run_swiglu_dropout_bwd(dh_bf16, y_bf16, M, F, d_rng, (uint32_t)dropped(p),
                                                              dy_bf16, (cudaStream_t)stream);
    return e == cudaSuccess ? MXQ_OK : fail_cuda(e);
}

int mxq_dropout(const void* x, const void* residual, int64_t n, const int64_t* d_rng, double p, int flags, void* out,
                mxq_stream_t stream) {
    if (flags & ~MXQ_OUT_F32) return MXQ_ERR_FLAGS;
    if (n != 0 && (!x || !out)) return MXQ_ERR_NULL;
    if (int r = check_dropout(n, 1, d_rng, p)) return r;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(out)) return MXQ_ERR_ALIGN;
    const cudaError_t e = mxq::ragged::run_dropout(x, residual, n, (flags & MXQ_OUT_F32) != 0, d_rng,
                                                   (uint32_t)dropped(p), out, (cudaStream_t)stream);
    return e == cudaSuccess ? MXQ_OK : fail_cuda(e);
}

}  // extern "C"
