// mxq_ragged_api.cu -- extern "C" entry points of the ragged grouped products
// (bf16, int8, fp8), of dropout and of a block's norms declared in
// include/mxq.h: host-side checks, then one or two launches on the caller's stream. Nothing here synchronizes or allocates.
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

int run_fp8(const mxq::ragged::Fp8Call& c, mxq_stream_t stream) {
    const cudaError_t e = mxq::ragged::run_fp8(c, (cudaStream_t)stream);
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

int check_norm(int64_t M, int64_t F, double scale) {
    if (!arch_ok()) return MXQ_ERR_ARCH;
    if (M < 0 || M > kMaxRows || F <= 0 || F % 8 || F > mxq::kNormMaxWidth) return MXQ_ERR_SHAPE;
    return std::isfinite((float)scale) ? MXQ_OK : MXQ_ERR_VALUE;
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

int mxq_ragged_gemm_fprop_swiglu(const void* x_bf16, int64_t ldx, const void* w_bf16, const void* bias_bf16, int64_t M,
                                 int64_t F, int64_t K, int E, const int64_t* d_m_splits, void* h, void* y_out,
                                 int32_t* d_status, mxq_stream_t stream) {
    if (!w_bf16 || (M != 0 && (!x_bf16 || !h))) return MXQ_ERR_NULL;
    if (int r = check_ragged(M, F, K, 8, 8, E, d_m_splits)) return r;
    if (2 * F > kMaxWidth || bad_stride(ldx, K)) return MXQ_ERR_SHAPE;
    if (!aligned16(x_bf16) || !aligned16(w_bf16) || !aligned16(bias_bf16) || !aligned16(h) || !aligned16(y_out))
        return MXQ_ERR_ALIGN;
    if (M == 0) return MXQ_OK;
    return run({mxq::ragged::kFpropSwiglu, x_bf16, ldx, w_bf16, 0, bias_bf16, M, F, K, E, d_m_splits, h, 0, 0, d_status,
                nullptr, y_out},
               stream);
}

int mxq_ragged_gemm_dgrad_swiglu(const void* dy_bf16, int64_t lddy, const void* w_bf16, const void* y1_bf16, int64_t M,
                                 int64_t N, int64_t F, int E, const int64_t* d_m_splits, void* dy1, void* h_out,
                                 int32_t* d_status, mxq_stream_t stream) {
    if (!w_bf16 || (M != 0 && (!dy_bf16 || !y1_bf16 || !dy1))) return MXQ_ERR_NULL;
    if (int r = check_ragged(M, N, F, 8, 8, E, d_m_splits)) return r;
    if (2 * F > kMaxWidth || bad_stride(lddy, N)) return MXQ_ERR_SHAPE;
    if (!aligned16(dy_bf16) || !aligned16(w_bf16) || !aligned16(y1_bf16) || !aligned16(dy1) || !aligned16(h_out))
        return MXQ_ERR_ALIGN;
    if (M == 0) return MXQ_OK;
    return run({mxq::ragged::kDgradSwiglu, dy_bf16, lddy, w_bf16, 0, nullptr, M, N, F, E, d_m_splits, dy1, 0, 0, d_status,
                y1_bf16, h_out},
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

int mxq_fp8_quantize_rows(const void* x_bf16, int64_t ldx, int64_t M, int64_t K, void* q, float* scale,
                          mxq_stream_t stream) {
    if (M != 0 && (!x_bf16 || !q || !scale)) return MXQ_ERR_NULL;
    if (!arch_ok()) return MXQ_ERR_ARCH;
    if (M < 0 || M > kMaxRows || K <= 0 || K > kMaxWidth || K % 16 || bad_stride(ldx, K)) return MXQ_ERR_SHAPE;
    if (!aligned16(x_bf16) || !aligned16(q) || !aligned4(scale)) return MXQ_ERR_ALIGN;
    const cudaError_t e = mxq::ragged::run_fp8_quantize_rows(x_bf16, M, K, ldx, q, scale, (cudaStream_t)stream);
    return e == cudaSuccess ? MXQ_OK : fail_cuda(e);
}

int mxq_fp8_quantize_weight(const void* w_bf16, int64_t N, int64_t K, int E, void* q, float* scale,
                            mxq_stream_t stream) {
    if (!w_bf16 || !q || !scale) return MXQ_ERR_NULL;
    if (!arch_ok()) return MXQ_ERR_ARCH;
    if (N <= 0 || K <= 0 || N > kMaxWidth || K > kMaxWidth || N % 8 || K % 16 || E < 1 || E > MXQ_MAX_EXPERTS)
        return MXQ_ERR_SHAPE;
    if (((N + 127) / 128) * ((K + 127) / 128) * E > 0x7FFFFFFF) return MXQ_ERR_SHAPE;
    if (!aligned16(w_bf16) || !aligned16(q) || !aligned4(scale)) return MXQ_ERR_ALIGN;
    const cudaError_t e = mxq::ragged::run_fp8_quantize_weight(w_bf16, N, K, E, q, scale, (cudaStream_t)stream);
    return e == cudaSuccess ? MXQ_OK : fail_cuda(e);
}

int mxq_fp8_gemm_fprop(const void* xq, const float* x_scale, const void* wq, const float* w_scale,
                       const void* bias_bf16, int64_t M, int64_t N, int64_t K, int E, const int64_t* d_m_splits,
                       int flags, void* y, int32_t* d_status, mxq_stream_t stream) {
    if (flags & ~MXQ_OUT_F32) return MXQ_ERR_FLAGS;
    if (!wq || !w_scale || (M != 0 && (!xq || !x_scale || !y))) return MXQ_ERR_NULL;
    if (int r = check_ragged(M, N, K, 8, 16, E, d_m_splits)) return r;
    if (!aligned16(xq) || !aligned4(x_scale) || !aligned16(wq) || !aligned4(w_scale) || !aligned16(bias_bf16) ||
        !aligned16(y))
        return MXQ_ERR_ALIGN;
    if (M == 0) return MXQ_OK;
    return run_fp8({mxq::ragged::kFprop, xq, x_scale, wq, w_scale, bias_bf16, M, N, K, E, d_m_splits, y,
                    (flags & MXQ_OUT_F32) != 0, d_status},
                   stream);
}

int mxq_fp8_gemm_dgrad(const void* dyq, const float* dy_scale, const void* wq, const float* w_scale, int64_t M,
                       int64_t N, int64_t K, int E, const int64_t* d_m_splits, int flags, void* dx, int32_t* d_status,
                       mxq_stream_t stream) {
    if (flags & ~MXQ_OUT_F32) return MXQ_ERR_FLAGS;
    if (!wq || !w_scale || (M != 0 && (!dyq || !dy_scale || !dx))) return MXQ_ERR_NULL;
    if (int r = check_ragged(M, N, K, 16, 16, E, d_m_splits)) return r;
    if (!aligned16(dyq) || !aligned4(dy_scale) || !aligned16(wq) || !aligned4(w_scale) || !aligned16(dx))
        return MXQ_ERR_ALIGN;
    if (M == 0) return MXQ_OK;
    return run_fp8({mxq::ragged::kDgrad, dyq, dy_scale, wq, w_scale, nullptr, M, N, K, E, d_m_splits, dx,
                    (flags & MXQ_OUT_F32) != 0, d_status},
                   stream);
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

int mxq_norm_residual_fwd(const void* x, const void* residual, const void* post_weight, const void* pre_weight,
                          const float* gate, int64_t M, int64_t F, double scale, double eps, int flags, void* res_out,
                          void* n_out, float* stats, int32_t* d_status,
                          mxq_stream_t stream) {
    if (flags & ~MXQ_OUT_F32) return MXQ_ERR_FLAGS;
    if (M != 0 && (!x || (!res_out && !n_out) || !n_out != !pre_weight)) return MXQ_ERR_NULL;
    if (int r = check_norm(M, F, scale)) return r;
    if (!(eps > 0.0 && std::isfinite((float)eps) && (float)eps > 0.0f)) return MXQ_ERR_VALUE;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(post_weight) || !aligned16(pre_weight) || !aligned4(gate) ||
        !aligned16(res_out) || !aligned16(n_out) || !aligned4(stats))
        return MXQ_ERR_ALIGN;
    const cudaError_t e = mxq::run_norm_fwd({x, residual, post_weight, pre_weight, gate, M, F, (float)scale, (float)eps,
                                             (flags & MXQ_OUT_F32) != 0, res_out, n_out, stats, d_status},
                                            (cudaStream_t)stream);
    return e == cudaSuccess ? MXQ_OK : fail_cuda(e);
}

int mxq_norm_residual_bwd(const void* dres, const void* dn, const void* x, const void* res, const float* stats,
                          const void* post_weight, const void* pre_weight, const float* gate, int64_t M, int64_t F,
                          double scale, int flags, void* dx, void* dresidual, float* dpost_weight, float* dpre_weight,
                          float* dgate, int32_t* d_status, void* ws, size_t ws_bytes, mxq_stream_t stream) {
    if (flags & ~MXQ_OUT_F32) return MXQ_ERR_FLAGS;
    if (!post_weight != !dpost_weight || !pre_weight != !dpre_weight) return MXQ_ERR_NULL;
    if (M != 0) {
        if (!dx && !dresidual) return MXQ_ERR_NULL;
        if ((!dres && !dn) || !dn != !pre_weight || !gate != !dgate) return MXQ_ERR_NULL;
        if ((pre_weight && !res) || ((post_weight || gate) && !x) || ((post_weight || pre_weight) && !stats))
            return MXQ_ERR_NULL;
    }
    if (int r = check_norm(M, F, scale)) return r;
    if (!aligned16(dres) || !aligned16(dn) || !aligned16(x) || !aligned16(res) || !aligned4(stats) ||
        !aligned16(post_weight) || !aligned16(pre_weight) || !aligned4(gate) || !aligned16(dx) || !aligned16(dresidual) ||
        !aligned16(dpost_weight) || !aligned16(dpre_weight) || !aligned4(dgate) || !aligned16(ws))
        return MXQ_ERR_ALIGN;
    if ((post_weight || pre_weight) && (!ws || ws_bytes < mxq::norm_bwd_workspace(M, F))) return MXQ_ERR_WORKSPACE;
    const cudaError_t e = mxq::run_norm_bwd({dres, dn, x, res, post_weight, pre_weight, gate, stats, M, F, (float)scale,
                                             (flags & MXQ_OUT_F32) != 0, dx, dresidual, dpost_weight, dpre_weight, dgate,
                                             static_cast<float*>(ws), d_status},
                                            (cudaStream_t)stream);
    return e == cudaSuccess ? MXQ_OK : fail_cuda(e);
}

}  // extern "C"
