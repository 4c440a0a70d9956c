// mxq_ragged.h -- launcher interfaces of the ragged grouped products and of
// dropout, between the C ABI (mxq_ragged_api.cu) and the kernels. Not
// installed; not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mxq {
namespace ragged {

// kFpropSwiglu: fprop of W1 (E, 2N, K), out = h (M, N), side = [g | u] (M, 2N) or null. kDgradSwiglu: dgrad through the
// activation, y = the saved [g | u] (M, 2K), out = its gradient (M, 2K), side = h (M, K) or null.
enum Mode { kFprop = 0, kDgrad = 1, kWgrad = 2, kFpropSwiglu = 3, kDgradSwiglu = 4 };
// the product that a mode is, its epilogue aside
__host__ __device__ constexpr Mode product_of(int mode) {
    return mode == kFpropSwiglu ? kFprop : mode == kDgradSwiglu ? kDgrad : (Mode)mode;
}

struct GemmCall {
    int mode;
    const void* tok;     // fprop: X (M, K); dgrad: dY (M, N); wgrad: X (M, K)
    int64_t ld_tok;      // its row stride in elements
    const void* mat;     // fprop, dgrad: W (E, N, K); wgrad: dY (M, N)
    int64_t ld_mat;      // wgrad: row stride of dY in elements
    const void* bias;    // fprop: (E, N) bf16 or null
    int64_t M, N, K;
    int E;
    const int64_t* m_splits;
    void* out;           // fprop (M, N), dgrad (M, K), wgrad (E, N, K)
    int out_f32;
    int accumulate;      // wgrad
    int32_t* status;
    const void* y = nullptr;  // the SwiGLU modes
    void* side = nullptr;
};
cudaError_t run_gemm(const GemmCall& c, cudaStream_t s);
// fprop and dgrad of at most kFewRows rows an expert on average
constexpr int kFewRows = 32;
cudaError_t run_gemm_few(const GemmCall& c, cudaStream_t s);
// CTAs (1, 2, 4 or 8) that share a tile's sum of `blocks` stages when a product has `tiles` one-SM tiles
int split_of(int64_t tiles, int64_t blocks);

struct Int8Call {
    const void* xq;      // (M, K) int8
    const float* xs;     // (M)
    const void* wq;      // (E, N, K) int8
    const float* ws;     // (E, N)
    const void* bias;    // (E, N) bf16 or null
    int64_t M, N, K;
    int E;
    const int64_t* m_splits;
    void* out;           // (M, N)
    int out_f32;
    int32_t* status;
};
cudaError_t run_int8(const Int8Call& c, cudaStream_t s);
// the int8 product, and fprop where its tiles leave SMs idle, of at most kVecRows rows an expert on average;
// int8: K up to kVecDepth
constexpr int kVecRows = 4;
constexpr int64_t kVecDepth = (1 << 17) - 16;  // |codes| <= 128: sums below 2^31
cudaError_t run_fprop_vec(const GemmCall& c, cudaStream_t s);
cudaError_t run_int8_vec(const Int8Call& c, cudaStream_t s);
cudaError_t run_int8_quantize(const void* x, int64_t M, int64_t K, int64_t ld, void* q, float* scale, cudaStream_t s);

// fp8 products with a scale for each block of kFp8Block values of a row and kFp8Block x kFp8Block of a weight.
constexpr int kFp8Block = 128;
struct Fp8Call {
    int mode;            // kFprop or kDgrad
    const void* tq;      // fprop: codes of X (M, K); dgrad: of dY (M, N)
    const float* ts;     // their scales (blocks of the sum, M)
    const void* wq;      // (E, N, K) codes
    const float* ws;     // (E, blocks of N, blocks of K)
    const void* bias;    // fprop: (E, N) bf16 or null
    int64_t M, N, K;
    int E;
    const int64_t* m_splits;
    void* out;           // fprop (M, N), dgrad (M, K)
    int out_f32;
    int32_t* status;
};
cudaError_t run_fp8(const Fp8Call& c, cudaStream_t s);
cudaError_t run_fp8_quantize_rows(const void* x, int64_t M, int64_t K, int64_t ld, void* q, float* scale, cudaStream_t s);
cudaError_t run_fp8_quantize_weight(const void* w, int64_t N, int64_t K, int E, void* q, float* scale, cudaStream_t s);

// Encodes a tensor map of int8, bf16 or fp32 elements (by their bytes) in up
// to five dimensions: dims and box innermost first, strides in bytes of
// dimensions 1 and up, the swizzle of 128, 64 or 0 (none) bytes. False on failure.
bool encode_tmap(CUtensorMap* m, const void* base, int elem_bytes, int rank, const int64_t* dims,
                 const int64_t* strides, const int* box, int swizzle_bytes = 128);
int sm_count();

// t of 65536 elements dropped; scale = 65536 / (65536 - t), 0 when t = 65536.
cudaError_t run_swiglu_dropout_fwd(const void* y, int64_t M, int64_t F, const int64_t* rng, uint32_t t, void* h,
                                   cudaStream_t s);
cudaError_t run_swiglu_dropout_bwd(const void* dh, const void* y, int64_t M, int64_t F, const int64_t* rng, uint32_t t,
                                   void* dy, cudaStream_t s);
cudaError_t run_dropout(const void* x, const void* residual, int64_t n, int f32, const int64_t* rng, uint32_t t,
                        void* out, cudaStream_t s);

}  // namespace ragged
}  // namespace mxq
