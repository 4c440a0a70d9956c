// mxq_dropout.cu -- dropout whose mask is made from a counter and never
// stored: the same {seed, offset} gives the same mask in the forward pass, in
// the backward pass and on any launch shape.
//
// Element i (row-major index of the (M, F) tensor that is dropped) is dropped
// when its 16-bit word is below t = round(65536 p), and scaled by
// 65536 / (65536 - t) otherwise, so that the expectation is kept exactly for
// the probability t / 65536 that is used. Its word is the (i mod 8)-th, low
// half first, of Philox 4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011) at the counter
// (i div 8, offset) under the key `seed`, all 64-bit, low word first. 16 bits
// an element halve the generator's work against 32.
//
// A dropped element is selected away, not multiplied by 0: an infinity or NaN
// in it does not reach the output or the gradient.
#include <cuda_bf16.h>

#include <algorithm>

#include "mxq_common.cuh"
#include "mxq_ragged.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace ragged {

// The eight 16-bit words of counter `block`, two per 32-bit word.
__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}
// Which elements are kept, as a threshold on a word shifted to the top of 32
// bits: half >= t is (half << 16) > ((t - 1) << 16 | 0xFFFF) whatever the low
// bits hold, for t = 1 .. 65536; `all` stands for t = 0. One shift (low halves
// only) and one comparison an element.
struct Keep {
    uint32_t above;
    bool all;
};
__host__ __device__ __forceinline__ Keep keep_of(uint32_t t) {
    return Keep{t ? ((t - 1) << 16 | 0xFFFFu) : 0u, t == 0};
}
__device__ __forceinline__ bool kept(const uint4& w, int j, const Keep& k) {
    const uint32_t x = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
    return ((j & 1) ? x : x << 16) > k.above || k.all;
}

// Position of a thread's 8-element vector in rows of `per` vectors, and its
// advance by `step` vectors, without a division in the loop.
struct Cursor {
    int64_t i, m;
    uint32_t f;
    int64_t dm;
    uint32_t df;
    __device__ Cursor(int64_t start, int64_t step, uint32_t per)
        : i(start), m(start / per), f((uint32_t)(start % per)), dm(step / per), df((uint32_t)(step % per)) {}
    __device__ void advance(int64_t step, uint32_t per) {
        i += step;
        m += dm;
        f += df;
        if (f >= per) {
            f -= per;
            ++m;
        }
    }
};

struct Rng {
    uint64_t seed, offset;
};
__device__ __forceinline__ Rng load_rng(const int64_t* rng) {
    return Rng{(uint64_t)rng[0], (uint64_t)rng[1]};
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16lo(ws[j]);
        f[2 * j + 1] = bf16hi(ws[j]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Bound by HBM: 6 bytes an element (10 in the gradient) against about 25 issued
// instructions, the generator's ten rounds shared by eight elements and two
// lanes to an instruction in the activation. 65536 x 1536: 95.5 us, 6.3 TB/s
// (122 us with an index division per vector and scalar steps); the gradient of
// 83968 x 1024: 128 us, 6.7 TB/s.
__global__ void __launch_bounds__(256) swiglu_dropout_fwd_kernel(const uint16_t* y, int64_t M, int64_t F,
                                                                 const int64_t* rng, Keep k, float scale,
                                                                 uint16_t* h) {
    wait_for_stream();
    const uint32_t per = (uint32_t)(F / 8);
    const int64_t vecs = M * per, step = (int64_t)gridDim.x * blockDim.x;
    Cursor c((int64_t)blockIdx.x * blockDim.x + threadIdx.x, step, per);
    if (c.i >= vecs) return;
    const Rng r = load_rng(rng);
    for (; c.i < vecs; c.advance(step, per)) {
        const uint4* row = reinterpret_cast<const uint4*>(y + c.m * 2 * F);
        const uint4 gw = row[c.f], uw = row[c.f + per];
        const uint4 w = philox((uint64_t)c.i, r.offset, r.seed);
        const uint32_t gs[4] = {gw.x, gw.y, gw.z, gw.w}, us[4] = {uw.x, uw.y, uw.z, uw.w};
        float o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = swiglu_h_x2(make_float2(bf16lo(gs[j]), bf16hi(gs[j])), make_float2(bf16lo(us[j]), bf16hi(us[j])));
            const float2 s = f2unpack(f2mul(f2pack(v.x, v.y), f2splat(scale)));
            o[2 * j] = kept(w, 2 * j, k) ? s.x : 0.0f;
            o[2 * j + 1] = kept(w, 2 * j + 1, k) ? s.y : 0.0f;
        }
        *reinterpret_cast<uint4*>(h + c.i * 8) = pack8(o);
    }
}

__global__ void __launch_bounds__(256) swiglu_dropout_bwd_kernel(const uint16_t* dh, const uint16_t* y, int64_t M,
                                                                 int64_t F, const int64_t* rng, Keep k, float scale,
                                                                 uint16_t* dy) {
    wait_for_stream();
    const uint32_t per = (uint32_t)(F / 8);
    const int64_t vecs = M * per, step = (int64_t)gridDim.x * blockDim.x;
    Cursor c((int64_t)blockIdx.x * blockDim.x + threadIdx.x, step, per);
    if (c.i >= vecs) return;
    const Rng r = load_rng(rng);
    for (; c.i < vecs; c.advance(step, per)) {
        const uint4* row = reinterpret_cast<const uint4*>(y + c.m * 2 * F);
        const uint4 gw = row[c.f], uw = row[c.f + per], dw = reinterpret_cast<const uint4*>(dh)[c.i];
        const uint4 w = philox((uint64_t)c.i, r.offset, r.seed);
        const uint32_t gs[4] = {gw.x, gw.y, gw.z, gw.w}, us[4] = {uw.x, uw.y, uw.z, uw.w}, ds[4] = {dw.x, dw.y, dw.z, dw.w};
        float dg[8], du[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 a, b;
            swiglu_grads_x2(f2unpack(f2mul(f2pack(bf16lo(ds[j]), bf16hi(ds[j])), f2splat(scale))),
                            make_float2(bf16lo(gs[j]), bf16hi(gs[j])), make_float2(bf16lo(us[j]), bf16hi(us[j])), a, b);
            const bool k0 = kept(w, 2 * j, k), k1 = kept(w, 2 * j + 1, k);
            dg[2 * j] = k0 ? a.x : 0.0f;
            dg[2 * j + 1] = k1 ? a.y : 0.0f;
            du[2 * j] = k0 ? b.x : 0.0f;
            du[2 * j + 1] = k1 ? b.y : 0.0f;
        }
        uint4* out = reinterpret_cast<uint4*>(dy + c.m * 2 * F);
        out[c.f] = pack8(dg);
        out[c.f + per] = pack8(du);
    }
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
    unpack8(*reinterpret_cast<const uint4*>(p), f);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = pack8(f);
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// One vector of eight elements at x, `residual` and out + 8 i.
template <typename T>
__device__ __forceinline__ void dropout8(const uint4 w, float (&v)[8], const T* residual, Keep k, float scale, T* out) {
    float a[8];
    if (residual) load8(residual, a);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = kept(w, j, k) ? __fmul_rn(v[j], scale) : 0.0f;
        if (residual) v[j] = __fadd_rn(v[j], a[j]);
    }
    store8(out, v);
}

// out may be x or residual: a thread reads its elements before it writes them. A block takes 256 kAhead consecutive
// vectors at a time and, where all are whole, reads x's before it draws a word.
template <typename T, int kAhead>
__global__ void __launch_bounds__(256) dropout_kernel(const T* x, const T* residual, int64_t n, const int64_t* rng,
                                                      Keep k, float scale, T* out) {
    wait_for_stream();
    const Rng r = load_rng(rng);
    const int64_t vecs = (n + 7) / 8, whole = n / 8;
    constexpr int kTile = 256 * kAhead;  // a block's consecutive vectors
    for (int64_t t = (int64_t)blockIdx.x * kTile; t < vecs; t += (int64_t)gridDim.x * kTile) {
        if (t + kTile <= whole) {
            float v[kAhead][8];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) load8(x + 8 * (t + 256 * u + threadIdx.x), v[u]);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int64_t at = t + 256 * u + threadIdx.x;
                dropout8(philox((uint64_t)at, r.offset, r.seed), v[u], residual ? residual + 8 * at : nullptr, k, scale,
                         out + 8 * at);
            }
            continue;
        }
        for (int64_t i = t + threadIdx.x; i < vecs && i < t + kTile; i += 256) {
            const uint4 w = philox((uint64_t)i, r.offset, r.seed);
            if (i < whole) {
                float v[8];
                load8(x + 8 * i, v);
                dropout8(w, v, residual ? residual + 8 * i : nullptr, k, scale, out + 8 * i);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (8 * i + j < n) {
                        float v = kept(w, j, k) ? __fmul_rn(to_f32(x[8 * i + j]), scale) : 0.0f;
                        if (residual) v = __fadd_rn(v, to_f32(residual[8 * i + j]));
                        from_f32(out + 8 * i + j, v);
                    }
            }
        }
    }
}

static unsigned grid_for(int64_t vecs) {
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>((vecs + 255) / 256, (int64_t)sm_count() * 8));
}
static float scale_of(uint32_t t) { return t >= 65536u ? 0.0f : (float)(65536.0 / (65536 - (int)t)); }

cudaError_t run_swiglu_dropout_fwd(const void* y, int64_t M, int64_t F, const int64_t* rng, uint32_t t, void* h,
                                   cudaStream_t s) {
    if (M == 0) return cudaSuccess;
    return launch(swiglu_dropout_fwd_kernel, grid_for(M * (F / 8)), 256, s, 0, (const uint16_t*)y, M, F, rng, keep_of(t),
                  scale_of(t), (uint16_t*)h);
}
cudaError_t run_swiglu_dropout_bwd(const void* dh, const void* y, int64_t M, int64_t F, const int64_t* rng, uint32_t t,
                                   void* dy, cudaStream_t s) {
    if (M == 0) return cudaSuccess;
    return launch(swiglu_dropout_bwd_kernel, grid_for(M * (F / 8)), 256, s, 0, (const uint16_t*)dh, (const uint16_t*)y, M, F,
                  rng, keep_of(t), scale_of(t), (uint16_t*)dy);
}
template <typename T, int kAhead>
static cudaError_t launch_dropout(const void* x, const void* residual, int64_t n, const int64_t* rng, uint32_t t, void* out,
                                  cudaStream_t s) {
    return launch(dropout_kernel<T, kAhead>, grid_for((n + 7) / 8), 256, s, 0, (const T*)x, (const T*)residual, n, rng,
                  keep_of(t), scale_of(t), (T*)out);
}
cudaError_t run_dropout(const void* x, const void* residual, int64_t n, int f32, const int64_t* rng, uint32_t t,
                        void* out, cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    // Beyond one vector a thread, more in flight. 40961 x 2048 without and with the residual, us: bf16 (floors 49
    // and 74) one vector 64 and 77, two 56 and 75, four 58 and 90; fp32 (99 and 148) one 124 and 171, two 113 and
    // 171, four 111 and 148. Vectors a whole grid apart instead of a block's own next ones: bf16 two 61 and 90.
    // Small calls are left at one: 7 x 16384 takes 1.9 us, with two 2.0 and 2.3, with four 2.4 and 3.0.
    const bool one = (n + 7) / 8 <= (int64_t)sm_count() * 8 * 256;
    if (f32)
        return one ? launch_dropout<float, 1>(x, residual, n, rng, t, out, s)
                   : launch_dropout<float, 4>(x, residual, n, rng, t, out, s);
    return one ? launch_dropout<__nv_bfloat16, 1>(x, residual, n, rng, t, out, s)
               : launch_dropout<__nv_bfloat16, 2>(x, residual, n, rng, t, out, s);
}

}  // namespace ragged
}  // namespace mxq
