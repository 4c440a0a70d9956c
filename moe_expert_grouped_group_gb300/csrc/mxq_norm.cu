// mxq_norm.cu -- RMS norms before and after a block, fused with the block's
// gate, the residual scale and the residual:
//   r' = r + c gate[m] N(x; w_post),  n = N(r'; w_pre),
//   N(v; w) = v w rstd(v),            rstd(v) = 1 / sqrt(mean(v^2) + eps)
// and the gradients. With D the gradient of r' (from the residual stream and
// through n), xh = x rstd(x), rh = r' rstd(r'), a = c gate:
//   D    = dr' + rstd(r') (dn w_pre - rh mean(dn w_pre rh))
//   dr   = D,  dw_pre = sum_m dn rh,  dw_post = sum_m a D xh
//   dx   = a rstd(x) (D w_post - xh mean(D w_post xh))
//   dgate = c sum_f D w_post xh       (without w_post: dx = a D, xh = x)
//
// Bound by HBM: every tensor is read or written once. A row belongs to a team
// of W warps that keeps it in registers from the loads to the stores; each
// thread always has the same columns, so that the weights' gradients grow in
// its registers while the team walks its rows. A team's two sums over the row
// are the only exchange. All arithmetic is fp32; r', n, dx, dr are rounded
// once. n comes from r' before its rounding.
//
// The weights' gradients leave a block as one partial row each, which a second
// kernel adds up, so that results are the same bits from run to run.
#include <cuda_bf16.h>

#include <algorithm>

#include "mxq_internal.h"
#include "mxq_ragged.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace norm {

using ragged::wait_for_stream;

// Eight consecutive elements as they lie in memory.
template <class T>
struct Pack;
template <>
struct Pack<__nv_bfloat16> {
    uint4 v;
    __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ void values(float (&f)[8]) const {
        f[0] = bf16lo(v.x), f[1] = bf16hi(v.x), f[2] = bf16lo(v.y), f[3] = bf16hi(v.y);
        f[4] = bf16lo(v.z), f[5] = bf16hi(v.z), f[6] = bf16lo(v.w), f[7] = bf16hi(v.w);
    }
    static __device__ void store(__nv_bfloat16* p, const float (&f)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(ragged::bf16x2_bits(f[0], f[1]), ragged::bf16x2_bits(f[2], f[3]),
                                                  ragged::bf16x2_bits(f[4], f[5]), ragged::bf16x2_bits(f[6], f[7]));
    }
};
template <>
struct Pack<float> {
    float4 a, b;
    __device__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ void values(float (&f)[8]) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    static __device__ void store(float* p, const float (&f)[8]) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
};

constexpr int kMaxWarps = 16, kMaxThreads = 32 * kMaxWarps;

// Where a thread stands: blocks of `teams` teams of W warps; with more than one team a team is one warp.
struct Team {
    int W, teams, team, tid;  // tid: thread of the team
    __device__ explicit Team(int W_) : W(W_), teams(blockDim.x / (32 * W_)), team(threadIdx.x / (32 * W_)) {
        tid = threadIdx.x - team * 32 * W;
    }
    // The sum of v over the team, the same bits in every thread. Called by all threads of a block alike; buf
    // alternates between two calls.
    __device__ float sum(float v, float (&buf)[kMaxWarps]) const {
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (W == 1) return v;
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        const int k = threadIdx.x & (kMaxWarps - 1);  // both halves of a warp add the same
        float s = k < W ? buf[k] : 0.0f;
#pragma unroll
        for (int o = kMaxWarps / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    }
};

template <class T>
struct Fwd {
    const T *x, *residual, *post, *pre;
    const float* gate;
    int64_t M;
    int F;
    float scale, eps;
    T *res, *n;
    float* stats;
};

template <class T, int NV>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(Fwd<T> p, int W) {
    __shared__ float buf[2][kMaxWarps];
    const Team t(W);
    const int step = 256 * W, f0 = 8 * t.tid;  // a thread's columns: f0 + i * step + 0 .. 7
    const float inv = 1.0f / (float)p.F;
    wait_for_stream();
    for (int64_t m = (int64_t)blockIdx.x * t.teams + t.team; m < p.M; m += (int64_t)gridDim.x * t.teams) {
        const int64_t at = m * p.F;
        Pack<T> x[NV], r[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i].zero();
            r[i].zero();
            if (f0 + i * step < p.F) {
                x[i].load(p.x + at + f0 + i * step);
                if (p.residual) r[i].load(p.residual + at + f0 + i * step);
            }
        }
        float a = p.scale, f[8], rstd = 1.0f;
        if (p.gate) a *= p.gate[m];
        if (p.post) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[i].values(f);
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(f[j], f[j], s);
            }
            rstd = 1.0f / sqrtf(fmaf(t.sum(s, buf[0]), inv, p.eps));
        }
        if (p.stats && t.tid == 0) p.stats[m] = rstd;
        float v[NV][8], s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float w[8];
            x[i].values(f);
            r[i].values(v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.0f;
            if (f0 + i * step >= p.F) continue;
            if (p.post) {
                Pack<T> k;
                k.load(p.post + f0 + i * step);
                k.values(w);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = fmaf(a, f[j] * rstd * w[j], v[i][j]);
                s = fmaf(v[i][j], v[i][j], s);
            }
            if (p.res) Pack<T>::store(p.res + at + f0 + i * step, v[i]);
        }
        if (p.pre) {
            rstd = 1.0f / sqrtf(fmaf(t.sum(s, buf[1]), inv, p.eps));
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (f0 + i * step < p.F) {
                    Pack<T> k;
                    float w[8];
                    k.load(p.pre + f0 + i * step);
                    k.values(w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = v[i][j] * rstd * w[j];
                    Pack<T>::store(p.n + at + f0 + i * step, f);
                }
        } else {
            rstd = 1.0f;
            if (W > 1) __syncthreads();  // buf[0] is read before the next row writes it
        }
        if (p.stats && t.tid == 0) p.stats[p.M + m] = rstd;
        if (!p.post && W > 1) __syncthreads();  // and buf[1]
    }
}

template <class T>
struct Bwd {
    const T *dres, *dn, *x, *res, *post, *pre;
    const float *gate, *stats;
    int64_t M;
    int F;
    float scale;
    T *dx, *dr;
    float *dgate, *partials;  // partials: (2, blocks, F): of w_post, of w_pre
};

// kHold: the row stays in registers from its one read. Otherwise (rows of more than 16 KB a tensor) each of the three
// passes over the row reads what it needs, the second and third time from L1 or L2. kSums: the weights' gradients
// grow in shared memory instead of registers.
template <class T, int NV, bool kHold, bool kSums>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(Bwd<T> p, int W) {
    __shared__ float buf[2][kMaxWarps];
    extern __shared__ __align__(16) float sums[];  // kSums: (2, F); teams > 1: (teams, F)
    const Team t(W);
    const int step = 256 * W, f0 = 8 * t.tid;
    const float inv = 1.0f / (float)p.F;
    constexpr int kRegs = kSums ? 1 : NV, kHeld = kHold ? NV : 1;
    float d_post[kRegs][8], d_pre[kRegs][8];
#pragma unroll
    for (int i = 0; i < kRegs; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) d_post[i][j] = d_pre[i][j] = 0.0f;
    if (kSums)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (f0 + i * step < p.F) {
                Pack<float>::store(sums + f0 + i * step, d_post[0]);
                Pack<float>::store(sums + p.F + f0 + i * step, d_pre[0]);
            }
    wait_for_stream();
    const bool dots = p.post || p.gate;
    // the values of a tensor's columns i, from registers or from memory
    const auto values = [&](const Pack<T>(&held)[kHeld], const T* from, int i, float (&f)[8]) {
        Pack<T> k = held[kHold ? i : 0];
        if (!kHold) {
            k.zero();
            if (from) k.load(from + f0 + i * step);
        }
        k.values(f);
    };
    const auto weights = [&](const T* w, int i, float (&f)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 1.0f;
        if (w) {
            Pack<T> k;
            k.load(w + f0 + i * step);
            k.values(f);
        }
    };
    const auto add = [&](float (&d)[kRegs][8], int row, int i, const float (&v)[8]) {
        if constexpr (kSums) {
            Pack<float> k;
            float f[8];
            k.load(sums + row * p.F + f0 + i * step);
            k.values(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += v[j];
            Pack<float>::store(sums + row * p.F + f0 + i * step, f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[i][j] += v[j];
        }
    };
    for (int64_t m = (int64_t)blockIdx.x * t.teams + t.team; m < p.M; m += (int64_t)gridDim.x * t.teams) {
        const int64_t at = m * p.F;
        const T *x_row = dots ? p.x + at : nullptr, *r_row = p.pre ? p.res + at : nullptr;
        const T *dn_row = p.pre ? p.dn + at : nullptr, *dr_row = p.dres ? p.dres + at : nullptr;
        Pack<T> x[kHeld], r[kHeld], dn[kHeld], dr[kHeld];
        if (kHold)
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                x[i].zero(), r[i].zero(), dn[i].zero(), dr[i].zero();
                if (f0 + i * step >= p.F) continue;
                if (r_row) r[i].load(r_row + f0 + i * step);
                if (dn_row) dn[i].load(dn_row + f0 + i * step);
                if (dr_row) dr[i].load(dr_row + f0 + i * step);
                if (x_row) x[i].load(x_row + f0 + i * step);
            }
        const float rstd1 = p.post ? p.stats[m] : 1.0f, rstd2 = p.pre ? p.stats[p.M + m] : 0.0f;
        const float a = p.gate ? p.scale * p.gate[m] : p.scale;
        float mean = 0.0f, dot = 0.0f, D[NV][8];
        if (p.pre) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (f0 + i * step >= p.F) continue;
                float rh[8], g[8], w[8];
                values(r, r_row, i, rh);
                values(dn, dn_row, i, g);
                weights(p.pre, i, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    rh[j] *= g[j] * rstd2;
                    s = fmaf(rh[j], w[j], s);
                }
                add(d_pre, 1, i, rh);
            }
            mean = t.sum(s, buf[0]) * inv;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (f0 + i * step >= p.F) continue;
            float rh[8], g[8], w[8], xh[8];
            values(r, r_row, i, rh);
            values(dn, dn_row, i, g);
            values(dr, dr_row, i, D[i]);
            weights(p.pre, i, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) D[i][j] = fmaf(rstd2, fmaf(-rh[j] * rstd2, mean, g[j] * w[j]), D[i][j]);
            if (p.dr) Pack<T>::store(p.dr + at + f0 + i * step, D[i]);
            if (!dots) continue;
            values(x, x_row, i, xh);
            weights(p.post, i, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[j] *= rstd1 * D[i][j];
                dot = fmaf(xh[j], w[j], dot);
                xh[j] *= a;
            }
            if (p.post) add(d_post, 0, i, xh);
        }
        if (dots) {
            dot = t.sum(dot, buf[1]);
            if (p.dgate && t.tid == 0) p.dgate[m] = p.scale * dot;
        } else if (W > 1) {
            __syncthreads();  // buf[0] is read before the next row writes it
        }
        if (!p.pre && W > 1) __syncthreads();  // and buf[1]
        if (!p.dx) continue;
        const float c = p.post ? dot * inv * rstd1 : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (f0 + i * step >= p.F) continue;
            float xv[8], w[8];
            values(x, x_row, i, xv);
            weights(p.post, i, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) xv[j] = a * rstd1 * fmaf(-xv[j], c, D[i][j] * w[j]);
            Pack<T>::store(p.dx + at + f0 + i * step, xv);
        }
    }
    // this block's part of the weights' gradients
    const auto leave = [&](const float (&d)[kRegs][8], int row, float* out) {
        if (t.teams > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kRegs; ++i)
                if (f0 + i * step < p.F) Pack<float>::store(sums + t.team * p.F + f0 + i * step, d[i]);
            __syncthreads();
            for (int f = threadIdx.x; f < p.F; f += blockDim.x) {
                float s = 0.0f;
                for (int k = 0; k < t.teams; ++k) s += sums[k * p.F + f];
                out[f] = s;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (f0 + i * step >= p.F) continue;
                float f[8];
                if constexpr (kSums) {
                    Pack<float> k;
                    k.load(sums + row * p.F + f0 + i * step);
                    k.values(f);
                    Pack<float>::store(out + f0 + i * step, f);
                } else {
                    Pack<float>::store(out + f0 + i * step, d[i]);
                }
            }
        }
    };
    if (p.post) leave(d_post, 0, p.partials + (int64_t)blockIdx.x * p.F);
    if (p.pre) leave(d_pre, 1, p.partials + ((int64_t)gridDim.x + blockIdx.x) * p.F);
}

// out[f] = the sum of a weight's partial rows: 32 columns a block, row k by warp k mod 8.
__global__ void __launch_bounds__(256) norm_weights_kernel(const float* partials, int blocks, int F, float* d_post,
                                                           float* d_pre) {
    __shared__ float s_sum[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, f = blockIdx.x * 32 + lane;
    float* out = blockIdx.y ? d_pre : d_post;
    wait_for_stream();
    if (!out) return;
    float s = 0.0f;
    if (f < F)
        for (int k = warp; k < blocks; k += 8) s += partials[((int64_t)blockIdx.y * blocks + k) * F + f];
    s_sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && f < F) {
        for (int k = 1; k < 8; ++k) s += s_sum[k][lane];
        out[f] = s;
    }
}

// ------------------------------------------------------------------ host side
// A team of W warps with nv vectors of eight columns a thread; teams > 1 share a block when a team is one warp.
struct Shape {
    int nv, W, teams;
};
static Shape shape_of(int64_t F) {
    Shape s;
    s.nv = F > 8192 ? 4 : F > 4096 ? 2 : 1;
    s.W = (int)((F + 256 * s.nv - 1) / (256 * s.nv));
    s.teams = s.W == 1 ? 8 : 1;
    return s;
}

template <class T>
static cudaError_t fwd(const NormFwd& c, cudaStream_t st) {
    const Fwd<T> p{(const T*)c.x, (const T*)c.residual, (const T*)c.post, (const T*)c.pre, c.gate, c.M, (int)c.F,
                   c.scale, c.eps, (T*)c.res, (T*)c.n, c.stats};
    const Shape s = shape_of(c.F);
    const unsigned threads = 32 * s.W * s.teams;
    const int64_t most = (int64_t)ragged::sm_count() * (2048 / threads);
    const unsigned grid = (unsigned)std::min<int64_t>((c.M + s.teams - 1) / s.teams, most);
    switch (s.nv) {
        case 1: return ragged::launch(norm_fwd_kernel<T, 1>, grid, threads, st, 0, p, s.W);
        case 2: return ragged::launch(norm_fwd_kernel<T, 2>, grid, threads, st, 0, p, s.W);
        default: return ragged::launch(norm_fwd_kernel<T, 4>, grid, threads, st, 0, p, s.W);
    }
}

// Blocks of the backward kernel, each of which leaves a partial row per weight: a rule on the shape alone (152 is this
// GPU's number of SMs), so that a workspace's size does not depend on the current device.
static int64_t bwd_blocks(int64_t M, int64_t F) {
    const Shape s = shape_of(F);
    const int threads = 32 * s.W * s.teams;
    return std::max<int64_t>(1, std::min<int64_t>((M + s.teams - 1) / s.teams, 152 * std::max(1, 768 / threads)));
}

template <class T, int NV>
static cudaError_t bwd_rows(const Bwd<T>& p, const Shape& s, unsigned grid, cudaStream_t st) {
    constexpr bool kHold = NV * sizeof(T) <= 4, kSums = NV == 4;
    const int smem = kSums ? 8 * p.F : s.teams > 1 ? 4 * s.teams * p.F : 0;
    if (kSums) {
        const cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<T, NV, kHold, kSums>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * kNormMaxWidth);
        if (e != cudaSuccess) return e;
    }
    return ragged::launch(norm_bwd_kernel<T, NV, kHold, kSums>, grid, 32 * s.W * s.teams, st, smem, p, s.W);
}

template <class T>
static cudaError_t bwd(const NormBwd& c, cudaStream_t st) {
    const Bwd<T> p{(const T*)c.dres, (const T*)c.dn, (const T*)c.x, (const T*)c.res, (const T*)c.post, (const T*)c.pre,
                   c.gate, c.stats, c.M, (int)c.F, c.scale, (T*)c.dx, (T*)c.dr, c.dgate, c.partials};
    const Shape s = shape_of(c.F);
    const unsigned grid = (unsigned)bwd_blocks(c.M, c.F);
    const cudaError_t e = s.nv == 1   ? bwd_rows<T, 1>(p, s, grid, st)
                          : s.nv == 2 ? bwd_rows<T, 2>(p, s, grid, st)
                                      : bwd_rows<T, 4>(p, s, grid, st);
    if (e != cudaSuccess || (!c.dpost && !c.dpre)) return e;
    return ragged::launch(norm_weights_kernel, dim3((unsigned)((c.F + 31) / 32), 2), 256, st, 0, (const float*)c.partials,
                          (int)grid, (int)c.F, c.dpost, c.dpre);
}

}  // namespace norm

size_t norm_bwd_workspace(int64_t M, int64_t F) {
    return (size_t)(2 * norm::bwd_blocks(M, F)) * (size_t)F * sizeof(float);
}
cudaError_t run_norm_fwd(const NormFwd& c, cudaStream_t s) {
    if (c.M == 0) return cudaSuccess;
    return c.f32 ? norm::fwd<float>(c, s) : norm::fwd<__nv_bfloat16>(c, s);
}
cudaError_t run_norm_bwd(const NormBwd& c, cudaStream_t s) {
    return c.f32 ? norm::bwd<float>(c, s) : norm::bwd<__nv_bfloat16>(c, s);
}

}  // namespace mxq
