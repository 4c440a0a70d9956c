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
// Bound by HBM: every tensor is read or written once. What it takes is loads in
// flight all the time: a row's two sums, one after the other, each leave the SM
// idle for a few hundred cycles. So rows come by bulk copies into a ring of
// shared memory, two rows ahead of the one that is computed.
//
// A row of more than kWarpWidth columns belongs to a cluster of 1 to 8 CTAs,
// eight columns to a thread; the CTAs' sums meet in each
// other's shared memory. Shorter rows belong to 8, 16 or 32 lanes of a warp,
// which in the backward kernel hold the next row in registers. A thread always has the same columns,
// so that the weights' gradients grow in its registers while it walks its
// rows; they leave a CTA as one partial row each, which a second kernel adds up
// in a fixed order. All arithmetic is fp32; r', n, dx, dr are rounded once. n
// comes from r' before its rounding.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "mxq_internal.h"
#include "mxq_ragged.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace norm {

using ragged::wait_for_stream;

__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// Eight fp32 values, two to a packed instruction. The backward rows compute that way, which leaves registers for half as
// many rows again on an SM (41k x 2048: 157 us against 178). The forward rows get no room by it, and a packed instruction
// takes as long as two: 120 us against 103.
struct V8 {
    uint64_t p[4];
    V8() = default;
    explicit __device__ V8(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = f2pack(f[2 * i], f[2 * i + 1]);
    }
    __device__ void split(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = f2unpack(p[i]);
            f[2 * i] = v.x, f[2 * i + 1] = v.y;
        }
    }
    __device__ void fill(float v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = f2splat(v);
    }
    __device__ float sum() const {
        const float2 s = f2unpack(f2add(f2add(p[0], p[1]), f2add(p[2], p[3])));
        return s.x + s.y;
    }
};
// Eight consecutive elements as they lie in memory.
template <class T>
struct Pack;
template <>
struct Pack<__nv_bfloat16> {
    uint4 v;
    __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ void load_shared(uint32_t a) { v = ld_shared(a); }
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
    __device__ void load_shared(uint32_t p) {
        const uint4 u = ld_shared(p), w = ld_shared(p + 16);
        a = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
        b = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
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

template <class T>
__device__ __forceinline__ V8 packed(const Pack<T>& k) {
    float f[8];
    k.values(f);
    return V8(f);
}
template <class T>
__device__ __forceinline__ void store8(T* p, const V8& v) {
    float f[8];
    v.split(f);
    Pack<T>::store(p, f);
}

constexpr int kWarpWidth = 256;  // widest row of a warp
constexpr int kThreads = 256;    // threads of a CTA for such rows
// Most threads of a CTA for wider ones, with eight columns each, and of one that shares its rows with others.
constexpr int kFwdThreads = 1024, kBwdThreads = 512, kShareThreads = 256;
constexpr int kMaxParts = 64;  // warps of a row

// Bulk copy into this CTA's shared memory, counted on its barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"((uint64_t)src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void async_load(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"((uint64_t)__cvta_generic_to_global(src)) : "memory");
}

// The rows of kTensors tensors on their way to this CTA, and what there is one number of for a row (its statistics, its
// gate): row n of the CTA's walk in stage n mod kStages
// (32 bits: no memory holds more rows). The numbers come the same way as the rows: read by every thread one row ahead into
// registers, they were waited for at once (gradients of 84k x 1024: 300 us against 174).
template <class T, int kTensors, int kStages>
struct Rows {
    const T* from[kTensors];  // this CTA's columns of row 0; null: not read
    const float* scalars[3];  // of row 0; null: not read
    int64_t M, F;
    uint32_t at, scalars_at, full, bytes, total;
    int width;
    __device__ uint32_t stage_bytes() const { return kTensors * width * (uint32_t)sizeof(T); }
    // by one thread
    __device__ void load(uint32_t n, int64_t m) const {
        if (m >= M) return;
        const int s = (int)(n % kStages);
        mbar_expect_tx(full + 8 * s, total);
#pragma unroll
        for (int i = 0; i < kTensors; ++i)
            if (from[i])
                bulk_load(at + s * stage_bytes() + i * width * (uint32_t)sizeof(T), from[i] + m * F, bytes, full + 8 * s);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (scalars[i]) async_load(scalars_at + 16 * s + 4 * i, scalars[i] + m);
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full + 8 * s) : "memory");
    }
    __device__ float scalar(uint32_t n, int i, float none) const {
        float v = none;
        if (scalars[i])
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(scalars_at + 16 * (int)(n % kStages) + 4 * i) : "memory");
        return v;
    }
    __device__ void get(uint32_t n, int i, int f, Pack<T>& p) const {
        const uint32_t a = at + (uint32_t)(n % kStages) * stage_bytes() + (i * width + f) * (uint32_t)sizeof(T);
        p.load_shared(a);
    }
    __device__ bool wait(uint32_t n, volatile int* abort_flag) const {
        return mbar_wait(full + 8 * (int)(n % kStages), (uint32_t)(n / kStages) & 1, abort_flag);
    }
    // After an expired wait, which lets the others return at once: the last rows are waited for again, so that no copy
    // is in flight when the CTA ends. n: rows of the walk.
    __device__ void drain(int64_t n) const {
        volatile int unused = 0;
        for (int64_t k = n > kStages ? n - kStages : 0; k < n; ++k)
            mbar_wait(full + 8 * (int)(k % kStages), (uint32_t)(k / kStages) & 1, &unused);
    }
};

// Sums over a row, which kC CTAs of W warps share: every warp sends its part to all CTAs, where all threads add the
// parts in the same order. Two buffers in turn: a warp sends the part after next only when it has the sum after this
// one, so when all warps have read this one.
template <int kC>
struct RowSum {
    uint32_t at, bar;  // [2][kMaxParts] floats; two barriers (kC > 1)
    int W, rank;
    uint32_t turn = 0;
    __device__ RowSum(uint32_t at_, uint32_t bar_, int W_, int rank_) : at(at_), bar(bar_), W(W_), rank(rank_) {}
    __device__ float sum(float v, volatile int* abort_flag) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const uint32_t side = turn & 1, phase = turn >> 1 & 1, to = at + (side * kMaxParts + rank * W + warp) * 4;
        ++turn;
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if constexpr (kC == 1) {
            if (lane == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
            __syncthreads();
        } else {
            if (threadIdx.x == 0) mbar_expect_tx(bar + 8 * side, 4 * kC * W);
            if (lane < kC)
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                                 ragged::mapa(to, lane)),
                             "r"(__float_as_uint(v)), "r"(ragged::mapa(bar + 8 * side, lane))
                             : "memory");
            ragged::mbar_wait_cluster(bar + 8 * side, phase, abort_flag);
            __syncwarp();
        }
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < (kC == 1 ? 1 : 2); ++k)
            if (lane + 32 * k < kC * W) {
                float x;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at + (side * kMaxParts + lane + 32 * k) * 4) : "memory");
                s += x;
            }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    }
};

// Dynamic shared memory: the ring, then the sums, the rows' numbers and the barriers.
constexpr int kStages = 3, kSumBytes = 2 * kMaxParts * 4, kScalarBytes = 16 * kStages, kTailBytes = kSumBytes + kScalarBytes + 64;
constexpr int smem_bytes(int tensors, int width, int size) { return kStages * tensors * width * size + kTailBytes; }
constexpr int kMostSmem = std::max(smem_bytes(2, 8 * kFwdThreads, 4), smem_bytes(4, 8 * kBwdThreads, 4));
static_assert(kMostSmem <= 232448 && (2 + kStages) * 8 <= 64, "shared memory");
constexpr int kSmThreads = 768;  // threads of an SM's CTAs in the backward kernel, by their registers

// What a thread does with its eight columns of a row, in the order of the formulas. Weights: 1 without one.
template <class T>
__device__ __forceinline__ void weights8(const T* w, int f, bool live, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.0f;
    if (w && live) {
        Pack<T> k;
        k.load(w + f);
        k.values(v);
    }
}

template <class T>
__device__ __forceinline__ V8 packed_weights8(const T* w, int f, bool live) {
    float v[8];
    weights8(w, f, live, v);
    return V8(v);
}

template <class T>
struct Fwd {
    const T *x, *residual, *post, *pre;
    const float* gate;
    int64_t M;
    int F;
    float scale, eps;
    T *res, *n;
    float* stats;
    int32_t* status;
};

// f: the thread's first column; sum(v) adds over the row; `mine`: this thread writes the row's statistics.
template <class T, class S>
__device__ __forceinline__ void fwd_row(const Fwd<T>& p, int64_t m, int f, bool live, bool mine, float gate, const Pack<T>& xp,
                                        const Pack<T>& rp, const float (&w_post)[8], const float (&w_pre)[8], float inv,
                                        S sum) {
    // rsqrtf is off by two units of the last place at most; 1 / sqrtf took every thread of a row through two long
    // sequences (41k x 2048: 118 us against 104)
    float x[8], v[8], rstd = 1.0f, s = 0.0f;
    xp.values(x);
    rp.values(v);
    if (p.post) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
        rstd = rsqrtf(fmaf(sum(s), inv, p.eps));
        s = 0.0f;
    }
    if (p.stats && mine) p.stats[m] = rstd;
    if (live) {
        const float a = p.scale * gate;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = fmaf(a, x[j] * rstd * w_post[j], v[j]);
            s = fmaf(v[j], v[j], s);
        }
        if (p.res) Pack<T>::store(p.res + m * p.F + f, v);
    }
    rstd = 1.0f;
    if (p.pre) {
        rstd = rsqrtf(fmaf(sum(s), inv, p.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= rstd * w_pre[j];
        if (live) Pack<T>::store(p.n + m * p.F + f, v);
    }
    if (p.stats && mine) p.stats[p.M + m] = rstd;
}

// Rows of up to kWarpWidth columns: kLanes lanes each. Many warps hide the loads here; with the next row in registers, as
// in the backward kernel, there were fewer (65536 x 256: 37 us against 30). 64 registers, not 40: 25 us.
template <class T, int kLanes>
__global__ void __launch_bounds__(kThreads, 4) norm_fwd_lanes_kernel(Fwd<T> p) {
    const int lane = threadIdx.x % kLanes, f = 8 * lane;
    const bool live = f < p.F;
    const float inv = 1.0f / (float)p.F;
    wait_for_stream();
    const int64_t step = (int64_t)gridDim.x * (kThreads / kLanes);
    int64_t m = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    // all lanes of a warp take as many turns: they share its shuffles
    for (int64_t first = m - threadIdx.x % 32 / kLanes; first < p.M; first += step, m += step) {
        Pack<T> x, r;
        x.zero(), r.zero();
        const bool mine = live && m < p.M;
        if (mine) {
            x.load(p.x + m * p.F + f);
            if (p.residual) r.load(p.residual + m * p.F + f);
        }
        const float gate = p.gate && m < p.M ? p.gate[m] : 1.0f;
        float w_post[8], w_pre[8];
        weights8(p.post, f, live, w_post);
        weights8(p.pre, f, live, w_pre);
        fwd_row(p, m, f, mine, lane == 0 && m < p.M, gate, x, r, w_post, w_pre, inv, [](float v) {
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            return v;
        });
    }
}

template <class T, int kC>
__global__ void __launch_bounds__(kFwdThreads) norm_fwd_kernel(Fwd<T> p, int width) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_abort;
    constexpr int kS = kStages;
    const int rank = kC > 1 ? (int)ragged::cta_rank() : 0, W = blockDim.x / 32;
    const int f0 = rank * width, mine = min(width, p.F - f0), f = 8 * (int)threadIdx.x;
    const bool live = f < mine;
    const float inv = 1.0f / (float)p.F;
    const uint32_t tail = smem_u32(smem) + kS * 2 * width * (uint32_t)sizeof(T), bars = tail + kSumBytes + kScalarBytes;
    volatile int* abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < 2 + kS; ++i) mbar_init(bars + 8 * i, i < 2 ? 1 : 2);  // the rows' numbers arrive by themselves
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_stream();
    __syncthreads();
    if (kC > 1) ragged::cluster_sync();
    const int64_t first = blockIdx.x / kC, step = gridDim.x / kC;
    const uint32_t bytes = mine * (uint32_t)sizeof(T);
    const Rows<T, 2, kS> rows{{p.x + f0, p.residual ? p.residual + f0 : nullptr}, {p.gate, nullptr, nullptr}, p.M, p.F,
                              smem_u32(smem), tail + kSumBytes, bars + 16, bytes, bytes * (1 + (p.residual != nullptr)), width};
    if (threadIdx.x == 0)
        for (int k = 0; k < kS; ++k) rows.load(k, first + k * step);
    RowSum<kC> sums(tail, bars, W, rank);
    float w_post[8], w_pre[8];
    weights8(p.post, f0 + f, live, w_post);
    weights8(p.pre, f0 + f, live, w_pre);
    uint32_t n = 0;
    for (int64_t m = first; m < p.M; m += step, ++n) {
        rows.wait(n, abort_flag);
        __syncwarp();
        Pack<T> x, r;
        x.zero(), r.zero();
        if (live) {
            rows.get(n, 0, f, x);
            if (p.residual) rows.get(n, 1, f, r);
        }
        // at a row's first exchange every thread has read the row before
        bool refill = threadIdx.x == 0 && n > 0;
        fwd_row(p, m, f0 + f, live, threadIdx.x == 0 && rank == 0, rows.scalar(n, 0, 1.0f), x, r, w_post, w_pre, inv, [&](float v) {
            v = sums.sum(v, abort_flag);
            if (refill) rows.load(n - 1 + kS, m + (kS - 1) * step);
            refill = false;
            return v;
        });
        if (!p.post && !p.pre) {
            __syncthreads();
            if (refill) rows.load(n - 1 + kS, m + (kS - 1) * step);
        }
    }
    __syncthreads();
    if (s_abort && threadIdx.x == 0) {
        rows.drain(n);
        if (p.status) atomicOr(p.status, MXQ_STATUS_WAIT_TIMEOUT);
    }
    if (kC > 1) ragged::cluster_sync();  // nothing is on its way to a CTA that has ended
}

template <class T>
struct Bwd {
    const T *dres, *dn, *x, *res, *post, *pre;
    const float *gate, *stats;
    int64_t M;
    int F;
    float scale;
    T *dx, *dr;
    float *dgate, *partials;  // partials: (2, parts, F): of w_post, of w_pre
    int32_t* status;
};

struct RowScalars {
    float rstd1, rstd2, gate;
    template <class T>
    __device__ void load(const Bwd<T>& p, int64_t m) {
        rstd1 = p.post ? p.stats[m] : 1.0f;
        rstd2 = p.pre ? p.stats[p.M + m] : 0.0f;
        gate = p.gate ? p.gate[m] : 1.0f;
    }
};

// get(i): dres (2) and x (3).
template <class T, class G, class S>
__device__ __forceinline__ void bwd_row(const Bwd<T>& p, int64_t m, int f, bool live, bool mine, const RowScalars& c,
                                        const Pack<T>& rp, const Pack<T>& np, G get, const V8& w_post, const V8& w_pre,
                                        V8& d_post, V8& d_pre, float inv, S sum) {
    V8 rh = packed(rp), g = packed(np), s;
    const float a = p.scale * c.gate;
    const uint64_t k2 = f2splat(c.rstd2);
    float mean = 0.0f;
    if (p.pre) {
        s.fill(0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rh.p[i] = f2mul(rh.p[i], k2);
            d_pre.p[i] = f2fma(g.p[i], rh.p[i], d_pre.p[i]);
            g.p[i] = f2mul(g.p[i], w_pre.p[i]);
            s.p[i] = f2mul(g.p[i], rh.p[i]);
        }
        mean = sum(s.sum()) * inv;
    }
    V8 D = packed(get(2));
    if (p.pre) {
        const uint64_t minus = f2splat(-mean);
#pragma unroll
        for (int i = 0; i < 4; ++i) D.p[i] = f2fma(k2, f2fma(rh.p[i], minus, g.p[i]), D.p[i]);
    }
    if (p.dr && live) store8(p.dr + m * p.F + f, D);
    float dot = 0.0f;
    V8 xh;
    xh.fill(0.0f);
    if (p.post || p.gate) {
        xh = packed(get(3));
        const uint64_t k1 = f2splat(c.rstd1), ka = f2splat(a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            xh.p[i] = f2mul(xh.p[i], k1);
            const uint64_t t = f2mul(D.p[i], xh.p[i]);
            d_post.p[i] = f2fma(ka, t, d_post.p[i]);
            s.p[i] = f2mul(t, w_post.p[i]);
        }
        dot = sum(s.sum());
        if (p.dgate && mine) p.dgate[m] = p.scale * dot;
    }
    if (!p.dx || !live) return;
    if (p.post) {
        const uint64_t minus = f2splat(-dot * inv), k = f2splat(a * c.rstd1);
#pragma unroll
        for (int i = 0; i < 4; ++i) D.p[i] = f2mul(k, f2fma(xh.p[i], minus, f2mul(D.p[i], w_post.p[i])));
    } else {
        const uint64_t k = f2splat(a);
#pragma unroll
        for (int i = 0; i < 4; ++i) D.p[i] = f2mul(k, D.p[i]);
    }
    store8(p.dx + m * p.F + f, D);
}

// Two blocks to an SM, whose warps hold the next rows in registers (65536 x 256, fp32: 69 us, with one block 82; of bf16 with
// two 44, with three and fewer registers 63).
template <class T, int kLanes>
__global__ void __launch_bounds__(kThreads, 2) norm_bwd_lanes_kernel(Bwd<T> p) {
    constexpr int kTeams = kThreads / kLanes;
    __shared__ __align__(16) float s_sum[kThreads / 32][kWarpWidth];
    const int lane = threadIdx.x % kLanes, f = 8 * lane;
    const bool live = f < p.F, dots = p.post || p.gate;
    const float inv = 1.0f / (float)p.F;
    wait_for_stream();
    const V8 w_post = packed_weights8(p.post, f, live), w_pre = packed_weights8(p.pre, f, live);
    V8 d_post, d_pre;
    d_post.fill(0.0f), d_pre.fill(0.0f);
    const int64_t step = (int64_t)gridDim.x * kTeams;
    int64_t m = (int64_t)blockIdx.x * kTeams + threadIdx.x / kLanes;
    const auto fetch = [&](int64_t row, Pack<T>(&v)[4], RowScalars& c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i].zero();
        c.rstd1 = c.rstd2 = c.gate = 0.0f;
        if (row >= p.M) return;
        const int64_t at = row * p.F + f;
        if (live) {
            if (p.pre) v[0].load(p.res + at), v[1].load(p.dn + at);
            if (p.dres) v[2].load(p.dres + at);
            if (dots) v[3].load(p.x + at);
        }
        c.load(p, row);
    };
    Pack<T> v[4], nv[4];
    RowScalars c, nc;
    fetch(m, v, c);
    for (int64_t first = m - threadIdx.x % 32 / kLanes; first < p.M; first += step, m += step) {
        fetch(m + step, nv, nc);
        // rows beyond the last are zeros and have no part in the sums
        bwd_row(p, m, f, live && m < p.M, lane == 0 && m < p.M, c, v[0], v[1],
                [&](int i) -> const Pack<T>& { return v[i]; }, w_post, w_pre, d_post, d_pre, inv, [](float s) {
#pragma unroll
                    for (int o = kLanes / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                    return s;
                });
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = nv[i];
        c = nc;
    }
    // the block's parts of the weights' gradients: over a warp's teams, then over the warps
    const auto leave = [&](V8& d, float* out) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int o = kLanes; o < 32; o <<= 1) d.p[i] = f2add(d.p[i], __shfl_xor_sync(0xffffffffu, d.p[i], o));
        __syncthreads();
        if (threadIdx.x % 32 < kLanes) store8(&s_sum[threadIdx.x / 32][f], d);
        __syncthreads();
        if ((int)threadIdx.x < p.F) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < kThreads / 32; ++k) s += s_sum[k][threadIdx.x];
            out[threadIdx.x] = s;
        }
    };
    if (p.post) leave(d_post, p.partials + (int64_t)blockIdx.x * p.F);
    if (p.pre) leave(d_pre, p.partials + ((int64_t)gridDim.x + blockIdx.x) * p.F);
}

template <class T, int kC>
__global__ void __launch_bounds__(kBwdThreads) norm_bwd_kernel(Bwd<T> p, int width) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_abort;
    constexpr int kS = kStages;
    const int rank = kC > 1 ? (int)ragged::cta_rank() : 0, W = blockDim.x / 32;
    const int f0 = rank * width, mine = min(width, p.F - f0), f = 8 * (int)threadIdx.x;
    const bool live = f < mine, dots = p.post || p.gate;
    const float inv = 1.0f / (float)p.F;
    const uint32_t tail = smem_u32(smem) + kS * 4 * width * (uint32_t)sizeof(T), bars = tail + kSumBytes + kScalarBytes;
    volatile int* abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < 2 + kS; ++i) mbar_init(bars + 8 * i, i < 2 ? 1 : 2);  // the rows' numbers arrive by themselves
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_stream();
    __syncthreads();
    if (kC > 1) ragged::cluster_sync();
    const int64_t first = blockIdx.x / kC, step = gridDim.x / kC;
    const uint32_t bytes = mine * (uint32_t)sizeof(T);
    const Rows<T, 4, kS> rows{{p.pre ? p.res + f0 : nullptr, p.pre ? p.dn + f0 : nullptr, p.dres ? p.dres + f0 : nullptr,
                               dots ? p.x + f0 : nullptr},
                              {p.post ? p.stats : nullptr, p.pre ? p.stats + p.M : nullptr, p.gate}, p.M, p.F,
                              smem_u32(smem), tail + kSumBytes, bars + 16, bytes,
                              bytes * (2 * (p.pre != nullptr) + (p.dres != nullptr) + dots), width};
    if (threadIdx.x == 0)
        for (int k = 0; k < kS; ++k) rows.load(k, first + k * step);
    RowSum<kC> sums(tail, bars, W, rank);
    const V8 w_post = packed_weights8(p.post, f0 + f, live), w_pre = packed_weights8(p.pre, f0 + f, live);
    V8 d_post, d_pre;
    d_post.fill(0.0f), d_pre.fill(0.0f);
    uint32_t n = 0;
    for (int64_t m = first; m < p.M; m += step, ++n) {
        rows.wait(n, abort_flag);
        __syncwarp();
        const RowScalars c{rows.scalar(n, 0, 1.0f), rows.scalar(n, 1, 0.0f), rows.scalar(n, 2, 1.0f)};
        const auto get = [&](int i) {
            Pack<T> v;
            v.zero();
            if (live && rows.from[i]) rows.get(n, i, f, v);
            return v;
        };
        // at a row's first exchange every thread has read the row before
        bool refill = threadIdx.x == 0 && n > 0;
        bwd_row(p, m, f0 + f, live, threadIdx.x == 0 && rank == 0, c, get(0), get(1), get, w_post, w_pre, d_post, d_pre, inv,
                [&](float s) {
                    s = sums.sum(s, abort_flag);
                    if (refill) rows.load(n - 1 + kS, m + (kS - 1) * step);
                    refill = false;
                    return s;
                });
        if (!p.pre && !dots) {
            __syncthreads();
            if (refill) rows.load(n - 1 + kS, m + (kS - 1) * step);
        }
    }
    __syncthreads();
    if (s_abort && threadIdx.x == 0) {
        rows.drain(n);
        if (p.status) atomicOr(p.status, MXQ_STATUS_WAIT_TIMEOUT);
    }
    const int64_t part = blockIdx.x / kC, parts = gridDim.x / kC;
    if (p.post && live) store8(p.partials + part * p.F + f0 + f, d_post);
    if (p.pre && live) store8(p.partials + (parts + part) * p.F + f0 + f, d_pre);
    if (kC > 1) ragged::cluster_sync();  // nothing is on its way to a CTA that has ended
}

// out[f] = the sum of a weight's partial rows: 32 columns a block, row k by warp k mod 32.
__global__ void __launch_bounds__(1024) norm_weights_kernel(const float* partials, int parts, int F, float* d_post,
                                                            float* d_pre) {
    __shared__ float s_sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, f = blockIdx.x * 32 + lane;
    float* out = blockIdx.y ? d_pre : d_post;
    wait_for_stream();
    if (!out) return;
    float s = 0.0f;
    if (f < F) {
        const float* from = partials + (int64_t)blockIdx.y * parts * F + f;
#pragma unroll 4
        for (int k = warp; k < parts; k += 32) s += from[(int64_t)k * F];
    }
    s_sum[lane][warp] = s;
    __syncthreads();
    s = s_sum[warp][lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && blockIdx.x * 32 + warp < F) out[blockIdx.x * 32 + warp] = s;
}

// ------------------------------------------------------------------ host side
// CTAs that share a row of F columns (0: lanes of a warp do), the columns and threads of each.
struct Shape {
    int ctas, width, threads;
};
static Shape shape_of(int64_t F, int most_threads) {
    if (F <= kWarpWidth) return {0, (int)F, kThreads};
    Shape s;
    s.ctas = 1;
    if (F > 8 * most_threads) most_threads = kShareThreads;
    while (s.ctas * 8 * most_threads < F) s.ctas *= 2;
    s.width = (int)((F / 8 + s.ctas - 1) / s.ctas * 8);
    s.threads = (s.width + 255) / 256 * 32;
    return s;
}

// `waves` times as many clusters as the device holds, no more than `clusters`, which is set to their number. The kernel's
// attribute and its co-residency are set and asked for once per device and number of threads.
template <auto kKernel, class P>
static cudaError_t launch_rows(const P& p, const Shape& s, int64_t& clusters, int waves, int smem, cudaStream_t st) {
    static std::atomic<int> cache[64][kFwdThreads / 32 + 1];
    int dev = 0, most = 0;
    cudaGetDevice(&dev);
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s.ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(s.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (dev >= 64 || (most = cache[dev][s.threads / 32].load(std::memory_order_acquire)) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(s.ctas * ragged::sm_count());
        // the widest rows of so many threads
        cfg.dynamicSmemBytes = (smem - kTailBytes) / s.width * (8 * s.threads) + kTailBytes;
        if (cudaOccupancyMaxActiveClusters(&most, (void*)kKernel, &cfg) != cudaSuccess || most <= 0) {
            cudaGetLastError();
            most = std::max(1, ragged::sm_count() / s.ctas);
        }
        if (dev < 64) cache[dev][s.threads / 32].store(most, std::memory_order_release);
        cfg.dynamicSmemBytes = smem;
    }
    clusters = std::min<int64_t>(clusters, (int64_t)waves * most);
    cfg.gridDim = dim3((unsigned)(clusters * s.ctas));
    cfg.stream = st;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kKernel, p, s.width);
}

template <class T, int kC>
static cudaError_t fwd_rows(const Fwd<T>& p, const Shape& s, cudaStream_t st) {
    int64_t clusters = p.M;
    // Blocks that start as others end even out short rows (bf16, us, with one wave and with four: 40961 x 2048 109 and 103,
    // 83968 x 1024 114 and 112; 8192 x 8192 93 and 100).
    const int waves = s.threads <= 256 ? 4 : 1;
    return launch_rows<norm_fwd_kernel<T, kC>>(p, s, clusters, kC == 1 ? waves : 1, smem_bytes(2, s.width, sizeof(T)), st);
}

template <class T>
static cudaError_t fwd(const NormFwd& c, cudaStream_t st) {
    const Fwd<T> p{(const T*)c.x, (const T*)c.residual, (const T*)c.post, (const T*)c.pre, c.gate, c.M, (int)c.F,
                   c.scale, c.eps, (T*)c.res, (T*)c.n, c.stats, c.status};
    const Shape s = shape_of(c.F, kFwdThreads);
    if (!s.ctas) {
        const int lanes = c.F <= 64 ? 8 : c.F <= 128 ? 16 : 32, teams = kThreads / lanes;
        const unsigned grid = (unsigned)std::min<int64_t>((c.M + teams - 1) / teams, (int64_t)ragged::sm_count() * 8);
        return lanes == 8    ? ragged::launch(norm_fwd_lanes_kernel<T, 8>, grid, kThreads, st, 0, p)
               : lanes == 16 ? ragged::launch(norm_fwd_lanes_kernel<T, 16>, grid, kThreads, st, 0, p)
                             : ragged::launch(norm_fwd_lanes_kernel<T, 32>, grid, kThreads, st, 0, p);
    }
    switch (s.ctas) {
        case 1: return fwd_rows<T, 1>(p, s, st);
        case 8: return fwd_rows<T, 8>(p, s, st);
        default: return cudaErrorInvalidConfiguration;  // no such width
    }
}

// The most blocks (clusters of them, for long rows) of the backward kernel, each of which leaves a partial row per
// weight: a rule on the shape alone (152 is this GPU's number of SMs), so that a workspace's size does not depend on the
// current device.
static int64_t bwd_parts(int64_t M, int64_t F) {
    const Shape s = shape_of(F, kBwdThreads);
    if (!s.ctas) {
        const int teams = kThreads / (F <= 64 ? 8 : F <= 128 ? 16 : 32);
        return std::max<int64_t>(1, std::min<int64_t>((M + teams - 1) / teams, 152 * 2));
    }
    return std::max<int64_t>(1, std::min<int64_t>(M, 152 * std::max(1, kSmThreads / s.threads) / s.ctas));
}

template <class T, int kC>
static cudaError_t bwd_rows(const Bwd<T>& p, const Shape& s, int64_t& parts, cudaStream_t st) {
    return launch_rows<norm_bwd_kernel<T, kC>>(p, s, parts, 1, smem_bytes(4, s.width, sizeof(T)), st);
}

template <class T>
static cudaError_t bwd(const NormBwd& c, cudaStream_t st) {
    const Bwd<T> p{(const T*)c.dres, (const T*)c.dn, (const T*)c.x, (const T*)c.res, (const T*)c.post, (const T*)c.pre,
                   c.gate, c.stats, c.M, (int)c.F, c.scale, (T*)c.dx, (T*)c.dr, c.dgate, c.partials, c.status};
    const Shape s = shape_of(c.F, kBwdThreads);
    int64_t parts = bwd_parts(c.M, c.F);
    cudaError_t e;
    if (!s.ctas) {
        const unsigned grid = (unsigned)parts;
        e = c.F <= 64    ? ragged::launch(norm_bwd_lanes_kernel<T, 8>, grid, kThreads, st, 0, p)
            : c.F <= 128 ? ragged::launch(norm_bwd_lanes_kernel<T, 16>, grid, kThreads, st, 0, p)
                         : ragged::launch(norm_bwd_lanes_kernel<T, 32>, grid, kThreads, st, 0, p);
    } else {
        e = s.ctas == 1   ? bwd_rows<T, 1>(p, s, parts, st)
            : s.ctas == 4 ? bwd_rows<T, 4>(p, s, parts, st)
            : s.ctas == 8 ? bwd_rows<T, 8>(p, s, parts, st)
                          : cudaErrorInvalidConfiguration;  // no such width
    }
    if (e != cudaSuccess || (!c.dpost && !c.dpre)) return e;
    return ragged::launch(norm_weights_kernel, dim3((unsigned)((c.F + 31) / 32), 2), 1024, st, 0, (const float*)c.partials,
                          (int)parts, (int)c.F, c.dpost, c.dpre);
}

}  // namespace norm

size_t norm_bwd_workspace(int64_t M, int64_t F) {
    return (size_t)(2 * norm::bwd_parts(M, F)) * (size_t)F * sizeof(float);
}
cudaError_t run_norm_fwd(const NormFwd& c, cudaStream_t s) {
    if (c.M == 0) return cudaSuccess;
    return c.f32 ? norm::fwd<float>(c, s) : norm::fwd<__nv_bfloat16>(c, s);
}
cudaError_t run_norm_bwd(const NormBwd& c, cudaStream_t s) {
    return c.f32 ? norm::bwd<float>(c, s) : norm::bwd<__nv_bfloat16>(c, s);
}

}  // namespace mxq
