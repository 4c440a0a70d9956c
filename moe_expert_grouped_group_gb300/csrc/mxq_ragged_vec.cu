// mxq_ragged_vec.cu -- the grouped products of single tokens: fprop in bf16 and
// the int8 product for experts with a handful of rows (kVecRows or fewer on
// average), where reading W once is all there is to do.
//
// No tensor core and no staging. A warp takes four output channels and up to
// eight tokens of an expert; its lanes hold 16 bytes each of the same 512 bytes
// of every row. int8 codes are added by 4-way integer products (dp4a), exact in
// 32 bits for any codes while K is below 2^17 (a longer K goes to the
// tensor-core shapes); bf16 values by fp32 multiply-adds, two k to an
// instruction. Tokens come from L1, shared by the warp's four channels: 16
// bytes a token for 64 bytes of W. The lanes' sums are added in a fixed order.
//
// What bounds it is HBM: 24 bytes of W a cycle and SM, 6 dp4a a token and cycle
// of the 64 an SM has, or 6 packed multiply-adds and 3 conversions a token of
// its 128. The tensor-core shapes pay more at their ends, and an int8 MMA with A
// in TMEM takes 130 cycles per 16 of K however few its columns are. W of 2048 x
// 4096, graph replay, us (tensor-core shape -> this one):
//   int8  1 expert x 1 row 11.5 -> 4.0   8 x 2 18.8 -> 10.3   64 x 2 112 -> 88 (6.0 TB/s)
//         8 x 4 18.7 -> 13.0   64 x 4 112 -> 114   8 x 8 19.3 -> 18.5   64 x 8 112 -> 151
//   bf16  1 expert x 1 row  7.7 -> 4.3   1 x 4 7.7 -> 5.9   4 x 4 11.6 -> 14.1   8 x 4 27.0 -> 32.8
// The rule goes by the average, the only thing the host knows. Its price is a crowded expert among empty ones, whose
// W is read (from L2) once for each eight of its rows: int8 with all rows on one expert
//         8 x 4 11.4 -> 10.9   64 x 1 11.8 -> 17.8   64 x 2 11.9 -> 34.8   64 x 4 19.5 -> 66.4
// and with Dirichlet(0.3) shares 8 x 4 18.8 -> 13.7, 64 x 2 59.0 -> 61.4, 64 x 4 66.5 -> 102.
#include <cuda_bf16.h>

#include <algorithm>

#include "mxq_internal.h"
#include "mxq_ragged.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace ragged {
namespace vec {

constexpr int ROWS = 8;       // tokens of a slice
constexpr int CHANNELS = 4;   // of a warp
constexpr int WARPS = 8, THREADS = 32 * WARPS;

struct Params {
    const uint8_t *x, *w;
    int64_t ldx, ldw;        // bytes of a row
    const float *xs, *ws;    // int8: scales
    const __nv_bfloat16* bias;
    int64_t M, N;
    int E;
    const int64_t* m_splits;
    void* out;
    int out_f32;
    int32_t* status;
};

__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

struct Int8 {
    using Acc = int;
    using Held = uint4;
    __host__ __device__ static constexpr int unroll(int) { return 2; }
    static __device__ __forceinline__ Held open(const uint4& w) { return w; }
    static __device__ __forceinline__ Acc zero() { return 0; }
    static __device__ __forceinline__ Acc add(const Held& a, const Held& b, Acc c) {
        c = __dp4a((int)a.x, (int)b.x, c);
        c = __dp4a((int)a.y, (int)b.y, c);
        c = __dp4a((int)a.z, (int)b.z, c);
        return __dp4a((int)a.w, (int)b.w, c);
    }
    static __device__ __forceinline__ int sum(Acc a) { return a; }
    static __device__ __forceinline__ float result(const Params& p, int v, int64_t row, int64_t at) {
        return __fmul_rn(__fmul_rn(__int2float_rn(v), p.xs[row]), p.ws[at]);
    }
};
struct Bf16 {
    using Acc = uint64_t;  // even and odd k
    struct Held {
        uint64_t v[4];
    };
    __host__ __device__ static constexpr int unroll(int tokens) { return tokens > 4 ? 1 : 2; }  // registers
    static __device__ __forceinline__ Held open(const uint4& w) {
        return Held{{f2pack(bf16lo(w.x), bf16hi(w.x)), f2pack(bf16lo(w.y), bf16hi(w.y)), f2pack(bf16lo(w.z), bf16hi(w.z)),
                     f2pack(bf16lo(w.w), bf16hi(w.w))}};
    }
    static __device__ __forceinline__ Acc zero() { return 0; }
    static __device__ __forceinline__ Acc add(const Held& a, const Held& b, Acc c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = f2fma(a.v[i], b.v[i], c);
        return c;
    }
    static __device__ __forceinline__ float sum(Acc a) {
        const float2 v = f2unpack(a);
        return __fadd_rn(v.x, v.y);
    }
    static __device__ __forceinline__ float result(const Params&, float v, int64_t, int64_t) { return v; }
};

// Sums of v[0 .. n-1] over the 32 lanes, in a fixed order: exchange-and-add rounds halve the values each lane
// keeps, then the rest of the lanes are added; lane l ends with the sum of value l * n / 32.
template <int n, int off = 16, class T, int kSize>
__device__ __forceinline__ T lane_sums(T (&v)[kSize], int lane) {
    if constexpr (off == 0) {
        return v[0];
    } else if constexpr (n > 1) {
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const T keep = up ? v[i + n / 2] : v[i], send = up ? v[i] : v[i + n / 2];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
        return lane_sums<n / 2, off / 2>(v, lane);
    } else {
        v[0] = v[0] + __shfl_xor_sync(0xffffffffu, v[0], off);
        return lane_sums<1, off / 2>(v, lane);
    }
}

// Channels f0 .. f0 + 3 (those below N) of expert e for kTokens tokens from row `row` on, of which `rows` are real.
template <class Op, int kTokens>
__device__ __forceinline__ void product(const Params& p, int e, int64_t row, int rows, int64_t f0, int lane) {
    // channels beyond N and tokens beyond the slice repeat the last ones and are not stored
    const int bytes = (int)p.ldw, last = (int)min((int64_t)CHANNELS, p.N - f0) - 1;
    const uint8_t* w = p.w + ((int64_t)e * p.N + f0) * p.ldw + 16 * lane;
    const uint8_t* x = p.x + row * p.ldx + 16 * lane;
    typename Op::Acc acc[CHANNELS][kTokens];
#pragma unroll
    for (int c = 0; c < CHANNELS; ++c)
#pragma unroll
        for (int t = 0; t < kTokens; ++t) acc[c][t] = Op::zero();
    constexpr int kUnroll = Op::unroll(kTokens);
#pragma unroll kUnroll
    for (int k = 16 * lane; k < bytes; k += 512, w += 512, x += 512) {
        uint4 raw[CHANNELS];
#pragma unroll
        for (int c = 0; c < CHANNELS; ++c) raw[c] = load_once(w + min(c, last) * p.ldw);
        typename Op::Held a[CHANNELS];
#pragma unroll
        for (int c = 0; c < CHANNELS; ++c) a[c] = Op::open(raw[c]);
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            const auto b = Op::open(*reinterpret_cast<const uint4*>(x + min(t, rows - 1) * p.ldx));
#pragma unroll
            for (int c = 0; c < CHANNELS; ++c) acc[c][t] = Op::add(a[c], b, acc[c][t]);
        }
    }
    constexpr int kValues = CHANNELS * kTokens, kLanes = 32 / kValues;  // lanes that end with the same sum
    decltype(Op::sum(Op::zero())) v[kValues];
#pragma unroll
    for (int i = 0; i < kValues; ++i) v[i] = Op::sum(acc[i % CHANNELS][i / CHANNELS]);
    const auto mine = lane_sums<kValues>(v, lane);
    const int t = lane / kLanes / CHANNELS;
    const int64_t f = f0 + lane / kLanes % CHANNELS;
    if (lane % kLanes == 0 && t < rows && f < p.N) {
        const int64_t at = (int64_t)e * p.N + f, o = (row + t) * p.N + f;
        float y = Op::result(p, mine, row + t, at);
        if (p.bias) y = __fadd_rn(y, __bfloat162float(p.bias[at]));
        if (p.out_f32) static_cast<float*>(p.out)[o] = y;
        else static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(y);
    }
}

template <class Op>
__global__ void __launch_bounds__(THREADS, 2) ragged_vec_kernel(Params p) {
    extern __shared__ int32_t s_tables[];
    int32_t *s_off = s_tables, *s_slices = s_tables + p.E + 1;
    const int bad = load_ragged(p.m_splits, p.E, p.M, ROWS, s_off, s_slices);
    if (bad) {
        report_status(p.status, bad);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t groups = (p.N + CHANNELS * WARPS - 1) / (CHANNELS * WARPS), total = s_slices[p.E] * groups;
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int slice = (int)(i / groups);
        const int e = owner_of(s_slices, p.E, slice);
        const Slice s = slice_of(s_off[e], s_off[e + 1] - s_off[e], s_slices[e + 1] - s_slices[e], slice - s_slices[e], 1);
        const int64_t f0 = (i % groups) * (CHANNELS * WARPS) + warp * CHANNELS;
        if (f0 >= p.N) continue;
        if (s.rows == 1) product<Op, 1>(p, e, s.row, 1, f0, lane);
        else if (s.rows == 2) product<Op, 2>(p, e, s.row, 2, f0, lane);
        else if (s.rows <= 4) product<Op, 4>(p, e, s.row, s.rows, f0, lane);
        else product<Op, 8>(p, e, s.row, s.rows, f0, lane);
    }
}

template <class Op>
static cudaError_t run(const Params& p, cudaStream_t s) {
    const int64_t units = (p.M / ROWS + std::min<int64_t>(p.E, p.M)) * ((p.N + CHANNELS * WARPS - 1) / (CHANNELS * WARPS));
    const unsigned grid = (unsigned)std::min<int64_t>(units, (int64_t)sm_count() * 2);
    return launch(ragged_vec_kernel<Op>, grid, THREADS, s, 8 * (p.E + 1), p);
}

}  // namespace vec

cudaError_t run_int8_vec(const Int8Call& c, cudaStream_t s) {
    return vec::run<vec::Int8>({static_cast<const uint8_t*>(c.xq), static_cast<const uint8_t*>(c.wq), c.K, c.K, c.xs, c.ws,
                                static_cast<const __nv_bfloat16*>(c.bias), c.M, c.N, c.E, c.m_splits, c.out, c.out_f32,
                                c.status},
                               s);
}

cudaError_t run_fprop_vec(const GemmCall& c, cudaStream_t s) {
    return vec::run<vec::Bf16>({static_cast<const uint8_t*>(c.tok), static_cast<const uint8_t*>(c.mat), 2 * c.ld_tok,
                                2 * c.K, nullptr, nullptr, static_cast<const __nv_bfloat16*>(c.bias), c.M, c.N, c.E,
                                c.m_splits, c.out, c.out_f32, c.status},
                               s);
}

}  // namespace ragged
}  // namespace mxq
