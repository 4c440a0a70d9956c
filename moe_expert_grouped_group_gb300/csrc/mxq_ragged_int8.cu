// mxq_ragged_int8.cu -- int8 grouped products of an MoE expert layer with one
// scale per token and per output channel, for expert counts that are multiples
// of nothing, and the quantizer of their tokens:
//   s_m = max(max_k |x[m,k]|, 2^-100) / 127,  q[m,k] = rint(x[m,k] (127 / max))
//   Y[m,n] = (sum_k xq[m,k] wq[e,n,k]) xs[m] ws[e,n] (+ b[e,n])
//
// GB300's int8 tensor rate is a small fraction of its 16-bit floating rate, so
// the codes travel as int8 (the bytes that a weight-bound call is made of) and
// are widened to f16 in shared memory, exactly: |q| <= 128 fits f16's 11
// significand bits. The products are then whole numbers below 2^14 and
// tcgen05.mma kind::f16 sums them in fp32.
//
// The tile walk, the operands' sides (features on the MMA's M, tokens on its
// N) and the edges are those of the bf16 products (mxq_ragged.cuh). Warp 0
// loads int8 boxes, warps 10..17 widen them into the 128-byte-swizzled
// operand stages, warp 1 issues the MMAs, warps 2..9 scale and store.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "mxq_internal.h"
#include "mxq_ragged.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace ragged {
namespace i8 {

constexpr int BK = 64;      // reduction depth of a stage
constexpr int BN = 256;     // widest MMA N
constexpr int RAWS = 3;     // int8 stages
constexpr int STAGES = 3;   // widened stages
constexpr int RAW_A = kFM * BK, RAW_BYTES = RAW_A + BN * BK;
constexpr int A_BYTES = kFM * BK * 2, STAGE_BYTES = A_BYTES + BN * BK * 2;
constexpr int EPI_WARPS = 8, CVT_WARPS = 8;
constexpr int THREADS = 64 + 32 * (EPI_WARPS + CVT_WARPS);
constexpr int TMEM_COLS = 512;
constexpr int RAW_REGION = STAGES * STAGE_BYTES;
constexpr int BAR_REGION = RAW_REGION + RAWS * RAW_BYTES;
constexpr int TABLE_REGION = BAR_REGION + 256;
__host__ __device__ constexpr int smem_bytes(int E) { return 1024 + TABLE_REGION + 8 * (E + 1); }
static_assert(smem_bytes(MXQ_MAX_EXPERTS) <= 232448, "shared memory over the per-block limit");

struct Params {
    const float *xs, *ws;
    const __nv_bfloat16* bias;
    int64_t M, N, K;
    int E;
    const int64_t* m_splits;
    void* out;
    int out_f32;
    int32_t* status;
};

// Four int8 -> four f16, exact. With its sign bit flipped a code is q + 128 in
// 0..255; under the high byte 0x64 that is the f16 1024 + 128 + q.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    const uint32_t u = w ^ 0x80808080u, bias = 0x64806480u;  // 1152, 1152
    uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), *reinterpret_cast<const __half2*>(&bias));
    __half2 b = __hsub2(*reinterpret_cast<__half2*>(&hi), *reinterpret_cast<const __half2*>(&bias));
    return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

__global__ void __launch_bounds__(THREADS, 1)
    ragged_int8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align<1024>(smem_raw);
    int32_t* s_off = reinterpret_cast<int32_t*>(smem + TABLE_REGION);
    int32_t* s_slices = s_off + p.E + 1;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int bad = load_ragged(p.m_splits, p.E, p.M, BN, s_off, s_slices);
    if (bad) {
        report_status(p.status, bad);
        return;
    }
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_REGION);
    const uint32_t rawf0 = smem_u32(bars), rawe0 = rawf0 + 8 * RAWS;
    const uint32_t full0 = rawe0 + 8 * RAWS, empty0 = full0 + 8 * STAGES;
    const uint32_t accf0 = empty0 + 8 * STAGES, acce0 = accf0 + 16;
    volatile int* abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int st = 0; st < RAWS; ++st) {
            mbar_init(rawf0 + 8 * st, 1);
            mbar_init(rawe0 + 8 * st, CVT_WARPS);
        }
        for (int st = 0; st < STAGES; ++st) {
            mbar_init(full0 + 8 * st, CVT_WARPS);
            mbar_init(empty0 + 8 * st, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, EPI_WARPS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmA) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmB) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    const Walk<kFprop, kFM, BN, 16> W(p.N, p.K, p.E, s_off, s_slices, nullptr);

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int64_t fills = 0;
            for (int64_t t = blockIdx.x; t < W.total; t += gridDim.x) {
                const Tile T = W.get(t);
                const int boxes = (T.n + 63) / 64;
                for (int r = 0; r < T.red; r += BK) {
                    if (!mbar_wait(rawe0 + 8 * stage, phase ^ 1, abort_flag)) {
                        drain_ring(rawf0, RAWS, fills);
                        goto done_producer;
                    }
                    const uint32_t fb = rawf0 + 8 * stage, a = smem_u32(smem + RAW_REGION + stage * RAW_BYTES);
                    mbar_expect_tx(fb, RAW_A + boxes * 64 * BK);
                    load_3d<1>(a, &tmA, fb, r, T.f0, T.e);
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d(a + RAW_A + i * 64 * BK, &tmB, fb, r, T.c0 + 64 * i);
                    ++fills;
                    if (++stage == RAWS) { stage = 0; phase ^= 1; }
                }
            }
        done_producer:;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, aphase = 0;
            const uint32_t base = smem_u32(smem);
            const uint64_t ad0 = smem_desc(base, 16, 1024), bd0 = smem_desc(base + A_BYTES, 16, 1024);
            bool ok = true;
            for (int64_t t = blockIdx.x; t < W.total && ok; t += gridDim.x) {
                const Tile T = W.get(t);
                const uint32_t id = idesc_f16(0, 0, 0, kFM, T.n);
                ok = mbar_wait(acce0 + 8 * buf, aphase ^ 1, abort_flag);
                for (int r = 0; r < T.red && ok; r += BK) {
                    ok = mbar_wait(full0 + 8 * stage, phase, abort_flag);
                    if (!ok) break;
                    fence_after();
                    const int steps = (min(BK, T.red - r) + 15) / 16;
                    const uint64_t so = (uint64_t)(stage * (STAGE_BYTES / 16));
                    for (int k = 0; k < steps; ++k)
                        mma_f16<1>(tmem + buf * BN, ad0 + so + 2 * k, bd0 + so + 2 * k, id, (r | k) != 0);
                    mma_commit<1>(empty0 + 8 * stage);
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (ok) mma_commit<1>(accf0 + 8 * buf);
                buf ^= 1;
                aphase ^= buf == 0;
            }
        }
    } else if (warp < 2 + EPI_WARPS) {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - 2) >> 2;
        int buf = 0;
        uint32_t aphase = 0;
        for (int64_t t = blockIdx.x; t < W.total; t += gridDim.x) {
            const Tile T = W.get(t);
            const int f = T.f0 + q * 32 + lane;
            const bool live = f < p.N;
            const bool ok = mbar_wait(accf0 + 8 * buf, aphase, abort_flag);
            __syncwarp();
            if (!ok || *abort_flag) break;
            fence_after();
            const float sw = live ? p.ws[(int64_t)T.e * p.N + f] : 0.0f;
            const float b = p.bias && live ? __bfloat162float(p.bias[(int64_t)T.e * p.N + f]) : 0.0f;
            for (int c = 32 * half; c < T.cols; c += 64) {
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + buf * BN + c, v);
                tmem_wait_ld();
                if (live) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (c + j >= T.cols) break;
                        const int64_t m = T.c0 + c + j;
                        const float y = __uint_as_float(v[j]) * __ldg(p.xs + m) * sw + b;
                        if (p.out_f32) static_cast<float*>(p.out)[m * p.N + f] = y;
                        else static_cast<__nv_bfloat16*>(p.out)[m * p.N + f] = __float2bfloat16_rn(y);
                    }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce0 + 8 * buf);
            buf ^= 1;
            aphase ^= buf == 0;
        }
    } else {
        // ------------------------------------------------------ int8 -> f16
        const int ct = (int)threadIdx.x - 32 * (2 + EPI_WARPS);
        int raw = 0, stage = 0;
        uint32_t rphase = 0, phase = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < W.total && ok; t += gridDim.x) {
            const Tile T = W.get(t);
            const int units = (kFM + T.n) * (BK / 16);  // 16-byte chunks of A's rows, then of B's
            for (int r = 0; r < T.red; r += BK) {
                ok = mbar_wait(rawf0 + 8 * raw, rphase, abort_flag) && mbar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                const uint8_t* src = smem + RAW_REGION + raw * RAW_BYTES;
                uint8_t* dst = smem + stage * STAGE_BYTES;
                for (int i = ct; i < units; i += 32 * CVT_WARPS) {
                    const uint4 w = *reinterpret_cast<const uint4*>(src + i * 16);
                    const uint2 a = widen4(w.x), b = widen4(w.y), c = widen4(w.z), d = widen4(w.w);
                    const int row = i >> 2, ch = (i & 3) * 2;  // 128-byte rows, chunk ^= row mod 8
                    uint8_t* o = dst + row * 128;
                    *reinterpret_cast<uint4*>(o + ((ch ^ (row & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
                    *reinterpret_cast<uint4*>(o + (((ch + 1) ^ (row & 7)) << 4)) = make_uint4(c.x, c.y, d.x, d.y);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(full0 + 8 * stage);
                    mbar_arrive(rawe0 + 8 * raw);
                }
                if (++raw == RAWS) { raw = 0; rphase ^= 1; }
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
        }
    }
    fence_before();
    __syncthreads();
    if (s_abort && threadIdx.x == 0 && p.status) atomicOr(p.status, MXQ_STATUS_WAIT_TIMEOUT);
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

// ------------------------------------------------------------ row quantizer
// One block per row. A row with an infinity or NaN has no scale: its scale is
// NaN and its codes are 0, so that its outputs are NaN and nothing else is.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const uint16_t* x, int64_t M, int64_t K, int64_t ld,
                                                            uint8_t* q, float* scale) {
    __shared__ uint32_t s_top[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const uint4* row = reinterpret_cast<const uint4*>(x + m * ld);
        uint32_t top = 0;  // two bf16 magnitudes: their bits order as the values do
        for (int64_t i = threadIdx.x; i < K / 8; i += 256) {
            const uint4 w = row[i];
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                         __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
        }
        top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
        __syncthreads();
        if (lane == 0) s_top[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, s_top[i]);
        const bool finite = top < 0x7F80u;
        const float amax = fmaxf(__uint_as_float(top << 16), 7.8886090522101181e-31f);  // 2^-100
        const float inv = finite ? __fdiv_rn(127.0f, amax) : 0.0f;
        for (int64_t i = threadIdx.x; i < K / 8; i += 256) {
            const uint4 w = row[i];
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int a = finite ? __float2int_rn(__fmul_rn(bf16lo(ws[j]), inv)) : 0;
                const int b = finite ? __float2int_rn(__fmul_rn(bf16hi(ws[j]), inv)) : 0;
                o[j >> 1] |= ((uint32_t)(a & 255) | (uint32_t)(b & 255) << 8) << (16 * (j & 1));
            }
            *reinterpret_cast<uint2*>(q + m * K + 8 * i) = make_uint2(o[0], o[1]);
        }
        if (threadIdx.x == 0) scale[m] = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FC00000u);
    }
}

}  // namespace i8

cudaError_t run_int8(const Int8Call& c, cudaStream_t s) {
    using namespace i8;
    Params p{c.xs, c.ws, static_cast<const __nv_bfloat16*>(c.bias), c.M, c.N, c.K, c.E, c.m_splits, c.out, c.out_f32,
             c.status};
    const int64_t da[3] = {c.K, c.N, c.E}, sa[2] = {c.K, c.K * c.N}, db[2] = {c.K, c.M}, sb[1] = {c.K};
    const int boxa[3] = {BK, kFM, 1}, boxb[2] = {BK, 64};
    CUtensorMap a, b;
    if (!encode_tmap(&a, c.wq, 1, 3, da, sa, boxa, 0) || !encode_tmap(&b, c.xq, 1, 2, db, sb, boxb, 0))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(ragged_int8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes(MXQ_MAX_EXPERTS));
    if (e != cudaSuccess) return e;
    const int64_t tiles = (c.M / BN + std::min<int64_t>(c.E, c.M)) * ((c.N + kFM - 1) / kFM);
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(tiles, sm_count()));
    ragged_int8_kernel<<<grid, THREADS, smem_bytes(c.E), s>>>(a, b, p);
    return cudaGetLastError();
}

cudaError_t run_int8_quantize(const void* x, int64_t M, int64_t K, int64_t ld, void* q, float* scale, cudaStream_t s) {
    if (M == 0) return cudaSuccess;
    const unsigned grid = (unsigned)std::min<int64_t>(M, (int64_t)sm_count() * 8);
    i8::quantize_rows_kernel<<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(x), M, K, ld, static_cast<uint8_t*>(q),
                                                  scale);
    return cudaGetLastError();
}

}  // namespace ragged
}  // namespace mxq
