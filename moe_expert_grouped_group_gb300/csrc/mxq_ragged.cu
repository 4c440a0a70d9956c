// mxq_ragged.cu -- bf16 grouped products of an MoE expert layer on GB300
// (sm_103a) for expert counts that are multiples of nothing:
//   fprop  Y[m,:]  = X[m,:]  . W[e(m)]^T (+ b[e(m)])
//   dgrad  dX[m,:] = dY[m,:] . W[e(m)]
//   wgrad  dW[e]   = dY_e^T . X_e
// fp32 accumulation in TMEM, one rounding to bf16 (or none, fp32 outputs).
//
// Which operand is which. fprop and dgrad put the weight's features on the
// MMA's M (128 TMEM lanes) and the tokens on its N, because N is a field of
// the instruction descriptor that may differ from tile to tile: a slice of an
// expert's rows costs MMA work in steps of 16 rows, not 128. The accumulator
// is the transpose of the output tile: lane = feature, column = token. wgrad
// puts dY's features on M, X's on N, and sums over the expert's rows.
//
// Majorness. X and dY of fprop / dgrad and W of fprop are K-major; W of dgrad
// and both operands of wgrad are MN-major. All are staged as 128-byte-wide
// boxes with the 128-byte swizzle: 64 elements of the contiguous dimension by
// up to 64 or 128 rows of the other.
//
// Edges. Widths of a tile beyond N or K read the tensor map's zero fill and
// are not stored. Token rows of a slice beyond its expert are the next
// expert's: in fprop and dgrad they are accumulator columns of their own that
// nobody stores; in wgrad they would enter the sum, so both operands' rows
// from m_e on are zeroed in shared memory, in the last block of an expert,
// before its MMAs (zeroing one operand would not do: 0 * inf is not 0).
//
// One persistent CTA per SM, warp-specialised: warp 0 issues TMA loads into a
// ring of 64-deep stages, warp 1 owns TMEM and issues the MMAs from one lane,
// warps 2..9 drain one of two accumulators while the MMAs fill the other.
// Every wait is bounded (about 2 s); on expiry MXQ_STATUS_WAIT_TIMEOUT is set.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "mxq_internal.h"
#include "mxq_ragged.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace ragged {

constexpr int BK = 64;   // reduction depth of a stage: 128 bytes of bf16
constexpr int BN = 256;  // widest MMA N
constexpr int STAGES = 4;
constexpr int A_BYTES = kFM * BK * 2;
constexpr int B_BYTES = BN * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int TMEM_COLS = 512;
constexpr int BAR_REGION = STAGES * STAGE_BYTES;
constexpr int TABLE_REGION = BAR_REGION + 256;
__host__ __device__ constexpr int smem_bytes(int E) { return 1024 + TABLE_REGION + 8 * (E + 1); }
static_assert(smem_bytes(MXQ_MAX_EXPERTS) <= 232448, "shared memory over the per-block limit");

struct Params {
    int64_t M, N, K;
    int E;
    const int64_t* m_splits;
    const __nv_bfloat16* bias;
    void* out;
    int out_f32, accumulate;
    int32_t* status;
};

// Store one value, or add it to what is there.
__device__ __forceinline__ void put(void* out, int64_t i, float v, bool f32, bool add) {
    if (f32) {
        float* o = static_cast<float*>(out) + i;
        *o = add ? *o + v : v;
    } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + i;
        *o = __float2bfloat16_rn(add ? __bfloat162float(*o) + v : v);
    }
}

template <int kMode>
__global__ void __launch_bounds__(THREADS, 1)
    ragged_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Params p) {
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
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
    const uint32_t accf0 = smem_u32(bars + 2 * STAGES), acce0 = smem_u32(bars + 2 * STAGES + 2);
    volatile int* abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int st = 0; st < STAGES; ++st) {
            mbar_init(full0 + 8 * st, 1);
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
    const Walk<kMode, BN> W(p.N, p.K, p.E, s_off, s_slices);
    constexpr bool a_mn = kMode != kFprop, b_mn = kMode == kWgrad;

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
                    if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag)) {
                        drain_ring(full0, STAGES, fills);
                        goto done_producer;
                    }
                    const uint32_t fb = full0 + 8 * stage, a = smem_u32(smem + stage * STAGE_BYTES), b = a + A_BYTES;
                    mbar_expect_tx(fb, A_BYTES + boxes * 8192);
                    if (kMode == kFprop) {
                        tma_load_3d(a, &tmA, fb, r, T.f0, T.e);
                    } else if (kMode == kDgrad) {
                        tma_load_3d(a, &tmA, fb, T.f0, r, T.e);
                        tma_load_3d(a + 8192, &tmA, fb, T.f0 + 64, r, T.e);
                    } else {
                        tma_load_2d(a, &tmA, fb, T.f0, T.red0 + r);
                        tma_load_2d(a + 8192, &tmA, fb, T.f0 + 64, T.red0 + r);
                    }
                    for (int i = 0; i < boxes; ++i) {
                        if (kMode == kWgrad) tma_load_2d(b + 8192 * i, &tmB, fb, T.c0 + 64 * i, T.red0 + r);
                        else tma_load_2d(b + 8192 * i, &tmB, fb, r, T.c0 + 64 * i);
                    }
                    ++fills;
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
        done_producer:;
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        int stage = 0, buf = 0;
        uint32_t phase = 0, aphase = 0;
        const uint32_t base = smem_u32(smem);
        // MN-major: 64-element chunks 8192 bytes apart, 8-row groups of the reduction 1024 apart
        const uint64_t ad0 = smem_desc(base, a_mn ? 8192 : 16, 1024);
        const uint64_t bd0 = smem_desc(base + A_BYTES, b_mn ? 8192 : 16, 1024);
        constexpr uint32_t a_step = (a_mn ? 2048 : 32) / 16, b_step = (b_mn ? 2048 : 32) / 16;  // 16 of the reduction
        bool ok = true;
        for (int64_t t = blockIdx.x; t < W.total && ok; t += gridDim.x) {
            const Tile T = W.get(t);
            if (T.red == 0) continue;  // wgrad of an empty expert: the epilogue writes zeros
            const uint32_t id = idesc_f16(1, a_mn, b_mn, kFM, T.n);
            ok = mbar_wait(acce0 + 8 * buf, aphase ^ 1, abort_flag);
            for (int r = 0; r < T.red && ok; r += BK) {
                ok = mbar_wait(full0 + 8 * stage, phase, abort_flag);
                if (!ok) break;
                const int left = min(BK, T.red - r), steps = (left + 15) / 16;
                if (kMode == kWgrad && (left & 15)) {
                    // rows left .. 16 * steps of every box belong to the next expert
                    const int per = (16 * steps - left) * 8, boxes = 2 + (T.n + 63) / 64;
                    uint8_t* s = smem + stage * STAGE_BYTES + left * 128;
                    for (int i = lane; i < per * boxes; i += 32)
                        *reinterpret_cast<uint4*>(s + i / per * 8192 + i % per * 16) = make_uint4(0u, 0u, 0u, 0u);
                    fence_async_smem();
                    __syncwarp();
                }
                fence_after();
                if (lane == 0) {
                    const uint64_t so = (uint64_t)(stage * (STAGE_BYTES / 16));
                    for (int k = 0; k < steps; ++k)
                        mma_f16(tmem + buf * BN, ad0 + so + k * a_step, bd0 + so + k * b_step, id, (r | k) != 0);
                    mma_commit(empty0 + 8 * stage);
                }
                __syncwarp();
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
            if (ok && lane == 0) mma_commit(accf0 + 8 * buf);
            __syncwarp();
            buf ^= 1;
            aphase ^= buf == 0;
        }
    } else {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - 2) >> 2;
        int buf = 0;
        uint32_t aphase = 0;
        for (int64_t t = blockIdx.x; t < W.total; t += gridDim.x) {
            const Tile T = W.get(t);
            const int f = T.f0 + q * 32 + lane;
            const bool live = f < (kMode == kDgrad ? p.K : p.N);
            const bool add = kMode == kWgrad && p.accumulate;
            if (T.red == 0) {
                if (!add && live)
                    for (int j = half; j < T.cols; j += 2)
                        put(p.out, ((int64_t)T.e * p.N + f) * p.K + T.c0 + j, 0.0f, p.out_f32, false);
                continue;
            }
            const bool ok = mbar_wait(accf0 + 8 * buf, aphase, abort_flag);
            __syncwarp();
            if (!ok || *abort_flag) break;
            fence_after();
            const float b =
                kMode == kFprop && p.bias && live ? __bfloat162float(p.bias[(int64_t)T.e * p.N + f]) : 0.0f;
            for (int c = 32 * half; c < T.cols; c += 64) {
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + buf * BN + c, v);
                tmem_wait_ld();
                if (live) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (c + j >= T.cols) break;
                        const int64_t i = kMode == kWgrad ? ((int64_t)T.e * p.N + f) * p.K + T.c0 + c + j
                                                          : (int64_t)(T.c0 + c + j) * (kMode == kDgrad ? p.K : p.N) + f;
                        put(p.out, i, __uint_as_float(v[j]) + b, p.out_f32, add);
                    }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce0 + 8 * buf);
            buf ^= 1;
            aphase ^= buf == 0;
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

// ------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode_tmap(CUtensorMap* m, const void* base, int elem_bytes, int rank, const int64_t* dims,
                 const int64_t* strides, const int* box, int swizzle_bytes) {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    if (!fn || !base || rank < 1 || rank > 3) return false;
    cuuint64_t d[3], s[2];
    cuuint32_t b[3], es[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = (cuuint64_t)dims[i];
        b[i] = (cuuint32_t)box[i];
        if (i) s[i - 1] = (cuuint64_t)strides[i - 1];
    }
    return fn(m, elem_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
              const_cast<void*>(base), d, s, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle_bytes == 0 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    static std::atomic<int> cache[64];
    int dev = 0, v = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && (v = cache[dev].load(std::memory_order_relaxed)) > 0) return v;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    if (dev < 64) cache[dev].store(v, std::memory_order_relaxed);
    return v;
}

template <int kMode>
static cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const Params& p, int64_t tiles, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(ragged_gemm_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes(MXQ_MAX_EXPERTS));
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(tiles, sm_count()));
    ragged_gemm_kernel<kMode><<<grid, THREADS, smem_bytes(p.E), s>>>(a, b, p);
    return cudaGetLastError();
}

cudaError_t run_gemm(const GemmCall& c, cudaStream_t s) {
    Params p{c.M, c.N, c.K, c.E, c.m_splits, static_cast<const __nv_bfloat16*>(c.bias), c.out, c.out_f32, c.accumulate,
             c.status};
    CUtensorMap a, b;
    bool ok;
    const int64_t feats = ((c.mode == kDgrad ? c.K : c.N) + kFM - 1) / kFM;
    int64_t tiles = (c.M / BN + std::min<int64_t>(c.E, c.M)) * feats;  // no fewer than the device counts
    if (c.mode == kWgrad) {
        tiles = feats * ((c.K + BN - 1) / BN) * c.E;
        // with M == 0 nothing is loaded: any valid address does
        const int64_t rows = std::max<int64_t>(c.M, 1);
        const int64_t da[2] = {c.N, rows}, sa[1] = {2 * c.ld_mat}, db[2] = {c.K, rows}, sb[1] = {2 * c.ld_tok};
        const int box[2] = {64, BK};
        ok = encode_tmap(&a, c.M ? c.mat : c.out, 2, 2, da, sa, box, 128) &&
             encode_tmap(&b, c.M ? c.tok : c.out, 2, 2, db, sb, box, 128);
    } else {
        const int64_t da[3] = {c.K, c.N, c.E}, sa[2] = {2 * c.K, 2 * c.K * c.N};
        const int64_t db[2] = {c.mode == kDgrad ? c.N : c.K, c.M}, sb[1] = {2 * c.ld_tok};
        const int boxa[3] = {64, c.mode == kDgrad ? BK : kFM, 1}, boxb[2] = {64, 64};
        ok = encode_tmap(&a, c.mat, 2, 3, da, sa, boxa, 128) && encode_tmap(&b, c.tok, 2, 2, db, sb, boxb, 128);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (c.mode == kFprop) return launch<kFprop>(a, b, p, tiles, s);
    if (c.mode == kDgrad) return launch<kDgrad>(a, b, p, tiles, s);
    return launch<kWgrad>(a, b, p, tiles, s);
}

}  // namespace ragged
}  // namespace mxq
