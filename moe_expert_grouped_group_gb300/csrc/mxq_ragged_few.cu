// mxq_ragged_few.cu -- bf16 fprop and dgrad for experts with few rows (the
// steps of serving, short tails of training): the products of mxq_ragged.cu on
// one-SM tiles of 128 features by up to 32 rows.
//
// What is left of such a product is reading W once. A stage is 16 KB of W and
// at most 4 KB of tokens, and eight are in flight. With fewer tiles than half
// the SMs the sum itself is split: a cluster of kSplit CTAs takes a tile, each
// a part of the reduction, and each then adds up its kSplit-th of the tile's
// columns, in rank order, from partial sums that the others store into its shared memory (st.async, which counts
// its bytes on the receiver's barrier; two buffers, used by alternate tiles).
// Sums stay in fp32 and come out the same bits from run to run.
//
// fp32 sums, one accumulator of FLUSH stages at a time, are added in registers
// as in the pair kernel's fp32 path; here that costs nothing that is noticed.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "mxq_internal.h"
#include "mxq_ragged.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace ragged {
namespace few {

constexpr int BK = 64;
constexpr int FLUSH = 8;
constexpr int STAGES = 8;
constexpr int WIDE = kFewRows, STEP = 16;
constexpr int A_BYTES = kFM * BK * 2, STAGE_BYTES = A_BYTES + WIDE * BK * 2;
constexpr int EPI_WARPS = 4;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int TMEM_COLS = 2 * WIDE;
constexpr int PART_REGION = STAGES * STAGE_BYTES;
constexpr int BAR_REGION = PART_REGION + kPartBytes;
constexpr int TABLE_REGION = BAR_REGION + 256;
__host__ __device__ constexpr int smem_bytes(int E) { return 1024 + TABLE_REGION + 8 * (E + 1); }
static_assert(smem_bytes(MXQ_MAX_EXPERTS) <= 232448, "shared memory over the per-block limit");
static_assert(8 * (2 * STAGES + 8) <= 256, "barrier region");

struct Params {
    int64_t M, N, K;
    int E;
    const int64_t* m_splits;
    const __nv_bfloat16* bias;
    void* out;
    int out_f32;
    int32_t* status;
};

template <int kMode, int kSplit>
__global__ void __launch_bounds__(THREADS, 1)
    ragged_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align<1024>(smem_raw);
    int32_t* s_off = reinterpret_cast<int32_t*>(smem + TABLE_REGION);
    int32_t* s_slices = s_off + p.E + 1;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = kSplit > 1 ? (int)cta_rank() : 0;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_REGION);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES;
    const uint32_t accf0 = empty0 + 8 * STAGES, acce0 = accf0 + 16, partf0 = acce0 + 16, parte0 = partf0 + 16;
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
            mbar_init(partf0 + 8 * b, 1);
            if (kSplit > 1) mbar_init(parte0 + 8 * b, (kSplit - 1) * EPI_WARPS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmA) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmB) : "memory");
    }
    // all CTAs of a cluster find the same fault and stop before any cluster-wide step
    const int bad = load_ragged(p.m_splits, p.E, p.M, WIDE, s_off, s_slices);
    if (bad) {
        report_status(p.status, bad);
        return;
    }
    if (warp == 1) tmem_alloc<1>(smem_u32(&s_tmem), TMEM_COLS);
    fence_before();
    __syncthreads();
    if (kSplit > 1) cluster_sync();  // the others' barriers exist before any partial sum is sent
    fence_after();
    const uint32_t tmem = s_tmem;
    const Walk<kMode, kFM, WIDE, STEP> W(p.N, p.K, p.E, s_off, s_slices, nullptr);
    const int64_t first = blockIdx.x / kSplit, stride = gridDim.x / kSplit;
    // this CTA's part of the reduction, the same for every tile
    const int red = (int)(kMode == kDgrad ? p.N : p.K), blocks = (red + BK - 1) / BK;
    const int rb = blocks * rank / kSplit * BK, re = min(red, blocks * (rank + 1) / kSplit * BK);
    constexpr bool a_mn = kMode == kDgrad;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0;
        int64_t fills = 0;
        for (int64_t t = first; t < W.total; t += stride) {
            const Tile T = W.get(t);
            for (int r = rb; r < re; r += BK) {
                if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag)) {
                    drain_ring(full0, STAGES, fills);
                    goto done_producer;
                }
                __syncwarp();
                const uint32_t fb = full0 + 8 * stage, a = smem_u32(smem) + stage * STAGE_BYTES;
                if (elect_one()) {
                    mbar_expect_tx(fb, STAGE_BYTES);
                    if (kMode == kFprop) {
                        load_3d<1>(a, &tmA, fb, r, T.f0, T.e);
                    } else {
                        load_3d<1>(a, &tmA, fb, T.f0, r, T.e);
                        load_3d<1>(a + 8192, &tmA, fb, T.f0 + 64, r, T.e);
                    }
                    load_2d<1>(a + A_BYTES, &tmB, fb, r, T.c0);
                }
                __syncwarp();
                ++fills;
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
        }
    done_producer:;
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        int stage = 0, buf = 0;
        uint32_t phase = 0, aphase = 0;
        const uint32_t base = smem_u32(smem);
        const uint64_t ad0 = smem_desc(base, a_mn ? 8192 : 16, 1024), bd0 = smem_desc(base + A_BYTES, 16, 1024);
        constexpr uint32_t a_step = (a_mn ? 2048 : 32) / 16, b_step = 32 / 16;
        for (int64_t t = first; t < W.total; t += stride) {
            const Tile T = W.get(t);
            const uint32_t id = idesc_f16(1, a_mn, 0, kFM, T.n);
            for (int r0 = rb; r0 < re; r0 += FLUSH * BK) {
                const int r1 = min(re, r0 + FLUSH * BK);
                const uint32_t d = tmem + buf * WIDE;
                if (!mbar_wait(acce0 + 8 * buf, aphase ^ 1, abort_flag)) goto done_mma;
                __syncwarp();
                for (int r = r0; r < r1; r += BK) {
                    const uint64_t ad = ad0 + (uint64_t)(stage * (STAGE_BYTES / 16));
                    const uint64_t bd = bd0 + (uint64_t)(stage * (STAGE_BYTES / 16));
                    if (!mbar_wait(full0 + 8 * stage, phase, abort_flag)) goto done_mma;
                    __syncwarp();
                    fence_after();
                    const int steps = re - r >= BK ? BK / 16 : (re - r + 15) / 16;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            if (k < steps) mma_f16<1>(d, ad + k * a_step, bd + k * b_step, id, r > r0 || k > 0);
                        mma_commit<1>(empty0 + 8 * stage);
                        if (r + BK >= r1) mma_commit<1>(accf0 + 8 * buf);
                    }
                    __syncwarp();
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                buf ^= 1;
                aphase ^= buf == 0;
            }
        }
    done_mma:;
    } else {
        // ------------------------------------------------------ epilogue: lane = feature
        const int q = warp & 3, l = q * 32 + lane;
        const int64_t ld = kMode == kFprop ? p.N : p.K;
        int buf = 0;
        uint32_t aphase = 0;
        SplitSum<kSplit> split(smem_u32(smem) + PART_REGION, partf0, parte0, rank);
        for (int64_t t = first; t < W.total; t += stride) {
            const Tile T = W.get(t);
            float acc[WIDE];
            bool ok = true;
            for (int r0 = rb; r0 < re; r0 += FLUSH * BK) {
                ok = mbar_wait(accf0 + 8 * buf, aphase, abort_flag);
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
                if (!ok) break;
                fence_after();
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + buf * WIDE, v);
                tmem_wait_ld();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce0 + 8 * buf);
                buf ^= 1;
                aphase ^= buf == 0;
#pragma unroll
                for (int j = 0; j < WIDE; ++j)
                    acc[j] = r0 == rb ? __uint_as_float(v[j]) : __fadd_rn(acc[j], __uint_as_float(v[j]));
            }
            if (!ok || !split.exchange(acc, l, lane, q == 0, t + 2 * stride < W.total, abort_flag)) break;
            if (T.f0 + l >= ld) continue;
            const float b = kMode == kFprop && p.bias ? __bfloat162float(p.bias[(int64_t)T.e * p.N + T.f0 + l]) : 0.0f;
#pragma unroll
            for (int j = 0; j < WIDE / kSplit; ++j) {
                const int c = rank * (WIDE / kSplit) + j;
                if (c >= T.cols) break;
                const int64_t at = (T.row0 + c) * ld + T.f0 + l;
                const float v = __fadd_rn(acc[j], b);
                if (p.out_f32) static_cast<float*>(p.out)[at] = v;
                else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
            }
        }
    }
    fence_before();
    __syncthreads();
    if (s_abort && threadIdx.x == 0 && p.status) atomicOr(p.status, MXQ_STATUS_WAIT_TIMEOUT);
    if (kSplit > 1) cluster_sync();  // nothing is on its way to a CTA that has ended
    if (warp == 1) {
        fence_after();
        tmem_dealloc<1>(tmem, TMEM_COLS);
    }
}

template <int kMode, int kSplit>
static cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const Params& p, int64_t tiles, cudaStream_t s) {
    return launch_persistent<kSplit, false, ragged_few_kernel<kMode, kSplit>>(THREADS, smem_bytes(MXQ_MAX_EXPERTS),
                                                                      smem_bytes(p.E), tiles, s, a, b, p);
}

template <int kMode>
static cudaError_t run(const GemmCall& c, cudaStream_t s) {
    const Params p{c.M, c.N, c.K, c.E, c.m_splits, static_cast<const __nv_bfloat16*>(c.bias), c.out, c.out_f32, c.status};
    const int64_t red = kMode == kDgrad ? c.N : c.K, feats = ((kMode == kFprop ? c.N : c.K) + kFM - 1) / kFM;
    const int64_t da[3] = {c.K, c.N, c.E}, sa[2] = {2 * c.K, 2 * c.K * c.N}, db[2] = {red, c.M}, sb[1] = {2 * c.ld_tok};
    const int boxa[3] = {64, kMode == kDgrad ? BK : kFM, 1}, boxb[2] = {BK, WIDE};
    CUtensorMap a, b;
    if (!encode_tmap(&a, c.mat, 2, 3, da, sa, boxa) || !encode_tmap(&b, c.tok, 2, 2, db, sb, boxb))
        return cudaErrorInvalidValue;
    const int64_t tiles = (c.M / WIDE + std::min<int64_t>(c.E, c.M)) * feats;  // no fewer than the device counts
    switch (split_of(tiles, (red + BK - 1) / BK)) {
        case 8: return launch<kMode, 8>(a, b, p, tiles, s);
        case 4: return launch<kMode, 4>(a, b, p, tiles, s);
        case 2: return launch<kMode, 2>(a, b, p, tiles, s);
        default: return launch<kMode, 1>(a, b, p, tiles, s);
    }
}

}  // namespace few

cudaError_t run_gemm_few(const GemmCall& c, cudaStream_t s) {
    return c.mode == kFprop ? few::run<kFprop>(c, s) : few::run<kDgrad>(c, s);
}

// As many CTAs to a tile as still leave every tile in one wave and four stages
// or more to each. 16 rows of 1 expert, 2048 x 4096: 13.0 us unsplit, 8.6 us
// split four ways (dgrad, 16 tiles: 20.5 and 10.7 us). Beyond one wave the
// exchange of partial sums (about 2.5 us a tile) costs more than a better
// filled last wave gives: 8 experts, 256 tiles, 27.8 us unsplit, 29.2 us split.
int split_of(int64_t tiles, int64_t blocks) {
    int s = 8;
    while (s > 1 && (tiles * s > sm_count() || blocks < 4 * s)) s /= 2;
    return s;
}

}  // namespace ragged
}  // namespace mxq
