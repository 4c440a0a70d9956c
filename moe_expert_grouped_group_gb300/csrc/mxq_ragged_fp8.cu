// mxq_ragged_fp8.cu -- e4m3 grouped products of an MoE expert layer whose
// operands carry one fp32 scale for 128 consecutive values of a token's row and
// one for 128 x 128 of a weight, for expert counts that are multiples of
// nothing, and the quantizers of both:
//   a = max(|v| over the block, 2^-100),  scale = a / 448,  q = e4m3(v (448 / a))
//   fprop  Y[m,n]  = sum_j xs[j,m] ws[e,n/128,j] (Xq[m,j] . Wq[e,n,j]) (+ b[e,n])
//   dgrad  dX[m,k] = sum_j ds[j,m] ws[e,j,k/128] (dYq[m,j] . Wq[e,j,k])
// j runs over the blocks of 128 of the sum. Scales of rows are stored (blocks,
// M), so that those of a tile's rows lie side by side.
//
// A scale that is no power of two cannot ride in the block-scaled MMA, and the
// product of two scales differs from block to block and row to row. So an
// accumulator holds one block (four MMAs of 32 k, kind::f8f6f4), and the
// epilogue's warps add it to sums in registers, one fused multiply-add an
// element, while the MMAs fill the other accumulator. The tile walk, the
// operands' sides (features on the MMA's M, tokens on its N), the edges and the
// pairs of SMs are those of the bf16 products (mxq_ragged.cuh, mxq_ragged.cu);
// a stage is 128 deep and has their 32 KB an SM.
//
// Accumulators are read as matrix fragments (two columns of a lane side by
// side), so a thread needs the scales of 8 columns of 32 rather than of all 32.
// A warp fetches the rows' scales some blocks ahead, multiplies them by the
// weight's, which is one number for a block and an SM's 128 features, and
// leaves them in shared memory in the order in which the fragments want them.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "mxq_internal.h"
#include "mxq_ragged.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace ragged {
namespace f8 {

constexpr int BK = kFp8Block;  // reduction depth of a stage: 128 bytes, one block of scales

// Instruction descriptor for kind::f8f6f4, e4m3 x e4m3 (formats 0) with fp32 accumulation; fields as in idesc_f16.
__device__ __forceinline__ uint32_t idesc_e4m3(uint32_t a_mn, uint32_t m, uint32_t n) {
    return (1u << 4) | (a_mn << 15) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
template <int kCG>
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, uint32_t accum) {
    if constexpr (kCG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(id), "r"(accum)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(id), "r"(accum)
            : "memory");
}

struct Params {
    const float *xs, *ws;
    const __nv_bfloat16* bias;
    int64_t M, N, K;
    int E;
    const int64_t* m_splits;
    void* out;
    int out_f32;
    int32_t* status;
    int64_t ws_rows, ws_cols;  // blocks of N and of K
};

// Index of the weight's scale for features f .. f + 127 and block j of the sum.
template <int kMode>
__device__ __forceinline__ int64_t weight_scale_at(const Params& p, int e, int f, int j) {
    const int64_t i = f / BK;
    return kMode == kFprop ? (e * p.ws_rows + i) * p.ws_cols + j : (e * p.ws_rows + j) * p.ws_cols + i;
}

// Where a slot of scales keeps column j: of 16 columns, the four that a thread's fragments hold (8b + 2c and the next,
// b = 0 and 1) lie side by side.
__device__ __forceinline__ int slot_of(int j) { return (j & ~15) + ((j >> 1 & 3) << 2) + ((j >> 3 & 1) << 1) + (j & 1); }

// The scales of the tiles' columns, block by block, through a ring of slots in shared memory.
template <int kWide, int kSlots>
struct Scales {
    static constexpr int kBytes = kSlots * kWide * 4, kBatch = 4, kPer = kWide / 32;
    uint32_t at, full, empty;
    int slot = 0;
    uint32_t phase = 0;
    __device__ Scales(uint32_t at_, uint32_t full_, uint32_t empty_) : at(at_), full(full_), empty(empty_) {}
    __device__ void step() {
        if (++slot == kSlots) { slot = 0; phase ^= 1; }
    }
    // Fills slots with blocks j0 .. j1 of T's columns; f: this CTA's first feature. kBatch blocks' loads are in flight
    // together: they take as long as a block or two of MMAs. A whole warp; false when a bounded wait has expired.
    template <int kMode>
    __device__ bool produce(const Params& p, const Tile& T, int f, int j0, int j1, int lane, volatile int* abort_flag) {
        for (int j = j0; j < j1; j += kBatch) {
            float v[kBatch][kPer], w[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                w[b] = 0.0f;
                if (j + b < j1 && f < (kMode == kFprop ? p.N : p.K)) w[b] = p.ws[weight_scale_at<kMode>(p, T.e, f, j + b)];
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int c = 32 * i + lane;
                    v[b][i] = 0.0f;
                    if (j + b < j1 && c < T.cols) v[b][i] = p.xs[(j + b) * p.M + T.row0 + c];
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (j + b >= j1) break;
                if (!__all_sync(0xffffffffu, mbar_wait(empty + 8 * slot, phase ^ 1, abort_flag))) return false;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 4 * (slot * kWide + slot_of(32 * i + lane))),
                                 "f"(v[b][i] * w[b])
                                 : "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(full + 8 * slot);
                step();
            }
        }
        return true;
    }
    // Scales of this thread's columns among 16 from column c on: 8b + 2 (lane mod 4) and the next, b = 0, 1
    __device__ float4 get(int c, int lane) const {
        float4 s;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(s.x), "=f"(s.y), "=f"(s.z), "=f"(s.w)
                     : "r"(at + 4 * (slot * kWide + c + 4 * (lane & 3)))
                     : "memory");
        return s;
    }
};

// Sums of 32 columns by this warp's 32 lanes as fragments: [16-lane half][2b + g]: lanes t/4 + 8g of the half, columns
// 8b + 2(t mod 4) and the next.
using Sums = uint64_t[2][8];

// sums += the accumulator's columns (loaded as fragments) times their scales
__device__ __forceinline__ void add_scaled(Sums& s, const uint32_t (&v)[2][16], float4 lo, float4 hi) {
    const uint64_t k[4] = {f2pack(lo.x, lo.y), f2pack(lo.z, lo.w), f2pack(hi.x, hi.y), f2pack(hi.z, hi.w)};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[h][i] = f2fma(f2pack(__uint_as_float(v[h][2 * i]), __uint_as_float(v[h][2 * i + 1])), k[i >> 1], s[h][i]);
}

// ------------------------------------------------------------ pairs of SMs
namespace pair {

constexpr int CG = 2;
constexpr int FEAT = kFM * CG;
constexpr int WIDE = 256, STEP = 16 * CG;
constexpr int BOX = 64;
constexpr int STAGES = 6;
constexpr int SLOTS = 8;
constexpr int EPI_FIRST = 4, EPI_WARPS = 8;
constexpr int THREADS = 32 * (EPI_FIRST + EPI_WARPS);
constexpr int CTL_REGS = 80, EPI_REGS = 208;
static_assert(EPI_FIRST * CTL_REGS + EPI_WARPS * EPI_REGS <= THREADS / 32 * (65536 / THREADS / 8 * 8),
              "the warps' registers are those that the block starts with");
constexpr int A_BYTES = kFM * BK, STAGE_BYTES = A_BYTES + WIDE / CG * BK;
constexpr int TMEM_COLS = 2 * WIDE;
constexpr int EPI_REGION = STAGES * STAGE_BYTES;  // staging of the bf16 epilogue, kBoxBytes a warp
using Ring = Scales<WIDE, SLOTS>;
constexpr int SCALE_REGION = EPI_REGION + EPI_WARPS * kBoxBytes;
constexpr int BAR_REGION = SCALE_REGION + Ring::kBytes;
constexpr int TABLE_REGION = BAR_REGION + 320;
__host__ __device__ constexpr int smem_bytes(int E) { return 1024 + TABLE_REGION + 8 * (E + 1); }
static_assert(smem_bytes(MXQ_MAX_EXPERTS) <= 232448, "shared memory over the per-block limit");
static_assert(BAR_REGION % 16 == 0 && 8 * (2 * STAGES + 2 * SLOTS + 6) + 16 <= 320, "barrier region");

template <int kMode>
__global__ void __launch_bounds__(THREADS, 1)
    ragged_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmHalf, Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align<1024>(smem_raw);
    int32_t* s_off = reinterpret_cast<int32_t*>(smem + TABLE_REGION);
    int32_t* s_slices = s_off + p.E + 1;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_REGION);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, sfull0 = empty0 + 8 * STAGES;
    const uint32_t sempty0 = sfull0 + 8 * SLOTS, accf0 = sempty0 + 8 * SLOTS, acce0 = accf0 + 16;
    const uint32_t ready = acce0 + 16, taken = ready + 8, answer = (taken + 8 + 15) & ~15u;
    volatile int* abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int st = 0; st < STAGES; ++st) {
            mbar_init(full0 + 8 * st, 1);
            mbar_init(empty0 + 8 * st, 1);
        }
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(sfull0 + 8 * i, 1);
            mbar_init(sempty0 + 8 * i, EPI_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, CG * EPI_WARPS);
        }
        mbar_init(ready, 1);
        mbar_init(taken, 7 + 2 * EPI_WARPS);  // the warps of both CTAs that call next()
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmA) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmB) : "memory");
    }
    // both CTAs of a pair find the same fault and stop before any cluster-wide step
    const int bad = load_ragged(p.m_splits, p.E, p.M, WIDE, s_off, s_slices);
    if (bad) {
        report_status(p.status, bad);
        return;
    }
    if (warp == 1) tmem_alloc<CG>(smem_u32(&s_tmem), TMEM_COLS);
    fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any load completes on rank 0's
    fence_after();
    const uint32_t tmem = s_tmem;
    const Walk<kMode, FEAT, WIDE, STEP> W(p.N, p.K, p.E, s_off, s_slices, nullptr);
    TileQueue queue(answer, ready, mapa(taken, 0));
    Ring ring(smem_u32(smem) + SCALE_REGION, sfull0, sempty0);
    int64_t t = blockIdx.x / CG;

    if (warp < EPI_FIRST) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTL_REGS));
        if (warp == 0) {
            // -------------------------------------------------- TMA producer
            int stage = 0;
            uint32_t phase = 0;
            int64_t fills = 0;
            do {
                if (t >= W.total) continue;
                const Tile T = W.get(t);
                const int half = T.n / CG;  // this CTA's columns of the tile: [rank * half, + half)
                // token rows: whole boxes, and half a box at the end where that is enough
                const bool half_box = (half - 1) % BOX < BOX / 2;
                const int boxes = half_box ? half / BOX : (half + BOX - 1) / BOX;
                const int f = T.f0 + rank * kFM, c = T.c0 + rank * half;
                const uint32_t bytes = A_BYTES + (2 * boxes + half_box) * (BOX / 2 * BK);
                for (int r = 0; r < T.red; r += BK) {
                    if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag)) {
                        if (rank == 0) drain_ring(full0, STAGES, fills);  // both CTAs' loads complete on rank 0's
                        goto done_producer;
                    }
                    __syncwarp();
                    const uint32_t own = full0 + 8 * stage, fb = mapa(own, 0);
                    const uint32_t a = smem_u32(smem) + stage * STAGE_BYTES, b = a + A_BYTES;
                    if (elect_one()) {
                        if (rank == 0) mbar_expect_tx(own, CG * bytes);
                        if (kMode == kFprop) load_3d<CG>(a, &tmA, fb, r, f, T.e);
                        else load_3d<CG>(a, &tmA, fb, f, r, T.e);
#pragma unroll
                        for (int i = 0; i < WIDE / CG / BOX; ++i)
                            if (i < boxes) load_2d<CG>(b + BOX * BK * i, &tmB, fb, r, c + BOX * i);
                        if (half_box) load_2d<CG>(b + BOX * BK * boxes, &tmHalf, fb, r, c + BOX * boxes);
                    }
                    __syncwarp();
                    ++fills;
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            } while (queue.next(t, lane, abort_flag) == TileQueue::kTile);
        done_producer:;
        } else if (warp == 1) {
            // -------------------------------------------------- MMA issuer (rank 0)
            if (rank == 0) {
                int stage = 0, buf = 0;
                uint32_t phase = 0, aphase = 0;
                const uint32_t base = smem_u32(smem);
                // MN-major A: one 128-byte chunk of features, 8-row groups of the reduction 1024 bytes apart
                const uint64_t ad0 = smem_desc(base, 16, 1024), bd0 = smem_desc(base + A_BYTES, 16, 1024);
                constexpr uint32_t a_step = (kMode == kDgrad ? 4096 : 32) / 16, b_step = 32 / 16;  // 32 of the sum
                do {
                    if (t >= W.total) continue;
                    const Tile T = W.get(t);
                    const uint32_t id = idesc_e4m3(kMode == kDgrad, FEAT, T.n);
                    for (int r = 0; r < T.red; r += BK) {
                        const uint64_t ad = ad0 + (uint64_t)(stage * (STAGE_BYTES / 16));
                        const uint64_t bd = bd0 + (uint64_t)(stage * (STAGE_BYTES / 16));
                        if (!mbar_wait(acce0 + 8 * buf, aphase ^ 1, abort_flag)) goto done_mma;
                        if (!mbar_wait(full0 + 8 * stage, phase, abort_flag)) goto done_mma;
                        __syncwarp();
                        fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < BK / 32; ++k)
                                mma_e4m3<CG>(tmem + buf * WIDE, ad + k * a_step, bd + k * b_step, id, k > 0);
                            mma_commit<CG>(accf0 + 8 * buf);
                            mma_commit<CG>(empty0 + 8 * stage);
                        }
                        __syncwarp();
                        if (++stage == STAGES) { stage = 0; phase ^= 1; }
                        buf ^= 1;
                        aphase ^= buf == 0;
                    }
                } while (queue.next(t, lane, abort_flag) == TileQueue::kTile);
            done_mma:;
            }
        } else if (warp == 2) {
            // -------------------------------------------------- scales
            do {
                if (t >= W.total) continue;
                const Tile T = W.get(t);
                if (!ring.template produce<kMode>(p, T, T.f0 + rank * kFM, 0, (T.red + BK - 1) / BK, lane, abort_flag)) break;
            } while (queue.next(t, lane, abort_flag) == TileQueue::kTile);
        } else {
            // -------------------------------------------------- next tiles
            for (uint32_t asked = 0;; asked ^= 1) {
                if (rank == 0 && !mbar_wait(taken, asked ^ 1, abort_flag)) break;
                __syncwarp();
                if (elect_one()) {
                    mbar_expect_tx(ready, 16);
                    if (rank == 0) queue.ask();
                }
                __syncwarp();
                if (queue.next(t, lane, abort_flag) != TileQueue::kTile) break;
            }
        }
    } else {
        // ------------------------------------------------------ epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
        const int q = warp & 3, group = (warp - EPI_FIRST) >> 2;  // two groups of four warps share the columns
        uint8_t* stage = smem + EPI_REGION + (warp - EPI_FIRST) * kBoxBytes;
        const int64_t ld = kMode == kFprop ? p.N : p.K;  // features
        constexpr int kChunks = WIDE / 64;               // 32-column chunks of a group
        int buf = 0;
        uint32_t aphase = 0;
        const uint32_t acce = mapa(acce0, 0);
        do {
            if (t >= W.total) continue;
            const Tile T = W.get(t);
            Sums acc[kChunks];
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[i][h][j] = 0;
            bool ok = true;
            for (int r = 0; r < T.red; r += BK) {
                ok = mbar_wait(ring.full + 8 * ring.slot, ring.phase, abort_flag) &&
                     mbar_wait(accf0 + 8 * buf, aphase, abort_flag);
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
                if (!ok) break;
                fence_after();
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    const int c = 64 * i + 32 * group;
                    if (c < T.cols) {
                        uint32_t v[2][16];
                        const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + buf * WIDE + c;
                        tmem_ld16x32(at, v[0]);
                        tmem_ld16x32(at + (16u << 16), v[1]);
                        const float4 lo = ring.get(c, lane), hi = ring.get(c + 16, lane);
                        tmem_wait_ld();
                        add_scaled(acc[i], v, lo, hi);
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(acce0 + 8 * buf);
                    else arrive_remote_relaxed(acce + 8 * buf);
                    mbar_arrive(ring.empty + 8 * ring.slot);
                }
                ring.step();
                buf ^= 1;
                aphase ^= buf == 0;
            }
            if (!ok) break;
            const int f0 = T.f0 + rank * kFM + 32 * q;
            const int live = (int)min((int64_t)32, ld - f0);  // may be negative: nothing to store
            float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (kMode == kFprop && p.bias) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int l = (lane >> 2) + 8 * g;
                    if (l < live) b[g] = __bfloat162float(p.bias[(int64_t)T.e * p.N + f0 + l]);
                }
            }
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int c0 = 64 * i + 32 * group;
                if (c0 >= T.cols) continue;
                if (p.out_f32) {
                    // eight lanes write 32 contiguous bytes
                    float* o = static_cast<float*>(p.out) + (T.row0 + c0) * ld + f0;
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int l = (lane >> 2) + 8 * g, c = 8 * j + 2 * (lane & 3);
                            const float2 v = f2unpack(acc[i][g >> 1][2 * j + (g & 1)]);
                            if (l < live && c0 + c < T.cols) o[c * ld + l] = v.x + b[g];
                            if (l < live && c0 + c + 1 < T.cols) o[(c + 1) * ld + l] = v.y + b[g];
                        }
                } else {
                    // transposed through the warp's stage: rows of 64 bytes, their 16-byte pieces exchanged by the
                    // row's bits 1 and 2
                    const int row = lane & 7;
                    const uint32_t at = smem_u32(stage) + row * 64 + (((lane >> 3) ^ (row >> 1)) << 4);
                    __syncwarp();  // the stage's last reads are done
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const float2 v = f2unpack(acc[i][g >> 1][2 * j + (g & 1)]);
                            w[g] = bf16x2_bits(v.x + b[g], v.y + b[g]);
                        }
                        stmatrix_trans(at + 512 * j, w);
                    }
                    __syncwarp();
                    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + (T.row0 + c0) * ld + f0;
                    const int piece = lane & 3;
                    if (piece * 8 < live)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int c = 8 * j + (lane >> 2);
                            if (c0 + c < T.cols)
                                *reinterpret_cast<uint4*>(o + c * ld + piece * 8) =
                                    *reinterpret_cast<const uint4*>(stage + c * 64 + ((piece ^ (c >> 1 & 3)) << 4));
                        }
                }
            }
        } while (queue.next(t, lane, abort_flag) == TileQueue::kTile);
    }
    fence_before();
    __syncthreads();
    if (s_abort && threadIdx.x == 0 && p.status) atomicOr(p.status, MXQ_STATUS_WAIT_TIMEOUT);
    cluster_sync();  // rank 0's MMAs have read this CTA's shared memory for the last time
    if (warp == 1) {
        fence_after();
        tmem_dealloc<CG>(tmem, TMEM_COLS);
    }
}

}  // namespace pair

// ------------------------------------------------------------ few rows
// One-SM tiles of 128 features by up to 32 rows: what is left is reading W once. As in the bf16 kernel for few rows
// (mxq_ragged_few.cu), a stage is 16 KB of W and at most 4 KB of tokens, eight are in flight, and where the tiles do not
// fill the SMs the sum is split over a cluster. An accumulator is 32 columns, so there are four.
namespace few {

constexpr int STAGES = 8, SLOTS = 16, BUFS = 4;
constexpr int WIDE = kFewRows, STEP = 16;
constexpr int A_BYTES = kFM * BK, STAGE_BYTES = A_BYTES + WIDE * BK;
constexpr int EPI_FIRST = 4, EPI_WARPS = 4;  // warp 3 is idle
constexpr int THREADS = 32 * (EPI_FIRST + EPI_WARPS);
constexpr int TMEM_COLS = BUFS * WIDE;
using Ring = Scales<WIDE, SLOTS>;
constexpr int PART_REGION = STAGES * STAGE_BYTES;
constexpr int SCALE_REGION = PART_REGION + kPartBytes;
constexpr int BAR_REGION = SCALE_REGION + Ring::kBytes;
constexpr int TABLE_REGION = BAR_REGION + 512;
__host__ __device__ constexpr int smem_bytes(int E) { return 1024 + TABLE_REGION + 8 * (E + 1); }
static_assert(smem_bytes(MXQ_MAX_EXPERTS) <= 232448, "shared memory over the per-block limit");
static_assert(8 * (2 * STAGES + 2 * SLOTS + 2 * BUFS + 4) <= 512, "barrier region");

template <int kMode, int kSplit>
__global__ void __launch_bounds__(THREADS, 1)
    ragged_fp8_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align<1024>(smem_raw);
    int32_t* s_off = reinterpret_cast<int32_t*>(smem + TABLE_REGION);
    int32_t* s_slices = s_off + p.E + 1;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = kSplit > 1 ? (int)cta_rank() : 0;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_REGION);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, sfull0 = empty0 + 8 * STAGES;
    const uint32_t sempty0 = sfull0 + 8 * SLOTS, accf0 = sempty0 + 8 * SLOTS, acce0 = accf0 + 8 * BUFS;
    const uint32_t partf0 = acce0 + 8 * BUFS, parte0 = partf0 + 16;
    volatile int* abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int st = 0; st < STAGES; ++st) {
            mbar_init(full0 + 8 * st, 1);
            mbar_init(empty0 + 8 * st, 1);
        }
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(sfull0 + 8 * i, 1);
            mbar_init(sempty0 + 8 * i, EPI_WARPS);
        }
        for (int b = 0; b < BUFS; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, EPI_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
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
    // this CTA's part of the reduction in blocks, the same for every tile
    const int red = (int)(kMode == kDgrad ? p.N : p.K), blocks = (red + BK - 1) / BK;
    const int jb = blocks * rank / kSplit, je = blocks * (rank + 1) / kSplit;
    Ring ring(smem_u32(smem) + SCALE_REGION, sfull0, sempty0);

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0;
        int64_t fills = 0;
        for (int64_t t = first; t < W.total; t += stride) {
            const Tile T = W.get(t);
            for (int j = jb; j < je; ++j) {
                if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag)) {
                    drain_ring(full0, STAGES, fills);
                    goto done_producer;
                }
                __syncwarp();
                const uint32_t fb = full0 + 8 * stage, a = smem_u32(smem) + stage * STAGE_BYTES;
                if (elect_one()) {
                    mbar_expect_tx(fb, STAGE_BYTES);
                    if (kMode == kFprop) load_3d<1>(a, &tmA, fb, j * BK, T.f0, T.e);
                    else load_3d<1>(a, &tmA, fb, T.f0, j * BK, T.e);
                    load_2d<1>(a + A_BYTES, &tmB, fb, j * BK, T.c0);
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
        const uint64_t ad0 = smem_desc(base, 16, 1024), bd0 = smem_desc(base + A_BYTES, 16, 1024);
        constexpr uint32_t a_step = (kMode == kDgrad ? 4096 : 32) / 16, b_step = 32 / 16;
        for (int64_t t = first; t < W.total; t += stride) {
            const Tile T = W.get(t);
            const uint32_t id = idesc_e4m3(kMode == kDgrad, kFM, T.n);
            for (int j = jb; j < je; ++j) {
                const uint64_t ad = ad0 + (uint64_t)(stage * (STAGE_BYTES / 16));
                const uint64_t bd = bd0 + (uint64_t)(stage * (STAGE_BYTES / 16));
                if (!mbar_wait(acce0 + 8 * buf, aphase ^ 1, abort_flag)) goto done_mma;
                if (!mbar_wait(full0 + 8 * stage, phase, abort_flag)) goto done_mma;
                __syncwarp();
                fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        mma_e4m3<1>(tmem + buf * WIDE, ad + k * a_step, bd + k * b_step, id, k > 0);
                    mma_commit<1>(empty0 + 8 * stage);
                    mma_commit<1>(accf0 + 8 * buf);
                }
                __syncwarp();
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
                if (++buf == BUFS) { buf = 0; aphase ^= 1; }
            }
        }
    done_mma:;
    } else if (warp == 2) {
        // ------------------------------------------------------ scales
        for (int64_t t = first; t < W.total; t += stride) {
            const Tile T = W.get(t);
            if (!ring.template produce<kMode>(p, T, T.f0, jb, je, lane, abort_flag)) break;
        }
    } else if (warp >= EPI_FIRST) {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3, l = q * 32 + lane;
        const int64_t ld = kMode == kFprop ? p.N : p.K;
        int buf = 0;
        uint32_t aphase = 0;
        SplitSum<kSplit> split(smem_u32(smem) + PART_REGION, partf0, parte0, rank);
        for (int64_t t = first; t < W.total; t += stride) {
            const Tile T = W.get(t);
            Sums acc;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[h][i] = 0;
            bool ok = true;
            for (int j = jb; j < je; ++j) {
                ok = mbar_wait(ring.full + 8 * ring.slot, ring.phase, abort_flag) &&
                     mbar_wait(accf0 + 8 * buf, aphase, abort_flag);
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
                if (!ok) break;
                fence_after();
                uint32_t v[2][16];
                const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + buf * WIDE;
                tmem_ld16x32(at, v[0]);
                tmem_ld16x32(at + (16u << 16), v[1]);
                const float4 lo = ring.get(0, lane), hi = ring.get(16, lane);
                tmem_wait_ld();
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(acce0 + 8 * buf);
                    mbar_arrive(ring.empty + 8 * ring.slot);
                }
                ring.step();
                if (++buf == BUFS) { buf = 0; aphase ^= 1; }
                add_scaled(acc, v, lo, hi);
            }
            // sums in the order [8-column block][column of the two][8-lane block], which a split divides
            float s[WIDE];
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float2 v = f2unpack(acc[g >> 1][2 * b + (g & 1)]);
                    s[8 * b + g] = v.x;
                    s[8 * b + 4 + g] = v.y;
                }
            if (!ok || !split.exchange(s, l, lane, q == 0, t + 2 * stride < W.total, abort_flag)) break;
            const int f0 = T.f0 + 32 * q + (lane >> 2);
            float b[4];
#pragma unroll
            for (int g = 0; g < 4; ++g)
                b[g] = kMode == kFprop && p.bias && f0 + 8 * g < ld
                           ? __bfloat162float(p.bias[(int64_t)T.e * p.N + f0 + 8 * g])
                           : 0.0f;
#pragma unroll
            for (int i = 0; i < WIDE / kSplit; ++i) {
                const int at = rank * (WIDE / kSplit) + i, g = i & 3;  // WIDE / kSplit is a multiple of 4
                const int c = 8 * (at >> 3) + 2 * (lane & 3) + (at >> 2 & 1), f = f0 + 8 * g;
                if (c >= T.cols || f >= ld) continue;
                const float v = __fadd_rn(s[i], b[g]);
                if (p.out_f32) static_cast<float*>(p.out)[(T.row0 + c) * ld + f] = v;
                else static_cast<__nv_bfloat16*>(p.out)[(T.row0 + c) * ld + f] = __float2bfloat16_rn(v);
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

}  // namespace few

// ------------------------------------------------------------ quantizers
// Scale and codes of a block from the bits of its largest magnitude (bf16, widened). A block that holds an infinity or
// NaN gets scale NaN and codes 0, so that what it enters is NaN.
struct BlockScale {
    float inv, scale;
    __device__ explicit BlockScale(uint32_t top) {
        const float amax = fmaxf(__uint_as_float(top << 16), 7.8886090522101181e-31f);  // 2^-100
        const bool finite = top < 0x7F80u;
        inv = finite ? __fdiv_rn(448.0f, amax) : 0.0f;
        scale = finite ? __fdiv_rn(amax, 448.0f) : __uint_as_float(0x7FC00000u);
    }
    __device__ uint32_t codes4(uint32_t a, uint32_t b) const {
        return cvt_e4m3x2(__fmul_rn(bf16lo(a), inv), __fmul_rn(bf16hi(a), inv)) |
               cvt_e4m3x2(__fmul_rn(bf16lo(b), inv), __fmul_rn(bf16hi(b), inv)) << 16;
    }
    // the codes of eight values; 0 * inf would be NaN
    __device__ uint2 codes(const uint4& w) const {
        return inv == 0.0f ? make_uint2(0u, 0u) : make_uint2(codes4(w.x, w.y), codes4(w.z, w.w));
    }
};
__device__ __forceinline__ uint32_t magnitude8(const uint4& w) {  // the largest of eight, in both halves' bits
    return __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
}

// Rows: a warp reads 256 columns (two blocks) of kRows rows at once; a block of eight warps makes 2 x 8 kRows scales,
// which leave through shared memory as runs of 8 kRows rows.
template <int kRows>
__global__ void __launch_bounds__(256) fp8_quantize_rows_kernel(const uint16_t* x, int64_t M, int64_t K, int64_t ld,
                                                                uint8_t* q, float* scale) {
    __shared__ float s_scale[2][8 * kRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t across = (K + 255) / 256, tiles = across * ((M + 8 * kRows - 1) / (8 * kRows));
    wait_for_stream();
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t m0 = t / across * (8 * kRows), k = t % across * 256 + 8 * lane;
        uint4 v[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t m = m0 + warp * kRows + i;
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (m < M && k < K) v[i] = *reinterpret_cast<const uint4*>(x + m * ld + k);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t m = m0 + warp * kRows + i;
            uint32_t top = magnitude8(v[i]);
#pragma unroll
            for (int o = 8; o; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
            const BlockScale s(max(top & 0xFFFFu, top >> 16));
            if (m < M && k < K) *reinterpret_cast<uint2*>(q + m * K + k) = s.codes(v[i]);
            if ((lane & 15) == 0) s_scale[lane >> 4][warp * kRows + i] = s.scale;
        }
        __syncthreads();
        if (threadIdx.x < 16 * kRows) {
            const int64_t j = t % across * 2 + threadIdx.x / (8 * kRows), m = m0 + threadIdx.x % (8 * kRows);
            if (m < M && j * BK < K) scale[j * M + m] = s_scale[threadIdx.x / (8 * kRows)][threadIdx.x % (8 * kRows)];
        }
        __syncthreads();
    }
}

// Weights: a block of 256 threads holds one 128 x 128 block in registers, 16 bytes of eight rows a thread.
__global__ void __launch_bounds__(256) fp8_quantize_weight_kernel(const uint16_t* w, int64_t N, int64_t K, int64_t across,
                                                                  int64_t down, uint8_t* q, float* scale) {
    __shared__ uint32_t s_top[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t b = blockIdx.x, j = b % across, i = b / across % down, e = b / across / down;
    const int64_t k = j * BK + 8 * (threadIdx.x & 15), n0 = i * BK + (threadIdx.x >> 4);
    wait_for_stream();
    uint4 v[8];
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        v[r] = make_uint4(0u, 0u, 0u, 0u);
        if (n0 + 16 * r < N && k < K) v[r] = *reinterpret_cast<const uint4*>(w + (e * N + n0 + 16 * r) * K + k);
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) top = __vmaxu2(top, magnitude8(v[r]));
    top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 8; ++r) top = max(top, s_top[r]);
    const BlockScale s(top);
#pragma unroll
    for (int r = 0; r < 8; ++r)
        if (n0 + 16 * r < N && k < K) *reinterpret_cast<uint2*>(q + (e * N + n0 + 16 * r) * K + k) = s.codes(v[r]);
    if (threadIdx.x == 0) scale[b] = s.scale;
}

// ------------------------------------------------------------------ host side
static Params params(const Fp8Call& c) {
    return {c.ts, c.ws, static_cast<const __nv_bfloat16*>(c.bias), c.M, c.N, c.K, c.E, c.m_splits, c.out, c.out_f32,
            c.status, (c.N + BK - 1) / BK, (c.K + BK - 1) / BK};
}

template <int kMode>
static cudaError_t run_pair(const Fp8Call& c, cudaStream_t s) {
    using namespace pair;
    const int64_t red = kMode == kDgrad ? c.N : c.K, feats = ((kMode == kFprop ? c.N : c.K) + FEAT - 1) / FEAT;
    const int64_t da[3] = {c.K, c.N, c.E}, sa[2] = {c.K, c.K * c.N}, db[2] = {red, c.M}, sb[1] = {red};
    const int boxa[3] = {BK, kFM, 1}, boxb[2] = {BK, BOX}, boxh[2] = {BK, BOX / 2};
    CUtensorMap a, b, half;
    if (!encode_tmap(&a, c.wq, 1, 3, da, sa, boxa) || !encode_tmap(&b, c.tq, 1, 2, db, sb, boxb) ||
        !encode_tmap(&half, c.tq, 1, 2, db, sb, boxh))
        return cudaErrorInvalidValue;
    const int64_t tiles = (c.M / WIDE + std::min<int64_t>(c.E, c.M)) * feats;  // no fewer than the device counts
    return launch_persistent<CG, true, ragged_fp8_kernel<kMode>>(THREADS, smem_bytes(MXQ_MAX_EXPERTS), smem_bytes(c.E),
                                                                 tiles, s, a, b, half, params(c));
}

template <int kMode, int kSplit>
static cudaError_t launch_few(const CUtensorMap& a, const CUtensorMap& b, const Fp8Call& c, int64_t tiles, cudaStream_t s) {
    return launch_persistent<kSplit, false, few::ragged_fp8_few_kernel<kMode, kSplit>>(
        few::THREADS, few::smem_bytes(MXQ_MAX_EXPERTS), few::smem_bytes(c.E), tiles, s, a, b, params(c));
}

template <int kMode>
static cudaError_t run_few(const Fp8Call& c, cudaStream_t s) {
    const int64_t red = kMode == kDgrad ? c.N : c.K, feats = ((kMode == kFprop ? c.N : c.K) + kFM - 1) / kFM;
    const int64_t da[3] = {c.K, c.N, c.E}, sa[2] = {c.K, c.K * c.N}, db[2] = {red, c.M}, sb[1] = {red};
    const int boxa[3] = {BK, kFM, 1}, boxb[2] = {BK, few::WIDE};
    CUtensorMap a, b;
    if (!encode_tmap(&a, c.wq, 1, 3, da, sa, boxa) || !encode_tmap(&b, c.tq, 1, 2, db, sb, boxb))
        return cudaErrorInvalidValue;
    const int64_t tiles = (c.M / few::WIDE + std::min<int64_t>(c.E, c.M)) * feats;  // no fewer than the device counts
    switch (split_of(tiles, (red + BK - 1) / BK)) {
        case 8: return launch_few<kMode, 8>(a, b, c, tiles, s);
        case 4: return launch_few<kMode, 4>(a, b, c, tiles, s);
        case 2: return launch_few<kMode, 2>(a, b, c, tiles, s);
        default: return launch_few<kMode, 1>(a, b, c, tiles, s);
    }
}

}  // namespace f8

cudaError_t run_fp8(const Fp8Call& c, cudaStream_t s) {
    if (c.M <= (int64_t)kFewRows * c.E) return c.mode == kFprop ? f8::run_few<kFprop>(c, s) : f8::run_few<kDgrad>(c, s);
    return c.mode == kFprop ? f8::run_pair<kFprop>(c, s) : f8::run_pair<kDgrad>(c, s);
}

cudaError_t run_fp8_quantize_rows(const void* x, int64_t M, int64_t K, int64_t ld, void* q, float* scale, cudaStream_t s) {
    if (M == 0) return cudaSuccess;
    const int64_t tiles = (K + 255) / 256 * ((M + 31) / 32);
    return launch(f8::fp8_quantize_rows_kernel<4>, (unsigned)std::min<int64_t>(tiles, (int64_t)sm_count() * 8), 256, s, 0,
                  static_cast<const uint16_t*>(x), M, K, ld, static_cast<uint8_t*>(q), scale);
}

cudaError_t run_fp8_quantize_weight(const void* w, int64_t N, int64_t K, int E, void* q, float* scale, cudaStream_t s) {
    const int64_t across = (K + f8::BK - 1) / f8::BK, down = (N + f8::BK - 1) / f8::BK;
    return launch(f8::fp8_quantize_weight_kernel, (unsigned)(across * down * E), 256, s, 0,
                  static_cast<const uint16_t*>(w), N, K, across, down, static_cast<uint8_t*>(q), scale);
}

}  // namespace ragged
}  // namespace mxq
