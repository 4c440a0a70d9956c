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
// element, while the MMAs fill the other accumulator. That is the bottleneck:
// everything an accumulator holds leaves TMEM once a block. Stamped in one CTA
// (16384 x 2048 by 4096 x 2048), a block takes its epilogue warps 730 to 760
// cycles: 150 for two barriers and the factor, 330 from the first load to the
// last with half of the FMAs, 210 for the other half; its MMAs take 512 at the
// pipe's rate. A tile's end takes 2300 more, of 14000: 780 to the staged rows, 620 for
// the proxy fence and the boxes, 900 to the next tile's first sums. Loads that
// run on from one block into the next (two at a time 128 us for the product,
// four 120 to 124, against 112), the next factor read a block ahead (112.5, but
// dgrad 117 against 107) and FMAs one at a time (118) were slower. Without any
// loads and FMAs the same kernel takes 95 us (dgrad 96): the rest is the MMAs,
// their feed and the tiles' ends, as in the MXFP8 product of this shape.
//
// The factor is the product of the two scales, rounded: callers keep it within
// fp32's range. Other results than infinite or NaN beyond it cost every call:
// a second factor for the blocks that need one, behind a flag, 117 -> 147 us (dgrad 104 -> 142);
// such rows made again from their codes at the tile's end dgrad 104 -> 110 and
// 8 experts x 2 rows 13.5 -> 15.2.
//
// Which operand is which. In the kernel for tiles of one SM (128 rows) or a
// pair (256) the tokens are on the MMA's M: a
// thread of the epilogue has one token, so one factor for a block and 128
// features, and reads TMEM 32 lanes at a time. With the features on M, as in
// the bf16 products, the factor differs from column to column: 256 factors a
// block from shared memory cost more than the FMAs (a warp's 128 columns with
// them 743 cycles, without 316), and fragment loads, which need few factors,
// take TMEM twice as long (560). The price is that a tile has 128 or 256 rows
// whatever the expert has. Experts with few rows on average go to the kernel
// below, whose tokens are on N.
//
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "mxq_internal.h"
#include "mxq_ragged.cuh"
#include "mxq_ragged.h"
#include "mxq_ragged_swiglu.cuh"

namespace mxq {
namespace ragged {
namespace f8 {

constexpr int BK = kFp8Block;  // reduction depth of a stage: 128 bytes, one block of scales

// Instruction descriptor for kind::f8f6f4, e4m3 x e4m3 (formats 0) with fp32 accumulation; fields as in idesc_f16.
__device__ __forceinline__ uint32_t idesc_e4m3(uint32_t a_mn, uint32_t b_mn, uint32_t m, uint32_t n) {
    return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
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

// In the kernel for few rows: the scales of the tiles' columns, block by block, through a ring of slots in shared memory. A slot keeps its columns in
// the order in which matrix fragments want them: of 16 columns, the four that a thread holds (8b + 2c and the next, b = 0
// and 1) side by side.
struct Scales {
    static constexpr int kWide = kFewRows, kSlots = 16;
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
                if (j + b < j1) w[b] = p.ws[weight_scale_at<kMode>(p, T.e, f, j + b)];
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
                for (int i = 0; i < kPer; ++i) {
                    const int c = 32 * i + lane;
                    const int to = (c & ~15) + ((c >> 1 & 3) << 2) + ((c >> 3 & 1) << 1) + (c & 1);
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 4 * (slot * kWide + to)), "f"(v[b][i] * w[b]) : "memory");
                }
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

// Sums of 32 columns by 16 lanes as a matrix fragment: [2b + g]: lane t/4 + 8g, columns 8b + 2(t mod 4) and the next.
using Sums = uint64_t[8];

// sums += the accumulator's columns (loaded as a fragment) times their scales
__device__ __forceinline__ void add_scaled(Sums& s, const uint32_t (&v)[16], float4 lo, float4 hi) {
    const uint64_t k[4] = {f2pack(lo.x, lo.y), f2pack(lo.z, lo.w), f2pack(hi.x, hi.y), f2pack(hi.z, hi.w)};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        s[i] = f2fma(f2pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), k[i >> 1], s[i]);
}

// ------------------------------------------------- pairs of SMs, and single ones
namespace wide {

constexpr int WIDE = 256;        // features of a tile, on the MMA's N: two blocks of the weight
constexpr int SLOTS = 8;         // blocks whose scales are on chip
constexpr int GROUP = 4;         // and that are handed over together; a tile begins at a new group
constexpr int AHEAD = 2;         // blocks whose scales' loads are in flight together
static_assert(SLOTS == 2 * GROUP && GROUP % AHEAD == 0, "the ring is two groups");
constexpr int EPI_FIRST = 4, EPI_WARPS = 8;
constexpr int THREADS = 32 * (EPI_FIRST + EPI_WARPS);
constexpr int CTL_REGS = 56, EPI_REGS = 224;
static_assert(EPI_FIRST * CTL_REGS + EPI_WARPS * EPI_REGS <= THREADS / 32 * (65536 / THREADS / 8 * 8),
              "the warps' registers are those that the block starts with");
constexpr int TMEM_COLS = 2 * WIDE;
constexpr int BOX_BYTES = 32 * 128;      // 32 rows of 128 bytes
constexpr int SLOT_BYTES = 2 * kFM * 4;  // a factor for each of this CTA's rows and each block of features

// Shared memory of a CTA. CG of them share a tile: each has 128 of its rows, and the codes of a CG-th of its features.
template <int CG>
struct Layout {
    static constexpr int ROWS = kFM * CG;  // token rows of a tile, on the MMA's M
    static constexpr int STAGES = CG == 2 ? 4 : 3;
    static constexpr int A_BYTES = kFM * BK, STAGE_BYTES = A_BYTES + WIDE / CG * BK;
    static constexpr int EPI_REGION = STAGES * STAGE_BYTES;  // staging of the epilogue, two boxes a warp
    static constexpr int SCALE_REGION = EPI_REGION + 2 * EPI_WARPS * BOX_BYTES;
    static constexpr int BAR_REGION = SCALE_REGION + SLOTS * SLOT_BYTES;
    static constexpr int BOARD_REGION = BAR_REGION + 256;  // a tile, see Board
    static constexpr int TABLE_REGION = BOARD_REGION + 64;
    __host__ __device__ static constexpr int smem_bytes(int E) { return 1024 + TABLE_REGION + 8 * (E + 1); }
    static_assert(1024 + TABLE_REGION + 8 * (MXQ_MAX_EXPERTS + 1) <= 232448, "shared memory over the per-block limit");
    static_assert(BAR_REGION % 1024 == 0 && 8 * (2 * STAGES + 4 + 8) + 16 <= 256, "barrier region");
};

struct Tile {
    int e, f0, row, rows, n;
};

// Slices of an expert run fastest, so that the CTAs of one wave share its weight (a tile's number is below 2^31: the
// outputs of more would not fit the device).
template <int kRows>
struct Walk {
    int feats, E;
    int64_t width, total;
    const int32_t *off, *slices;
    __device__ Walk(int64_t width_, int E_, const int32_t* off_, const int32_t* slices_)
        : E(E_), width(width_), off(off_), slices(slices_) {
        feats = (int)((width + WIDE - 1) / WIDE);
        total = (int64_t)slices[E] * feats;
    }
    __device__ Tile get(int64_t t) const {
        Tile T;
        T.e = owner_of(slices, E, (int32_t)((uint32_t)t / (uint32_t)feats));
        const uint32_t count = slices[T.e + 1] - slices[T.e], r = (uint32_t)(t - (int64_t)slices[T.e] * feats);
        const int f = (int)(r / count), i = (int)(r - f * count);
        T.f0 = f * WIDE;
        T.row = off[T.e] + i * kRows;
        T.rows = min(kRows, off[T.e + 1] - T.row);
        T.n = width - T.f0 > WIDE / 2 ? WIDE : WIDE / 2;
        return T;
    }
};

// The next tile of a CTA, as its last control warp finds it: where a tile lies takes several hundred cycles of divisions,
// so it is computed once, ahead, and left here for the other warps. A tile with e < 0 ends the kernel.
struct Board {
    uint32_t at, full, empty;
    uint32_t phase = 0;
    __device__ Board(uint32_t at_, uint32_t full_, uint32_t empty_) : at(at_), full(full_), empty(empty_) {}
    // Leaves T and waits until all have taken it, so that a CTA holds one tile more than it works on. A whole warp; false
    // when a bounded wait has expired.
    __device__ bool put(const Tile& T, int lane, volatile int* abort_flag) {
        if (lane == 0) {
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(T.e), "r"(T.f0), "r"(T.row), "r"(T.rows)
                         : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 16), "r"(T.n) : "memory");
            mbar_arrive(full);
        }
        __syncwarp();
        const bool ok = __all_sync(0xffffffffu, mbar_wait(empty, phase, abort_flag)) != 0;
        phase ^= 1;
        return ok;
    }
    // The next tile, for a whole warp; e < 0 at the end or when a bounded wait has expired.
    __device__ Tile take(int lane, volatile int* abort_flag) {
        Tile T;
        T.e = -1;
        if (!__all_sync(0xffffffffu, mbar_wait(full, phase, abort_flag))) return T;
        phase ^= 1;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(T.e), "=r"(T.f0), "=r"(T.row), "=r"(T.rows)
                     : "r"(at)
                     : "memory");
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(T.n) : "r"(at + 16) : "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(empty);
        return T;
    }
};

// 16-byte piece i (of 8) of a row of 128 bytes under the 128-byte swizzle
__device__ __forceinline__ uint32_t box_piece(uint32_t box, int row, int i) { return box + row * 128 + ((i ^ (row & 7)) << 4); }

template <int kMode, int CG>
__global__ void __launch_bounds__(THREADS, 1)
    ragged_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmOut, Params p) {
    using L = Layout<CG>;
    constexpr int ROWS = L::ROWS, STAGES = L::STAGES, A_BYTES = L::A_BYTES, STAGE_BYTES = L::STAGE_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align<1024>(smem_raw);
    int32_t* s_off = reinterpret_cast<int32_t*>(smem + L::TABLE_REGION);
    int32_t* s_slices = s_off + p.E + 1;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 1 ? 0 : cta_rank();

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_REGION);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, accf0 = empty0 + 8 * STAGES, acce0 = accf0 + 16;
    const uint32_t sfull0 = acce0 + 16, sempty0 = sfull0 + 16, bfull = sempty0 + 16, bempty = bfull + 8, ready = bempty + 8, taken = ready + 8;
    const uint32_t answer = (taken + 8 + 15) & ~15u;
    volatile int* abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int st = 0; st < STAGES; ++st) {
            mbar_init(full0 + 8 * st, 1);
            mbar_init(empty0 + 8 * st, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, CG * EPI_WARPS);
            mbar_init(sfull0 + 8 * b, 1);
            mbar_init(sempty0 + 8 * b, EPI_WARPS);
        }
        mbar_init(bfull, 1);
        mbar_init(bempty, 2 + EPI_WARPS + (rank == 0));  // loads, scales, the epilogue; the MMAs
        mbar_init(ready, 1);
        mbar_init(taken, CG);  // one warp of each CTA asks for tiles
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmA) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmB) : "memory");
    }
    // both CTAs of a pair find the same fault and stop before any cluster-wide step
    const int bad = load_ragged(p.m_splits, p.E, p.M, ROWS, s_off, s_slices);
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
    const int red = (int)(kMode == kFprop ? p.K : p.N);      // terms of a sum
    const int64_t ld = kMode == kFprop ? p.N : p.K;          // features
    const int blocks = (red + BK - 1) / BK;
    Board board(smem_u32(smem) + L::BOARD_REGION, bfull, bempty);

    if (warp < EPI_FIRST) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTL_REGS));
        if (warp == 0) {
            // -------------------------------------------------- TMA producer
            int stage = 0;
            uint32_t phase = 0;
            int64_t fills = 0;
            for (;;) {
                const Tile T = board.take(lane, abort_flag);
                if (T.e < 0) break;
                const int m = T.row + rank * kFM, f = T.f0 + rank * (T.n / CG);
                for (int r = 0; r < red; r += BK) {
                    if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag)) goto done_producer;
                    __syncwarp();
                    const uint32_t own = full0 + 8 * stage, fb = CG == 1 ? own : mapa(own, 0);
                    const uint32_t a = smem_u32(smem) + stage * STAGE_BYTES, b = a + A_BYTES;
                    if (elect_one()) {
                        if (rank == 0) mbar_expect_tx(own, CG * STAGE_BYTES);
                        load_2d<CG>(a, &tmA, fb, r, m);
#pragma unroll
                        for (int g = 0; g < 2 / CG; ++g) {  // 128 features each
                            if (kMode == kFprop) load_3d<CG>(b + g * kFM * BK, &tmB, fb, r, f + g * kFM, T.e);
                            else load_3d<CG>(b + g * kFM * BK, &tmB, fb, f + g * kFM, r, T.e);
                        }
                    }
                    __syncwarp();
                    ++fills;
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
        done_producer:
            // a bounded wait expired: no copy may be in flight when the block ends (both CTAs' loads complete on rank 0's)
            if (*abort_flag && rank == 0) drain_ring(full0, STAGES, fills);
        } else if (warp == 1) {
            // -------------------------------------------------- MMA issuer (rank 0)
            if (rank == 0) {
                int stage = 0, buf = 0;
                uint32_t phase = 0, aphase = 0;
                const uint32_t base = smem_u32(smem);
                // MN-major B: 128-byte chunks of features (one, or two for a single CTA), 8-row groups of the reduction 1024
                // bytes apart
                const uint64_t ad0 = smem_desc(base, 16, 1024);
                const uint64_t bd0 = smem_desc(base + A_BYTES, kMode == kDgrad ? kFM * BK : 16, 1024);
                constexpr uint32_t a_step = 32 / 16, b_step = (kMode == kDgrad ? 4096 : 32) / 16;  // 32 of the sum
                for (;;) {
                    const Tile T = board.take(lane, abort_flag);
                    if (T.e < 0) break;
                    const uint32_t id = idesc_e4m3(0, kMode == kDgrad, ROWS, T.n);
                    for (int r = 0; r < red; r += BK) {
                        const uint64_t ad = ad0 + (uint64_t)(stage * (STAGE_BYTES / 16));
                        const uint64_t bd = bd0 + (uint64_t)(stage * (STAGE_BYTES / 16));
                        if (!mbar_wait(full0 + 8 * stage, phase, abort_flag)) goto done_mma;
                        if (!mbar_wait(acce0 + 8 * buf, aphase ^ 1, abort_flag)) goto done_mma;
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
                }
            done_mma:;
            }
        } else if (warp == 2) {
            // -------------------------------------------------- scales
            const uint32_t at = smem_u32(smem) + L::SCALE_REGION + 4 * lane;
            int group = 0;
            uint32_t phase = 0;
            for (;;) {
                const Tile T = board.take(lane, abort_flag);
                if (T.e < 0) break;
                const int rows = T.rows - 128 * (int)rank;  // of this CTA
                const float* xs = p.xs + T.row + 128 * (int)rank + lane;
                for (int j0 = 0; j0 < blocks; j0 += AHEAD) {
                    float x[AHEAD][4], w[AHEAD][2];
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            w[j][g] = 0.0f;
                            const int f = T.f0 + g * BK;
                            if (j0 + j < blocks && f < ld) w[j][g] = p.ws[weight_scale_at<kMode>(p, T.e, f, j0 + j)];
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x[j][i] = 0.0f;
                            if (j0 + j < blocks && 32 * i + lane < rows) x[j][i] = xs[(j0 + j) * p.M + 32 * i];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j) {
                        if (j0 + j >= blocks) break;
                        const int in_group = (j0 + j) % GROUP;
                        if (in_group == 0 && !__all_sync(0xffffffffu, mbar_wait(sempty0 + 8 * group, phase ^ 1, abort_flag)))
                            goto done_scales;
#pragma unroll
                        for (int g = 0; g < 2; ++g)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + (group * GROUP + in_group) * SLOT_BYTES +
                                                                             512 * g + 128 * i),
                                             "f"(x[j][i] * w[j][g])
                                             : "memory");
                        if (in_group == GROUP - 1 || j0 + j == blocks - 1) {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(sfull0 + 8 * group);
                            group ^= 1;
                            phase ^= group == 0;
                        }
                    }
                }
            }
        done_scales:;
        } else {
            // -------------------------------------------------- tiles
            const Walk<ROWS> W(ld, p.E, s_off, s_slices);
            TileQueue queue(answer, ready, mapa(taken, 0), CG);
            int64_t t = blockIdx.x / CG;
            for (uint32_t asked = 0;; asked ^= 1) {
                if (t < W.total && !board.put(W.get(t), lane, abort_flag)) break;
                if (rank == 0 && !mbar_wait(taken, asked ^ 1, abort_flag)) break;
                __syncwarp();
                if (elect_one()) {
                    mbar_expect_tx(ready, 16);
                    if (rank == 0) queue.ask();
                }
                __syncwarp();
                if (queue.next(t, lane, abort_flag) != TileQueue::kTile) {
                    board.put(Tile{-1, 0, 0, 0, 0}, lane, abort_flag);
                    break;
                }
            }
        }
    } else {
        // ------------------------------------------------------ epilogue: lane = token row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
        // two groups of four warps: a group has one of the tile's two blocks of features
        const int q = warp & 3, group = (warp - EPI_FIRST) >> 2;
        const uint32_t stage = smem_u32(smem) + L::EPI_REGION + (warp - EPI_FIRST) * 2 * BOX_BYTES;
        constexpr int kParts = WIDE / 32;  // 16 columns each
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + group * (WIDE / 2);
        const uint32_t acce = mapa(acce0, 0);  // this CTA's own too, for rank 0
        const uint32_t scales = smem_u32(smem) + L::SCALE_REGION + 512 * group + 4 * (32 * q + lane);
        int buf = 0, group_at = 0;
        uint32_t aphase = 0, sphase = 0;
        for (;;) {
            const Tile T = board.take(lane, abort_flag);
            if (T.e < 0) break;
            uint64_t acc[kParts][8];  // sums of two columns each
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i][j] = 0;
            // One block at a time: four in a row, unrolled, no longer fit the instruction cache (750 cycles each).
#pragma unroll 1
            for (int j = 0; j < blocks; ++j) {
                // after an expired wait the others return at once; the tile is then not stored
                const int in_group = j % GROUP;
                const bool group_ends = in_group == GROUP - 1 || j == blocks - 1;
                if (in_group == 0) mbar_wait(sfull0 + 8 * group_at, sphase, abort_flag);
                float factor;
                asm volatile("ld.shared.f32 %0, [%1];"
                             : "=f"(factor)
                             : "r"(scales + (group_at * GROUP + in_group) * SLOT_BYTES)
                             : "memory");
                mbar_wait(accf0 + 8 * buf, aphase, abort_flag);
                __syncwarp();
                fence_after();
                const uint64_t k = f2splat(factor);
                // Four parts out of TMEM at a time: the accumulator is free when the last has been read, before the last four
                // are added (two at a time, one on its way while the other is added: 113 us against 110.5).
                uint32_t v[4][16];
                const auto load = [&](int i) { tmem_ld16(lanes + buf * WIDE + 16 * i, v[i & 3]); };
                const auto add = [&](int i) {
#pragma unroll
                    for (int l = 0; l < 8; ++l)
                        acc[i][l] = f2fma(f2pack(__uint_as_float(v[i & 3][2 * l]), __uint_as_float(v[i & 3][2 * l + 1])), k,
                                          acc[i][l]);
                };
                static_assert(kParts == 8, "eight parts");
                load(0), load(1), load(2), load(3);
                tmem_wait_ld();
                add(0), load(4), add(1), load(5);
                tmem_wait_ld();
                add(2), load(6), add(3), load(7);
                tmem_wait_ld();
                fence_before();
                __syncwarp();
                arrive_relaxed_if(lane == 0, acce + 8 * buf);
                add(4), add(5), add(6), add(7);
                if (group_ends) {
                    if (lane == 0) mbar_arrive(sempty0 + 8 * group_at);  // behind the arrive above: all lanes have read
                    group_at ^= 1;
                    sphase ^= group_at == 0;
                }
                buf ^= 1;
                aphase ^= buf == 0;
            }
            if (__any_sync(0xffffffffu, *abort_flag)) break;
            const int f0 = T.f0 + group * BK, row = T.row + 128 * (int)rank + 32 * q;
            const int live = (int)min((int64_t)BK, ld - f0);  // features; may be negative: nothing to store
            const int rows = min(32, T.rows - 128 * (int)rank - 32 * q);
            if (live <= 0 || rows <= 0) continue;
            if (kMode == kFprop && p.bias) {
                const __nv_bfloat16* bias = p.bias + (int64_t)T.e * p.N + f0;
#pragma unroll
                for (int i = 0; i < kParts; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (16 * i + 8 * h >= live) continue;
                        const uint4 b = *reinterpret_cast<const uint4*>(bias + 16 * i + 8 * h);
                        const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int l = 0; l < 4; ++l)
                            acc[i][4 * h + l] = f2add(acc[i][4 * h + l], f2pack(bf16lo(u[l]), bf16hi(u[l])));
                    }
            }
            // Rows of 128 bytes through shared memory, 64 bf16 or 32 fp32, two boxes at a time: by TMA where all 32 rows are
            // the slice's, which nothing waits for.
            const auto store_boxes = [&](int column, int width, auto put) {
                if (lane < 2) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
                put(0, stage);
                put(1, stage + BOX_BYTES);
                if (rows == 32) {
                    fence_async_smem();
                    __syncwarp();
                    if (lane < 2 && column + lane * width < live)
                        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                                         (uint64_t)&tmOut),
                                     "r"(f0 + column + lane * width), "r"(row), "r"(stage + lane * BOX_BYTES)
                                     : "memory");
                    if (lane < 2) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                } else {
                    __syncwarp();
                    const int size = p.out_f32 ? 4 : 2, piece = lane & 7;
                    for (int i = 0; i < 2; ++i) {
                        const int at = (column + i * width) * size + piece * 16;  // bytes of the row
                        uint8_t* o = static_cast<uint8_t*>(p.out) + ((int64_t)row * ld + f0) * size + at;
                        if (at < live * size)
                            for (int m = lane >> 3; m < rows; m += 4)
                                *reinterpret_cast<uint4*>(o + m * ld * size) =
                                    ld_shared(box_piece(stage + i * BOX_BYTES, m, piece));
                    }
                    __syncwarp();
                }
            };
            if (p.out_f32) {
#pragma unroll
                for (int i = 0; i < kParts; i += 4)
                    store_boxes(16 * i, 32, [&](int half, uint32_t box) {
#pragma unroll
                        for (int h = 0; h < 8; ++h) {
                            const int part = i + 2 * half + (h >> 2);
                            const float2 a = f2unpack(acc[part][2 * (h & 3)]), b = f2unpack(acc[part][2 * (h & 3) + 1]);
                            st_shared(box_piece(box, lane, h), make_uint4(__float_as_uint(a.x), __float_as_uint(a.y),
                                                                          __float_as_uint(b.x), __float_as_uint(b.y)));
                        }
                    });
            } else {
                store_boxes(0, 64, [&](int half, uint32_t box) {
#pragma unroll
                    for (int h = 0; h < 8; ++h) {
                        uint32_t u[4];
#pragma unroll
                        for (int l = 0; l < 4; ++l) {
                            const float2 a = f2unpack(acc[4 * half + (h >> 1)][4 * (h & 1) + l]);
                            u[l] = bf16x2_bits(a.x, a.y);
                        }
                        st_shared(box_piece(box, lane, h), make_uint4(u[0], u[1], u[2], u[3]));
                    }
                });
            }
        }
        // the last boxes are written before the block leaves its shared memory
        if (lane < 2) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
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

}  // namespace wide

// ------------------------------------------------------------ few rows
// One-SM tiles of 128 features by up to 32 rows: what is left is reading W once. As in the bf16 kernel for few rows
// (mxq_ragged_few.cu), a stage is 16 KB of W and at most 4 KB of tokens, eight are in flight, and where the tiles do not
// fill the SMs the sum is split over a cluster. An accumulator is 32 columns, so there are four.
namespace few {

constexpr int STAGES = 8, SLOTS = Scales::kSlots, BUFS = 4;
constexpr int WIDE = kFewRows, STEP = 16;
constexpr int A_BYTES = kFM * BK, STAGE_BYTES = A_BYTES + WIDE * BK;
constexpr int EPI_FIRST = 4, EPI_WARPS = 4;  // warp 3 is idle
constexpr int THREADS = 32 * (EPI_FIRST + EPI_WARPS);
constexpr int TMEM_COLS = BUFS * WIDE;
constexpr int PART_REGION = STAGES * STAGE_BYTES;
constexpr int SCALE_REGION = PART_REGION + kPartBytes;
constexpr int BAR_REGION = SCALE_REGION + Scales::kBytes;
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
    // this CTA's part of the reduction in blocks, the same for every tile
    const int red = (int)(kMode == kDgrad ? p.N : p.K), blocks = (red + BK - 1) / BK;
    const int jb = blocks * rank / kSplit, je = blocks * (rank + 1) / kSplit;
    const int64_t first = blockIdx.x / kSplit, stride = gridDim.x / kSplit;
    let_next_begin();  // 8 experts x 2 rows, call after call: 17.4 -> 16.5 us
    // While the counts are on their way, the first blocks of the weight that this CTA needs if every expert has rows, as
    // it mostly is where there are as many rows as experts (8 experts x 2 rows behind the quantizer, 2048 x 4096, cold:
    // 19.7 -> 19.2 us; 64 experts of 2048 x 1024 27.2 -> 26.2 us).
    if (kSplit == 1 && warp == 1 && p.M >= p.E) {
        const int feats = (int)(((kMode == kFprop ? p.N : p.K) + kFM - 1) / kFM);
        const int64_t e = first / feats;
        const int f = (int)(first - e * feats) * kFM, j = jb + lane;
        if (e < p.E && lane < STAGES && j < je) {
            if (kMode == kFprop) prefetch_3d(&tmA, j * BK, f, (int)e);
            else prefetch_3d(&tmA, f, j * BK, (int)e);
        }
        __syncwarp();
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
    Scales ring(smem_u32(smem) + SCALE_REGION, sfull0, sempty0);

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
            const uint32_t id = idesc_e4m3(kMode == kDgrad, 0, kFM, T.n);
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
            if (!ring.produce<kMode>(p, T, T.f0, jb, je, lane, abort_flag)) break;
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
            Sums acc[2];
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
                add_scaled(acc[0], v[0], lo, hi);
                add_scaled(acc[1], v[1], lo, hi);
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
// which leave through shared memory as runs of 8 kRows rows. Six blocks to an SM (131072 x 7168: 444 us, floor 423; five,
// what the compiler takes by itself, 457; eight 456).
template <int kRows>
__global__ void __launch_bounds__(256, 6) fp8_quantize_rows_kernel(const uint16_t* x, int64_t M, int64_t K, int64_t ld,
                                                                uint8_t* q, float* scale) {
    __shared__ float s_scale[2][8 * kRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t across = (K + 255) / 256, tiles = across * ((M + 8 * kRows - 1) / (8 * kRows));
    let_next_begin();  // the product's blocks (the same case without: 20.2 us)
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

// Weights: a block of 256 threads holds one 128 x 128 block in registers, 16 bytes of eight rows a thread. Bound by HBM
// (128 x 2048 x 7168: 843 us, 6.68 TB/s, two bytes read for one written: a plain copy, one for one, reaches 6.67) when the compiler has the registers of three blocks to an SM and issues a thread's
// eight loads together; with those of four, what it takes by itself, 1009 us, of six 1095.
__global__ void __launch_bounds__(256, 3) fp8_quantize_weight_kernel(const uint16_t* w, int64_t N, int64_t K, int64_t across,
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

template <int kMode, int CG>
static cudaError_t run_wide(const Fp8Call& c, cudaStream_t s) {
    using namespace wide;
    using L = Layout<CG>;
    const int64_t red = kMode == kDgrad ? c.N : c.K, width = kMode == kFprop ? c.N : c.K, size = c.out_f32 ? 4 : 2;
    const int64_t da[2] = {red, c.M}, sa[1] = {red}, db[3] = {c.K, c.N, c.E}, sb[2] = {c.K, c.K * c.N};
    const int64_t dd[2] = {width, c.M}, sd[1] = {size * width};
    const int boxa[2] = {BK, kFM}, boxb[3] = {BK, kFM, 1}, boxd[2] = {128 / (int)size, 32};
    CUtensorMap a, b, out;
    if (!encode_tmap(&a, c.tq, 1, 2, da, sa, boxa) || !encode_tmap(&b, c.wq, 1, 3, db, sb, boxb) ||
        !encode_tmap(&out, c.out, (int)size, 2, dd, sd, boxd))
        return cudaErrorInvalidValue;
    // no fewer than the device counts
    const int64_t tiles = (c.M / L::ROWS + std::min<int64_t>(c.E, c.M)) * ((width + WIDE - 1) / WIDE);
    return launch_persistent<CG, true, ragged_fp8_kernel<kMode, CG>>(THREADS, L::smem_bytes(MXQ_MAX_EXPERTS),
                                                                     L::smem_bytes(c.E), tiles, s, a, b, out, params(c));
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
    // By the rows of an expert on average: the counts are on the device. W of 2048 x 4096, us, fprop and dgrad.
    // Up to 16, or as many as one tile of the kernel for few rows holds, that kernel; against tiles of 128 rows: one expert
    // of 32 rows 8.2 and 7.8 against 11.5 and 15.8; 8 experts of 16 13.5 and 12.6 against 12.9 and 16.7, of 32 18.8 and 22.7
    // against 13.4 and 17.0 (Dirichlet(100) shares); 64 experts of 16 85 and 84 against 86 and 89, of 24 in Dirichlet(0.3)
    // shares 100 and 94 against 74 and 73.
    // Up to 128 tiles of one SM, against pairs: 8 experts of 48 rows 13.3 and 16.8 against 20.5 and 18.0, of 128 in flat
    // Dirichlet shares 21 and 18.5 against 27 and 29; 64 experts of 48 88.8 and 91 against 114 and 107, of 128 even rows 96
    // and 98 against 119 and 113. Beyond, the counts decide: 64 experts of 208 rows 132 and 128 against 123 and 117 even,
    // 136 and 137 against 158 and 144 in flat Dirichlet shares; 48 experts of 208 (1424 x 2064) 60 against 56; 8 of 2048 even
    // 116 and 107 against 111 and 98.
    const bool fprop = c.mode == kFprop;
    if (c.M <= std::max<int64_t>((int64_t)16 * c.E, f8::few::WIDE))
        return fprop ? f8::run_few<kFprop>(c, s) : f8::run_few<kDgrad>(c, s);
    if (c.M <= (int64_t)128 * c.E) return fprop ? f8::run_wide<kFprop, 1>(c, s) : f8::run_wide<kDgrad, 1>(c, s);
    return fprop ? f8::run_wide<kFprop, 2>(c, s) : f8::run_wide<kDgrad, 2>(c, s);
}

cudaError_t run_fp8_quantize_rows(const void* x, int64_t M, int64_t K, int64_t ld, void* q, float* scale, cudaStream_t s) {
    if (M == 0) return cudaSuccess;
    const int64_t tiles = (K + 255) / 256 * ((M + 31) / 32);
    // many short blocks: one that starts loads while others store (131072 x 7168: 502 us with as many as run at once, 460 with these)
    return launch(f8::fp8_quantize_rows_kernel<4>, (unsigned)std::min<int64_t>(tiles, (int64_t)sm_count() * 64), 256, s, 0,
                  static_cast<const uint16_t*>(x), M, K, ld, static_cast<uint8_t*>(q), scale);
}

cudaError_t run_fp8_quantize_weight(const void* w, int64_t N, int64_t K, int E, void* q, float* scale, cudaStream_t s) {
    const int64_t across = (K + f8::BK - 1) / f8::BK, down = (N + f8::BK - 1) / f8::BK;
    return launch(f8::fp8_quantize_weight_kernel, (unsigned)(across * down * E), 256, s, 0,
                  static_cast<const uint16_t*>(w), N, K, across, down, static_cast<uint8_t*>(q), scale);
}

}  // namespace ragged
}  // namespace mxq
