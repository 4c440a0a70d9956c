// mxq_ragged.cu -- bf16 grouped products of an MoE expert layer on GB300
// (sm_103a) for expert counts that are multiples of nothing:
//   fprop  Y[m,:]  = X[m,:]  . W[e(m)]^T (+ b[e(m)])
//   dgrad  dX[m,:] = dY[m,:] . W[e(m)]
//   wgrad  dW[e]   = dY_e^T . X_e
// fp32 sums, one rounding to bf16 (or none, fp32 outputs).
//
// Which operand is which. The output's contiguous dimension is put on the
// MMA's M (TMEM lanes), its rows on the MMA's N (accumulator columns): W and
// the tokens in fprop and dgrad, X and dY in wgrad. N is a field of the
// instruction descriptor that may differ from tile to tile, so a slice of an
// expert's rows costs MMA work in steps of 32 rows, not 128.
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
// fp32 results. The tensor core truncates as it adds to its fp32 accumulator:
// over 2048 rows a wgrad entry came out 2.1e-6 off (relative 2-norm; an fp32
// matrix product 3.9e-7). Outputs that are not rounded to bf16 are therefore
// summed in registers, one accumulator of FLUSH stages at a time (kRegs).
//
// Long sums to bf16. A step of 16 terms may lose up to 2^-23 of the sum, in the
// same direction for terms of one sign: 2^-12, a sixteenth of bf16's rounding,
// in one accumulator of kTruncDepth = 2^15 terms, and some 2^-8 in one of 2^20.
// So a tile with more terms (an expert's rows in wgrad; K or N otherwise) is
// summed in pieces of LONG_FLUSH stages in one accumulator, which the epilogue's
// warps add up in the other one, where the tile's epilogue then finds the sum.
// The MMAs wait while a piece is added, which at 128 stages a piece is not
// noticed (2 experts, 131072 rows, 2048 x 2048: 649 us in one accumulator, 648
// to 666 so). Sums in registers beside the shorter tiles' code did not fit: the
// spills took adding to bf16 dW from 67 to 186 us.
//
// A pair of SMs (a cluster of two CTAs, cta_group::2) shares a tile of 256
// features by up to 256 rows, each staging half of both operands: 32 KB a stage
// and SM for the MMA work that costs one SM alone 48 KB. Experts with few rows
// go to mxq_ragged_few.cu.
//
// Tiles are dealt by the hardware: the grid is a cluster per tile, and a
// cluster that has started takes further ones from the queue of those not yet
// launched (TileQueue). wgrad's experts come heaviest first. Against a static
// deal: 128 experts, 128k rows 2815 -> 2625 us; 48 uneven experts (dgrad) 84.6
// -> 79.3 us; even experts the same.
//
// Warp-specialised: warp 0 issues TMA loads into a ring of 64-deep stages, warp
// 1 owns TMEM and issues the MMAs (rank 0 of a pair), warps 2..9 drain one of
// two accumulators while the MMAs fill the other, warp 10 zeroes its CTA's
// share of an expert's last rows (wgrad), warp 11 asks for the next tile. The
// loading and issuing warps stay converged and elect a lane for each stage's
// instructions, whose operands the compiler then keeps in uniform registers:
// from one lane alone, issuing took longer (681 cycles a stage) than the MMAs
// (512), and so did the loads.
//
// What bounds it: 8 experts x 2048 rows, 2048 x 4096: 152 us, 1808 TFLOP/s,
// 565 cycles a stage; there the operand feed (32 KB an SM and stage, 58 bytes
// a cycle) and the tensor pipe's clock under the power limit (1.65 to 1.75 GHz)
// meet. Uneven counts pay for slices that are not whole (16k rows: 178 us).
//
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

constexpr int BK = 64;    // reduction depth of a stage: 128 bytes of bf16
constexpr int FLUSH = 8;  // stages an accumulator holds before it is added to the registers (kRegs)
constexpr int LONG_FLUSH = 128;  // and before it is added to the other accumulator (more than kTruncDepth terms)
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 128 + 32 * EPI_WARPS;

constexpr int CG = 2;                         // CTAs, and SMs, of a tile
constexpr int FEAT = kFM * CG;                // features of a tile
constexpr int WIDE = 256, STEP = 16 * CG;     // widest MMA N and its granularity
constexpr int BOX = 64;                       // token rows of a K-major box
constexpr int STAGES = 6;
constexpr int A_BYTES = kFM * BK * 2, STAGE_BYTES = A_BYTES + WIDE / CG * BK * 2;
constexpr int TMEM_COLS = 2 * WIDE;
constexpr int EPI_REGION = STAGES * STAGE_BYTES;  // staging of the bf16 epilogue, a buffer a warp
constexpr int BAR_REGION = EPI_REGION + EPI_WARPS * kEpiBytes;
constexpr int TABLE_REGION = BAR_REGION + 256;
__host__ __device__ constexpr int smem_bytes(int E) { return 1024 + TABLE_REGION + 12 * (E + 1); }
static_assert(smem_bytes(MXQ_MAX_EXPERTS) <= 232448, "shared memory over the per-block limit");
static_assert(BAR_REGION % 8 == 0 && 8 * (4 * STAGES + 6) + 16 <= 256, "barrier region");

struct Params {
    int64_t M, N, K;
    int E;
    const int64_t* m_splits;
    const __nv_bfloat16* bias;
    void* out;
    int out_f32, accumulate;
    int32_t* status;
};

template <int kMode, bool kRegs>
__global__ void __launch_bounds__(THREADS, 1)
    ragged_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmHalf, const __grid_constant__ CUtensorMap tmOut,
                       Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align<1024>(smem_raw);
    int32_t* s_off = reinterpret_cast<int32_t*>(smem + TABLE_REGION);
    int32_t* s_slices = s_off + p.E + 1;
    int32_t* s_order = s_slices + p.E + 1;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_REGION);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES, tail0 = empty0 + 8 * STAGES;
    const uint32_t fix0 = tail0 + 8 * STAGES, accf0 = fix0 + 8 * STAGES, acce0 = accf0 + 16;
    const uint32_t ready = acce0 + 16, taken = ready + 8, answer = (taken + 8 + 15) & ~15u;
    volatile int* abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int st = 0; st < STAGES; ++st) {
            mbar_init(full0 + 8 * st, 1);
            mbar_init(empty0 + 8 * st, 1);
            mbar_init(tail0 + 8 * st, 1);
            mbar_init(fix0 + 8 * st, CG);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, CG * EPI_WARPS);
        }
        mbar_init(ready, 1);
        mbar_init(taken, 5 + 2 * EPI_WARPS + (kMode == kWgrad ? 2 : 0));  // the warps of both CTAs that call next()
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
    if (kMode == kWgrad) {
        for (int e = threadIdx.x; e < p.E; e += THREADS) {
            const int m = s_off[e + 1] - s_off[e];
            int before = 0;
            for (int f = 0; f < p.E; ++f) {
                const int o = s_off[f + 1] - s_off[f];
                before += o > m || (o == m && f < e);
            }
            s_order[before] = e;
        }
    }
    if (warp == 1) tmem_alloc<CG>(smem_u32(&s_tmem), TMEM_COLS);
    fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any load completes on rank 0's
    fence_after();
    const uint32_t tmem = s_tmem;
    const Walk<kMode, FEAT, WIDE, STEP> W(p.N, p.K, p.E, s_off, s_slices, s_order);
    TileQueue queue(answer, ready, mapa(taken, 0));
    int64_t t = blockIdx.x / CG;
    constexpr bool a_mn = kMode != kFprop, b_mn = kMode == kWgrad;
    // An expert's last block of rows in wgrad, when it ends inside a step of 16: its loads complete on each
    // CTA's own tail[st], warp 10 of both CTAs zeroes the rows up to the next multiple of 16 and arrives on
    // rank 0's fix[st], and the MMAs wait for that instead of full[st]. The parities of full, tail and fix
    // of a stage therefore follow their own uses, not the ring's laps.
    auto ragged_end = [](const Tile& T, int r) { return kMode == kWgrad && T.red - r < BK && ((T.red - r) & 15) != 0; };
    auto long_sum = [](const Tile& T) { return !kRegs && T.red > kTruncDepth; };
    auto piece = [&](const Tile& T) { return kRegs ? FLUSH * BK : long_sum(T) ? LONG_FLUSH * BK : T.red; };
    auto zero_rows = [&](const Tile& T, int r, int stage) {
        // a 16-byte chunk a lane, four rows at a time, box by box
        const int left = (T.red - r) & 15, boxes = 2 + (T.n / CG + 63) / 64;
        uint8_t* s = smem + stage * STAGE_BYTES + (T.red - r + (lane >> 3)) * 128 + (lane & 7) * 16;
        for (int i = 0; i < boxes; ++i)
            for (int row = left + (lane >> 3), at = i * 8192; row < 16; row += 4, at += 512)
                *reinterpret_cast<uint4*>(s + at) = make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
        __syncwarp();
    };

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        int stage = 0;
        uint32_t phase = 0;
        uint32_t used = 0, full_uses = 0, tail_uses = 0, tail_last = 0;  // bits of stages
        do {
            if (t >= W.total) continue;
            const Tile T = W.get(t);
            const int half = T.n / CG;  // this CTA's columns of the tile: [rank * half, + half)
            // rows of the other operand: whole boxes, and half a box at the end where that is enough
            const bool half_box = kMode != kWgrad && (half - 1) % BOX < BOX / 2;
            const int boxes = half_box ? half / BOX : (half + BOX - 1) / BOX;
            const int f = T.f0 + rank * kFM, c = T.c0 + rank * half;
            const uint32_t bytes = A_BYTES + (2 * boxes + half_box) * (BOX * BK);
            for (int r = 0; r < T.red; r += BK) {
                if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, abort_flag)) {
                    // a bounded wait expired: no copy may be in flight when the block ends
                    volatile int unused = 0;
                    for (int st = 0; st < STAGES; ++st) {
                        const bool tail = tail_last >> st & 1;
                        if ((used >> st & 1) && (tail || rank == 0))  // rank 1's full loads complete on rank 0's
                            mbar_wait((tail ? tail0 : full0) + 8 * st, ((tail ? tail_uses : full_uses) >> st & 1) ^ 1,
                                      &unused);
                    }
                    goto done_producer;
                }
                __syncwarp();
                const bool tail = ragged_end(T, r);
                const uint32_t own = (tail ? tail0 : full0) + 8 * stage, bit = 1u << stage;
                const uint32_t fb = mapa(own, tail ? rank : 0);
                const uint32_t a = smem_u32(smem) + stage * STAGE_BYTES, b = a + A_BYTES;
                if (elect_one()) {
                    if (tail) mbar_expect_tx(own, bytes);
                    else if (rank == 0) mbar_expect_tx(own, CG * bytes);
                    if (kMode == kFprop) {
                        load_3d<CG>(a, &tmA, fb, r, f, T.e);
                    } else if (kMode == kDgrad) {
                        load_3d<CG>(a, &tmA, fb, f, r, T.e);
                        load_3d<CG>(a + 8192, &tmA, fb, f + 64, r, T.e);
                    } else {
                        load_2d<CG>(a, &tmA, fb, f, T.red0 + r);
                        load_2d<CG>(a + 8192, &tmA, fb, f + 64, T.red0 + r);
                    }
#pragma unroll
                    for (int i = 0; i < WIDE / CG / BOX; ++i) {
                        const uint32_t dst = b + BOX * BK * 2 * i;
                        if (i < boxes) {
                            if (kMode == kWgrad) load_2d<CG>(dst, &tmB, fb, c + BOX * i, T.red0 + r);
                            else load_2d<CG>(dst, &tmB, fb, r, c + BOX * i);
                        }
                    }
                    if (half_box) load_2d<CG>(b + BOX * BK * 2 * boxes, &tmHalf, fb, r, c + BOX * boxes);
                }
                __syncwarp();
                used |= bit;
                if (tail) {
                    tail_uses ^= bit;
                    tail_last |= bit;
                } else {
                    full_uses ^= bit;
                    tail_last &= ~bit;
                }
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
        } while (queue.next(t, lane, abort_flag) == TileQueue::kTile);
    done_producer:;
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer (rank 0)
        if (rank == 0) {
            int stage = 0, buf = 0;
            uint32_t acc_uses = 0, full_uses = 0, fix_uses = 0;  // bits of accumulators and stages: parities
            const uint32_t base = smem_u32(smem);
            // MN-major: 64-element chunks 8192 bytes apart, 8-row groups of the reduction 1024 apart
            const uint64_t ad0 = smem_desc(base, a_mn ? 8192 : 16, 1024);
            const uint64_t bd0 = smem_desc(base + A_BYTES, b_mn ? 8192 : 16, 1024);
            constexpr uint32_t a_step = (a_mn ? 2048 : 32) / 16, b_step = (b_mn ? 2048 : 32) / 16;  // 16 of the sum
            do {
                if (t >= W.total) continue;
                const Tile T = W.get(t);
                const uint32_t id = idesc_f16(1, a_mn, b_mn, FEAT, T.n);
                for (int r0 = 0, r1; r0 < T.red; r0 = r1) {
                    r1 = min(T.red, r0 + piece(T));
                    const uint32_t d = tmem + buf * WIDE;
                    if (!mbar_wait(acce0 + 8 * buf, (acc_uses >> buf & 1) ^ 1, abort_flag)) goto done_mma;
                    __syncwarp();
                    acc_uses ^= 1u << buf;
                    for (int r = r0; r < r1; r += BK) {
                        const uint64_t ad = ad0 + (uint64_t)(stage * (STAGE_BYTES / 16));
                        const uint64_t bd = bd0 + (uint64_t)(stage * (STAGE_BYTES / 16));
                        if (ragged_end(T, r)) {
                            if (!mbar_wait(fix0 + 8 * stage, fix_uses >> stage & 1, abort_flag)) goto done_mma;
                            fix_uses ^= 1u << stage;
                        } else {
                            if (!mbar_wait(full0 + 8 * stage, full_uses >> stage & 1, abort_flag)) goto done_mma;
                            full_uses ^= 1u << stage;
                        }
                        __syncwarp();
                        fence_after();
                        const int steps = T.red - r >= BK ? BK / 16 : (T.red - r + 15) / 16;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < BK / 16; ++k)
                                if (k < steps) mma_f16<CG>(d, ad + k * a_step, bd + k * b_step, id, r > r0 || k > 0);
                            mma_commit<CG>(empty0 + 8 * stage);
                            if (r + BK >= r1) mma_commit<CG>(accf0 + 8 * buf);
                        }
                        __syncwarp();
                        if (++stage == STAGES) stage = 0;
                    }
                    if (!long_sum(T)) buf ^= 1;
                }
                if (long_sum(T)) acc_uses ^= 2u >> buf;  // the epilogue's use of the other accumulator
            } while (queue.next(t, lane, abort_flag) == TileQueue::kTile);
        done_mma:;
        }
    } else if (warp == 2 + EPI_WARPS) {
        // ------------------------------------------------------ rows of the next expert (wgrad)
        if (kMode == kWgrad) {
            int stage = 0;
            uint32_t uses = 0;  // bits of stages: parity of tail[st]
            do {
                if (t >= W.total) continue;
                const Tile T = W.get(t);
                if (T.red == 0) continue;
                const int last = (T.red - 1) / BK, at = (stage + last) % STAGES;
                if (ragged_end(T, last * BK)) {
                    if (!__all_sync(0xffffffffu, mbar_wait(tail0 + 8 * at, uses >> at & 1, abort_flag))) break;
                    uses ^= 1u << at;
                    zero_rows(T, last * BK, at);
                    if (lane == 0) {
                        if (rank == 0) mbar_arrive(fix0 + 8 * at);
                        else arrive_remote(mapa(fix0 + 8 * at, 0));
                    }
                }
                stage = (at + 1) % STAGES;
            } while (queue.next(t, lane, abort_flag) == TileQueue::kTile);
        }
    } else if (warp == 3 + EPI_WARPS) {
        // ------------------------------------------------------ next tiles
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
    } else {
        // ------------------------------------------------------ epilogue
        const int q = warp & 3, group = (warp - 2) >> 2;  // two groups of four warps share the columns
        uint8_t* stage = smem + EPI_REGION + (warp - 2) * (kMode == kWgrad ? kBoxBytes : kEpiBytes);
        const int64_t ld = kMode == kFprop ? p.N : p.K;  // features
        int buf = 0;
        uint32_t acc_uses = 0;  // bits of accumulators: parities
        auto filled = [&] {
            const bool ok = mbar_wait(accf0 + 8 * buf, acc_uses >> buf & 1, abort_flag);
            acc_uses ^= 1u << buf;
            return __all_sync(0xffffffffu, ok && !*abort_flag) != 0;
        };
        auto drained = [&](int b) {
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) mbar_arrive(acce0 + 8 * b);
                else arrive_remote_relaxed(mapa(acce0 + 8 * b, 0));
            }
        };
        do {
            if (t >= W.total) continue;
            const Tile T = W.get(t);
            const int f0 = T.f0 + rank * kFM;
            const int live = (int)min((int64_t)kFM, ld - f0);  // may be negative: nothing to store
            if (kMode == kWgrad && T.red == 0) {
                // an empty expert: 16-byte stores of zero, a row piece of 128 features at a time
                if (!p.accumulate) {
                    const int size = p.out_f32 ? 4 : 2, per = live * size / 16;
                    for (int c = q + 4 * group; c < T.cols; c += 8)
                        for (int i = lane; i < per; i += 32)
                            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + ((T.row0 + c) * ld + f0) * size +
                                                      16 * i) = make_uint4(0u, 0u, 0u, 0u);
                }
                continue;
            }
            if constexpr (kRegs) {
                constexpr int kChunks = WIDE / 64;  // 32-column chunks of a group
                float acc[kChunks][32];
                bool ok = true;
                for (int r0 = 0; r0 < T.red && ok; r0 += FLUSH * BK) {
                    ok = filled();
                    if (!ok) break;
                    fence_after();
#pragma unroll
                    for (int i = 0; i < kChunks; ++i) {
                        const int c = 64 * i + 32 * group;
                        if (c < T.cols) {
#pragma unroll
                            for (int h = 0; h < 32; h += 16) {
                                uint32_t v[16];
                                tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + buf * WIDE + c + h, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    acc[i][h + j] = r0 == 0 ? __uint_as_float(v[j])
                                                            : __fadd_rn(acc[i][h + j], __uint_as_float(v[j]));
                            }
                        }
                    }
                    drained(buf);
                    buf ^= 1;
                }
                if (!ok) break;
                const int l = q * 32 + lane;
                // dW as boxes by TMA where it is added to, where stores would need a test for each column, and after
                // short sums, whose epilogue nothing hides (8 experts, 4096 x 2048, us by boxes and by the warps: 512
                // rows each 74.2 and 79.8, 16 rows 55.9 and 58.0; 128 experts 1000 x 1000 104 and 114; 2048 rows each
                // 200 and 196)
                if (kMode == kWgrad && (p.accumulate || T.red <= FLUSH * BK || T.cols != WIDE)) {
#pragma unroll
                    for (int i = 0; i < kChunks; ++i)
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            const int c = 64 * i + 32 * group + h;
                            if (c < T.cols)
                                store_box_f32(&acc[i][h], lane, stage, &tmOut, f0 + 32 * q, T.c0 + c, T.e, live > 32 * q,
                                              p.accumulate);
                        }
                } else if (l < live) {
                    const float b =
                        kMode == kFprop && p.bias ? __bfloat162float(p.bias[(int64_t)T.e * p.N + f0 + l]) : 0.0f;
                    auto each = [&](auto&& put) {
#pragma unroll
                        for (int i = 0; i < kChunks; ++i)
#pragma unroll
                            for (int j = 0; j < 32; ++j) put(64 * i + 32 * group + j, __fadd_rn(acc[i][j], b));
                    };
                    const int64_t at = T.row0 * ld + f0 + l;
                    float* o = static_cast<float*>(p.out) + at;
                    if (T.cols == WIDE) {  // whole tiles: nothing but stores, 128 bytes a warp
                        each([&](int c, float v) { o[c * ld] = v; });
                    } else {
                        each([&](int c, float v) {
                            if (c < T.cols) o[c * ld] = v;
                        });
                    }
                }
            } else {
                // dW's old values are read while the sums are made
                constexpr int kBoxes = kMode == kWgrad ? WIDE / 64 : 1;
                uint4 old[kBoxes][4];
                if (kMode == kWgrad && p.accumulate) {
#pragma unroll
                    for (int i = 0; i < kBoxes; ++i) {
                        const int c = 64 * i + 32 * group;
                        load_rows_bf16(static_cast<const __nv_bfloat16*>(p.out) + (T.row0 + c) * ld + f0 + 32 * q, ld,
                                       live - 32 * q, T.cols - c, lane, old[i]);
                    }
                }
                const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
                int from = buf;  // the accumulator that holds the sums
                bool ok = true;
                if (long_sum(T)) {
                    from ^= 1;
                    for (int r0 = 0; r0 < T.red; r0 += piece(T)) {
                        ok = filled();
                        if (!ok) break;
                        fence_after();
                        for (int c = 32 * group; c < T.cols; c += 64)
#pragma unroll
                            for (int h = 0; h < 32; h += 16) {
                                uint32_t v[16], s[16];
                                tmem_ld16(lanes + buf * WIDE + c + h, v);
                                tmem_ld16(lanes + from * WIDE + c + h, s);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    if (r0 > 0)
                                        v[j] = __float_as_uint(__fadd_rn(__uint_as_float(s[j]), __uint_as_float(v[j])));
                                tmem_st16(lanes + from * WIDE + c + h, v);
                            }
                        tmem_wait_st();
                        drained(buf);
                    }
                } else {
                    ok = filled();
                    buf ^= 1;
                }
                if (!ok) break;
                fence_after();
                float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (kMode == kFprop && p.bias) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int l = q * 32 + (lane >> 2) + 8 * g;
                        if (l < live) b[g] = __bfloat162float(p.bias[(int64_t)T.e * p.N + f0 + l]);
                    }
                }
                const uint32_t acc = lanes + from * WIDE;
                if constexpr (kMode == kWgrad) {
#pragma unroll
                    for (int i = 0; i < kBoxes; ++i) {
                        const int c = 64 * i + 32 * group;
                        if (c < T.cols)
                            store_box_bf16(acc + c, lane, stage, &tmOut, f0 + 32 * q, T.c0 + c, T.e, live > 32 * q,
                                           p.accumulate, old[i]);
                    }
                } else {
                    for (int c = 32 * group; c < T.cols; c += 64)
                        store_columns_bf16(acc + c, lane, stage,
                                           static_cast<__nv_bfloat16*>(p.out) + (T.row0 + c) * ld + f0 + 32 * q, ld,
                                           live - 32 * q, T.cols - c, [&](float v, int l, int) { return v + b[l >> 3]; });
                }
                drained(from);
            }
        } while (queue.next(t, lane, abort_flag) == TileQueue::kTile);
        if (kMode == kWgrad) {  // the last boxes are written before the block leaves its shared memory
            if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            __syncwarp();
        }
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
    return fn(m, elem_bytes == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
              : elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
              rank,
              const_cast<void*>(base), d, s, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle_bytes == 0    ? CU_TENSOR_MAP_SWIZZLE_NONE
              : swizzle_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                    : CU_TENSOR_MAP_SWIZZLE_128B,
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

template <int kMode, bool kRegs>
static cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& half, const CUtensorMap& out,
                          const Params& p, int64_t tiles, cudaStream_t s) {
    return launch_persistent<CG, true, ragged_gemm_kernel<kMode, kRegs>>(THREADS, smem_bytes(MXQ_MAX_EXPERTS), smem_bytes(p.E),
                                                                   tiles, s, a, b, half, out, p);
}

template <int kMode>
static cudaError_t run_mode(const GemmCall& c, cudaStream_t s) {
    const Params p{c.M, c.N, c.K, c.E, c.m_splits, static_cast<const __nv_bfloat16*>(c.bias), c.out, c.out_f32,
                   c.accumulate, c.status};
    CUtensorMap a, b, half, out;  // half: b in boxes of half the rows; out: dW
    bool ok;
    const int64_t feats = ((kMode == kFprop ? c.N : c.K) + FEAT - 1) / FEAT;
    int64_t tiles = (c.M / WIDE + std::min<int64_t>(c.E, c.M)) * feats;  // no fewer than the device counts
    if (kMode == kWgrad) {
        tiles = feats * ((c.N + WIDE - 1) / WIDE) * c.E;
        // with M == 0 nothing is loaded: any valid address does
        const int64_t rows = std::max<int64_t>(c.M, 1);
        const int64_t da[2] = {c.K, rows}, sa[1] = {2 * c.ld_tok}, db[2] = {c.N, rows}, sb[1] = {2 * c.ld_mat};
        const int boxa[2] = {64, BK}, boxb[2] = {BOX, BK};
        ok = encode_tmap(&a, c.M ? c.tok : c.out, 2, 2, da, sa, boxa) &&
             encode_tmap(&b, c.M ? c.mat : c.out, 2, 2, db, sb, boxb);
        half = b;
        const int size = c.out_f32 ? 4 : 2;
        const int64_t dd[3] = {c.K, c.N, c.E}, sd[2] = {size * c.K, size * c.K * c.N};
        const int boxd[3] = {32, c.out_f32 ? 16 : 32, 1};
        ok = ok && encode_tmap(&out, c.out, size, 3, dd, sd, boxd, c.out_f32 ? 0 : 64);
    } else {
        const int64_t da[3] = {c.K, c.N, c.E}, sa[2] = {2 * c.K, 2 * c.K * c.N};
        const int64_t db[2] = {kMode == kDgrad ? c.N : c.K, c.M}, sb[1] = {2 * c.ld_tok};
        const int boxa[3] = {64, kMode == kDgrad ? BK : kFM, 1}, boxb[2] = {BK, BOX}, boxh[2] = {BK, BOX / 2};
        ok = encode_tmap(&a, c.mat, 2, 3, da, sa, boxa) && encode_tmap(&b, c.tok, 2, 2, db, sb, boxb) &&
             encode_tmap(&half, c.tok, 2, 2, db, sb, boxh);
    }
    if (kMode != kWgrad) out = a;  // not read
    if (!ok) return cudaErrorInvalidValue;
    return c.out_f32 ? launch<kMode, true>(a, b, half, out, p, tiles, s)
                     : launch<kMode, false>(a, b, half, out, p, tiles, s);
}

cudaError_t run_gemm(const GemmCall& c, cudaStream_t s) {
    if (c.mode == kWgrad) return run_mode<kWgrad>(c, s);
    // One-SM tiles up to as many rows as one holds, on average. W of 2048 x 4096, us, fprop and dgrad, one SM against
    // pairs: 8 experts of 16 rows each 26.2 and 23.7 against 27.4 and 25.5, of 32 26.6 and 24.0 against 27.4 and 25.7,
    // of 40 39.9 and 38.1 against 27.8 and 25.9; 64 experts of 32 168 and 163 against 170 and 159. Uneven counts need
    // more one-SM tiles: 32 rows on average in Dirichlet(0.3) shares 30.7 and 38.0 against 26.7 and 25.5 (8 experts),
    // 194 and 182 against 135 and 134 (64); all on one expert 20.9 and 20.2 against 15.9 and 23.9 (8), 130 and 124
    // against 27 and 25 (64).
    if (c.M <= (int64_t)kFewRows * c.E) {
        // dot products where the one-SM tiles would leave SMs idle (2048 x 4096, us: 1 row of 1 expert 4.3
        // against 7.7, 4 rows 5.9 against 7.7; 8 experts fill the SMs: 1 row each 26.2 and 26.3, 4 rows 32.8
        // and 27.0)
        const int64_t tiles = std::min<int64_t>(c.E, c.M) * ((c.N + kFM - 1) / kFM);
        if (c.mode == kFprop && c.M <= (int64_t)kVecRows * c.E && tiles <= sm_count()) return run_fprop_vec(c, s);
        return run_gemm_few(c, s);
    }
    return c.mode == kFprop ? run_mode<kFprop>(c, s) : run_mode<kDgrad>(c, s);
}

}  // namespace ragged
}  // namespace mxq
