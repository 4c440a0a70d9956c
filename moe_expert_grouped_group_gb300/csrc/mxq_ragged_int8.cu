// mxq_ragged_int8.cu -- int8 grouped products of an MoE expert layer with one
// scale per token and per output channel, for expert counts that are multiples
// of nothing, and the quantizer of their tokens:
//   s_m = max(max_k |x[m,k]|, 2^-100) / 127,  q[m,k] = rint(x[m,k] (127 / max))
//   Y[m,n] = (sum_k xq[m,k] wq[e,n,k]) xs[m] ws[e,n] (+ b[e,n])
//
// GB300's int8 tensor rate is a small fraction of its 16-bit floating rate, so
// the codes travel as int8 (the bytes that a weight-bound call is made of) and
// are widened to f16 on chip, exactly: |q| <= 128 fits f16's 11 significand
// bits. The products are then whole numbers up to 2^14 and tcgen05.mma
// kind::f16 sums them in fp32, exactly while sums stay within 2^24: 1024 of K
// whatever the codes. Past that the tensor core truncates, up to 2^-23 of the
// sum per 16 of K (codes of one sign: 3e-6 at K = 4096, 2e-3 at 2^17). So sums
// that may pass 2^24 are drained every 1024 of K and added in registers
// (kDeep): as 32-bit integers, exact, while no sum can leave them (K up to
// kVecDepth), in fp32 beyond. fp32 outputs take that shape where K > 1024 and
// so are the same bits as those of the dot products, whatever shares the call.
// bf16 outputs take it where K > kTruncDepth = 2^15: below, the truncation is under 2^-12 of
// the sum of the products' magnitudes, a sixteenth of bf16's rounding, and
// zero-mean codes, whose sums stay within 2^24, have none.
//
// What kDeep costs: a pair's sums fill the registers at 128 columns, half of
// what an MMA with A in TMEM takes in the same time, against which the epilogue
// is hidden by a second accumulator. fp32, 8 experts, 16384 rows, us, in one
// truncating accumulator and as it is: 2048 x 4096 253 and 310, 7168 x 2048 320
// and 482 (bf16: 193 and 293). One set of converting warps leaves the epilogue
// its registers; with two it spilled (2048 x 4096 a tenth slower). Few rows: 8
// experts x 16 19.9 and 20.9, 64 x 16 113 and 118.
//
// The tile walk, the operands' sides (features on the MMA's M, tokens on its
// N), the edges and the two shapes (pairs of SMs; one SM for few rows) are
// those of the bf16 products (mxq_ragged.cuh, mxq_ragged.cu). A handful of rows
// an expert goes to mxq_ragged_vec.cu.
//
// The widened weights go to TMEM, the widened tokens to shared memory: with
// both in shared memory a 256 x 256 tile of a pair moves 96 KB and more through
// it per 64 of K (load, read, write back twice as wide, read by the MMA), 750
// cycles against the MMA's 512. An MMA that reads A from TMEM takes about 130
// cycles per 16 of K however few its columns are, so the pair shape gives it
// 256; its accumulator and three slots of weights then fill TMEM, and a tile's
// epilogue is not hidden behind the next tile's MMAs: eight warps keep it
// short, and its scales are fetched before the sums are done. The few-rows
// shape (one SM, up to 32 tokens) has room for two accumulators.
//
// Warp 0 loads 128-deep int8 stages; sets of four warps for the weights and
// four for the tokens take turns, so that one set's latencies hide behind the
// others' work; warp 1 issues the MMAs; the epilogue's warps scale and store.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "mxq_internal.h"
#include "mxq_ragged.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace ragged {
namespace i8 {

constexpr int BK = 128;  // depth of an int8 stage
constexpr int HK = 64;   // half of it: 128 bytes of f16
constexpr int CVT_WARPS = 4;  // of a set: for the weights, and as many for the tokens
constexpr int CHUNK = 1024;  // of K whose sums are whole numbers in fp32: |codes| <= 128

template <int kCG, bool kDeep>
struct Shape {
    static constexpr int kFeat = kFM * kCG;
    static constexpr int kWide = kCG == 1 ? kFewRows : kDeep ? 128 : 256;
    static constexpr int kStep = 16 * kCG;
    static constexpr int kBox = 32;                  // token rows of a box
    static constexpr int kTok = kWide / kCG;         // token rows of a stage in one CTA
    static constexpr int kRaws = kCG == 2 ? 3 : 8;   // int8 stages
    static constexpr int kRaw = (kFM + kTok) * BK;   // weights, then tokens
    static constexpr int kSets = kCG == 1 ? 3 : kDeep ? 1 : 2;  // of converting warps
    static constexpr int kSlots = 3;                 // of widened operands
    static constexpr int kHalf = kTok * HK * 2;      // widened tokens of half a slot
    static constexpr int kSlot = 2 * kHalf;
    static constexpr int kBufs = kWide == 256 ? 1 : 2;  // accumulators
    static constexpr int kTmemA = kBufs * kWide;     // the weights' slots follow them
    static constexpr int kSlotCols = BK / 2;         // of its weights in TMEM
    static constexpr int kTmem = kCG == 2 ? 512 : 256;
    static constexpr int kRawAt = kSlots * kSlot;
    static constexpr int kEpi = kRawAt + kRaws * kRaw;
    // warps: 0 loads, 1 MMAs, two idle; the epilogue; the weights' sets; the tokens' sets
    static constexpr int kEpiWarps = kCG == 2 ? 8 : 4;
    static constexpr int kEpiFirst = 4, kCvtFirst = kEpiFirst + kEpiWarps, kTokFirst = kCvtFirst + kSets * CVT_WARPS;
    static constexpr int kThreads = 32 * (kTokFirst + kSets * CVT_WARPS);
    // registers a thread: at launch, and then of the first four warps, the epilogue's, the weights' and the tokens'
    static constexpr int kStartRegs = 65536 / kThreads / 8 * 8, kCtlRegs = 56;
    static constexpr int kEpiRegs = kCG == 1 ? 96 : kDeep ? 136 : 88;
    static constexpr int kWeiRegs = kCG == 1 ? 64 : kDeep ? 80 : 72, kTokRegs = kCG == 1 ? 56 : 64;
    static_assert(4 * kCtlRegs + kEpiWarps * kEpiRegs + kSets * CVT_WARPS * (kWeiRegs + kTokRegs) <=
                      kThreads / 32 * kStartRegs,
                  "the warps' registers are those that the block starts with");
    static constexpr int kBars = kEpi + kEpiWarps * kEpiBytes;
    static constexpr int kTables = kBars + 256;
    __host__ __device__ static constexpr int smem(int E) { return 1024 + kTables + 8 * (E + 1); }
    static_assert(1024 + kTables + 8 * (MXQ_MAX_EXPERTS + 1) <= 232448, "shared memory over the per-block limit");
    static_assert(kBars % 8 == 0 && 8 * (2 * (kRaws + kSlots) + 4) <= 256, "barrier region");
    static_assert(kRaws >= kSlots && kSlots >= kSets, "see the order of the conversion's waits");
    static_assert(kHalf % 1024 == 0 && kRaw % 1024 == 0, "the 128-byte swizzle repeats every 1024 bytes");
    static_assert(kTmemA + kSlots * kSlotCols <= kTmem, "TMEM columns");
};

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
// 0..255; under the high byte 0x64 that is the f16 1024 + 128 + q. Bytes 0 and
// 2 come first, then 1 and 3: both operands' sums run over k in the same order.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    const uint32_t bias = 0x64806480u;  // 1152, 1152
    uint32_t lo = (w & 0x00FF00FFu) ^ 0x64806480u, hi = (w >> 8 & 0x00FF00FFu) ^ 0x64806480u;
    __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), *reinterpret_cast<const __half2*>(&bias));
    __half2 b = __hsub2(*reinterpret_cast<__half2*>(&hi), *reinterpret_cast<const __half2*>(&bias));
    return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

// Sums of a column's pieces of CHUNK, as the bits of an integer (`whole`) or of an fp32 value.
struct Pieces {
    bool whole;
    __device__ __forceinline__ static uint32_t add_whole(uint32_t sum, uint32_t v, bool first) {
        const uint32_t i = (uint32_t)__float2int_rn(__uint_as_float(v));
        return first ? i : sum + i;
    }
    __device__ __forceinline__ static uint32_t add_fp32(uint32_t sum, uint32_t v, bool first) {
        return first ? v : __float_as_uint(__fadd_rn(__uint_as_float(sum), __uint_as_float(v)));
    }
    template <int n>
    __device__ __forceinline__ void add(uint32_t* sum, const uint32_t (&v)[n], bool first) const {
        if (whole) {
#pragma unroll
            for (int j = 0; j < n; ++j) sum[j] = add_whole(sum[j], v[j], first);
        } else {
#pragma unroll
            for (int j = 0; j < n; ++j) sum[j] = add_fp32(sum[j], v[j], first);
        }
    }
    template <int n>
    __device__ __forceinline__ void finish(uint32_t* sum) const {
        if (whole)
#pragma unroll
            for (int j = 0; j < n; ++j) sum[j] = __float_as_uint(__int2float_rn((int)sum[j]));
    }
};

// The steps of every shape, and of the dot products: each one fp32 rounding.
__device__ __forceinline__ float scaled(float sum, float xs, float ws, float bias) {
    return __fadd_rn(__fmul_rn(__fmul_rn(sum, xs), ws), bias);
}

template <int kCG, bool kF32, bool kDeep>
__global__ void __launch_bounds__(Shape<kCG, kDeep>::kThreads, 1)
    ragged_int8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Params p) {
    using S = Shape<kCG, kDeep>;
    constexpr int RAWS = S::kRaws, SETS = S::kSets, SLOTS = S::kSlots;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align<1024>(smem_raw);
    int32_t* s_off = reinterpret_cast<int32_t*>(smem + S::kTables);
    int32_t* s_slices = s_off + p.E + 1;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kCG == 2 ? cta_rank() : 0;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
    const uint32_t rawf0 = smem_u32(bars), rawe0 = rawf0 + 8 * RAWS;
    const uint32_t full0 = rawe0 + 8 * RAWS, empty0 = full0 + 8 * SLOTS;
    const uint32_t accf0 = empty0 + 8 * SLOTS, acce0 = accf0 + 16;
    volatile int* abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int st = 0; st < RAWS; ++st) {
            mbar_init(rawf0 + 8 * st, 1);
            mbar_init(rawe0 + 8 * st, 2 * CVT_WARPS);
        }
        for (int st = 0; st < SLOTS; ++st) {
            mbar_init(full0 + 8 * st, kCG * 2 * CVT_WARPS);
            mbar_init(empty0 + 8 * st, 1);
        }
        for (int b = 0; b < S::kBufs; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, kCG * S::kEpiWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmA) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmB) : "memory");
    }
    const int bad = load_ragged(p.m_splits, p.E, p.M, S::kWide, s_off, s_slices);
    if (bad) {
        report_status(p.status, bad);
        return;
    }
    if (warp == 1) tmem_alloc<kCG>(smem_u32(&s_tmem), S::kTmem);
    fence_before();
    __syncthreads();
    if (kCG == 2) cluster_sync();
    fence_after();
    const uint32_t tmem = s_tmem;
    const Walk<kFprop, S::kFeat, S::kWide, S::kStep> W(p.N, p.K, p.E, s_off, s_slices, nullptr);
    const int64_t first = blockIdx.x / kCG, stride = gridDim.x / kCG;

    if (warp < S::kEpiFirst) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kCtlRegs));
        if (warp == 0) {
            // -------------------------------------------------- TMA producer: this CTA's int8 boxes
            int stage = 0;
            uint32_t phase = 0;
            int64_t fills = 0;
            for (int64_t t = first; t < W.total; t += stride) {
                const Tile T = W.get(t);
                const int half = T.n / kCG, boxes = (half + S::kBox - 1) / S::kBox;  // this CTA's rows
                const int f = T.f0 + rank * kFM, c = T.c0 + rank * half;
                for (int r = 0; r < T.red; r += BK) {
                    if (!mbar_wait(rawe0 + 8 * stage, phase ^ 1, abort_flag)) {
                        drain_ring(rawf0, RAWS, fills);
                        goto done_producer;
                    }
                    __syncwarp();
                    const uint32_t fb = rawf0 + 8 * stage, a = smem_u32(smem) + S::kRawAt + stage * S::kRaw;
                    if (elect_one()) {
                        mbar_expect_tx(fb, (kFM + boxes * S::kBox) * BK);
                        load_3d<1>(a, &tmA, fb, r, f, T.e);
                        for (int i = 0; i < boxes; ++i)
                            load_2d<1>(a + (kFM + i * S::kBox) * BK, &tmB, fb, r, c + S::kBox * i);
                    }
                    __syncwarp();
                    ++fills;
                    if (++stage == RAWS) { stage = 0; phase ^= 1; }
                }
            }
        done_producer:;
        } else if (warp == 1 && rank == 0) {
            // -------------------------------------------------- MMA issuer (rank 0)
            int slot = 0, buf = 0;
            uint32_t phase = 0, aphase = 0;
            const uint64_t bd0 = smem_desc(smem_u32(smem), 16, 1024);
            for (int64_t t = first; t < W.total; t += stride) {
                const Tile T = W.get(t);
                const uint32_t id = idesc_f16(0, 0, 0, S::kFeat, T.n);
                for (int r0 = 0; r0 < T.red; r0 += kDeep ? CHUNK : T.red) {
                    const int r1 = kDeep ? min(T.red, r0 + CHUNK) : T.red;
                    const uint32_t d = tmem + buf * S::kWide;
                    if (!mbar_wait(acce0 + 8 * buf, aphase ^ 1, abort_flag)) goto done_mma;
                    __syncwarp();
                    for (int r = r0; r < r1; r += BK) {
                        const uint32_t at = tmem + S::kTmemA + slot * S::kSlotCols;
                        const uint64_t off = (uint64_t)(slot * (S::kSlot / 16));
                        if (!mbar_wait(full0 + 8 * slot, phase, abort_flag)) goto done_mma;
                        __syncwarp();
                        fence_after();
                        const int steps = T.red - r >= BK ? BK / 16 : (T.red - r + 15) / 16;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < BK / 16; ++k)
                                if (k < steps)
                                    mma_f16_tmem<kCG>(d, at + 8 * k, bd0 + off + (k >> 2) * (S::kHalf / 16) + 2 * (k & 3),
                                                      id, r > r0 || k > 0);
                            mma_commit<kCG>(empty0 + 8 * slot);
                            if (r + BK >= r1) mma_commit<kCG>(accf0 + 8 * buf);
                        }
                        __syncwarp();
                        if (++slot == SLOTS) { slot = 0; phase ^= 1; }
                    }
                    if (++buf == S::kBufs) { buf = 0; aphase ^= 1; }
                }
            }
        done_mma:;
        }
    } else if (warp < S::kCvtFirst) {
        // ------------------------------------------------------ epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kEpiRegs));
        const int q = warp & 3, group = (warp - S::kEpiFirst) >> 2;
        constexpr int kGroups = S::kEpiWarps / 4;
        uint8_t* stage = smem + S::kEpi + (warp - S::kEpiFirst) * kEpiBytes;
        int buf = 0;
        uint32_t aphase = 0;
        for (int64_t t = first; t < W.total; t += stride) {
            const Tile T = W.get(t);
            const int f0 = T.f0 + rank * kFM + 32 * q;  // of this warp's 32 lanes
            const int live = (int)min((int64_t)32, p.N - f0);
            const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
            // scales and bias are fetched while the sums are made
            const float* xs = p.xs + T.row0;
            auto ready = [&] {
                const bool ok = mbar_wait(accf0 + 8 * buf, aphase, abort_flag);
                fence_after();
                return __all_sync(0xffffffffu, ok && !*abort_flag) != 0;
            };
            auto drained = [&] {
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(acce0 + 8 * buf);
                    else arrive_remote_relaxed(mapa(acce0 + 8 * buf, 0));
                }
                if (++buf == S::kBufs) { buf = 0; aphase ^= 1; }
            };
            // kDeep: the sums of this warp's columns, 32 of every 32 * kGroups
            constexpr int kMine = S::kWide / (32 * kGroups);
            const Pieces pieces{p.K <= kVecDepth};
            auto each_piece = [&](auto&& take) {  // take(column's place in kMine, column, first piece)
                for (int r0 = 0; r0 < T.red; r0 += CHUNK) {
                    if (!ready()) return false;
#pragma unroll
                    for (int i = 0; i < kMine; ++i)
                        if (32 * (group + kGroups * i) < T.cols)
                            take(i, lanes + buf * S::kWide + 32 * (group + kGroups * i), r0 == 0);
                    drained();
                }
                return true;
            };
            if constexpr (kF32) {
                const int64_t at = (int64_t)T.e * p.N + f0 + lane;
                const float sw = lane < live ? p.ws[at] : 0.0f;
                const float b = p.bias && lane < live ? __bfloat162float(p.bias[at]) : 0.0f;
                auto store = [&](const uint32_t* v, int c) {
                    if (lane >= live) return;
                    float* o = static_cast<float*>(p.out) + (T.row0 + c) * p.N + f0 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < T.cols) o[j * p.N] = scaled(__uint_as_float(v[j]), xs[c + j], sw, b);
                };
                if constexpr (kDeep) {
                    uint32_t sum[kMine][32];
                    const bool ok = each_piece([&](int i, uint32_t at, bool first) {
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            uint32_t v[16];
                            tmem_ld16(at + h, v);
                            tmem_wait_ld();
                            pieces.add(&sum[i][h], v, first);
                        }
                    });
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        pieces.finish<32>(sum[i]);
                        store(sum[i], 32 * (group + kGroups * i));
                    }
                } else {
                    if (!ready()) break;
                    for (int c = 32 * group; c < T.cols; c += 32 * kGroups) {
                        uint32_t v[32];
                        tmem_ld32(lanes + buf * S::kWide + c, v);
                        tmem_wait_ld();
                        store(v, c);
                    }
                    drained();
                }
            } else {
                float sw[4], b[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int l = (lane >> 2) + 8 * g;
                    const int64_t at = (int64_t)T.e * p.N + f0 + l;
                    sw[g] = l < live ? p.ws[at] : 0.0f;
                    b[g] = p.bias && l < live ? __bfloat162float(p.bias[at]) : 0.0f;
                }
                // this thread's token scales in 32 columns: columns 8b + 2 (lane mod 4) and the next
                float sx[8];
                auto scales = [&](int c) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int col = c + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
                        sx[i] = col < T.cols ? xs[col] : 0.0f;
                    }
                };
                auto store = [&](auto&& v, int c) {
                    store_columns_bf16(v, lane, stage, static_cast<__nv_bfloat16*>(p.out) + (T.row0 + c) * p.N + f0, p.N,
                                       live, T.cols - c, [&](float v, int l, int col) {
                                           return scaled(v, sx[(col >> 3) * 2 + (col & 1)], sw[l >> 3], b[l >> 3]);
                                       });
                };
                if constexpr (kDeep) {
                    uint32_t sum[kMine][2][16];
                    const bool ok = each_piece([&](int i, uint32_t at, bool first) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t v[16];
                            tmem_ld16x32(at + ((uint32_t)(16 * h) << 16), v);
                            tmem_wait_ld();
                            pieces.add(sum[i][h], v, first);
                        }
                    });
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        const int c = 32 * (group + kGroups * i);
                        if (c >= T.cols) break;
                        pieces.finish<16>(sum[i][0]);
                        pieces.finish<16>(sum[i][1]);
                        scales(c);
                        store(sum[i], c);
                    }
                } else {
                    scales(32 * group);
                    if (!ready()) break;
                    for (int c = 32 * group; c < T.cols; c += 32 * kGroups) {
                        float s[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) s[i] = sx[i];
                        scales(c + 32 * kGroups);
                        store_columns_bf16(lanes + buf * S::kWide + c, lane, stage,
                                           static_cast<__nv_bfloat16*>(p.out) + (T.row0 + c) * p.N + f0, p.N, live,
                                           T.cols - c, [&](float v, int l, int col) {
                                               return scaled(v, s[(col >> 3) * 2 + (col & 1)], sw[l >> 3], b[l >> 3]);
                                           });
                    }
                    drained();
                }
            }
        }
    } else {
        // ------------------------------------------------------ int8 -> f16, this CTA's rows
        // A set's turn is every kSets-th stage: wait for the next slot and for the stage, load the codes into
        // registers, widen them into the slot, free the stage. The slot comes first: its last MMAs are
        // those of SLOTS stages ago, so all earlier stages have been loaded, and with no fewer than SLOTS of
        // them a stage's barrier cannot be more than one phase behind what a set waits for, although the other
        // sets' phases are not its own.
        // The stage is freed when its codes have been used, behind a fence: TMA writes the next fill through
        // another proxy, and an arrival that only followed the loads overtook those that waited behind the
        // epilogue's stores (fp32, K = 7168: codes of the next fill in 1 call of 100). Freed between the loads and
        // the widening, with the fence there, 16384 rows take 218 us in place of 213.
        const bool weights = warp < S::kTokFirst;
        const int set = (warp - (weights ? S::kCvtFirst : S::kTokFirst)) / CVT_WARPS;
        const uint32_t lead_full = kCG == 2 ? mapa(full0, 0) : 0;
        int raw = 0, turn = 0, slot = 0;
        uint32_t rphase = 0, phase = 0;
        auto convert = [&](auto&& load, auto&& widen) {
            for (int64_t t = first; t < W.total; t += stride) {
                const Tile T = W.get(t);
                for (int r = 0; r < T.red; r += BK) {
                    if (turn == set) {
                        const bool ok = mbar_wait(empty0 + 8 * slot, phase ^ 1, abort_flag) &&
                                        mbar_wait(rawf0 + 8 * raw, rphase, abort_flag);
                        if (!__all_sync(0xffffffffu, ok)) return;
                        load(smem + S::kRawAt + raw * S::kRaw);
                        widen();
                        if (weights) fence_async_smem();  // the tokens' writes end with one
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(rawe0 + 8 * raw);
                            if (rank == 0) mbar_arrive(full0 + 8 * slot);
                            else arrive_remote(lead_full + 8 * slot);
                        }
                    }
                    if (++turn == SETS) turn = 0;
                    if (++slot == SLOTS) { slot = 0; phase ^= 1; }
                    if (++raw == RAWS) { raw = 0; rphase ^= 1; }
                }
            }
        };
        if (weights) {
            if constexpr (S::kWeiRegs < S::kStartRegs)
                asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kWeiRegs));
            // lane = feature: 128 codes of its swizzled row (16-byte chunk ^= row mod 8)
            const int q = warp & 3;
            const uint32_t quarter = tmem + ((uint32_t)(32 * q) << 16) + S::kTmemA;
            uint4 w[BK / 16];
            convert(
                [&](const uint8_t* src) {
#pragma unroll
                    for (int i = 0; i < BK / 16; ++i)
                        w[i] = *reinterpret_cast<const uint4*>(src + (32 * q + lane) * BK + ((i ^ (lane & 7)) << 4));
                },
                [&] {
                    fence_after();  // the slot's last MMAs come before the writes
#pragma unroll
                    for (int i = 0; i < BK / 16; ++i)
                        tmem_st8(quarter + slot * S::kSlotCols + 8 * i, widen4(w[i].x), widen4(w[i].y), widen4(w[i].z),
                                 widen4(w[i].w));
                    tmem_wait_st();
                    fence_before();
                });
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kTokRegs));
            // rows beyond the slice are widened too: what they hold is never stored
            constexpr int kUnits = S::kTok * (BK / 16) / (32 * CVT_WARPS);  // 16-byte chunks a thread
            // Eight lanes (a quarter warp) take four chunks of one row's first half of K and four of the next
            // row's second half: no two of them meet in a bank, neither here nor where they write.
            const int ct = (int)threadIdx.x & (32 * CVT_WARPS - 1), second = ct >> 2 & 1, cc = ct & 3;
            auto row_of = [&](int u) { return (((ct >> 3) + u * 4 * CVT_WARPS) & ~1) + second; };
            const int half = second ^ (ct >> 3 & 1);
            uint4 w[kUnits];
            convert(
                [&](const uint8_t* src) {
#pragma unroll
                    for (int u = 0; u < kUnits; ++u)
                        w[u] = *reinterpret_cast<const uint4*>(src + (kFM + row_of(u)) * BK +
                                                               (((4 * half + cc) ^ (row_of(u) & 7)) << 4));
                },
                [&] {
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) {
                        const uint2 a = widen4(w[u].x), b = widen4(w[u].y), c = widen4(w[u].z), d = widen4(w[u].w);
                        uint8_t* o = smem + slot * S::kSlot + half * S::kHalf + row_of(u) * 128;
                        const int at = (2 * cc) ^ (row_of(u) & 7);
                        *reinterpret_cast<uint4*>(o + (at << 4)) = make_uint4(a.x, a.y, b.x, b.y);
                        *reinterpret_cast<uint4*>(o + ((at ^ 1) << 4)) = make_uint4(c.x, c.y, d.x, d.y);
                    }
                    fence_async_smem();
                });
        }
    }
    fence_before();
    __syncthreads();
    if (s_abort && threadIdx.x == 0 && p.status) atomicOr(p.status, MXQ_STATUS_WAIT_TIMEOUT);
    if (kCG == 2) cluster_sync();
    if (warp == 1) {
        fence_after();
        tmem_dealloc<kCG>(tmem, S::kTmem);
    }
}

// ------------------------------------------------------------ row quantizer
// A row with an infinity or NaN has no scale: its scale is NaN and its codes
// are 0, so that its outputs are NaN and nothing else is. bf16 magnitudes are
// compared as bits, two at a time: they order as the values do.
__device__ __forceinline__ uint32_t top2(uint32_t top, const uint4& w) {
    return __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                  __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
}
struct RowScale {
    float inv, scale;
    bool finite;
    __device__ explicit RowScale(uint32_t top) {  // bits of the row's largest magnitude
        finite = top < 0x7F80u;
        const float amax = fmaxf(__uint_as_float(top << 16), 7.8886090522101181e-31f);  // 2^-100
        inv = finite ? __fdiv_rn(127.0f, amax) : 0.0f;
        scale = finite ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FC00000u);
    }
    __device__ uint2 codes(const uint4& w) const {
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int a = finite ? __float2int_rn(__fmul_rn(bf16lo(ws[j]), inv)) : 0;
            const int b = finite ? __float2int_rn(__fmul_rn(bf16hi(ws[j]), inv)) : 0;
            o[j >> 1] |= ((uint32_t)(a & 255) | (uint32_t)(b & 255) << 8) << (16 * (j & 1));
        }
        return make_uint2(o[0], o[1]);
    }
};

// Rows of at most kLanes * kVec * 8 elements: kLanes lanes hold a row in
// registers, so it is read once and no block waits. 16384 x 2048: 27.8 us with
// the block kernel below, 14.1 to 17.4 us with this one; 1000000 x 128: 884 and 74 us.
template <int kLanes, int kVec>
__global__ void __launch_bounds__(256) quantize_rows_lanes_kernel(const uint16_t* x, int64_t M, int64_t K, int64_t ld,
                                                                  uint8_t* q, float* scale) {
    wait_for_stream();
    const int l = threadIdx.x % kLanes, vecs = (int)(K / 8);
    const int64_t step = (int64_t)gridDim.x * (256 / kLanes);
    for (int64_t m0 = (int64_t)blockIdx.x * (256 / kLanes); m0 < M; m0 += step) {
        const int64_t m = m0 + threadIdx.x / kLanes;
        const bool live = m < M;
        const uint4* row = reinterpret_cast<const uint4*>(x + m * ld);
        uint4 w[kVec];
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            w[v] = live && l + v * kLanes < vecs ? row[l + v * kLanes] : make_uint4(0u, 0u, 0u, 0u);
            top = top2(top, w[v]);
        }
        top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const RowScale s(top);
#pragma unroll
        for (int v = 0; v < kVec; ++v)
            if (live && l + v * kLanes < vecs) *reinterpret_cast<uint2*>(q + m * K + 8 * (l + v * kLanes)) = s.codes(w[v]);
        if (live && l == 0) scale[m] = s.scale;
    }
}

// Longer rows: a block each, read twice (the second time from cache). 16384 x 4096: 51.7 us, x 7168: 67.7 us; 131072 x
// 7168: 437 us (floors, at 3 bytes an element: 30, 52 and 415).
__global__ void __launch_bounds__(256) quantize_rows_kernel(const uint16_t* x, int64_t M, int64_t K, int64_t ld,
                                                            uint8_t* q, float* scale) {
    wait_for_stream();
    __shared__ uint32_t s_top[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const uint4* row = reinterpret_cast<const uint4*>(x + m * ld);
        uint32_t top = 0;
        for (int64_t i = threadIdx.x; i < K / 8; i += 256) top = top2(top, row[i]);
        top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
        __syncthreads();
        if (lane == 0) s_top[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, s_top[i]);
        const RowScale s(top);
        for (int64_t i = threadIdx.x; i < K / 8; i += 256) *reinterpret_cast<uint2*>(q + m * K + 8 * i) = s.codes(row[i]);
        if (threadIdx.x == 0) scale[m] = s.scale;
    }
}

}  // namespace i8

template <int kCG, bool kF32, bool kDeep>
static cudaError_t launch_int8(const CUtensorMap& a, const CUtensorMap& b, const i8::Params& p, int64_t tiles,
                               cudaStream_t s) {
    using S = i8::Shape<kCG, kDeep>;
    return launch_persistent<kCG, false, i8::ragged_int8_kernel<kCG, kF32, kDeep>>(S::kThreads, S::smem(MXQ_MAX_EXPERTS),
                                                                     S::smem(p.E), tiles, s, a, b, p);
}

template <int kCG, bool kDeep>
static cudaError_t run_int8_shape(const Int8Call& c, cudaStream_t s) {
    using S = i8::Shape<kCG, kDeep>;
    const i8::Params p{c.xs, c.ws, static_cast<const __nv_bfloat16*>(c.bias), c.M, c.N, c.K, c.E, c.m_splits, c.out,
                       c.out_f32, c.status};
    const int64_t da[3] = {c.K, c.N, c.E}, sa[2] = {c.K, c.K * c.N}, db[2] = {c.K, c.M}, sb[1] = {c.K};
    const int boxa[3] = {i8::BK, kFM, 1}, boxb[2] = {i8::BK, S::kBox};
    CUtensorMap a, b;
    if (!encode_tmap(&a, c.wq, 1, 3, da, sa, boxa) || !encode_tmap(&b, c.xq, 1, 2, db, sb, boxb))
        return cudaErrorInvalidValue;
    const int64_t tiles = (c.M / S::kWide + std::min<int64_t>(c.E, c.M)) * ((c.N + S::kFeat - 1) / S::kFeat);
    return c.out_f32 ? launch_int8<kCG, true, kDeep>(a, b, p, tiles, s) : launch_int8<kCG, false, kDeep>(a, b, p, tiles, s);
}

cudaError_t run_int8(const Int8Call& c, cudaStream_t s) {
    if (c.M <= (int64_t)kVecRows * c.E && c.K <= kVecDepth) return run_int8_vec(c, s);
    // One-SM tiles up to as many rows as one holds, on average. W of 2048 x 4096, bf16, us, one SM against pairs: 8
    // experts of 32 rows each 19.0 against 24.6, of 48 34.3 against 24.8; 64 experts of 32 113 against 145, of 48 211
    // against 146. Uneven counts need more one-SM tiles: 32 rows on average in Dirichlet(0.3) shares 26.4 against 26.0
    // (8 experts), 157 against 120 (64); all on one expert 19.0 against 17.7 (8), 111 against 31 (64).
    const bool deep = c.K > (c.out_f32 ? i8::CHUNK : kTruncDepth);
    if (c.M <= (int64_t)kFewRows * c.E) return deep ? run_int8_shape<1, true>(c, s) : run_int8_shape<1, false>(c, s);
    return deep ? run_int8_shape<2, true>(c, s) : run_int8_shape<2, false>(c, s);
}

cudaError_t run_int8_quantize(const void* x, int64_t M, int64_t K, int64_t ld, void* q, float* scale, cudaStream_t s) {
    if (M == 0) return cudaSuccess;
    const auto run = [&](auto kernel, int64_t rows) {
        const unsigned grid = (unsigned)std::min<int64_t>((M + rows - 1) / rows, (int64_t)sm_count() * 8);
        return launch(kernel, grid, 256, s, 0, static_cast<const uint16_t*>(x), M, K, ld, static_cast<uint8_t*>(q), scale);
    };
    if (K <= 128) return run(i8::quantize_rows_lanes_kernel<8, 2>, 32);
    if (K <= 512) return run(i8::quantize_rows_lanes_kernel<32, 2>, 8);
    if (K <= 2048) return run(i8::quantize_rows_lanes_kernel<32, 8>, 8);
    return run(i8::quantize_rows_kernel, 1);
}

}  // namespace ragged
}  // namespace mxq
