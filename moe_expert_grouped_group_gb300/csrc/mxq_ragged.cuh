// mxq_ragged.cuh -- what the ragged grouped products (mxq_ragged.cu and
// mxq_ragged_few.cu, bf16; mxq_ragged_int8.cu; mxq_ragged_vec.cu) share: the
// tables of a ragged grouping, the tile walk and queue, split sums, the bf16
// epilogue, the tcgen05 wrappers for 16-bit floating operands, the launchers.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "mxq_common.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace ragged {

constexpr int kFM = 128;  // MMA M: rows of A (features) per CTA
// Terms of a sum rounded to bf16 beyond which it is not left to one accumulator, which truncates: up to 2^-23 of the
// sum per 16 terms, 2^-12 at this length.
constexpr int64_t kTruncDepth = 1 << 15;

// ------------------------------------------------------------ PTX wrappers
// These kernels are launched so that they may begin while the stream's previous
// kernel ends (launch() below): before this wait they touch nothing but their
// parameters and shared memory, after it everything earlier in the stream has
// completed and is visible. It takes the launch latency off a chain of short
// kernels (16 rows, 8 experts, 2048 x 4096: 28.7 -> 26.0 us a call).
// A kernel that begins early runs beside the one that writes its inputs, so
// nothing global is read-only for its lifetime: no __ldg, ld.global.nc or const
// __restrict__ here (the compiler may take such loads before the wait), only
// plain loads behind it.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory matrix descriptor (tcgen05): start>>4 [0,14), LBO>>4 [16,30),
// SBO>>4 [32,46), version 1 [46,48), layout [61,64) (2 = 128-byte swizzle).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor for kind::f16 with fp32 accumulation: D format f32
// [4,6) = 1; A and B formats [7,10) and [10,13) (0 = f16, 1 = bf16); majorness
// of A [15] and B [16] (1 = MN-major); N>>3 [17,23); M>>4 [24,29).
__device__ __forceinline__ uint32_t idesc_f16(uint32_t fmt, uint32_t a_mn, uint32_t b_mn, uint32_t m, uint32_t n) {
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (a_mn << 15) | (b_mn << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// kCG = 1: one SM's tile; 2: a tile of a pair of SMs (a cluster of two CTAs), issued by its rank 0.
template <int kCG>
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, uint32_t accum) {
    if constexpr (kCG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(id), "r"(accum)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(id), "r"(accum)
            : "memory");
}
// The same with A in TMEM: lane = row of A (of this CTA, for a pair), two consecutive k in each column.
template <int kCG>
__device__ __forceinline__ void mma_f16_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t accum) {
    if constexpr (kCG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem), "l"(b), "r"(id), "r"(accum)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem), "l"(b), "r"(id), "r"(accum)
            : "memory");
}
// Arrive on `bar` (in both CTAs of a pair) when the MMAs issued so far have completed.
template <int kCG>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (kCG == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                bar),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
}
template <int kCG>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
    if constexpr (kCG == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <int kCG>
__device__ __forceinline__ void tmem_dealloc(uint32_t tmem, uint32_t cols) {
    if constexpr (kCG == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}
// TMA loads into this CTA's shared memory; `bar` may be the pair's rank 0's (a cluster address) when kCG = 2.
template <int kCG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    if constexpr (kCG == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
            "%4}], [%2];" ::"r"(dst),
            "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y)
            : "memory");
    else
        tma_load_2d(dst, map, bar, x, y);
}
template <int kCG>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    if constexpr (kCG == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
            "%4, %5}], [%2];" ::"r"(dst),
            "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
            "%5}], [%2];" ::"r"(dst),
            "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
}
// True in one lane of a converged warp, always the same. Behind this predicate (unlike behind a test of the
// lane's number) the compiler keeps what is equal in all lanes, the MMAs' descriptors, in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// shared::cluster address of the variable at shared::cta address `a` in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t mapa(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
// Remote arrive after a completed tcgen05.ld: nothing of this CTA's memory is handed over, so no release.
__device__ __forceinline__ void arrive_remote_relaxed(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// mbar_wait on what other CTAs of the cluster have sent or released.
__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_try_cluster(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t i = 0;; ++i) {
        if (mbar_try_cluster(bar, parity)) return true;
        if ((i & 63) == 63) {
            if (*abort_flag) return false;
            if (globaltimer() - t0 > kWaitNs) {
                *abort_flag = 1;
                return false;
            }
        }
    }
}
// Remote arrive that follows this warp's earlier accesses to its own CTA's shared memory or TMEM, which
// fence.proxy.async or tcgen05.wait::st has completed: an answer of the tile queue that has been read, or writes
// that a pair's MMA reads through this SM. What was accessed is on this SM, so the arrive needs no cluster-wide
// release, which would wait for this warp's global stores as well: 800 to 1500 cycles an arrive.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// Remote arrive behind plain shared-memory loads: it may not overtake them (0.2 us each).
__device__ __forceinline__ void arrive_remote_release(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// 32 consecutive accumulator columns of this warp's 32 TMEM lanes
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// 16 consecutive accumulator columns of this warp's 32 TMEM lanes
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// 32 consecutive accumulator columns of 16 TMEM lanes, as a matrix fragment: registers 4i .. 4i+3 of
// thread t hold lanes t/4 (first two) and t/4 + 8 at columns 8i + 2(t mod 4) and the next.
__device__ __forceinline__ void tmem_ld16x32(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Writes 8 consecutive columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, uint2 a, uint2 b, uint2 c, uint2 d) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(a.x), "r"(a.y),
                 "r"(b.x), "r"(b.y), "r"(c.x), "r"(c.y), "r"(d.x), "r"(d.y)
                 : "memory");
}
// Writes 16 consecutive columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// ------------------------------------------------------------ bf16 epilogue
// The accumulator is the transpose of the output tile (lane = feature, column =
// output row), so each warp takes its 32 lanes by 32 columns through a staging
// buffer of its own: matrix fragments out of TMEM, two columns rounded and
// packed at a time, transposed on the way into shared memory (stmatrix
// .trans), then 64-byte row pieces, eight rows to a store instruction. Rows
// are 80 bytes apart: eight consecutive rows start in different banks. Four
// warps writing 256-byte pieces together, at barriers, measured the same.
constexpr int kEpiRow = 80, kEpiBytes = 32 * kEpiRow;

// Columns 0 .. 31 of 32 accumulator lanes at tmem as matrix fragments.
__device__ __forceinline__ void load_columns(uint32_t tmem, uint32_t (&v)[2][16]) {
    tmem_ld16x32(tmem, v[0]);
    tmem_ld16x32(tmem + (16u << 16), v[1]);
    tmem_wait_ld();
}
// They, rounded and packed two columns at a time: [8-column block b][8-lane block g] for stmatrix .trans. A value is
// passed through f(value, b, g, which of the two columns).
template <class F>
__device__ __forceinline__ void columns_bf16(const uint32_t (&v)[2][16], uint32_t (&w)[4][4], F f) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int r = 4 * b + 2 * (g & 1);
            w[b][g] = bf16x2_bits(f(__uint_as_float(v[g >> 1][r]), b, g, 0), f(__uint_as_float(v[g >> 1][r + 1]), b, g, 1));
        }
}

__device__ __forceinline__ void stmatrix_trans(uint32_t row, const uint32_t (&w)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(row), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_trans(uint32_t row, uint32_t (&w)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(row)
                 : "memory");
}

// The same columns, each value passed through f(value, lane in 0..31, column in 0..31), to
// out + column * ld + lane for lanes < live and columns < cols. Called by a warp; `stage` is its own.
template <class F>
__device__ __forceinline__ void store_columns_bf16(const uint32_t (&x)[2][16], int lane, uint8_t* stage,
                                                   __nv_bfloat16* out, int64_t ld, int live, int cols, F f) {
    uint32_t w[4][4];
    columns_bf16(x, w, [&](float v, int b, int g, int half) {
        return f(v, (lane >> 2) + 8 * g, 8 * b + 2 * (lane & 3) + half);
    });
    __syncwarp();  // the stage's last reads are done
    const uint32_t at = smem_u32(stage) + (lane & 7) * kEpiRow + (lane >> 3) * 16;
#pragma unroll
    for (int b = 0; b < 4; ++b) stmatrix_trans(at + 8 * b * kEpiRow, w[b]);
    __syncwarp();
    const int piece = lane & 3;
    if (piece * 8 < live)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = i * 8 + (lane >> 2);
            if (j < cols)
                *reinterpret_cast<uint4*>(out + j * ld + piece * 8) =
                    *reinterpret_cast<const uint4*>(stage + j * kEpiRow + piece * 16);
        }
}
template <class F>
__device__ __forceinline__ void store_columns_bf16(uint32_t tmem, int lane, uint8_t* stage, __nv_bfloat16* out,
                                                   int64_t ld, int live, int cols, F f) {
    uint32_t v[2][16];
    load_columns(tmem, v);
    store_columns_bf16(v, lane, stage, out, ld, live, cols, f);
}

// 32 rows of 32 bf16 at out, 64 contiguous bytes to four lanes; 0 beyond live and cols.
__device__ __forceinline__ void load_rows_bf16(const __nv_bfloat16* out, int64_t ld, int live, int cols, int lane,
                                               uint4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = i * 8 + (lane >> 2), x = (lane & 3) * 8;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (x < live && j < cols) v[i] = *reinterpret_cast<const uint4*>(out + j * ld + x);
    }
}
// The same columns without f as one box of a tensor map (32 lanes x 32 columns, 64-byte swizzle), at column x of
// row y of matrix z; what lies outside the tensor is not written. For outputs whose rows all belong to the
// call's matrix, so dW: its rows leave as 64 contiguous bytes without the warp's own reads and address
// arithmetic (8 experts' dW of 4096 x 2048 from 16 rows each: 30.4 us against 37.6 with store_columns_bf16;
// boxes of 64 x 32 by two warps at a barrier 31.7). `stage` is the warp's own, 512 bytes aligned; it is reused
// once the last box has been read. The caller waits for the last writes. With add, `old` (load_rows_bf16) passes
// through the stage into the fragments' layout and is added in fp32, before the one rounding (the same dW: 67 us,
// floor 40; 16 loads at a time after the sums 697).
constexpr int kBoxBytes = 2048;
__device__ __forceinline__ void store_box_bf16(uint32_t tmem, int lane, uint8_t* stage, const CUtensorMap* map, int x,
                                               int y, int z, bool inside, bool add, const uint4 (&old)[4]) {
    // rows of 64 bytes, their 16-byte pieces exchanged by the row's bits 1 and 2
    const int row = lane & 7;
    const uint32_t at = smem_u32(stage) + row * 64 + (((lane >> 3) ^ (row >> 1)) << 4);
    uint32_t v[2][16], w[4][4];
    if (add) {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = i * 8 + (lane >> 2);
            *reinterpret_cast<uint4*>(stage + j * 64 + (((lane & 3) ^ (j >> 1 & 3)) << 4)) = old[i];
        }
        __syncwarp();
        uint32_t o[4][4];
#pragma unroll
        for (int b = 0; b < 4; ++b) ldmatrix_trans(at + 512 * b, o[b]);
        load_columns(tmem, v);
        columns_bf16(v, w, [&](float v, int b, int g, int half) {
            return v + __uint_as_float(half ? o[b][g] & 0xffff0000u : o[b][g] << 16);
        });
    } else {
        load_columns(tmem, v);
        columns_bf16(v, w, [](float v, int, int, int) { return v; });
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    __syncwarp();
#pragma unroll
    for (int b = 0; b < 4; ++b) stmatrix_trans(at + 512 * b, w[b]);
    fence_async_smem();
    __syncwarp();
    if (lane == 0 && inside) {
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                         (uint64_t)map),
                     "r"(x), "r"(y), "r"(z), "r"(smem_u32(stage))
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// 16 columns of 32 fp32 lanes, one to a thread, as one box (32 lanes x 16 columns, no swizzle) written over the
// matrix or added to it. The add is one fp32 addition, rounded to nearest in L2 (subnormals kept), each
// element's only one of the call, so its result is that of the warp's own read, add and store. Those took 802 us
// on 8 experts' dW of 4096 x 2048 from 16 rows each, every read waiting for the store before it; this 104 (268 MB
// read and written: 79 at the copy rate).
__device__ __forceinline__ void store_box_f32(const float* v, int lane, uint8_t* stage, const CUtensorMap* map, int x,
                                              int y, int z, bool inside, bool add) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
    const uint32_t at = smem_u32(stage);
#pragma unroll
    for (int j = 0; j < 16; ++j) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 128 * j + 4 * lane), "f"(v[j]) : "memory");
    fence_async_smem();
    __syncwarp();
    if (lane == 0 && inside) {
        if (add)
            asm volatile(
                "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                    (uint64_t)map),
                "r"(x), "r"(y), "r"(z), "r"(at)
                : "memory");
        else
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                             (uint64_t)map),
                         "r"(x), "r"(y), "r"(z), "r"(at)
                         : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// ------------------------------------------------------------ ragged grouping
// Tables in shared memory: off[0..E], the first token row of each expert, and
// slices[0..E], the exclusive count of token slices of at most `width` rows.
// Validates m_e >= 0 and sum == M (each m_e is compared with M before it is
// added, so the sum cannot wrap) and returns a status bit mask. Called by all
// threads of the block; all of them wait for the stream and fetch counts, so
// that many experts cost one memory latency, then one warp sums them.
__device__ __forceinline__ int load_ragged(const int64_t* d_m_splits, int E, int64_t M, int width,
                                           int32_t* off, int32_t* slices) {
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    wait_for_stream();
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const int64_t v = d_m_splits[e];
        const bool fits = v >= 0 && v <= M;
        if (!fits) atomicOr(&s_bad, v < 0 ? MXQ_STATUS_SPLIT_NEGATIVE : MXQ_STATUS_SPLIT_SUM);
        off[e] = fits ? (int32_t)v : 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int64_t rows = 0, tiles = 0;  // totals of the experts before `base`, the same in every lane
        for (int base = 0; base < E; base += 32) {
            const int e = base + lane;
            const int64_t v = e < E ? off[e] : 0, t = (v + width - 1) / width;
            int64_t vs = v, ts = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t vu = __shfl_up_sync(0xffffffffu, vs, o), tu = __shfl_up_sync(0xffffffffu, ts, o);
                if (lane >= o) {
                    vs += vu;
                    ts += tu;
                }
            }
            if (e < E) {  // a wrong sum may not fit 32 bits: the caller stops on the status then
                off[e] = (int32_t)(rows + vs - v);
                slices[e] = (int32_t)(tiles + ts - t);
            }
            rows += __shfl_sync(0xffffffffu, vs, 31);
            tiles += __shfl_sync(0xffffffffu, ts, 31);
        }
        if (lane == 0) {
            off[E] = (int32_t)rows;
            slices[E] = (int32_t)tiles;
            if (rows != M) s_bad |= MXQ_STATUS_SPLIT_SUM;
        }
    }
    __syncthreads();
    return s_bad;
}

// The e with table[e] <= i < table[e + 1].
__device__ __forceinline__ int owner_of(const int32_t* table, int E, int32_t i) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (table[mid + 1] > i) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// A slice of an expert's rows: the expert's m rows, in units of `step` rows
// (the MMA's N granularity), are dealt evenly to ceil(m / width) slices, so a
// remainder of a few rows costs a few columns of MMA work and never a
// near-empty full tile.
struct Slice {
    int row, rows, n;  // first token row, rows of the expert in it, MMA N
};
__device__ __forceinline__ Slice slice_of(int off, int m, int count, int i, int step) {
    const int64_t units = (m + step - 1) / step;
    const int u0 = (int)(units * i / count), u1 = (int)(units * (i + 1) / count);
    Slice s;
    s.n = (u1 - u0) * step;
    s.row = off + u0 * step;
    s.rows = min(s.n, m - u0 * step);
    return s;
}

// One output tile: out[row0 + c][f0 + l] for accumulator column c, lane l.
struct Tile {
    int e;
    int f0;        // first output column (feature), on the MMA's M
    int c0;        // first row of the other operand: fprop, dgrad: a token row; wgrad: a row of dW[e]
    int cols;      // accumulator columns to store
    int n;         // MMA N
    int red0;      // wgrad: first token row of the sum
    int red;       // length of the sum
    int64_t row0;  // first output row
};

// The tiles of a product in the order in which a grid takes them: kFeat
// features by at most kWide columns, kWide's granularity kStep. `order` (wgrad)
// lists the experts, heaviest first.
template <int kMode, int kFeat, int kWide, int kStep>
struct Walk {
    int64_t N, K, total;
    int E, feats;  // tiles along the MMA's M
    int wide;      // wgrad: tiles along its N
    const int32_t *off, *slices, *order;

    __device__ Walk(int64_t N_, int64_t K_, int E_, const int32_t* off_, const int32_t* slices_, const int32_t* order_)
        : N(N_), K(K_), E(E_), off(off_), slices(slices_), order(order_) {
        feats = (int)(((kMode == kFprop ? N : K) + kFeat - 1) / kFeat);
        wide = (int)((N + kWide - 1) / kWide);
        total = kMode == kWgrad ? (int64_t)E * feats * wide : (int64_t)slices[E] * feats;
    }
    __device__ Tile get(int64_t t) const {
        Tile T;
        if (kMode == kWgrad) {
            const int per = feats * wide, r = (int)(t % per);
            T.e = order[t / per];
            T.f0 = r / wide * kFeat;
            T.c0 = r % wide * kWide;
            T.cols = (int)min((int64_t)kWide, N - T.c0);
            T.n = (T.cols + kStep - 1) / kStep * kStep;
            T.red0 = off[T.e];
            T.red = off[T.e + 1] - T.red0;
            T.row0 = T.e * N + T.c0;
        } else {
            // slices of an expert run fastest, so that the CTAs of one wave share its weight rows
            T.e = owner_of(slices, E, (int32_t)(t / feats));
            const int count = slices[T.e + 1] - slices[T.e];
            const int64_t r = t - (int64_t)slices[T.e] * feats;
            const Slice s = slice_of(off[T.e], off[T.e + 1] - off[T.e], count, (int)(r % count), kStep);
            T.f0 = (int)(r / count) * kFeat;
            T.c0 = s.row;
            T.cols = s.rows;
            T.n = s.n;
            T.red0 = 0;
            T.red = (int)(kMode == kDgrad ? N : K);
            T.row0 = s.row;
        }
        return T;
    }
};

// ------------------------------------------------------------ split sums
// A tile of 128 features by kFewRows columns whose sum is split over a cluster
// of kSplit CTAs: rank r gets columns [r * kOwn, + kOwn) of all partial sums
// and adds them in rank order. Buffers of alternate tiles: [2][kSplit] of 128
// lanes by kOwn columns, 32 KB for every kSplit. partf[2]: bytes received;
// parte[2]: arrivals of the owners' warps that have read what this CTA sent.
constexpr int kPartBytes = 2 * kFM * kFewRows * 4;

__device__ __forceinline__ void st_async(uint32_t cluster_dst, uint32_t cluster_bar, float a, float b, float c, float d) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(cluster_dst),
        "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)), "r"(__float_as_uint(d)),
        "r"(cluster_bar)
        : "memory");
}

template <int kSplit>
struct SplitSum {
    static constexpr int kOwn = kFewRows / kSplit, kPart = kFM * kOwn * 4;
    uint32_t buf, partf, parte;
    int rank;
    uint32_t tile = 0;

    __device__ SplitSum(uint32_t buf_, uint32_t partf_, uint32_t parte_, int rank_)
        : buf(buf_), partf(partf_), parte(parte_), rank(rank_) {}

    // v: this CTA's partial sums of lane l on entry, the whole sums of its kOwn columns in v[0 .. kOwn - 1]
    // on return. Called by the four warps that hold the 128 lanes; `first` is true in one of them; `again`: the
    // cluster has a tile after the next one, which fills this tile's buffer again. False when a bounded wait has
    // expired.
    __device__ bool exchange(float (&v)[kFewRows], int l, int lane, bool first, bool again, volatile int* abort_flag) {
        if constexpr (kSplit > 1) {
            const uint32_t side = tile & 1, phase = tile >> 1 & 1;
            ++tile;
            bool ok = mbar_wait_cluster(parte + 8 * side, phase ^ 1, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) return false;
            if (first && lane == 0) mbar_expect_tx(partf + 8 * side, (kSplit - 1) * kPart);
            const uint32_t mine = buf + (side * kSplit + rank) * kPart + l * kOwn * 4;
#pragma unroll
            for (int j = 0; j < kSplit; ++j)
                if (j != rank) {
                    const uint32_t dst = mapa(mine, j), bar = mapa(partf + 8 * side, j);
#pragma unroll
                    for (int i = 0; i < kOwn; i += 4)
                        st_async(dst + 4 * i, bar, v[j * kOwn + i], v[j * kOwn + i + 1], v[j * kOwn + i + 2],
                                 v[j * kOwn + i + 3]);
                }
            float own[kOwn];
#pragma unroll
            for (int j = 0; j < kSplit; ++j)
#pragma unroll
                for (int i = 0; i < kOwn; ++i) own[i] = j == 0 || j == rank ? v[j * kOwn + i] : own[i];
            ok = mbar_wait_cluster(partf + 8 * side, phase, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) return false;
#pragma unroll
            for (int j = 0; j < kSplit; ++j) {
                const uint32_t src = buf + (side * kSplit + j) * kPart + l * kOwn * 4;
#pragma unroll
                for (int i = 0; i < kOwn; i += 4) {
                    float4 a = make_float4(own[i], own[i + 1], own[i + 2], own[i + 3]);
                    if (j != rank)
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w)
                                     : "r"(src + 4 * i)
                                     : "memory");
                    v[i] = j ? __fadd_rn(v[i], a.x) : a.x;
                    v[i + 1] = j ? __fadd_rn(v[i + 1], a.y) : a.y;
                    v[i + 2] = j ? __fadd_rn(v[i + 2], a.z) : a.z;
                    v[i + 3] = j ? __fadd_rn(v[i + 3], a.w) : a.w;
                }
            }
            __syncwarp();
            if (again && lane == 0)
                for (int j = 0; j < kSplit; ++j)
                    if (j != rank) arrive_remote_release(mapa(parte + 8 * side, j));
        }
        return true;
    }
};

// ------------------------------------------------------------ tile queue
// A grid of one cluster per tile, most of which never start: a cluster that
// has a tile in hand takes the next one from the hardware's queue of clusters
// not yet launched (clusterlaunchcontrol). So tiles of uneven cost go to
// whichever SMs are free, with no counter in memory. One warp of a pair's rank
// 0 asks; the answer arrives in both CTAs. It asks when every warp has taken
// the last answer, that is while the tile before is being computed, so a
// cluster holds one tile more than it works on.
struct TileQueue {
    uint32_t answer, ready, taken;  // 16 bytes; barrier of this CTA; barrier of rank 0 (cluster address)
    uint32_t phase = 0;
    enum Result { kDone = 0, kTile = 1, kAbort = 2 };

    __device__ TileQueue(uint32_t answer_, uint32_t ready_, uint32_t taken_)
        : answer(answer_), ready(ready_), taken(taken_) {}

    // The next tile of this cluster, for a whole warp.
    __device__ Result next(int64_t& tile, int lane, volatile int* abort_flag) {
        const bool ok = mbar_wait(ready, phase, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) return kAbort;
        phase ^= 1;
        uint32_t valid, first;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t.reg .b32 y, z, w;\n\t"
            "ld.shared.b128 a, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t"
            "mov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, a;\n\t}"
            : "=&r"(valid), "=&r"(first)
            : "r"(answer)
            : "memory");
        fence_async_smem();  // read before the next answer is written
        __syncwarp();
        if (lane == 0) arrive_remote(taken);
        tile = first / 2;
        return valid ? kTile : kDone;
    }
    // Asks for the next cluster; the answer goes to `answer` and `ready` of both CTAs.
    __device__ void ask() const {
        asm volatile(
            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 "
            "[%0], [%1];" ::"r"(answer),
            "r"(ready)
            : "memory");
    }
};

// On a bounded wait's expiry: wait, again at most about 2 s each, for the last
// fills of the ring, so that no copy is in flight when the block ends.
__device__ __forceinline__ void drain_ring(uint32_t full0, int stages, int64_t fills) {
    volatile int unused = 0;
    for (int64_t i = fills > stages ? fills - stages : 0; i < fills; ++i)
        mbar_wait(full0 + 8 * (int)(i % stages), (uint32_t)(i / stages) & 1, &unused);
}

// ------------------------------------------------------------------ host side
// Launches a kernel of clusters of kCG CTAs: one cluster per tile for a kernel
// with a TileQueue, otherwise as many as fit the device and no more than
// `tiles`. The kernel's attribute and co-residency are set and asked for once
// per device.
template <int kCG, bool kQueue, auto kKernel, class... Args>
static cudaError_t launch_persistent(int threads, int smem_max, int smem, int64_t tiles, cudaStream_t s,
                                     const Args&... args) {
    static std::atomic<int> cache[64];
    int dev = 0, most = 0;
    cudaGetDevice(&dev);
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCG;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(threads);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (dev >= 64 || (most = cache[dev].load(std::memory_order_acquire)) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_max);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(kCG * (sm_count() / kCG));
        cfg.dynamicSmemBytes = smem_max;
        if (cudaOccupancyMaxActiveClusters(&most, (void*)kKernel, &cfg) != cudaSuccess || most <= 0) {
            cudaGetLastError();
            most = sm_count() / kCG;
        }
        if (dev < 64) cache[dev].store(most, std::memory_order_release);
    }
    cfg.numAttrs = 2;
    if (!kQueue) tiles = std::min<int64_t>(tiles, most);
    if (tiles > ((int64_t)1 << 30) / kCG) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)(kCG * std::max<int64_t>(1, tiles)));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kKernel, args...);
}

// Launches a kernel that begins with wait_for_stream().
template <class... Params, class... Args>
static cudaError_t launch(void (*kernel)(Params...), unsigned grid, unsigned threads, cudaStream_t s, int smem,
                          Args... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace ragged
}  // namespace mxq
