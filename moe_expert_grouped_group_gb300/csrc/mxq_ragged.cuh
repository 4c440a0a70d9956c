// mxq_ragged.cuh -- what the ragged grouped products (mxq_ragged.cu, bf16;
// mxq_ragged_int8.cu, int8) share: the tables of a ragged grouping, the tile
// walk and the tcgen05 wrappers for 16-bit floating operands.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mxq_common.cuh"
#include "mxq_ragged.h"

namespace mxq {
namespace ragged {

constexpr int kFM = 128;        // MMA M: rows of A (weight features) per CTA
constexpr int kBoxBytes = 128;  // inner extent of every operand box: the 128-byte swizzle span

// ------------------------------------------------------------ PTX wrappers
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
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(id), "r"(accum)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(dst),
        "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
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
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// ------------------------------------------------------------ ragged grouping
// Tables in shared memory: off[0..E], the first token row of each expert, and
// slices[0..E], the exclusive count of token slices of at most `width` rows.
// Validates m_e >= 0 and sum == M (each m_e is compared with M before it is
// added, so the sum cannot wrap) and returns a status bit mask. Called by all
// threads of the block; all of them fetch counts, so that many experts cost
// one memory latency, then one warp sums them.
__device__ __forceinline__ int load_ragged(const int64_t* __restrict__ d_m_splits, int E, int64_t M, int width,
                                           int32_t* off, int32_t* slices) {
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
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

// A slice of an expert's rows: the expert's m rows are cut evenly into
// ceil(m / width) slices, each a multiple of `step` rows wide (the MMA's N
// granularity) but the last, so a remainder of a few rows costs a few columns
// of MMA work spread over all slices and never a near-empty full tile.
struct Slice {
    int row, rows, n;  // first token row, rows of the expert in it, MMA N
};
__device__ __forceinline__ Slice slice_of(int off, int m, int count, int i, int step) {
    const int even = (m + count - 1) / count;
    Slice s;
    s.n = (even + step - 1) / step * step;
    s.row = off + i * s.n;
    s.rows = min(s.n, m - i * s.n);
    return s;
}

// One output tile.
struct Tile {
    int e;
    int f0;    // first feature on the MMA's M
    int c0;    // fprop, dgrad: first token row; wgrad: first column of dW
    int cols;  // columns to store
    int n;     // MMA N
    int red0;  // wgrad: first token row of the sum
    int red;   // length of the sum
};

// The tiles of a product in the order in which a grid takes them, kWide the
// widest MMA N.
template <int kMode, int kWide>
struct Walk {
    int64_t N, K, total;
    int E, feats;  // tiles along the MMA's M
    int wide;      // wgrad: tiles along its N
    const int32_t *off, *slices;

    __device__ Walk(int64_t N_, int64_t K_, int E_, const int32_t* off_, const int32_t* slices_)
        : N(N_), K(K_), E(E_), off(off_), slices(slices_) {
        feats = (int)(((kMode == kDgrad ? K : N) + kFM - 1) / kFM);
        wide = (int)((K + kWide - 1) / kWide);
        total = kMode == kWgrad ? (int64_t)E * feats * wide : (int64_t)slices[E] * feats;
    }
    __device__ Tile get(int64_t t) const {
        Tile T;
        if (kMode == kWgrad) {
            const int per = feats * wide, r = (int)(t % per);
            T.e = (int)(t / per);
            T.f0 = r / wide * kFM;
            T.c0 = r % wide * kWide;
            T.cols = (int)min((int64_t)kWide, K - T.c0);
            T.n = (T.cols + 15) / 16 * 16;
            T.red0 = off[T.e];
            T.red = off[T.e + 1] - T.red0;
        } else {
            // slices of an expert run fastest, so that the CTAs of one wave share its weight rows
            T.e = owner_of(slices, E, (int32_t)(t / feats));
            const int count = slices[T.e + 1] - slices[T.e];
            const int64_t r = t - (int64_t)slices[T.e] * feats;
            const Slice s = slice_of(off[T.e], off[T.e + 1] - off[T.e], count, (int)(r % count), 16);
            T.f0 = (int)(r / count) * kFM;
            T.c0 = s.row;
            T.cols = s.rows;
            T.n = s.n;
            T.red0 = 0;
            T.red = (int)(kMode == kDgrad ? N : K);
        }
        return T;
    }
};

// On a bounded wait's expiry: wait, again at most about 2 s each, for the last
// fills of the ring, so that no copy is in flight when the block ends.
__device__ __forceinline__ void drain_ring(uint32_t full0, int stages, int64_t fills) {
    volatile int unused = 0;
    for (int64_t i = fills > stages ? fills - stages : 0; i < fills; ++i)
        mbar_wait(full0 + 8 * (int)(i % stages), (uint32_t)(i / stages) & 1, &unused);
}

}  // namespace ragged
}  // namespace mxq
