// mxq_ragged_swiglu.cuh -- SwiGLU in the epilogues of the ragged bf16 products
// (mxq_ragged.cu, mxq_ragged_few.cu).
//
// fprop, [g | u] = X W1^T + b1, h = silu(g) u. The rows of W1 come onto the
// MMA's M in blocks of eight, eight of the gate and then the same eight of up
// (one tensor map of five dimensions does that), so a matrix fragment holds g
// and u of a feature in the same thread, and h is made from the sums before
// they are rounded. A tile has half as many features of h as it has lanes.
//
// dgrad, dh = dY W2 and the gradient [dg | du] of the saved [g | u]: dh stays in
// the accumulator; the tile's part of [g | u] is read as rows, 64 contiguous
// bytes to four lanes, and passes through the warp's stage into the fragments'
// layout. The first 32 columns' part is read while the sums are made, the next
// ones' while the ones before are computed.
//
// The fp32 steps of SwiGLU are those of mxq_common.cuh; every result is rounded
// to bf16 once.
#pragma once

#include "mxq_ragged.cuh"

namespace mxq {
namespace ragged {

constexpr int kGateRows = 8;  // consecutive lanes of gate features, and then of up features

__device__ __forceinline__ void load_5d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int chunk, int e) {
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %4, "
        "%5, %6}], [%2];" ::"r"(dst),
        "l"((uint64_t)map), "r"(bar), "r"(x), "r"(0), "r"(chunk), "r"(e)
        : "memory");
}
__device__ __forceinline__ void load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int chunk, int e) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %4, %5, "
        "%6}], [%2];" ::"r"(dst),
        "l"((uint64_t)map), "r"(bar), "r"(x), "r"(0), "r"(chunk), "r"(e)
        : "memory");
}
// W1 (E, 2F, K) for them: rows of 64 elements of 8 gate features, the same 8 of up, the next 8, ...
static inline bool encode_gate_up(CUtensorMap* m, const void* w, int64_t E, int64_t F, int64_t K, int chunks) {
    const int64_t d[5] = {K, kGateRows, 2, F / kGateRows, E};
    const int64_t s[4] = {2 * K, 2 * K * F, 2 * K * kGateRows, 4 * K * F};
    const int box[5] = {64, kGateRows, 2, chunks, 1};
    return encode_tmap(m, w, 2, 5, d, s, box);
}

// rows of 64 bytes of a warp's stage, their 16-byte pieces exchanged by the row's bits 1 and 2
__device__ __forceinline__ uint32_t stage_piece(uint32_t stage, int row, int piece) {
    return stage + row * 64 + ((piece ^ (row >> 1 & 3)) << 4);
}
__device__ __forceinline__ void st_shared(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
// 32 rows of 32 bf16 (four lanes' 16-byte pieces) -> fragments [8-column block][8-lane block]
__device__ __forceinline__ void rows_to_fragments(const uint4 (&rows)[4], uint32_t stage, int lane, uint32_t (&w)[4][4]) {
    __syncwarp();  // the stage's last reads are done
#pragma unroll
    for (int i = 0; i < 4; ++i) st_shared(stage_piece(stage, i * 8 + (lane >> 2), lane & 3), rows[i]);
    __syncwarp();
#pragma unroll
    for (int b = 0; b < 4; ++b) ldmatrix_trans(stage_piece(stage, 8 * b + (lane & 7), lane >> 3), w[b]);
}
// Fragments -> rows at out + column * ld, lanes < live and columns < cols
__device__ __forceinline__ void fragments_to_rows(const uint32_t (&w)[4][4], uint32_t stage, int lane, __nv_bfloat16* out,
                                                  int64_t ld, int live, int cols) {
    __syncwarp();
#pragma unroll
    for (int b = 0; b < 4; ++b) stmatrix_trans(stage_piece(stage, 8 * b + (lane & 7), lane >> 3), w[b]);
    __syncwarp();
    const int piece = lane & 3;
    if (piece * 8 < live)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = i * 8 + (lane >> 2);
            if (c < cols) *reinterpret_cast<uint4*>(out + c * ld + piece * 8) = ld_shared(stage_piece(stage, c, piece));
        }
}
__device__ __forceinline__ float2 bf16x2_values(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }

// fprop: columns 0 .. 31 of the accumulator lanes at tmem, 16 features of h. bg, bu: the biases of features lane / 4 and
// lane / 4 + 8. To h + column * F and, if y is not null, y + column * 2F (gate) and F further (up), for features < live
// and columns < cols.
__device__ __forceinline__ void store_swiglu(uint32_t tmem, int lane, uint32_t stage, __nv_bfloat16* h, __nv_bfloat16* y,
                                             int64_t F, int live, int cols, const float (&bg)[2], const float (&bu)[2]) {
    uint32_t v[2][16], hw[4][2], gu[4][4];  // [8-column block][8-feature block], of y: gate blocks, then up blocks
    load_columns(tmem, v);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t* r = &v[k][4 * b];
            const float2 g = make_float2(__fadd_rn(__uint_as_float(r[0]), bg[k]), __fadd_rn(__uint_as_float(r[1]), bg[k]));
            const float2 u = make_float2(__fadd_rn(__uint_as_float(r[2]), bu[k]), __fadd_rn(__uint_as_float(r[3]), bu[k]));
            const float2 o = swiglu_h_x2(g, u);
            hw[b][k] = bf16x2_bits(o.x, o.y);
            gu[b][k] = bf16x2_bits(g.x, g.y);
            gu[b][2 + k] = bf16x2_bits(u.x, u.y);
        }
    if (y) {
        // rows of 64 bytes: 16 gate features, then 16 up features
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 4; ++b) stmatrix_trans(stage_piece(stage, 8 * b + (lane & 7), lane >> 3), gu[b]);
        __syncwarp();
        const int piece = lane & 3, f = (piece & 1) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = i * 8 + (lane >> 2);
            if (f < live && c < cols)
                *reinterpret_cast<uint4*>(y + c * 2 * F + (piece >> 1) * F + f) = ld_shared(stage_piece(stage, c, piece));
        }
    }
    // rows of 32 bytes, two side by side: columns c and c + 16
    __syncwarp();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint32_t w[4] = {hw[b][0], hw[b][1], hw[b + 2][0], hw[b + 2][1]};
        stmatrix_trans(stage_piece(stage, 8 * b + (lane & 7), lane >> 3), w);
    }
    __syncwarp();
    const int piece = lane & 3, f = (piece & 1) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = i * 8 + (lane >> 2), c = row + 16 * (piece >> 1);
        if (f < live && c < cols) *reinterpret_cast<uint4*>(h + c * F + f) = ld_shared(stage_piece(stage, row, piece));
    }
}

// dgrad: columns 0 .. 31 of 32 accumulator lanes at tmem are dh; gate, up: the rows of [g | u] (load_rows_bf16). To
// d + column * 2F (dg) and F further (du) and, if h is not null, silu(g) u to h + column * F, for lanes < live and
// columns < cols. `next()` is called when gate and up have been read.
template <class F_>
__device__ __forceinline__ void store_swiglu_grads(uint32_t tmem, int lane, uint32_t stage, uint4 (&gate)[4], uint4 (&up)[4],
                                                   __nv_bfloat16* d, __nv_bfloat16* h, int64_t F, int live, int cols,
                                                   F_ next) {
    uint32_t v[2][16], g[4][4], u[4][4];
    rows_to_fragments(gate, stage, lane, g);
    rows_to_fragments(up, stage, lane, u);
    next();
    load_columns(tmem, v);
    if (h) {
        uint32_t w[4][4];
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 o = swiglu_h_x2(bf16x2_values(g[b][k]), bf16x2_values(u[b][k]));
                w[b][k] = bf16x2_bits(o.x, o.y);
            }
        fragments_to_rows(w, stage, lane, h, F, live, cols);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = 4 * b + 2 * (k & 1);
            const float2 dh = make_float2(__uint_as_float(v[k >> 1][r]), __uint_as_float(v[k >> 1][r + 1]));
            float2 dg, du;
            swiglu_grads_x2(dh, bf16x2_values(g[b][k]), bf16x2_values(u[b][k]), dg, du);
            g[b][k] = bf16x2_bits(dg.x, dg.y);
            u[b][k] = bf16x2_bits(du.x, du.y);
        }
    fragments_to_rows(g, stage, lane, d, 2 * F, live, cols);
    fragments_to_rows(u, stage, lane, d + F, 2 * F, live, cols);
}

}  // namespace ragged
}  // namespace mxq
