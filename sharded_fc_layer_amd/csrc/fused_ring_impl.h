// The ring kernel's main loop (gemm_w4_ring_impl.h: 256 x BN block tiles, one
// wave per SIMD, 64-value stages through three A and two B tiles of LDS) under
// the fused operators' epilogues. Built per epilogue in fused_ring_*.hip, each
// through fused_ring_table.inc. KIND and VEC: see ring_elementwise.
//
// Bound by the matrix units and the epilogue that follows them, since a block
// has its CU to itself: 8192 x 2048 x 8192 with a bias, gelu by tanh and Z kept
// takes 229 us, 1200 TFLOP/s (a tile: 72 thousand cycles of main loop, 24 of
// epilogue); the statistics of 8192 x 16384 x 16032 2.8 ms, 1530 TFLOP/s.
#pragma once

#include "fused_ring_epilogue.h"
#include "gemm_w4_common.h"

// Each operand's descriptor starts at the block's tile (and at its group's
// matrix or rows) and ends with the last row that the tile may read, so that
// only one tile's rows, or one group's, have to lie within 2 GiB.
#define FCR_SETUP                                                                                                   \
    const TilePos pos = tile_position<256, BN, GRP>(g);                                                             \
    if (!pos.any) return; /* the whole block */                                                                     \
    W4Setup w;                                                                                                      \
    w.lane = threadIdx.x & 63;                                                                                      \
    w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);                                                      \
    w.wm0 = (w.wave >> 1) * 128;                                                                                    \
    w.wn0 = (w.wave & 1) * (BN / 2);                                                                                \
    w.slice = 0, w.m0 = 0, w.n0 = 0;                                                                                \
    w.kbeg = 0, w.kend = pos.kend - pos.kbeg;                                                                       \
    w.nkt = (int)((w.kend + BKP - 1) / BKP);                                                                        \
    const int64_t a0_ = pos.row0 + pos.m0, rows_ = pos.M - pos.m0 < 256 ? pos.M - pos.m0 : 256;                     \
    const int64_t cols_ = g.N - pos.n0 < BN ? g.N - pos.n0 : BN;                                                    \
    const uint16_t* pa_ = g.A + (A_OC ? pos.kbeg * g.lda + a0_ : a0_ * g.lda + pos.kbeg);                           \
    const uint16_t* pb_ = g.B + (GRP == GRP_ROWS ? (int64_t)pos.e * g.b_stride : 0) +                               \
                          (B_OC ? pos.kbeg * g.ldb + pos.n0 : pos.n0 * g.ldb + pos.kbeg);                           \
    w.ra = __builtin_amdgcn_make_buffer_rsrc(                                                                       \
        (void*)pa_, 0, (int)(2 * (A_OC ? w.kend * g.lda - a0_ : rows_ * g.lda - pos.kbeg)), kRsrcWord3);            \
    w.rb = __builtin_amdgcn_make_buffer_rsrc(                                                                       \
        (void*)pb_, 0, (int)(2 * (B_OC ? w.kend * g.ldb - pos.n0 : cols_ * g.ldb - pos.kbeg)), kRsrcWord3);
#define FCR_ROWS (pos.M - pos.m0)
#define FCR_COLS (g.N - pos.n0)
#define FCR_SHORT (GRP == GRP_RED)
#define FCR_EPILOGUE ring_epilogue<MODE, GRP, TN, KIND, VEC>(g, pos, wave >> 1, wave & 1, lane, acc, stage);

namespace fcs {
namespace {

template <EpiMode MODE, GroupMode GRP, bool A_OC, bool B_OC, int BN, int HEAD, int NA, int KIND, bool VEC>
__global__ __launch_bounds__(kW4Threads) __attribute__((amdgpu_waves_per_eu(1, 1))) void fused_ring_kernel(
    FusedArgs g) {
    constexpr bool STAMP = false;
#include "gemm_w4_ring_body.inc"
}

}  // namespace
}  // namespace fcs
