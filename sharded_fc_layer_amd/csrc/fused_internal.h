// Internal interface between the fused operators' C ABI (fused_api.hip) and
// their gfx950 kernels. Not installed, not part of the ABI.
#pragma once

#include "fcshard.h"
#include "fcshard_internal.h"

namespace fcs {

// FC_OK when the current device is a gfx950 (defined in fcshard_api.hip).
fc_status current_device_status();

// What a product does with its fp32 results.
enum EpiMode : int {
    EPI_STORE = 0,  // C = v, or C += v (fp32), or a split slice's partial plane
    EPI_ACT = 1,    // z = v + bias; Z = z; C = act(z) + R
    EPI_DACT = 2,   // C = v * act'(Z); column sums of C per block of rows
    EPI_STATS = 3,  // per row and block of columns: maximum and sum of exponentials; the target's value
    EPI_DLOGIT = 4, // C = w / s (exp(v - lse) - [column = target]), s of weight_scale
    EPI_GLU = 5,    // z = v + bias over 2 N columns [gate | up]; Z = z; C = act(gate) * up, N columns
    EPI_DGLU = 6,   // C = [v * up * act'(gate) | v * act(gate)], 2 N columns, Z = [gate | up]; Y = act(gate) * up; column sums of C
    EPI_LOGITS = 7, // per row and block of columns: maximum, sum of exponentials, their mean logit; C = v or none; the target's value
    kNumEpiModes = 8
};

// Which rows a product's tiles cover.
enum GroupMode : int {
    GRP_NONE = 0,  // one product
    GRP_ROWS = 1,  // rows offsets[e] .. offsets[e + 1] - 1 of A and C take matrix e of B
    GRP_RED = 2,   // C matrix e reduces over rows offsets[e] .. offsets[e + 1] - 1 of A and B
};

// One product with its epilogue, in kernel terms (see GemmArgs). Only the
// fields of the launch's modes are read.
struct FusedArgs : GemmArgs {
    // one past the last value of each operand that may be read (set by launch_fused)
    const uint16_t* a_end = nullptr;
    const uint16_t* b_end = nullptr;
    int out_f32 = 0;      // C is fp32 (else bf16)
    int vec_out = 0;      // ring kernel: the rows of C, R, Y and Z start on 16-byte boundaries, N is a multiple of 8
    int act = 0;          // fc_act
    const uint16_t* bias = nullptr;  // N values, or none
    const uint16_t* R = nullptr;     // M x N, or none
    uint16_t* Z = nullptr;           // EPI_ACT: written, or none; EPI_DACT: read
    float* colpart = nullptr;        // EPI_DACT: column sums, one row of N per block of rows, or none
    const int64_t* targets = nullptr;
    int64_t v0 = 0;       // vocabulary index of column 0
    int64_t ignore = 0;   // target of a row that takes no part
    const float* lse = nullptr;
    const float* gw = nullptr;       // EPI_DLOGIT: the rows' weights
    float* wscale = nullptr;         // EPI_DLOGIT: s, written; EPI_STORE: a factor of v, or none
    float* stat = nullptr;           // EPI_STATS: [block of columns][M] maxima, then as many sums
    float* tlogit = nullptr;
    float inv_t = 1.0f;              // EPI_DLOGIT, EPI_LOGITS: one over the temperature, a factor of the logits
    const uint32_t* need = nullptr;  // EPI_LOGITS, ring kernel: bit p % 32 of need[p / 32][row]: the logits of part p are read (none: all)
    uint16_t* Y = nullptr;           // EPI_DGLU: M x N, written, or none
    int stagger = 0;      // ring kernel: how far the four phases of the first blocks start apart, in 10 ns
    const int64_t* offsets = nullptr;  // E + 1 values on the device
    int E = 1;
    int64_t T = 0;        // rows that offsets may reach
    int64_t b_stride = 0, c_stride = 0;  // elements between the groups' matrices of B (GRP_ROWS), of C (GRP_RED)
};

// General kernel (fused_gemm.hip): block tiles kFusedTiles[tile], any M, N and
// K >= 0, operands at any element's address. Where the rows of both start on
// 16-byte boundaries (lda, ldb multiples of 8, aligned bases) they go straight
// into LDS; a reduction-contiguous operand then has zeros from K to the next
// multiple of 8, which the ring kernel needs too.
struct FusedTile {
    int bm, bn, wave_rows, wave_cols;  // the 4 waves' grid within the tile
};
constexpr int kNumFusedTiles = 4;
constexpr int kRingTile = 2;  // the ring kernel's tile: see ring_takes
extern const FusedTile kFusedTiles[kNumFusedTiles];
typedef void (*FusedFn)(FusedArgs);
// The general kernel's instances (fused_gemm_*.hip) by way of loading; nullptr
// for a combination that no operator uses.
template <bool ANY>
FusedFn fused_kernel(EpiMode mode, GroupMode grp, int tile, bool a_oc, bool b_oc);
template <>
FusedFn fused_kernel<false>(EpiMode mode, GroupMode grp, int tile, bool a_oc, bool b_oc);
template <>
FusedFn fused_kernel<true>(EpiMode mode, GroupMode grp, int tile, bool a_oc, bool b_oc);
// The ring kernel's (fused_ring_*.hip), 256 x 256 block tiles: one product, or
// an expert layer's (EPI_STORE).
template <EpiMode MODE, int KIND>
FusedFn fused_ring(int head, bool vec, bool a_oc, bool b_oc);
template <int KIND>
FusedFn fused_ring_grouped(GroupMode grp, int head, bool vec, bool b_oc);
#define FCU_DECLARE_RING(MODE, KIND) \
    template <>                      \
    FusedFn fused_ring<MODE, KIND>(int head, bool vec, bool a_oc, bool b_oc);
FCU_DECLARE_RING(EPI_STORE, 0)
FCU_DECLARE_RING(EPI_STORE, 1)
FCU_DECLARE_RING(EPI_ACT, 0)
FCU_DECLARE_RING(EPI_ACT, 1)
FCU_DECLARE_RING(EPI_ACT, 2)
FCU_DECLARE_RING(EPI_DACT, 0)
FCU_DECLARE_RING(EPI_DACT, 1)
FCU_DECLARE_RING(EPI_DACT, 2)
FCU_DECLARE_RING(EPI_STATS, 0)
FCU_DECLARE_RING(EPI_DLOGIT, 0)
FCU_DECLARE_RING(EPI_LOGITS, 0)
FCU_DECLARE_RING(EPI_LOGITS, 1)
FCU_DECLARE_RING(EPI_GLU, 0)
FCU_DECLARE_RING(EPI_GLU, 1)
FCU_DECLARE_RING(EPI_GLU, 2)
FCU_DECLARE_RING(EPI_DGLU, 0)
FCU_DECLARE_RING(EPI_DGLU, 1)
FCU_DECLARE_RING(EPI_DGLU, 2)
#undef FCU_DECLARE_RING
template <>
FusedFn fused_ring_grouped<0>(GroupMode grp, int head, bool vec, bool b_oc);
template <>
FusedFn fused_ring_grouped<1>(GroupMode grp, int head, bool vec, bool b_oc);

// Whether the ring kernel can run a product: an output-contiguous operand has
// to lie within 2 GiB, as do 256 rows of a reduction-contiguous one and 128 of
// the output; without ragged reductions, at least one whole stage of 64 values.
bool ring_takes(GroupMode grp, bool a_oc, bool b_oc, int64_t N, int64_t K, int64_t lda, int64_t ldb);
hipError_t launch_fused(EpiMode mode, GroupMode grp, int tile, bool a_oc, bool b_oc, const FusedArgs& g,
                        hipStream_t s);

// EPI_ACT, EPI_GLU (at most 32 rows) and EPI_LOGITS (16; parts of 32 columns), both operands reduction-contiguous (fused_skinny.hip)
hipError_t launch_fused_skinny(const FusedArgs& g, hipStream_t s);
hipError_t launch_fused_skinny_glu(const FusedArgs& g, hipStream_t s);
hipError_t launch_fused_skinny_logits(const FusedArgs& g, hipStream_t s);

// dst (rows x ld) = src (rows x cols) with zeros in columns cols .. ld - 1;
// any cols and src alignment; ld a multiple of 8, dst 16-byte aligned.
// rows = 0: no copy.
struct PadCopy {
    const uint16_t* src;
    uint16_t* dst;
    int64_t rows, cols, ld;
};
hipError_t launch_pad_any(const PadCopy& a, const PadCopy& b, hipStream_t s);

// out[j] = sum over p < parts of part[p * N + j], in that order
hipError_t launch_colsum_parts(const float* part, float* out, int64_t N, int parts, hipStream_t s);

// The epilogue of a split reduction: v = sum of the slices' planes (M rows of
// pld values, a multiple of 4) in order, then what `mode` says.
hipError_t launch_split_epilogue(EpiMode mode, const FusedArgs& g, const float* planes, int64_t pld, int splits,
                                 hipStream_t s);
// rows of its column-sum partials (EPI_DACT); its blocks of columns (EPI_STATS)
int split_epilogue_parts(int64_t M);
int split_stats_parts(int64_t N);

// dZ = dY * act'(Z) (dZ and Z may be none) and the column sums of the products
hipError_t launch_act_bwd(const uint16_t* dY, const uint16_t* Z, int act, uint16_t* dZ, float* part, int64_t M,
                          int64_t N, int parts, hipStream_t s);

// lse, target value and loss of every row from EPI_STATS' partials
hipError_t launch_xent_finish(const float* stat, int parts, const int64_t* targets, int64_t v0, int64_t ignore,
                              int64_t M, int64_t N, float* lse, float* tlogit, float* loss, hipStream_t s);

// ---- gated layers (fused_glu.hip)

// The epilogues of gated products from the planes of a plain one (EPI_GLU: of
// 2 N columns). EPI_DGLU leaves split_epilogue_parts(M) rows of 2 N column sums.
hipError_t launch_split_glu(EpiMode mode, const FusedArgs& g, const float* planes, int64_t pld, int splits,
                            hipStream_t s);
// dZ = [dY * up * act'(gate) | dY * act(gate)] and Y = act(gate) * up from Z =
// [gate | up] (dZ and Y may be none), and the column sums of dZ in glu_bwd_parts rows
int glu_bwd_parts(int64_t M, int64_t N);
hipError_t launch_glu_bwd(const uint16_t* dY, const uint16_t* Z, int act, uint16_t* dZ, uint16_t* Y, float* part,
                          int64_t M, int64_t N, hipStream_t s);

// ---- the vocabulary's logits (fused_vocab.hip)

// EPI_LOGITS from the planes of a plain product: the sum of a row's planes
// goes to plane 0, the statistics of each kLogitCols columns to g.stat.
constexpr int kLogitCols = 256;
hipError_t launch_row_logits(const FusedArgs& g, float* planes, int64_t pld, int splits, hipStream_t s);

// M rows of logits with their statistics (EPI_LOGITS: 3 x parts x M values,
// `width` columns to a part, a power of two from 32 to 256).
struct RowLogits {
    const float* z;  // M x ld, or none
    int64_t ld;
    const float* stat;
    int parts, width;
    int64_t M, N, v0;
    float inv_t;
};
constexpr int kMaxTop = 128;  // most alternatives and most listed tokens of a row

// What fc_logprob returns of these rows.
struct LogprobOut {
    const int64_t* targets;  // or none
    int64_t ignore;
    const float* tlogit;
    float *logp, *entropy, *lse, *top_logp;  // logp and entropy may be none
    int64_t* top_ids;
    int k;
};
hipError_t launch_logprob_finish(const RowLogits& r, const LogprobOut& o, hipStream_t s);

// A teacher's n listed tokens of each row.
struct Listed {
    const int64_t* ids;      // M x n
    const float* tlogits;    // M x n
    int n;
    const float* slogits;    // M x n: the student's logits there
    const float* p;          // M x n (launch_listed_prep)
};
// need[p / 32][row], a bit for each part of `width` columns (FusedArgs::need): where the listed tokens lie
hipError_t launch_listed_need(const Listed& t, int64_t M, int64_t N, int64_t v0, int width, int parts, uint32_t* need,
                              hipStream_t s);
hipError_t launch_distill_finish(const RowLogits& r, const Listed& t, float* lse, float* slogits, float* loss,
                                 hipStream_t s);
// For the gradient: p = the listed tokens' probabilities, a token's summed at
// its first place (-1 at the others and where none is); gw = grad / T; targets
// = -1 in rows that count, INT64_MIN in the others.
hipError_t launch_listed_prep(const Listed& t, const float* grad, float inv_t, int64_t M, float* p, float* gw,
                              int64_t* targets, hipStream_t s);
// Columns v0 .. v0 + c - 1 of D (bf16, rows of ld) at the listed tokens:
// gw / *scale (exp(z / T - lse) - p).
hipError_t launch_listed_grad(const Listed& t, const float* lse, const float* gw, float inv_t, const float* scale,
                              uint16_t* D, int64_t ld, int64_t v0, int64_t c, int64_t M, hipStream_t s);

// The two gradients of a loss over a vocabulary projection (fused_api.hip):
// D = gw (exp(z / T - lse) - [column = target]), and at the listed tokens as above.
struct LogitsBwd {
    const void *X, *W;
    int w_order;
    const int64_t* targets;
    int64_t v0, ignore;
    const float *lse, *gw;
    float inv_t = 1.0f;
    const Listed* listed = nullptr;
    void *dX, *dW;
    int dx_f32, dw_dtype;
    int64_t M, K, N;
};
int64_t logits_bwd_ws_bytes(int64_t M, int64_t K, int64_t N, int w_order, bool aligned);
hipError_t run_logits_bwd(const LogitsBwd& b, char* ws, hipStream_t s);

}  // namespace fcs
