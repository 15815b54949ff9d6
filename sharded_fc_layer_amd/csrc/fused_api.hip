// C ABI of the fused operators: argument checks, the choice of kernel and
// workspace layout for each product, and the launches.
//
// Every plan here is a function of sizes, orders, types and operand alignment
// alone, so that the workspace queries and the calls agree. Nothing is
// allocated, kept or synchronized: workspaces are the caller's.
#include <algorithm>
#include <initializer_list>

#include "fused_internal.h"

namespace fcs {
namespace {

constexpr int64_t kMaxSize = (int64_t)1 << 22;   // largest M, K, N, T: 128 rows of it stay within 2 GiB
constexpr int64_t kMaxCount = (int64_t)1 << 46;  // largest element count of the experts' weights
constexpr int kMaxExperts = 1 << 20;

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

bool bad_order(int o) { return o != FC_ROW_MAJOR && o != FC_COL_MAJOR; }
bool bad_act(int a) { return a < FC_ACT_NONE || a > FC_ACT_SILU; }
bool bad_size(int64_t v) { return v < 1 || v > kMaxSize; }

struct Span {
    const void* p;
    int64_t bytes;
};
bool meets(const Span& a, const Span& b) {
    if (!a.p || !b.p) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}
// outputs must not meet each other or an input
bool overlapping(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& i : ins)
            if (meets(*o, i)) return true;
        for (auto q = o + 1; q != outs.end(); ++q)
            if (meets(*o, *q)) return true;
    }
    return false;
}
bool off(const void* p, int64_t a) { return (uintptr_t)p % (uintptr_t)a != 0; }

// An operand as the kernels read it: in place, or, where the ring kernel would
// find rows that do not start on 16-byte boundaries, copied into the workspace
// with rows padded to whole 128-byte lines. The copy's padding is zeros, which
// a reduction may run into.
struct Operand {
    int64_t rows, cols;
    bool copy;
    int64_t ld, off;  // row length as read; workspace offset of the copy
};
bool fits(int64_t cols, bool aligned) { return cols % 8 == 0 && aligned; }
int64_t ring_ld(int64_t cols, bool aligned) { return fits(cols, aligned) ? cols : up(cols, 64); }
Operand operand(int64_t rows, int64_t cols, bool aligned, bool ring, int64_t* ws) {
    Operand o{rows, cols, ring && !fits(cols, aligned), cols, 0};
    if (o.copy) {
        o.ld = up(cols, 64);
        o.off = *ws;
        *ws += up(rows * o.ld * 2, 256);
    }
    return o;
}
// Both operands' places: the caller's memory, or the copies (one launch).
hipError_t place(const Operand& a, const void* pa, const uint16_t** oa, const Operand& b, const void* pb,
                 const uint16_t** ob, char* ws, hipStream_t s) {
    auto one = [ws](const Operand& o, const void* src, const uint16_t** out) {
        *out = o.copy ? reinterpret_cast<const uint16_t*>(ws + o.off) : static_cast<const uint16_t*>(src);
        return PadCopy{static_cast<const uint16_t*>(src), const_cast<uint16_t*>(*out), o.copy ? o.rows : 0, o.cols,
                       o.copy ? o.ld : 0};
    };
    const PadCopy ca = one(a, pa, oa), cb = one(b, pb, ob);
    return a.copy || b.copy ? launch_pad_any(ca, cb, s) : hipSuccess;
}

// Tile and reduction slices of one product. The ring kernel's round of 256
// tiles of 256 x 256 takes about as long as 0.7 rounds of the general
// kernel's 512 tiles of 128 x 128. A product of the general kernel with fewer
// tiles than the chip holds blocks (two per CU) splits a long reduction, 256
// values to a slice at least.
struct Shape {
    int tile, splits;
    int64_t k_split;
};
constexpr int kSkinny = -1;  // Shape::tile: the kernel for a few rows
// row length of fp32 planes: whole vectors and lines whatever N is
int64_t plane_ld(int64_t N) { return up(N, 64); }
// the planes of a split reduction
int64_t planes_bytes(const Shape& sh, int64_t M, int64_t N) {
    return sh.splits > 1 ? (int64_t)sh.splits * M * plane_ld(N) * 4 : 0;
}
int64_t tiles_of(int tile, int64_t M, int64_t N) {
    const FusedTile& t = kFusedTiles[tile];
    return ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
}
bool ring_pays(int64_t ring_tiles, int64_t tiles) {
    return ring_tiles >= 96 && (ring_tiles + 255) / 256 * 7 <= (tiles + 511) / 512 * 10;
}
Shape shape_of(int64_t M, int64_t N, int64_t K, bool a_oc, bool b_oc, int64_t lda, int64_t ldb, bool may_split) {
    Shape sh{a_oc || M > 64 ? 0 : M <= 32 ? 1 : 3, 1, up(K, 64)};
    if (M > 64 && ring_takes(GRP_NONE, a_oc, b_oc, N, K, lda, ldb) &&
        ring_pays(tiles_of(kRingTile, M, N), tiles_of(0, M, N))) {
        sh.tile = kRingTile;
        return sh;
    }
    const int64_t tiles = tiles_of(sh.tile, M, N);
    if (may_split && tiles < 256) {
        const int64_t want = std::min<int64_t>({512 / tiles, K / 256, 16});
        if (want > 1) {
            sh.k_split = up((K + want - 1) / want, 32);
            sh.splits = (int)((K + sh.k_split - 1) / sh.k_split);
        }
    }
    return sh;
}


// FusedArgs::vec_out for rows of ld values
int vec_rows(int64_t ld, const void* C, const void* R, const void* Z) {
    return ld % 8 == 0 && !off(C, 16) && !off(R, 16) && !off(Z, 16);
}

bool bad_ws(const void* ws, int64_t have, int64_t need) { return need > 0 && (!ws || have < need || off(ws, 256)); }

fc_status done(hipError_t e) { return e == hipSuccess ? FC_OK : FC_E_HIP; }

// The common end of a split product: the slices' planes, then the epilogue.
hipError_t run_product(EpiMode mode, const Shape& sh, bool a_oc, bool b_oc, FusedArgs g, float* planes,
                       hipStream_t s) {
    g.k_split = sh.k_split;
    g.splits = sh.splits;
    g.c_split_stride = 0;
    if (sh.tile == kSkinny) return launch_fused_skinny(g, s);
    if (sh.splits == 1) return launch_fused(mode, GRP_NONE, sh.tile, a_oc, b_oc, g, s);
    FusedArgs p = g;
    p.C = planes;
    p.ldc = plane_ld(g.N);
    p.out_f32 = 1;
    p.vec_out = 1;
    p.accumulate = 0;
    p.c_split_stride = g.M * p.ldc;
    const hipError_t e = launch_fused(EPI_STORE, GRP_NONE, sh.tile, a_oc, b_oc, p, s);
    return e != hipSuccess ? e : launch_split_epilogue(mode, g, planes, p.ldc, sh.splits, s);
}

// ---------------------------------------------------------------- act

struct ActPlan {
    Operand A, B;
    Shape sh;
    int64_t planes, parts_off, total;
    int parts;  // rows of column-sum partials
};

// the forward product (M x N over K) and, with `grad`, the backward-data one
// (output M x N = the layer's M x K, reduction over its outputs)
ActPlan act_plan(int64_t M, int64_t N, int64_t K, bool a_oc, bool b_oc, bool aligned, bool grad) {
    ActPlan p;
    int64_t ws = 0;
    const int64_t acols = a_oc ? M : K, bcols = b_oc ? N : K;
    p.sh = shape_of(M, N, K, a_oc, b_oc, ring_ld(acols, aligned), ring_ld(bcols, aligned), true);
    if (!grad && M <= 32 && !a_oc && !b_oc) p.sh = Shape{kSkinny, 1, K};
    const bool ring = p.sh.tile == kRingTile;
    p.A = operand(a_oc ? K : M, acols, aligned, ring, &ws);
    p.B = operand(b_oc ? K : N, bcols, aligned, ring, &ws);
    p.planes = ws;
    ws += planes_bytes(p.sh, M, N);
    p.parts_off = ws;
    p.parts = 0;
    if (grad) {
        const FusedTile& t = kFusedTiles[p.sh.tile];
        p.parts = p.sh.splits > 1 ? split_epilogue_parts(M) : (int)((M + t.bm - 1) / t.bm) * t.wave_rows;
        ws += up((int64_t)p.parts * N * 4, 256);
    }
    p.total = ws;
    return p;
}

bool bad_sizes(int64_t M, int64_t K, int64_t N) {
    return bad_size(M) || bad_size(K) || bad_size(N);
}

int bwd_act_parts(int64_t M, int64_t N) {
    // about 2048 blocks, at least 16 rows to each
    const int64_t cols = (N + 255) / 256;
    return (int)std::max<int64_t>(1, std::min<int64_t>({(M + 15) / 16, 2048 / cols, 65535}));
}

// --------------------------------------------------------------- xent

struct XentFwdPlan {
    Operand A, B;
    Shape sh;
    int parts;
    int64_t planes, stat, total;
};
XentFwdPlan xent_fwd_plan(int64_t M, int64_t K, int64_t N, bool b_oc, bool aligned) {
    XentFwdPlan p;
    int64_t ws = 0;
    const int64_t bcols = b_oc ? N : K;
    p.sh = shape_of(M, N, K, false, b_oc, ring_ld(K, aligned), ring_ld(bcols, aligned), true);
    const bool ring = p.sh.tile == kRingTile;
    p.A = operand(M, K, aligned, ring, &ws);
    p.B = operand(b_oc ? K : N, bcols, aligned, ring, &ws);
    p.planes = ws;
    ws += planes_bytes(p.sh, M, N);
    const FusedTile& t = kFusedTiles[p.sh.tile];
    p.parts = p.sh.splits > 1 ? split_stats_parts(N) : (int)((N + t.bn - 1) / t.bn) * t.wave_cols;
    p.stat = ws;
    ws += up((int64_t)2 * p.parts * M * 4, 256);
    p.total = ws;
    return p;
}

// The vocabulary is taken in pieces whose gradient of the logits (bf16)
// holds about kPieceBytes: it is written once and read by two products.
constexpr int64_t kPieceBytes = (int64_t)256 << 20;
struct XentBwdPlan {
    Operand A, B;
    int64_t piece, d_ld, d_off;  // columns of a piece (a multiple of 256 but for the last); its buffer
    int pieces;
    Shape logits, dx, dw;        // for a whole piece
    int64_t planes, sum_off, total;  // split products' planes; dX summed over several pieces
};
XentBwdPlan xent_bwd_plan(int64_t M, int64_t K, int64_t N, bool b_oc, bool aligned) {
    XentBwdPlan p;
    int64_t ws = 0;
    p.piece = std::min<int64_t>(N, std::max<int64_t>(256, kPieceBytes / (2 * M) / 256 * 256));
    p.pieces = (int)((N + p.piece - 1) / p.piece);
    p.d_ld = up(p.piece, 64);
    const int64_t bcols = b_oc ? N : K, lda = ring_ld(K, aligned), ldb = ring_ld(bcols, aligned);
    p.logits = shape_of(M, p.piece, K, false, b_oc, lda, ldb, p.pieces == 1);
    p.dx = shape_of(M, K, p.piece, false, !b_oc, p.d_ld, ldb, p.pieces == 1);
    p.dw = shape_of(K, p.piece, M, true, true, lda, p.d_ld, p.pieces == 1);
    if (512 * N >= (int64_t)1 << 31 && p.dw.tile == kRingTile) p.dw.tile = 0;  // its rows are N wide in dW
    const bool ring = p.logits.tile == kRingTile || p.dx.tile == kRingTile || p.dw.tile == kRingTile;
    p.A = operand(M, K, aligned, ring, &ws);
    p.B = operand(b_oc ? K : N, bcols, aligned, ring, &ws);
    p.d_off = ws;
    ws += up(M * p.d_ld * 2, 256);
    p.planes = ws;
    ws += std::max({planes_bytes(p.logits, M, p.piece), planes_bytes(p.dx, M, K), planes_bytes(p.dw, K, p.piece)});
    p.sum_off = ws;
    if (p.pieces > 1) ws += M * plane_ld(K) * 4;
    p.total = ws;
    return p;
}

// ------------------------------------------------------------ grouped

struct GroupedPlan {
    Operand A, B;
    int tile;
    int64_t total;
};
GroupedPlan grouped_plan(int op, int64_t T, int64_t E, int64_t K, int64_t N, int w_order, bool aligned) {
    GroupedPlan p;
    int64_t ws = 0;
    const bool red = op == FC_OP_BWD_WEIGHT, fwd = op == FC_OP_FWD, b_oc = red || fwd == (w_order == FC_ROW_MAJOR);
    const int64_t acols = op == FC_OP_BWD_DATA ? N : K, bcols = red || w_order == FC_ROW_MAJOR ? N : K;
    const int64_t n = op == FC_OP_BWD_DATA ? K : N, k = red ? T : fwd ? K : N;  // output columns, reduction
    const int64_t lda = ring_ld(acols, aligned), ldb = ring_ld(bcols, aligned);
    p.tile = red || T > 64 * E ? 0 : T <= 32 * E ? 1 : 3;
    // The experts' weights would be copied for the ring kernel: that takes as
    // long as its product over some 300 rows of each.
    const bool copies = !red && !fits(bcols, aligned);
    if (p.tile == 0 && !(copies && T < 300 * E) && ring_takes(red ? GRP_RED : GRP_ROWS, red, b_oc, n, k, lda, ldb)) {
        // (a group ends with a partly filled tile: half a tile's rows are lost on average)
        const int64_t ring = red ? E * tiles_of(kRingTile, K, N) : tiles_of(kRingTile, T + 128 * E, n);
        const int64_t small = red ? E * tiles_of(0, K, N) : tiles_of(0, T + 64 * E, n);
        if (ring_pays(ring, small)) p.tile = kRingTile;
    }
    p.A = operand(T, acols, aligned, p.tile == kRingTile, &ws);
    p.B = operand(red ? T : w_order == FC_ROW_MAJOR ? E * K : E * N, bcols, aligned, p.tile == kRingTile, &ws);
    p.total = ws;
    return p;
}

bool bad_grouped_sizes(int64_t T, int64_t E, int64_t K, int64_t N) {
    return bad_size(T) || E < 1 || E > kMaxExperts || bad_size(K) || bad_size(N) || E > kMaxCount / (K * N);
}

fc_status grouped_call(int op, const void* P, const void* Q, int w_order, const int64_t* offsets, void* out,
                       int dtype, int64_t T, int64_t E, int64_t K, int64_t N, void* ws, int64_t ws_bytes,
                       void* stream) {
    if (!P || !Q || !offsets || !out) return FC_E_INVALID;
    if (bad_order(w_order) || dtype < FC_OUT_BF16 || dtype > FC_OUT_F32_ACCUMULATE) return FC_E_INVALID;
    if (op != FC_OP_BWD_WEIGHT && dtype == FC_OUT_F32_ACCUMULATE) return FC_E_INVALID;
    if (bad_grouped_sizes(T, E, K, N)) return FC_E_INVALID;
    const bool f32 = dtype != FC_OUT_BF16;
    const int64_t esz = f32 ? 4 : 2;
    if (off(P, 2) || off(Q, 2) || off(offsets, 8) || off(out, esz)) return FC_E_INVALID;
    const int64_t pbytes = T * (op == FC_OP_BWD_DATA ? N : K) * 2;
    const int64_t qbytes = op == FC_OP_BWD_WEIGHT ? T * N * 2 : E * K * N * 2;
    const int64_t obytes = esz * (op == FC_OP_FWD ? T * N : op == FC_OP_BWD_DATA ? T * K : E * K * N);
    const bool aligned = !off(P, 16) && !off(Q, 16);
    const GroupedPlan pl = grouped_plan(op, T, E, K, N, w_order, aligned);
    if (bad_ws(ws, ws_bytes, pl.total)) return FC_E_INVALID;
    if (overlapping({{out, obytes}, {pl.total ? ws : nullptr, pl.total}},
                    {{P, pbytes}, {Q, qbytes}, {offsets, 8 * (E + 1)}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();  // the launchers report it: drop what an earlier, unrelated call left
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    FusedArgs g;
    hipError_t e;
    if ((e = place(pl.A, P, &g.A, pl.B, Q, &g.B, base, s)) != hipSuccess) return done(e);
    g.C = out;
    g.lda = pl.A.ld, g.ldb = pl.B.ld;
    g.out_f32 = f32;
    g.accumulate = dtype == FC_OUT_F32_ACCUMULATE;
    g.k_split = 0, g.splits = 1, g.c_split_stride = 0;
    g.offsets = offsets, g.E = (int)E, g.T = T;
    if (op == FC_OP_BWD_WEIGHT) {
        g.M = K, g.N = N, g.K = T;
        g.ldc = N;
        g.c_stride = K * N;
        g.vec_out = vec_rows(N, out, nullptr, nullptr);
        return done(launch_fused(EPI_STORE, GRP_RED, pl.tile, true, true, g, s));
    }
    const bool fwd = op == FC_OP_FWD;
    g.M = T, g.N = fwd ? N : K, g.K = fwd ? K : N;
    g.ldc = g.N;
    g.b_stride = (w_order == FC_ROW_MAJOR ? K : N) * pl.B.ld;
    g.vec_out = vec_rows(g.N, out, nullptr, nullptr);
    const bool b_oc = fwd == (w_order == FC_ROW_MAJOR);
    return done(launch_fused(EPI_STORE, GRP_ROWS, pl.tile, false, b_oc, g, s));
}

}  // namespace
}  // namespace fcs

using namespace fcs;

extern "C" {

int64_t fc_fwd_act_ws_bytes(int64_t M, int64_t K, int64_t N, fc_order x_order, fc_order w_order, int aligned) {
    if (bad_sizes(M, K, N) || bad_order(x_order) || bad_order(w_order)) return -1;
    return act_plan(M, N, K, x_order == FC_COL_MAJOR, w_order == FC_ROW_MAJOR, aligned != 0, false).total;
}

fc_status fc_fwd_act(const void* X, fc_order x_order, const void* W, fc_order w_order, const void* bias,
                     const void* R, fc_act act, void* Z, void* Y, fc_out_dtype y_dtype, int64_t M, int64_t K,
                     int64_t N, void* ws, int64_t ws_bytes, void* stream) {
    if (!X || !W || !Y) return FC_E_INVALID;
    if (bad_order(x_order) || bad_order(w_order) || bad_act(act)) return FC_E_INVALID;
    if (y_dtype != FC_OUT_BF16 && y_dtype != FC_OUT_F32) return FC_E_INVALID;
    if (bad_sizes(M, K, N)) return FC_E_INVALID;
    const bool f32 = y_dtype == FC_OUT_F32;
    if (off(X, 2) || off(W, 2) || off(bias, 2) || off(R, 2) || off(Z, 2) || off(Y, f32 ? 4 : 2)) return FC_E_INVALID;
    const bool aligned = !off(X, 16) && !off(W, 16);
    const bool a_oc = x_order == FC_COL_MAJOR, b_oc = w_order == FC_ROW_MAJOR;
    const ActPlan pl = act_plan(M, N, K, a_oc, b_oc, aligned, false);
    if (bad_ws(ws, ws_bytes, pl.total)) return FC_E_INVALID;
    if (overlapping({{Y, M * N * (f32 ? 4 : 2)}, {Z, M * N * 2}, {pl.total ? ws : nullptr, pl.total}},
                    {{X, M * K * 2}, {W, K * N * 2}, {bias, N * 2}, {R, M * N * 2}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    FusedArgs g;
    hipError_t e;
    if ((e = place(pl.A, X, &g.A, pl.B, W, &g.B, base, s)) != hipSuccess) return done(e);
    g.C = Y;
    g.M = M, g.N = N, g.K = K;
    g.lda = pl.A.ld, g.ldb = pl.B.ld, g.ldc = N;
    g.accumulate = 0;
    g.out_f32 = f32;
    g.vec_out = vec_rows(N, Y, R, Z);
    g.act = act;
    g.bias = static_cast<const uint16_t*>(bias);
    g.R = static_cast<const uint16_t*>(R);
    g.Z = static_cast<uint16_t*>(Z);
    return done(run_product(EPI_ACT, pl.sh, a_oc, b_oc, g, reinterpret_cast<float*>(base + pl.planes), s));
}

int64_t fc_bwd_data_act_ws_bytes(int64_t M, int64_t K, int64_t N, fc_order w_order, int aligned) {
    if (bad_sizes(M, K, N) || bad_order(w_order)) return -1;
    return act_plan(M, K, N, false, w_order == FC_COL_MAJOR, aligned != 0, true).total;
}

fc_status fc_bwd_data_act(const void* dY, const void* W, fc_order w_order, const void* Z, fc_act act, void* dX,
                          fc_out_dtype dx_dtype, float* db, int64_t M, int64_t K, int64_t N, void* ws,
                          int64_t ws_bytes, void* stream) {
    if (!dY || !W || !Z || !dX) return FC_E_INVALID;
    if (bad_order(w_order) || bad_act(act)) return FC_E_INVALID;
    if (dx_dtype != FC_OUT_BF16 && dx_dtype != FC_OUT_F32) return FC_E_INVALID;
    if (bad_sizes(M, K, N)) return FC_E_INVALID;
    const bool f32 = dx_dtype == FC_OUT_F32;
    if (off(dY, 2) || off(W, 2) || off(Z, 2) || off(db, 4) || off(dX, f32 ? 4 : 2)) return FC_E_INVALID;
    const bool aligned = !off(dY, 16) && !off(W, 16);
    const bool b_oc = w_order == FC_COL_MAJOR;
    const ActPlan pl = act_plan(M, K, N, false, b_oc, aligned, true);
    if (bad_ws(ws, ws_bytes, pl.total)) return FC_E_INVALID;
    if (overlapping({{dX, M * K * (f32 ? 4 : 2)}, {db, K * 4}, {ws, pl.total}},
                    {{dY, M * N * 2}, {W, K * N * 2}, {Z, M * K * 2}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    FusedArgs g;
    hipError_t e;
    if ((e = place(pl.A, dY, &g.A, pl.B, W, &g.B, base, s)) != hipSuccess) return done(e);
    g.C = dX;
    g.M = M, g.N = K, g.K = N;
    g.lda = pl.A.ld, g.ldb = pl.B.ld, g.ldc = K;
    g.accumulate = 0;
    g.out_f32 = f32;
    g.vec_out = vec_rows(K, dX, nullptr, Z);
    g.act = act;
    g.Z = static_cast<uint16_t*>(const_cast<void*>(Z));  // read only
    g.colpart = db ? reinterpret_cast<float*>(base + pl.parts_off) : nullptr;
    e = run_product(EPI_DACT, pl.sh, false, b_oc, g, reinterpret_cast<float*>(base + pl.planes), s);
    if (e == hipSuccess && db) e = launch_colsum_parts(g.colpart, db, K, pl.parts, s);
    return done(e);
}

int64_t fc_bwd_act_ws_bytes(int64_t M, int64_t N) {
    if (bad_size(M) || bad_size(N)) return -1;
    return up((int64_t)bwd_act_parts(M, N) * N * 4, 256);
}

fc_status fc_bwd_act(const void* dY, const void* Z, fc_act act, void* dZ, float* db, int64_t M, int64_t N, void* ws,
                     int64_t ws_bytes, void* stream) {
    if (!dY || (!dZ && !db) || bad_act(act) || (!Z && act != FC_ACT_NONE)) return FC_E_INVALID;
    if (bad_size(M) || bad_size(N)) return FC_E_INVALID;
    if (off(dY, 2) || off(Z, 2) || off(dZ, 2) || off(db, 4)) return FC_E_INVALID;
    const int64_t need = db ? fc_bwd_act_ws_bytes(M, N) : 0;
    if (bad_ws(ws, ws_bytes, need)) return FC_E_INVALID;
    if (overlapping({{dZ, M * N * 2}, {db, N * 4}, {need ? ws : nullptr, need}}, {{dY, M * N * 2}, {Z, M * N * 2}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int parts = bwd_act_parts(M, N);
    float* part = db ? static_cast<float*>(ws) : nullptr;
    hipError_t e = launch_act_bwd(static_cast<const uint16_t*>(dY), static_cast<const uint16_t*>(Z), act,
                                  static_cast<uint16_t*>(dZ), part, M, N, parts, s);
    if (e == hipSuccess && db) e = launch_colsum_parts(part, db, N, parts, s);
    return done(e);
}

int64_t fc_xent_fwd_ws_bytes(int64_t M, int64_t K, int64_t N, fc_order w_order, int aligned) {
    if (bad_sizes(M, K, N) || bad_order(w_order)) return -1;
    return xent_fwd_plan(M, K, N, w_order == FC_ROW_MAJOR, aligned != 0).total;
}

fc_status fc_xent_fwd(const void* X, const void* W, fc_order w_order, const int64_t* targets, int64_t vocab_start,
                      int64_t ignore_index, float* lse, float* tlogit, float* loss, int64_t M, int64_t K, int64_t N,
                      void* ws, int64_t ws_bytes, void* stream) {
    if (!X || !W || !targets || !lse || !tlogit) return FC_E_INVALID;
    if (bad_order(w_order) || bad_sizes(M, K, N) || vocab_start < 0) return FC_E_INVALID;
    if (off(X, 2) || off(W, 2) || off(targets, 8) || off(lse, 4) || off(tlogit, 4) || off(loss, 4))
        return FC_E_INVALID;
    const bool aligned = !off(X, 16) && !off(W, 16), b_oc = w_order == FC_ROW_MAJOR;
    const XentFwdPlan pl = xent_fwd_plan(M, K, N, b_oc, aligned);
    if (bad_ws(ws, ws_bytes, pl.total)) return FC_E_INVALID;
    if (overlapping({{lse, M * 4}, {tlogit, M * 4}, {loss, M * 4}, {ws, pl.total}},
                    {{X, M * K * 2}, {W, K * N * 2}, {targets, M * 8}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    FusedArgs g;
    hipError_t e;
    if ((e = place(pl.A, X, &g.A, pl.B, W, &g.B, base, s)) != hipSuccess) return done(e);
    g.C = nullptr;
    g.M = M, g.N = N, g.K = K;
    g.lda = pl.A.ld, g.ldb = pl.B.ld, g.ldc = N;
    g.accumulate = 0;
    g.targets = targets, g.v0 = vocab_start, g.ignore = ignore_index;
    g.stat = reinterpret_cast<float*>(base + pl.stat);
    g.tlogit = tlogit;
    if ((e = run_product(EPI_STATS, pl.sh, false, b_oc, g, reinterpret_cast<float*>(base + pl.planes), s)) != hipSuccess) return done(e);
    return done(launch_xent_finish(g.stat, pl.parts, targets, vocab_start, ignore_index, M, N, lse, tlogit, loss, s));
}

int64_t fc_xent_bwd_ws_bytes(int64_t M, int64_t K, int64_t N, fc_order w_order, int aligned) {
    if (bad_sizes(M, K, N) || bad_order(w_order)) return -1;
    return xent_bwd_plan(M, K, N, w_order == FC_ROW_MAJOR, aligned != 0).total;
}

fc_status fc_xent_bwd(const void* X, const void* W, fc_order w_order, const int64_t* targets, int64_t vocab_start,
                      int64_t ignore_index, const float* lse, const float* grad, void* dX, fc_out_dtype dx_dtype,
                      void* dW, fc_out_dtype dw_dtype, int64_t M, int64_t K, int64_t N, void* ws, int64_t ws_bytes,
                      void* stream) {
    if (!X || !W || !targets || !lse || !grad || !dX || !dW) return FC_E_INVALID;
    if (bad_order(w_order) || bad_sizes(M, K, N) || vocab_start < 0) return FC_E_INVALID;
    if (dx_dtype != FC_OUT_BF16 && dx_dtype != FC_OUT_F32) return FC_E_INVALID;
    if (dw_dtype < FC_OUT_BF16 || dw_dtype > FC_OUT_F32_ACCUMULATE) return FC_E_INVALID;
    const bool xf32 = dx_dtype == FC_OUT_F32, wf32 = dw_dtype != FC_OUT_BF16;
    if (off(X, 2) || off(W, 2) || off(targets, 8) || off(lse, 4) || off(grad, 4) || off(dX, xf32 ? 4 : 2) ||
        off(dW, wf32 ? 4 : 2))
        return FC_E_INVALID;
    const bool aligned = !off(X, 16) && !off(W, 16), w_row = w_order == FC_ROW_MAJOR;
    const XentBwdPlan pl = xent_bwd_plan(M, K, N, w_row, aligned);
    if (bad_ws(ws, ws_bytes, pl.total)) return FC_E_INVALID;
    if (overlapping({{dX, M * K * (xf32 ? 4 : 2)}, {dW, K * N * (wf32 ? 4 : 2)}, {ws, pl.total}},
                    {{X, M * K * 2}, {W, K * N * 2}, {targets, M * 8}, {lse, M * 4}, {grad, M * 4}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    const uint16_t *x, *w;
    hipError_t e;
    if ((e = place(pl.A, X, &x, pl.B, W, &w, base, s)) != hipSuccess) return done(e);
    uint16_t* D = reinterpret_cast<uint16_t*>(base + pl.d_off);
    float* planes = reinterpret_cast<float*>(base + pl.planes);
    float* sum = reinterpret_cast<float*>(base + pl.sum_off);
    for (int p = 0; p < pl.pieces; ++p) {
        const int64_t c0 = (int64_t)p * pl.piece, c = std::min(pl.piece, N - c0);
        const uint16_t* wp = w + (w_row ? c0 : c0 * pl.B.ld);
        // the piece's logits again, and their gradient
        FusedArgs g;
        g.A = x, g.B = wp, g.C = D;
        g.M = M, g.N = c, g.K = K;
        g.lda = pl.A.ld, g.ldb = pl.B.ld, g.ldc = pl.d_ld;
        g.accumulate = 0;
        g.targets = targets, g.v0 = vocab_start + c0, g.ignore = ignore_index;
        g.lse = lse, g.gw = grad;
        if ((e = run_product(EPI_DLOGIT, pl.logits, false, w_row, g, planes, s)) != hipSuccess) return done(e);
        // dW = X^T D, this piece's columns
        FusedArgs h;
        h.A = x, h.B = D;
        h.C = static_cast<char*>(dW) + c0 * (wf32 ? 4 : 2);
        h.M = K, h.N = c, h.K = M;
        h.lda = pl.A.ld, h.ldb = pl.d_ld, h.ldc = N;
        h.out_f32 = wf32;
        h.accumulate = dw_dtype == FC_OUT_F32_ACCUMULATE;
        h.vec_out = vec_rows(N, h.C, nullptr, nullptr);
        if ((e = run_product(EPI_STORE, pl.dw, true, true, h, planes, s)) != hipSuccess) return done(e);
        // dX = D W^T: in one go, or summed over the pieces in 32 bits
        FusedArgs d;
        d.A = D, d.B = wp;
        d.M = M, d.N = K, d.K = c;
        d.lda = pl.d_ld, d.ldb = pl.B.ld;
        const bool last = pl.pieces == 1;
        d.ldc = last ? K : plane_ld(K);
        d.C = last ? dX : sum;
        d.out_f32 = last ? xf32 : 1;
        d.accumulate = p > 0;
        d.vec_out = vec_rows(d.ldc, d.C, nullptr, nullptr);
        Shape sh = pl.dx;
        if (sh.splits == 1) sh.k_split = up(c, 64);
        if (sh.tile == kRingTile && c < 64) sh.tile = 0;  // a last piece of less than one stage
        if ((e = run_product(EPI_STORE, sh, false, !w_row, d, planes, s)) != hipSuccess) return done(e);
    }
    if (pl.pieces > 1) {
        FusedArgs d;
        d.C = dX;
        d.M = M, d.N = K, d.ldc = K;
        d.accumulate = 0;
        d.out_f32 = xf32;
        d.vec_out = vec_rows(K, dX, nullptr, nullptr);
        e = launch_split_epilogue(EPI_STORE, d, sum, plane_ld(K), 1, s);
    }
    return done(e);
}

int64_t fc_grouped_ws_bytes(fc_op op, int64_t T, int64_t E, int64_t K, int64_t N, fc_order w_order, int aligned) {
    if (op < FC_OP_FWD || op > FC_OP_BWD_WEIGHT || bad_order(w_order) || bad_grouped_sizes(T, E, K, N)) return -1;
    return grouped_plan(op, T, E, K, N, w_order, aligned != 0).total;
}

fc_status fc_grouped_fwd(const void* X, const void* W, fc_order w_order, const int64_t* offsets, void* Y,
                         fc_out_dtype y_dtype, int64_t T, int64_t E, int64_t K, int64_t N, void* ws,
                         int64_t ws_bytes, void* stream) {
    return grouped_call(FC_OP_FWD, X, W, w_order, offsets, Y, y_dtype, T, E, K, N, ws, ws_bytes, stream);
}

fc_status fc_grouped_bwd_data(const void* dY, const void* W, fc_order w_order, const int64_t* offsets, void* dX,
                              fc_out_dtype dx_dtype, int64_t T, int64_t E, int64_t K, int64_t N, void* ws,
                              int64_t ws_bytes, void* stream) {
    return grouped_call(FC_OP_BWD_DATA, dY, W, w_order, offsets, dX, dx_dtype, T, E, K, N, ws, ws_bytes, stream);
}

fc_status fc_grouped_bwd_weight(const void* X, const void* dY, const int64_t* offsets, void* dW,
                                fc_out_dtype dw_dtype, int64_t T, int64_t E, int64_t K, int64_t N, void* ws,
                                int64_t ws_bytes, void* stream) {
    return grouped_call(FC_OP_BWD_WEIGHT, X, dY, FC_ROW_MAJOR, offsets, dW, dw_dtype, T, E, K, N, ws, ws_bytes,
                        stream);
}

}  // extern "C"
