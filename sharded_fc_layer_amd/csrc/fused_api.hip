// C ABI of the fused operators: argument checks, the choice of kernel and
// workspace layout for each product, and the launches.
//
// Every plan here is a function of sizes, orders, types and operand alignment
// alone, so that the workspace queries and the calls agree. Nothing is
// allocated, kept or synchronized: workspaces are the caller's.
#include "fused_plan.h"

namespace fcs {
namespace {

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
    p.sh = shape_of(M, N, K, a_oc, b_oc, acols, bcols, aligned);
    if (!grad && M <= 32 && !a_oc && !b_oc && skinny_pays(M, N, K)) p.sh = Shape{kSkinny, 1, K, 0};
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
    p.sh = shape_of(M, N, K, false, b_oc, K, bcols, aligned);
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
    int64_t scale_off, planes, sum_off, total;  // weight_scale; split products' planes; dX summed over several pieces
};
XentBwdPlan xent_bwd_plan(int64_t M, int64_t K, int64_t N, bool b_oc, bool aligned) {
    XentBwdPlan p;
    int64_t ws = 0;
    p.piece = std::min<int64_t>(N, std::max<int64_t>(256, kPieceBytes / (2 * M) / 256 * 256));
    p.pieces = (int)((N + p.piece - 1) / p.piece);
    p.d_ld = up(p.piece, 64);
    const int64_t bcols = b_oc ? N : K, lda = ring_ld(K, aligned), ldb = ring_ld(bcols, aligned);
    // each product's better kernel; the copies, if the operands need them, serve all three
    const bool split = p.pieces == 1, copies = !fits(K, aligned) || !fits(bcols, aligned);
    const Shape small[3] = {small_shape(M, p.piece, K, false, copies, split),
                            small_shape(M, K, p.piece, false, !fits(bcols, aligned), split),
                            small_shape(K, p.piece, M, true, !fits(K, aligned), split)};
    Shape ring[3] = {ring_shape(M, p.piece, K, false, b_oc, lda, ldb), ring_shape(M, K, p.piece, false, !b_oc, p.d_ld, ldb),
                     ring_shape(K, p.piece, M, true, true, lda, p.d_ld)};
    if (512 * N >= (int64_t)1 << 31) ring[2].us = 1e30;  // dW's rows are N wide
    Shape* to[3] = {&p.logits, &p.dx, &p.dw};
    double gain = 0;
    for (int i = 0; i < 3; ++i) {
        *to[i] = ring[i].us < small[i].us ? ring[i] : small[i];
        gain += (small[i].us - to[i]->us) * p.pieces;
    }
    const int64_t bytes = (fits(K, aligned) ? 0 : M * K * 2) + (fits(bcols, aligned) ? 0 : N * K * 2);
    const bool ring_any = gain > 0 && (!copies || gain > copy_us(bytes));
    if (!ring_any)
        for (int i = 0; i < 3; ++i) *to[i] = small[i];
    p.A = operand(M, K, aligned, ring_any, &ws);
    p.B = operand(b_oc ? K : N, bcols, aligned, ring_any, &ws);
    p.d_off = ws;
    ws += up(M * p.d_ld * 2, 256);
    p.scale_off = ws;
    ws += 256;
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
    int tile, slices;
    int64_t k_split, planes, total;
};
GroupedPlan grouped_plan(int op, int64_t T, int64_t E, int64_t K, int64_t N, int w_order, bool aligned) {
    GroupedPlan p;
    int64_t ws = 0;
    const bool red = op == FC_OP_BWD_WEIGHT, fwd = op == FC_OP_FWD, b_oc = red || fwd == (w_order == FC_ROW_MAJOR);
    const int64_t acols = op == FC_OP_BWD_DATA ? N : K, bcols = red || w_order == FC_ROW_MAJOR ? N : K;
    const int64_t n = op == FC_OP_BWD_DATA ? K : N, k = red ? T : fwd ? K : N;  // output columns, reduction
    const int64_t lda = ring_ld(acols, aligned), ldb = ring_ld(bcols, aligned);
    // (a group ends with a partly filled tile: half a tile's rows are lost on average)
    p.tile = red || T > 64 * E ? 0 : T <= 32 * E ? 1 : 3;
    p.slices = 1, p.k_split = k;
    const int64_t mean = std::max<int64_t>(1, T / E);  // a group's reduction, of the weights' gradient
    int64_t tiles;
    if (red)
        tiles = E * tiles_of(0, K, N);
    else if (p.tile == 0)
        tiles = tiles_of(0, T + 64 * E, n);
    else  // groups of a tile's rows or fewer
        tiles = std::min(T, E) * ((n + 127) / 128);
    const bool any = !fits(acols, aligned) || !fits(bcols, aligned);
    const double moved = 2.0 * (double)T * (double)(K + N) + 2.0 * (double)std::min(T, E) * (double)K * (double)N;
    double us = small_us(p.tile, tiles, red ? mean : k, any, moved);
    if (ring_takes(red ? GRP_RED : GRP_ROWS, red, b_oc, n, k, lda, ldb)) {
        const int64_t rtiles = red ? E * tiles_of(kRingTile, K, N) : tiles_of(kRingTile, T + 128 * E, n);
        const int64_t bytes = (fits(acols, aligned) ? 0 : T * acols * 2) +
                              (fits(bcols, aligned) ? 0 : (red ? T * N : E * K * N) * 2);
        const double ring = ring_us(rtiles, red ? mean : k, red, moved) + (bytes ? copy_us(bytes) : 0);
        if (ring < us) p.tile = kRingTile, us = ring;
    }
    // a few rows against long reductions: slices, as for one product
    if (!red && p.tile != kRingTile && tiles < 256) {
        for (int s = 2; s <= 16; ++s) {
            const int64_t k_split = up((k + s - 1) / s, 32);
            if (k_split < 128) break;
            const int slices = (int)((k + k_split - 1) / k_split);
            const double t = small_us(p.tile, tiles * slices, k_split, any, moved) + planes_us(slices, T, n);
            if (t < us) p.slices = slices, p.k_split = k_split, us = t;
        }
    }
    p.A = operand(T, acols, aligned, p.tile == kRingTile, &ws);
    p.B = operand(red ? T : w_order == FC_ROW_MAJOR ? E * K : E * N, bcols, aligned, p.tile == kRingTile, &ws);
    p.planes = ws;
    if (p.slices > 1) ws += (int64_t)p.slices * T * plane_ld(n) * 4;
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
    GroupedPlan pl = grouped_plan(op, T, E, K, N, w_order, aligned);
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
    g.k_split = pl.k_split;
    if (pl.slices == 1) return done(launch_fused(EPI_STORE, GRP_ROWS, pl.tile, false, b_oc, g, s));
    FusedArgs p = g;
    p.C = base + pl.planes;
    p.ldc = plane_ld(g.N);
    p.out_f32 = 1;
    p.splits = pl.slices;
    p.c_split_stride = T * p.ldc;
    e = launch_fused(EPI_STORE, GRP_ROWS, pl.tile, false, b_oc, p, s);
    return done(e != hipSuccess ? e
                                : launch_split_epilogue(EPI_STORE, g, static_cast<const float*>(p.C), p.ldc, pl.slices, s));
}

}  // namespace

int64_t logits_bwd_ws_bytes(int64_t M, int64_t K, int64_t N, int w_order, bool aligned) {
    return xent_bwd_plan(M, K, N, w_order == FC_ROW_MAJOR, aligned).total;
}

hipError_t run_logits_bwd(const LogitsBwd& b, char* base, hipStream_t s) {
    const int64_t M = b.M, K = b.K, N = b.N;
    const bool w_row = b.w_order == FC_ROW_MAJOR, wf32 = b.dw_dtype != FC_OUT_BF16;
    XentBwdPlan pl = xent_bwd_plan(M, K, N, w_row, !off(b.X, 16) && !off(b.W, 16));
    const uint16_t *x, *w;
    hipError_t e;
    if ((e = place(pl.A, b.X, &x, pl.B, b.W, &w, base, s)) != hipSuccess) return e;
    uint16_t* D = reinterpret_cast<uint16_t*>(base + pl.d_off);
    float* planes = reinterpret_cast<float*>(base + pl.planes);
    float* sum = reinterpret_cast<float*>(base + pl.sum_off);
    float* scale = reinterpret_cast<float*>(base + pl.scale_off);
    for (int p = 0; p < pl.pieces; ++p) {
        const int64_t c0 = (int64_t)p * pl.piece, c = std::min(pl.piece, N - c0);
        const uint16_t* wp = w + (w_row ? c0 : c0 * pl.B.ld);
        // the piece's logits again, and their gradient
        FusedArgs g;
        g.A = x, g.B = wp, g.C = D;
        g.M = M, g.N = c, g.K = K;
        g.lda = pl.A.ld, g.ldb = pl.B.ld, g.ldc = pl.d_ld;
        g.accumulate = 0;
        g.targets = b.targets, g.v0 = b.v0 + c0, g.ignore = b.ignore;
        g.lse = b.lse, g.gw = b.gw, g.inv_t = b.inv_t, g.wscale = scale;
        if ((e = run_product(EPI_DLOGIT, pl.logits, false, w_row, g, planes, s)) != hipSuccess) return e;
        if (b.listed && (e = launch_listed_grad(*b.listed, b.lse, b.gw, b.inv_t, scale, D, pl.d_ld, g.v0, c, M, s)) != hipSuccess)
            return e;
        // dW = X^T D, this piece's columns
        FusedArgs h;
        h.A = x, h.B = D;
        h.C = static_cast<char*>(b.dW) + c0 * (wf32 ? 4 : 2);
        h.M = K, h.N = c, h.K = M;
        h.lda = pl.A.ld, h.ldb = pl.d_ld, h.ldc = N;
        h.out_f32 = wf32;
        h.accumulate = b.dw_dtype == FC_OUT_F32_ACCUMULATE;
        h.vec_out = vec_rows(N, h.C, nullptr, nullptr);
        h.wscale = scale;
        if ((e = run_product(EPI_STORE, pl.dw, true, true, h, planes, s)) != hipSuccess) return e;
        // dX = D W^T: in one go, or summed over the pieces in 32 bits
        FusedArgs d;
        d.A = D, d.B = wp;
        d.M = M, d.N = K, d.K = c;
        d.lda = pl.d_ld, d.ldb = pl.B.ld;
        const bool last = pl.pieces == 1;
        d.ldc = last ? K : plane_ld(K);
        d.C = last ? b.dX : sum;
        d.out_f32 = last ? b.dx_f32 : 1;
        d.accumulate = p > 0;
        d.vec_out = vec_rows(d.ldc, d.C, nullptr, nullptr);
        d.wscale = scale;
        Shape sh = pl.dx;
        if (sh.splits == 1) sh.k_split = up(c, 64);
        if (sh.tile == kRingTile && c < 64) sh.tile = 0;  // a last piece of less than one stage
        if ((e = run_product(EPI_STORE, sh, false, !w_row, d, planes, s)) != hipSuccess) return e;
    }
    if (pl.pieces > 1) {
        FusedArgs d;
        d.C = b.dX;
        d.M = M, d.N = K, d.ldc = K;
        d.accumulate = 0;
        d.out_f32 = b.dx_f32;
        d.vec_out = vec_rows(K, b.dX, nullptr, nullptr);
        e = launch_split_epilogue(EPI_STORE, d, sum, plane_ld(K), 1, s);
    }
    return e;
}

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
    ActPlan pl = act_plan(M, N, K, a_oc, b_oc, aligned, false);
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
    ActPlan pl = act_plan(M, K, N, false, b_oc, aligned, true);
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
    XentFwdPlan pl = xent_fwd_plan(M, K, N, b_oc, aligned);
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
    return logits_bwd_ws_bytes(M, K, N, w_order, aligned != 0);
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
    const int64_t need = logits_bwd_ws_bytes(M, K, N, w_order, !off(X, 16) && !off(W, 16));
    if (bad_ws(ws, ws_bytes, need)) return FC_E_INVALID;
    if (overlapping({{dX, M * K * (xf32 ? 4 : 2)}, {dW, K * N * (wf32 ? 4 : 2)}, {ws, need}},
                    {{X, M * K * 2}, {W, K * N * 2}, {targets, M * 8}, {lse, M * 4}, {grad, M * 4}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    LogitsBwd b;
    b.X = X, b.W = W, b.w_order = w_order;
    b.targets = targets, b.v0 = vocab_start, b.ignore = ignore_index;
    b.lse = lse, b.gw = grad;
    b.dX = dX, b.dx_f32 = xf32, b.dW = dW, b.dw_dtype = dw_dtype;
    b.M = M, b.K = K, b.N = N;
    return done(run_logits_bwd(b, static_cast<char*>(ws), static_cast<hipStream_t>(stream)));
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
