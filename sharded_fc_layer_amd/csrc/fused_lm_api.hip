// C ABI of the gated layers, log probabilities and distillation: argument
// checks, plans, and the launches (fused_plan.h says how products are planned).
#include "fused_plan.h"

namespace fcs {
namespace {

// -------------------------------------------------------------- gated

// The few-row kernel against the general one (us, W from memory; from the
// caches): 2048 -> 8192 one row 16.0 and 19.8 (12.4; 16.2), 16 rows 19.4 and
// 22.5 (14.9; 17.4), 32 rows 23.1 and 23.0; 4096 -> 14336 one row 49.6 and 55.8
// (39.3; 35.1), 4 rows 51.9 and 60.6 (40.2; 34.8), 16 rows 60.5 and 57.2. Rows
// on odd elements are slower to read: 1001 -> 1531 one row 8.0 and 11.3, 32 rows
// 11.7 and 14.5, 511 -> 4000 8.5 and 12.5, 12.1 and 14.8, but 2047 -> 4000 18.9
// and 18.8, 30.8 and 21.6, 4095 -> 14336 114 and 78.
bool few_rows_pay(int64_t M, int64_t N, int64_t K, bool aligned) {
    const bool odd = K % 2 != 0 || !aligned;
    return N <= (M <= 8 ? 16384 : M <= 16 ? 8192 : 4096) && K >= 256 && (!odd || N * K <= 1 << 22);
}

// A gated product: the plain one of 2 N columns (forward) or of N (its data
// gradient, `grad`), whose epilogue reads or writes 2 N columns of Z.
struct GluPlan {
    Operand A, B;
    Shape sh;
    bool fused;  // the epilogue in the product's kernel, else from planes
    int64_t planes, parts_off, total;
    int parts;  // rows of column-sum partials, 2 N wide
};
GluPlan glu_plan(int64_t M, int64_t N, int64_t K, bool b_oc, bool aligned, bool grad) {
    GluPlan p;
    int64_t ws = 0;
    const int64_t cols = grad ? N : 2 * N, bcols = b_oc ? cols : K, ldb = ring_ld(bcols, aligned);
    const int64_t limit = (int64_t)1 << 31;
    // (the two halves of W are read through one descriptor; Z's rows are 2 N wide)
    const bool near = grad || 2 * (b_oc ? K : cols) * ldb < limit;
    p.sh = low_shape(M, cols, K, !fits(K, aligned) || !fits(bcols, aligned) || (b_oc && !grad && N % 8 != 0), true);
    p.fused = near && p.sh.splits == 1;
    if (!near) p.sh.us += planes_us(1, M, cols);
    // the large tiles: fused where rows of N values are whole vectors, else with planes
    Shape ring = ring_shape(M, cols, K, false, b_oc, ring_ld(K, aligned), ldb);
    const bool ring_fused = near && N % 8 == 0 && 512 * 2 * N < limit;
    const int64_t copies = (fits(K, aligned) ? 0 : M * K * 2) + (fits(bcols, aligned) ? 0 : cols * K * 2);
    if (copies) ring.us += copy_us(copies);
    if (!ring_fused) ring.us += planes_us(1, M, cols);
    if (512 * plane_ld(cols) < limit && ring.us < p.sh.us) p.sh = ring, p.fused = ring_fused;
    if (!grad && M <= 32 && !b_oc && few_rows_pay(M, N, K, aligned)) p.sh = Shape{kSkinny, 1, K, 0}, p.fused = true;
    const bool large = p.sh.tile == kRingTile;
    p.A = operand(M, K, aligned, large, &ws);
    p.B = operand(b_oc ? K : cols, bcols, aligned, large, &ws);
    p.planes = ws;
    if (!p.fused) ws += up((int64_t)p.sh.splits * M * plane_ld(cols) * 4, 256);
    p.parts_off = ws;
    p.parts = 0;
    if (grad) {
        const FusedTile& t = kFusedTiles[p.sh.tile];
        p.parts = p.fused ? (int)((M + t.bm - 1) / t.bm) * t.wave_rows : split_epilogue_parts(M);
    }
    // (a launch that falls back from the large tiles to the first ones leaves more rows)
    const int rows = large && grad && p.fused ? (int)((M + 127) / 128) * 2 : p.parts;
    ws += up((int64_t)rows * 2 * N * 4, 256);
    p.total = ws;
    return p;
}
// The product with its epilogue.
hipError_t run_glu(EpiMode mode, const GluPlan& pl, bool b_oc, FusedArgs g, int64_t cols, char* base, hipStream_t s) {
    if (!pl.fused) return run_planes(mode, pl.sh, false, b_oc, g, cols, reinterpret_cast<float*>(base + pl.planes), s);
    if (pl.sh.tile == kSkinny) return launch_fused_skinny_glu(g, s);
    g.k_split = pl.sh.k_split, g.splits = 1, g.c_split_stride = 0;
    return launch_fused(mode, GRP_NONE, pl.sh.tile, false, b_oc, g, s);
}

int64_t glu_bwd_bytes(int64_t M, int64_t N) { return up((int64_t)glu_bwd_parts(M, N) * 2 * N * 4, 256); }

// ---------------------------------------------------------- vocabulary

bool bad_temperature(float t) { return !(t >= 0x1p-10f && t <= 0x1p10f); }

// A row's logits and their statistics, a chunk of rows at a time: the workspace
// holds the chunk's logits.
constexpr int64_t kLogitBytes = (int64_t)1024 << 20;
// The few-row kernel against the general one (us, W from memory, k = 0): one
// row, 2048 -> 8000: 13.8 and 17.0, 32000: 32.7 and 38.9, 128000: 102 and 134,
// 4096 -> 128256: 205 and 232; 8 rows 14.7 and 17.7, 34.5 and 37.8, 110 and 121,
// 211 and 229; 16 rows 15.1 and 17.7, 36.9 and 38.0, 120 and 123, and over 4096
// (32000) 64.4 and 62.5; 32 rows of 32000 45.5 and 39.0. Where W stays in the
// caches it loses up to an eighth (32000: 28.5 and 25.5). Rows on odd elements are
// read one by one (2047 -> 32000: 78 and 49).
bool few_logit_rows_pay(int64_t M, int64_t K, bool aligned) {
    return M <= (K <= 2048 ? 16 : 8) && K >= 256 && K % 2 == 0 && aligned;
}
struct LogitsPlan {
    Operand A, B;
    Shape sh;
    bool keep;     // the logits are stored: they are read again, or a split reduction's planes
    int64_t rows;  // of a chunk: a multiple of 256, or all
    int64_t z_ld, z_off, stat_off, t_off, need_off, total;
    int parts, width;
    bool need;     // of listed tokens: which parts are stored
};
LogitsPlan logits_plan(int64_t M, int64_t K, int64_t N, bool b_oc, bool aligned, bool read_again, bool listed) {
    LogitsPlan p;
    int64_t ws = 0;
    p.z_ld = plane_ld(N);
    // (three statistics for 32 columns or more, where no logits are kept)
    const int64_t row_bytes = read_again ? 4 * p.z_ld : 12 * ((N + 31) / 32);
    const int64_t fit = std::max<int64_t>(256, kLogitBytes / row_bytes / 256 * 256);
    const int64_t bcols = b_oc ? N : K;
    p.rows = std::min(M, fit);
    p.sh = shape_of(p.rows, N, K, false, b_oc, K, bcols, aligned, true);
    if (512 * p.z_ld >= (int64_t)1 << 31 && p.sh.tile == kRingTile)
        p.sh = small_shape(p.rows, N, K, false, !fits(K, aligned) || !fits(bcols, aligned), false);
    if (!b_oc && few_logit_rows_pay(M, K, aligned)) p.sh = Shape{kSkinny, 1, K, 0};
    const bool ring = p.sh.tile == kRingTile, split = p.sh.splits > 1, few = p.sh.tile == kSkinny;
    p.keep = read_again || split;
    p.A = operand(M, K, aligned, ring, &ws);
    p.B = operand(b_oc ? K : N, bcols, aligned, ring, &ws);
    const FusedTile& t = kFusedTiles[few ? 0 : p.sh.tile];
    p.width = split ? kLogitCols : few ? 32 : t.bn / t.wave_cols;
    p.parts = split || few ? (int)((N + p.width - 1) / p.width) : (int)((N + t.bn - 1) / t.bn) * t.wave_cols;
    p.z_off = ws;
    if (p.keep) ws += p.sh.splits * p.rows * p.z_ld * 4;
    p.stat_off = ws;
    ws += up((int64_t)3 * p.parts * p.rows * 4, 256);
    p.t_off = ws;
    ws += up(p.rows * 4, 256);
    p.need = listed && ring;
    p.need_off = ws;
    if (p.need) ws += up((int64_t)((p.parts + 31) / 32) * p.rows * 4, 256);
    p.total = ws;
    return p;
}

// Rows m0 .. m0 + rows - 1: their logits' statistics (and the logits), for the kernels that follow.
struct LogitsCall {
    int w_order;
    const int64_t* targets;  // or none
    int64_t v0;
    float inv_t;
    int64_t K, N;
    const Listed* listed;    // of these rows, or none
};
hipError_t run_logits(const LogitsPlan& pl, const LogitsCall& c, const uint16_t* x, const uint16_t* w, int64_t m0,
                      int64_t rows, char* base, RowLogits* out, hipStream_t s) {
    FusedArgs g;
    g.A = x + m0 * pl.A.ld, g.B = w;
    g.M = rows, g.N = c.N, g.K = c.K;
    g.lda = pl.A.ld, g.ldb = pl.B.ld;
    g.accumulate = 0;
    g.targets = c.targets ? c.targets + m0 : nullptr, g.v0 = c.v0;
    g.inv_t = c.inv_t;
    g.stat = reinterpret_cast<float*>(base + pl.stat_off);
    g.tlogit = reinterpret_cast<float*>(base + pl.t_off);
    float* z = reinterpret_cast<float*>(base + pl.z_off);
    *out = RowLogits{z, pl.z_ld, g.stat, pl.parts, pl.width, rows, c.N, c.v0, c.inv_t};
    const bool b_oc = c.w_order == FC_ROW_MAJOR;
    if (pl.sh.splits > 1) return run_planes(EPI_LOGITS, pl.sh, false, b_oc, g, c.N, z, s);
    if (pl.need && c.listed) {
        uint32_t* need = reinterpret_cast<uint32_t*>(base + pl.need_off);
        const hipError_t e = launch_listed_need(*c.listed, rows, c.N, c.v0, pl.width, pl.parts, need, s);
        if (e != hipSuccess) return e;
        g.need = need;
    }
    g.C = pl.keep ? z : nullptr;
    g.ldc = pl.z_ld;
    if (pl.sh.tile == kSkinny) return launch_fused_skinny_logits(g, s);
    g.k_split = pl.sh.k_split, g.splits = 1, g.c_split_stride = 0;
    return launch_fused(EPI_LOGITS, GRP_NONE, pl.sh.tile, false, b_oc, g, s);
}

}  // namespace
}  // namespace fcs

using namespace fcs;

extern "C" {

int64_t fc_fwd_glu_ws_bytes(int64_t M, int64_t K, int64_t N, fc_order w_order, int aligned) {
    if (bad_sizes(M, K, N) || bad_order(w_order)) return -1;
    return glu_plan(M, N, K, w_order == FC_ROW_MAJOR, aligned != 0, false).total;
}

fc_status fc_fwd_glu(const void* X, const void* W, fc_order w_order, const void* bias, fc_act act, void* Z, void* Y,
                     fc_out_dtype y_dtype, int64_t M, int64_t K, int64_t N, void* ws, int64_t ws_bytes, void* stream) {
    if (!X || !W || !Y) return FC_E_INVALID;
    if (bad_order(w_order) || bad_act(act) || bad_sizes(M, K, N)) return FC_E_INVALID;
    if (y_dtype != FC_OUT_BF16 && y_dtype != FC_OUT_F32) return FC_E_INVALID;
    const bool f32 = y_dtype == FC_OUT_F32;
    if (off(X, 2) || off(W, 2) || off(bias, 2) || off(Z, 2) || off(Y, f32 ? 4 : 2)) return FC_E_INVALID;
    const bool aligned = !off(X, 16) && !off(W, 16), b_oc = w_order == FC_ROW_MAJOR;
    GluPlan pl = glu_plan(M, N, K, b_oc, aligned, false);
    if (bad_ws(ws, ws_bytes, pl.total)) return FC_E_INVALID;
    if (overlapping({{Y, M * N * (f32 ? 4 : 2)}, {Z, M * N * 4}, {pl.total ? ws : nullptr, pl.total}},
                    {{X, M * K * 2}, {W, K * N * 4}, {bias, N * 4}}))
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
    g.act = act;
    g.bias = static_cast<const uint16_t*>(bias);
    g.Z = static_cast<uint16_t*>(Z);
    g.vec_out = vec_rows(N, Y, nullptr, Z);
    return done(run_glu(EPI_GLU, pl, b_oc, g, 2 * N, base, s));
}

int64_t fc_bwd_data_glu_ws_bytes(int64_t M, int64_t K, int64_t N, fc_order w_order, int aligned) {
    if (bad_sizes(M, K, N) || bad_order(w_order)) return -1;
    return glu_plan(M, K, N, w_order == FC_COL_MAJOR, aligned != 0, true).total;
}

fc_status fc_bwd_data_glu(const void* dY, const void* W, fc_order w_order, const void* Z, fc_act act, void* dZ, void* H,
                          float* db, int64_t M, int64_t K, int64_t N, void* ws, int64_t ws_bytes, void* stream) {
    if (!dY || !W || !Z || !dZ) return FC_E_INVALID;
    if (bad_order(w_order) || bad_act(act) || bad_sizes(M, K, N)) return FC_E_INVALID;
    if (off(dY, 2) || off(W, 2) || off(Z, 2) || off(dZ, 2) || off(H, 2) || off(db, 4)) return FC_E_INVALID;
    const bool aligned = !off(dY, 16) && !off(W, 16), b_oc = w_order == FC_COL_MAJOR;
    GluPlan pl = glu_plan(M, K, N, b_oc, aligned, true);
    if (bad_ws(ws, ws_bytes, pl.total)) return FC_E_INVALID;
    if (overlapping({{dZ, M * K * 4}, {H, M * K * 2}, {db, K * 8}, {ws, pl.total}},
                    {{dY, M * N * 2}, {W, K * N * 2}, {Z, M * K * 4}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    FusedArgs g;
    hipError_t e;
    if ((e = place(pl.A, dY, &g.A, pl.B, W, &g.B, base, s)) != hipSuccess) return done(e);
    g.C = dZ;
    g.M = M, g.N = K, g.K = N;
    g.lda = pl.A.ld, g.ldb = pl.B.ld, g.ldc = 2 * K;
    g.accumulate = 0;
    g.act = act;
    g.Z = static_cast<uint16_t*>(const_cast<void*>(Z));  // read only
    g.Y = static_cast<uint16_t*>(H);
    g.colpart = db ? reinterpret_cast<float*>(base + pl.parts_off) : nullptr;
    g.vec_out = vec_rows(K, dZ, H, Z);
    // (the large tiles fall back to the first ones where outputs are not aligned: their partial rows)
    const int parts = pl.fused && pl.sh.tile == kRingTile && !g.vec_out ? (int)((M + 127) / 128) * 2 : pl.parts;
    e = run_glu(EPI_DGLU, pl, b_oc, g, K, base, s);
    if (e == hipSuccess && db) e = launch_colsum_parts(g.colpart, db, 2 * K, parts, s);
    return done(e);
}

int64_t fc_bwd_glu_ws_bytes(int64_t M, int64_t N) {
    if (bad_size(M) || bad_size(N)) return -1;
    return glu_bwd_bytes(M, N);
}

fc_status fc_bwd_glu(const void* dY, const void* Z, fc_act act, void* dZ, void* Y, float* db, int64_t M, int64_t N,
                     void* ws, int64_t ws_bytes, void* stream) {
    if (!dY || !Z || (!dZ && !Y && !db) || bad_act(act)) return FC_E_INVALID;
    if (bad_size(M) || bad_size(N)) return FC_E_INVALID;
    if (off(dY, 2) || off(Z, 2) || off(dZ, 2) || off(Y, 2) || off(db, 4)) return FC_E_INVALID;
    const int64_t need = db ? glu_bwd_bytes(M, N) : 0;
    if (bad_ws(ws, ws_bytes, need)) return FC_E_INVALID;
    if (overlapping({{dZ, M * N * 4}, {Y, M * N * 2}, {db, N * 8}, {need ? ws : nullptr, need}},
                    {{dY, M * N * 2}, {Z, M * N * 4}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    hipStream_t s = static_cast<hipStream_t>(stream);
    float* part = db ? static_cast<float*>(ws) : nullptr;
    hipError_t e = launch_glu_bwd(static_cast<const uint16_t*>(dY), static_cast<const uint16_t*>(Z), act,
                                  static_cast<uint16_t*>(dZ), static_cast<uint16_t*>(Y), part, M, N, s);
    if (e == hipSuccess && db) e = launch_colsum_parts(part, db, 2 * N, glu_bwd_parts(M, N), s);
    return done(e);
}

int64_t fc_logprob_ws_bytes(int64_t M, int64_t K, int64_t N, fc_order w_order, int top_k, int aligned) {
    if (bad_sizes(M, K, N) || bad_order(w_order) || top_k < 0 || top_k > kMaxTop || top_k > N) return -1;
    return logits_plan(M, K, N, w_order == FC_ROW_MAJOR, aligned != 0, top_k > 0, false).total;
}

fc_status fc_logprob(const void* X, const void* W, fc_order w_order, const int64_t* targets, int64_t vocab_start,
                     int64_t ignore_index, float temperature, float* logp, float* entropy, float* lse, float* top_logp,
                     int64_t* top_ids, int top_k, int64_t M, int64_t K, int64_t N, void* ws, int64_t ws_bytes,
                     void* stream) {
    if (!X || !W || !lse || !targets != !logp) return FC_E_INVALID;
    if (bad_order(w_order) || bad_sizes(M, K, N) || vocab_start < 0 || bad_temperature(temperature)) return FC_E_INVALID;
    if (top_k < 0 || top_k > kMaxTop || top_k > N || (top_k > 0 && (!top_logp || !top_ids))) return FC_E_INVALID;
    if (off(X, 2) || off(W, 2) || off(targets, 8) || off(logp, 4) || off(entropy, 4) || off(lse, 4) ||
        off(top_logp, 4) || off(top_ids, 8))
        return FC_E_INVALID;
    const bool aligned = !off(X, 16) && !off(W, 16);
    LogitsPlan pl = logits_plan(M, K, N, w_order == FC_ROW_MAJOR, aligned, top_k > 0, false);
    if (bad_ws(ws, ws_bytes, pl.total)) return FC_E_INVALID;
    if (overlapping({{logp, M * 4}, {entropy, M * 4}, {lse, M * 4}, {top_k ? top_logp : nullptr, M * top_k * 4},
                     {top_k ? top_ids : nullptr, M * top_k * 8}, {ws, pl.total}},
                    {{X, M * K * 2}, {W, K * N * 2}, {targets, M * 8}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    const uint16_t *x, *w;
    hipError_t e;
    if ((e = place(pl.A, X, &x, pl.B, W, &w, base, s)) != hipSuccess) return done(e);
    const LogitsCall call{w_order, targets, vocab_start, 1.0f / temperature, K, N, nullptr};
    for (int64_t m0 = 0; m0 < M; m0 += pl.rows) {
        RowLogits r;
        if ((e = run_logits(pl, call, x, w, m0, std::min(pl.rows, M - m0), base, &r, s)) != hipSuccess) return done(e);
        const LogprobOut o{targets ? targets + m0 : nullptr, ignore_index, reinterpret_cast<const float*>(base + pl.t_off),
                           logp ? logp + m0 : nullptr, entropy ? entropy + m0 : nullptr, lse + m0,
                           top_k ? top_logp + m0 * top_k : nullptr, top_k ? top_ids + m0 * top_k : nullptr, top_k};
        if ((e = launch_logprob_finish(r, o, s)) != hipSuccess) return done(e);
    }
    return FC_OK;
}

int64_t fc_distill_fwd_ws_bytes(int64_t M, int64_t K, int64_t N, fc_order w_order, int aligned) {
    if (bad_sizes(M, K, N) || bad_order(w_order)) return -1;
    return logits_plan(M, K, N, w_order == FC_ROW_MAJOR, aligned != 0, true, true).total;
}

fc_status fc_distill_fwd(const void* X, const void* W, fc_order w_order, const int64_t* ids, const float* tlogits,
                         int top_n, int64_t vocab_start, float temperature, float* lse, float* slogits, float* loss,
                         int64_t M, int64_t K, int64_t N, void* ws, int64_t ws_bytes, void* stream) {
    if (!X || !W || !ids || !tlogits || !lse || !slogits || !loss) return FC_E_INVALID;
    if (bad_order(w_order) || bad_sizes(M, K, N) || vocab_start < 0 || bad_temperature(temperature)) return FC_E_INVALID;
    if (top_n < 1 || top_n > kMaxTop) return FC_E_INVALID;
    if (off(X, 2) || off(W, 2) || off(ids, 8) || off(tlogits, 4) || off(lse, 4) || off(slogits, 4) || off(loss, 4))
        return FC_E_INVALID;
    const bool aligned = !off(X, 16) && !off(W, 16);
    LogitsPlan pl = logits_plan(M, K, N, w_order == FC_ROW_MAJOR, aligned, true, true);
    if (bad_ws(ws, ws_bytes, pl.total)) return FC_E_INVALID;
    if (overlapping({{lse, M * 4}, {slogits, M * top_n * 4}, {loss, M * 4}, {ws, pl.total}},
                    {{X, M * K * 2}, {W, K * N * 2}, {ids, M * top_n * 8}, {tlogits, M * top_n * 4}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    const uint16_t *x, *w;
    hipError_t e;
    if ((e = place(pl.A, X, &x, pl.B, W, &w, base, s)) != hipSuccess) return done(e);
    for (int64_t m0 = 0; m0 < M; m0 += pl.rows) {
        const Listed t{ids + m0 * top_n, tlogits + m0 * top_n, top_n, nullptr, nullptr};
        const LogitsCall call{w_order, nullptr, vocab_start, 1.0f / temperature, K, N, &t};
        RowLogits r;
        if ((e = run_logits(pl, call, x, w, m0, std::min(pl.rows, M - m0), base, &r, s)) != hipSuccess) return done(e);
        if ((e = launch_distill_finish(r, t, lse + m0, slogits + m0 * top_n, loss + m0, s)) != hipSuccess) return done(e);
    }
    return FC_OK;
}

// the gradient's own workspace, then the rows' targets and weights and the listed probabilities
static int64_t listed_bytes(int64_t M, int top_n) { return up(M * 8, 256) + up(M * 4, 256) + up(M * top_n * 4, 256); }

int64_t fc_distill_bwd_ws_bytes(int64_t M, int64_t K, int64_t N, fc_order w_order, int top_n, int aligned) {
    if (bad_sizes(M, K, N) || bad_order(w_order) || top_n < 1 || top_n > kMaxTop) return -1;
    return logits_bwd_ws_bytes(M, K, N, w_order, aligned != 0) + listed_bytes(M, top_n);
}

fc_status fc_distill_bwd(const void* X, const void* W, fc_order w_order, const int64_t* ids, const float* tlogits,
                         int top_n, int64_t vocab_start, float temperature, const float* slogits, const float* lse,
                         const float* grad, void* dX, fc_out_dtype dx_dtype, void* dW, fc_out_dtype dw_dtype, int64_t M,
                         int64_t K, int64_t N, void* ws, int64_t ws_bytes, void* stream) {
    if (!X || !W || !ids || !tlogits || !slogits || !lse || !grad || !dX || !dW) return FC_E_INVALID;
    if (bad_order(w_order) || bad_sizes(M, K, N) || vocab_start < 0 || bad_temperature(temperature)) return FC_E_INVALID;
    if (top_n < 1 || top_n > kMaxTop) return FC_E_INVALID;
    if (dx_dtype != FC_OUT_BF16 && dx_dtype != FC_OUT_F32) return FC_E_INVALID;
    if (dw_dtype < FC_OUT_BF16 || dw_dtype > FC_OUT_F32_ACCUMULATE) return FC_E_INVALID;
    const bool xf32 = dx_dtype == FC_OUT_F32, wf32 = dw_dtype != FC_OUT_BF16;
    if (off(X, 2) || off(W, 2) || off(ids, 8) || off(tlogits, 4) || off(slogits, 4) || off(lse, 4) || off(grad, 4) ||
        off(dX, xf32 ? 4 : 2) || off(dW, wf32 ? 4 : 2))
        return FC_E_INVALID;
    const bool aligned = !off(X, 16) && !off(W, 16);
    const int64_t own = logits_bwd_ws_bytes(M, K, N, w_order, aligned), need = own + listed_bytes(M, top_n);
    if (bad_ws(ws, ws_bytes, need)) return FC_E_INVALID;
    if (overlapping({{dX, M * K * (xf32 ? 4 : 2)}, {dW, K * N * (wf32 ? 4 : 2)}, {ws, need}},
                    {{X, M * K * 2}, {W, K * N * 2}, {ids, M * top_n * 8}, {tlogits, M * top_n * 4},
                     {slogits, M * top_n * 4}, {lse, M * 4}, {grad, M * 4}}))
        return FC_E_INVALID;
    const fc_status st = current_device_status();
    if (st != FC_OK) return st;
    (void)hipGetLastError();
    hipStream_t s = static_cast<hipStream_t>(stream);
    char* base = static_cast<char*>(ws);
    int64_t* targets = reinterpret_cast<int64_t*>(base + up(own, 256));
    float* gw = reinterpret_cast<float*>(targets) + up(M * 8, 256) / 4;
    float* p = gw + up(M * 4, 256) / 4;
    const Listed t{ids, tlogits, top_n, slogits, p};
    hipError_t e = launch_listed_prep(t, grad, 1.0f / temperature, M, p, gw, targets, s);
    if (e != hipSuccess) return done(e);
    LogitsBwd b;
    b.X = X, b.W = W, b.w_order = w_order;
    b.targets = targets, b.v0 = vocab_start, b.ignore = INT64_MIN;
    b.lse = lse, b.gw = gw;
    b.inv_t = 1.0f / temperature, b.listed = &t;
    b.dX = dX, b.dx_f32 = xf32, b.dW = dW, b.dw_dtype = dw_dtype;
    b.M = M, b.K = K, b.N = N;
    return done(run_logits_bwd(b, base, s));
}

}  // extern "C"
