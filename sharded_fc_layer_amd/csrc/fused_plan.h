// Plans of the fused operators' products, shared by their C ABI files
// (fused_*api.hip): argument checks, operands' places, the estimated times
// that choose a kernel, a tile and reduction slices, and the launch of a
// product. Host code; every function is internal to its file.
//
// Every plan is a function of sizes, orders, types and operand alignment
// alone, so that the workspace queries and the calls agree. Nothing is
// allocated, kept or synchronized: workspaces are the caller's.
#pragma once

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
// Both operands' places: the caller's memory, or the copies (one launch). A
// plan says `aligned` of both or of neither; an operand that fits as it is
// stays where it is, whatever the other one does.
hipError_t place(Operand& a, const void* pa, const uint16_t** oa, Operand& b, const void* pb, const uint16_t** ob,
                 char* ws, hipStream_t s) {
    auto one = [ws](Operand& o, const void* src, const uint16_t** out) {
        if (o.copy && fits(o.cols, !off(src, 16))) o.copy = false, o.ld = o.cols;
        *out = o.copy ? reinterpret_cast<const uint16_t*>(ws + o.off) : static_cast<const uint16_t*>(src);
        return PadCopy{static_cast<const uint16_t*>(src), const_cast<uint16_t*>(*out), o.copy ? o.rows : 0, o.cols,
                       o.copy ? o.ld : 0};
    };
    const PadCopy ca = one(a, pa, oa), cb = one(b, pb, ob);
    return a.copy || b.copy ? launch_pad_any(ca, cb, s) : hipSuccess;
}

// Tile and reduction slices of one product.
struct Shape {
    int tile, splits;
    int64_t k_split;
    double us;  // estimated time
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

// Estimated times in microseconds, fitted to measurements on one MI355X
// (outputs 128 x 128 to 8192 x 8192, reductions 40 to 4104):
//  * a round of up to 256 ring tiles takes 15 and 1.1 for each 64-value stage,
//    of which a reduction that is not head plus periods has up to 5 more (136
//    tiles: 19.2 at a reduction of 72, 49.5 at 2056; 1024 tiles at 2048: 213);
//  * a round of the general kernel's tiles 5 and 0.65 for each 32-value stage
//    with a block to a CU, 7 and 1.0 with two, from memory (168 tiles at 3904: 73;
//    4096 tiles at 2048: 577; operands that lie in the caches take 0.37 to 0.5);
//    where rows start anywhere 2 more and 1.3 of the stages' time; tiles of 32
//    or 64 rows 0.4 of it (391 tiles of 64 rows at 2048: 36 with W in the
//    caches, 55 from memory, where the next bound says 44);
//  * neither reads, writes or copies faster than 5 TB/s (16 experts' weights of
//    403 MB against 48 rows: 70);
//  * a launch 3; a split reduction's second launch 4, its planes at 6 TB/s (252
//    tiles of three slices at 1001: 18.7 and 6.6);
//  * copies 3, read and written at 3.5 TB/s.
double ring_us(int64_t tiles, int64_t K, bool ragged, double bytes) {
    const int64_t n = (K + 63) / 64;
    const bool head = !ragged && K % 64 == 0 && (n % 6 == 2 || n % 6 == 4) && n > 6;
    const double stages = ragged ? (double)n + 2.5 : head ? (double)n : (double)up(n, 6);
    return 3 + std::max((double)((tiles + 255) / 256) * (15 + 1.1 * stages), bytes / 5e6);
}
double small_us(int tile, int64_t blocks, int64_t K, bool any, double bytes) {
    const double stages = (double)((K + 31) / 32) * (tile == 0 ? 1.0 : 0.4) * (any ? 1.3 : 1.0), more = any ? 2 : 0;
    const double us = blocks <= 256 ? 5 + more + 0.65 * stages : (double)((blocks + 511) / 512) * (7 + more + 1.0 * stages);
    return 3 + std::max(us, bytes / 5e6);
}
double planes_us(int64_t slices, int64_t M, int64_t N) {
    return 4 + (double)slices * (double)M * (double)plane_ld(N) * 8 / 6e6;
}
// what a product reads
double operand_bytes(int64_t M, int64_t N, int64_t K) { return 2.0 * (double)K * (double)(M + N); }
double copy_us(int64_t bytes) { return 3 + (double)bytes * 2 / 3.5e6; }

// The general kernel's best form with a tile. A product with few tiles may split
// a long reduction, 128 values to a slice at least.
Shape tile_shape(int tile, int64_t M, int64_t N, int64_t K, bool any, bool may_split) {
    const int64_t tiles = tiles_of(tile, M, N);
    const double bytes = operand_bytes(M, N, K);
    Shape best{tile, 1, up(K, 64), small_us(tile, tiles, K, any, bytes)};
    if (!may_split || tiles > 256) return best;
    for (int s = 2; s <= 16; ++s) {
        const int64_t k_split = up((K + s - 1) / s, 32);
        if (k_split < 128) break;
        const int slices = (int)((K + k_split - 1) / k_split);
        const double us = small_us(tile, tiles * slices, k_split, any, bytes) + planes_us(slices, M, N);
        if (us < best.us) best = Shape{tile, slices, k_split, us};
    }
    return best;
}
// ... with the tile that the rows say
Shape small_shape(int64_t M, int64_t N, int64_t K, bool a_oc, bool any, bool may_split) {
    return tile_shape(a_oc || M > 64 ? 0 : M <= 32 ? 1 : 3, M, N, K, any, may_split);
}
// ... with lower tiles as well where they give no CU a second block: for the
// gated layers and the logits, whose epilogues weigh more. Measured (us,
// weights in the caches) with tiles of 128, 64 and 32 rows: gradient of 1500 x
// 600 -> 1100 31.8, 19.7 (216 tiles); 200 x 2048 -> 5632 25.0, 19.3 (176), 26.7
// (308); 256 x 2048 -> 2 x 2048 19.3, 16.7, 14.2 (256); 100 x 1024 -> 2 x 4096
// 17.6, 13.7, 12.4 (256); but 200 x 2048 -> 2 x 5632 21.5, 26.6 (352), and logits
// of 200 x 1024 -> 16000 24.4, 27.6 (500). With slices: 500 x 4096 -> 2 x 1000
// 32.6 (3 slices), 30.7 (4), 44.2 (1).
Shape low_shape(int64_t M, int64_t N, int64_t K, bool any, bool may_split) {
    Shape best = small_shape(M, N, K, false, any, may_split);
    for (int tile : {3, 1}) {
        if (tiles_of(tile, M, N) > 256) continue;
        const Shape sh = tile_shape(tile, M, N, K, any, may_split);
        if (sh.us <= best.us) best = sh;
    }
    return best;
}
// The ring kernel's, if it takes the product, without any copies it needs.
Shape ring_shape(int64_t M, int64_t N, int64_t K, bool a_oc, bool b_oc, int64_t lda, int64_t ldb) {
    const bool takes = ring_takes(GRP_NONE, a_oc, b_oc, N, K, lda, ldb);
    return Shape{kRingTile, 1, up(K, 64), takes ? ring_us(tiles_of(kRingTile, M, N), K, false, operand_bytes(M, N, K)) : 1e30};
}
// The better of both for one product, whose operands' rows are acols and bcols values.
Shape shape_of(int64_t M, int64_t N, int64_t K, bool a_oc, bool b_oc, int64_t acols, int64_t bcols, bool aligned,
               bool low = false) {
    const bool any = !fits(acols, aligned) || !fits(bcols, aligned);
    const Shape small = low ? low_shape(M, N, K, any, true) : small_shape(M, N, K, a_oc, any, true);
    Shape ring = ring_shape(M, N, K, a_oc, b_oc, ring_ld(acols, aligned), ring_ld(bcols, aligned));
    const int64_t bytes = (fits(acols, aligned) ? 0 : M * K * 2) + (fits(bcols, aligned) ? 0 : N * K * 2);
    if (bytes) ring.us += copy_us(bytes);
    return ring.us < small.us ? ring : small;
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
    p.wscale = nullptr;
    p.c_split_stride = g.M * p.ldc;
    const hipError_t e = launch_fused(EPI_STORE, GRP_NONE, sh.tile, a_oc, b_oc, p, s);
    return e != hipSuccess ? e : launch_split_epilogue(mode, g, planes, p.ldc, sh.splits, s);
}

// A product of `cols` columns left in its planes (one, or a split reduction's),
// then the epilogue that reads them.
hipError_t run_planes(EpiMode mode, const Shape& sh, bool a_oc, bool b_oc, const FusedArgs& g, int64_t cols,
                      float* planes, hipStream_t s) {
    FusedArgs p = g;
    p.C = planes;
    p.N = cols;
    p.ldc = plane_ld(cols);
    p.out_f32 = 1;
    p.vec_out = 1;
    p.accumulate = 0;
    p.wscale = nullptr;
    p.k_split = sh.k_split, p.splits = sh.splits;
    p.c_split_stride = sh.splits > 1 ? g.M * p.ldc : 0;
    const hipError_t e = launch_fused(EPI_STORE, GRP_NONE, sh.tile, a_oc, b_oc, p, s);
    if (e != hipSuccess) return e;
    return mode == EPI_LOGITS ? launch_row_logits(g, planes, p.ldc, sh.splits, s)
                              : launch_split_glu(mode, g, planes, p.ldc, sh.splits, s);
}

// The few-row kernel against the general one (24 rows, outputs 28000: 16.7
// against 4.8 us at a reduction of 72, 38.5 against 28.3 at 2056; one row, 8192
// outputs, 2048: 7.0 against 12.3): it reads a narrow W at once, but its blocks
// of 16 columns cost more where they are many.
bool skinny_pays(int64_t M, int64_t N, int64_t K) { return N <= (M <= 16 ? 16384 : 8192) && K >= 256; }

bool bad_sizes(int64_t M, int64_t K, int64_t N) {
    return bad_size(M) || bad_size(K) || bad_size(N);
}

int bwd_act_parts(int64_t M, int64_t N) {
    // about 2048 blocks, at least 16 rows to each
    const int64_t cols = (N + 255) / 256;
    return (int)std::max<int64_t>(1, std::min<int64_t>({(M + 15) / 16, 2048 / cols, 65535}));
}

}  // namespace
}  // namespace fcs
