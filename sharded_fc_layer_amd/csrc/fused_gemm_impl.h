// The general kernel of the fused operators: one tile of a product and its
// epilogue. Built in fused_gemm_*.hip, through fused_gemm_table.inc.
//
// Structure (256 threads = 4 wave64s, block tile BM x BN, 32-value reduction
// stages in a ring of S = 4 LDS slots): global data goes straight into LDS with
// 16 bytes per lane, chunks past the tile's rows or the end of the reduction
// read zeros through an out-of-range offset; stage t + S is requested as soon
// as every wave has read stage t. Eight slots measured the same with a block to
// a CU, and slower with more (48 rows of 16 experts, 2048 x 6144: 62 us against
// 99, since fewer blocks fit a CU). Layouts, swizzles and operand reads are
// those of gemm_common.h. Each stage's buffer descriptor starts at that
// stage's first row or column, so operands may be of any size. A reduction
// length may differ from block to block (ragged groups) and may be zero. ANY:
// rows of the operands start at any element (AnyLoads).
//
// Bound by the time of a stage, mostly its loads' (1900 x 2100 outputs over
// 2000: 36.3 us, 440 TFLOP/s), and with few rows by reading B (48 rows that
// all 16 of those experts have a share of: 403 MB in 70 us, 5.8 TB/s; W with
// its reduction contiguous 76).
#pragma once

#include <type_traits>

#include "fused_epilogue.h"

namespace fcs {
namespace {

// Loads of one operand tile of R rows (output index) x 32 reduction values,
// shared by the 4 waves in instructions of 64 chunks of 16 bytes. A tile of
// 32 rows has two of them, which waves 2 and 3 repeat (the same bytes into
// the same place), so that every wave counts the same loads.
template <int R, bool OC>
struct StageLoads {
    static constexpr int kAll = R / 16, kInstr = kAll >= 4 ? kAll / 4 : 1;
    static_assert(!OC || R == 128, "output-contiguous tiles have 128 rows");
    uint32_t base[kInstr];  // byte offset within a stage, or kOOB
    int kk[kInstr];         // reduction index of the chunk within a stage
    static constexpr __device__ int slot(int wave, int j) { return (wave * kInstr + j) % kAll; }

    __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int64_t rows) {
#pragma unroll
        for (int j = 0; j < kInstr; ++j) {
            if (!OC) {
                const int i = slot(wave, j) * 16 + (lane >> 2);
                const int c = (lane & 3) ^ ((lane >> 4) & 3);
                kk[j] = 8 * c;
                base[j] = i < rows ? (uint32_t)((i * ld + 8 * c) * 2) : kOOB;
            } else {
                constexpr int CPR = R / 8, RPI = 64 / CPR;
                const int k = slot(wave, j) * RPI + lane / CPR;
                const int c = (lane % CPR) ^ oc_swizzle(k);
                kk[j] = k;
                base[j] = 8 * c < rows ? (uint32_t)((k * ld + 8 * c) * 2) : kOOB;
            }
        }
    }

    // `p`: the tile's first row at the stage's first reduction value; `left`:
    // reduction values from there to the end (none: every chunk reads zeros,
    // and nothing is read at p)
    __device__ __forceinline__ void issue(const uint16_t* p, char* region, int left, int wave) const {
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, 0x7FFFFFFF, kRsrcWord3);
#pragma unroll
        for (int j = 0; j < kInstr; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)(region + slot(wave, j) * 1024), 16,
                                                     kk[j] < left ? base[j] : kOOB, 0, 0, 0);
    }
};

// The same tile of an operand whose rows start anywhere: through registers
// (gfx950 takes global vectors at any element's address), into the same places
// in LDS. Q sets of registers, so that loads have Q stages to land.
//
// All stages but the last load without masks: rows and columns outside the
// product load others' values instead (the last row there is, the first
// columns; a chunk across the last column runs into the next row), which only
// reach results that nobody stores. The last stage, after which no row may
// follow, reads zeros past the end of the reduction, and takes a chunk that
// would run past the operand's last value (`end`) one by one.
template <int R, bool OC, int Q>
struct AnyLoads {
    typedef StageLoads<R, OC> Places;
    static constexpr int kInstr = Places::kInstr;
    uint32_t at[kInstr];        // element offset within a stage
    int kk[kInstr], n[kInstr];  // reduction index; values inside the product (OC: columns, else row there or not)
    u16x8 v[Q][kInstr];

    __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int64_t rows) {
#pragma unroll
        for (int j = 0; j < kInstr; ++j) {
            if (!OC) {
                const int i = Places::slot(wave, j) * 16 + (lane >> 2);
                kk[j] = 8 * ((lane & 3) ^ ((lane >> 4) & 3));
                n[j] = i < rows;
                at[j] = (uint32_t)((i < rows ? i : rows - 1) * ld + kk[j]);
            } else {
                constexpr int CPR = R / 8, RPI = 64 / CPR;
                kk[j] = Places::slot(wave, j) * RPI + lane / CPR;
                const int c = 8 * ((lane % CPR) ^ oc_swizzle(kk[j]));
                n[j] = c >= rows ? 0 : rows - c < 8 ? (int)(rows - c) : 8;
                at[j] = (uint32_t)(kk[j] * ld + (c < rows ? c : 0));
            }
        }
    }
    // `left` values of the reduction from the stage's first on
    __device__ __forceinline__ void load(int set, const uint16_t* p, int left, const uint16_t* end) {
        if (left >= kBK + (OC ? 8 : 0)) {  // (a chunk spans up to 8 rows of a very narrow operand)
#pragma unroll
            for (int j = 0; j < kInstr; ++j) v[set][j] = *reinterpret_cast<const u16x8_any*>(p + at[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kInstr; ++j) {
                const int there = OC ? (kk[j] < left ? n[j] : 0) : n[j] ? left - kk[j] : 0;
                u16x8 w{0, 0, 0, 0, 0, 0, 0, 0};
                if (there > 0) {
                    if (p + at[j] + 8 <= end)
                        w = *reinterpret_cast<const u16x8_any*>(p + at[j]);
                    else
                        w = load8(p + at[j], there);
                }
                if constexpr (!OC) {  // values past the end of the reduction: zeros
#pragma unroll
                    for (int e = 1; e < 8; ++e) w[e] = e < there ? w[e] : (uint16_t)0;
                }
                v[set][j] = w;
            }
        }
    }
    __device__ __forceinline__ void store(int set, char* region, int wave, int lane) const {
#pragma unroll
        for (int j = 0; j < kInstr; ++j)
            *reinterpret_cast<u16x8*>(region + Places::slot(wave, j) * 1024 + lane * 16) = v[set][j];
    }
};

template <EpiMode MODE, GroupMode GRP, int BM, int BN, int WR, int WC, bool A_OC, bool B_OC, bool ANY>
__global__ __launch_bounds__(kThreads) void fused_gemm_kernel(FusedArgs g) {
    static_assert(WR * WC == 4, "four waves");
    constexpr int S = kStages;
    constexpr int WTM = BM / WR, WTN = BN / WC, TM = WTM / 32, TN = WTN / 32;
    constexpr int kABytes = BM * kBK * 2, kStageBytes = (BM + BN) * kBK * 2;
    typedef StageLoads<BM, A_OC> LoadA;
    typedef StageLoads<BN, B_OC> LoadB;
    constexpr int L = LoadA::kInstr + LoadB::kInstr;
    __shared__ __attribute__((aligned(1024))) char smem[S * kStageBytes];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave_m = wave / WC, wave_n = wave % WC;
    const int wm0 = wave_m * WTM, wn0 = wave_n * WTN;

    const TilePos t = tile_position<BM, BN, GRP>(g);
    if (!t.any) return;  // the whole block: no wave waits for another yet
    const int nkt = (int)((t.kend - t.kbeg + kBK - 1) / kBK);

    // the tile's first row (column) of each operand at reduction value 0
    const int64_t a0 = t.row0 + t.m0;
    const uint16_t* pa = g.A + (A_OC ? a0 : a0 * g.lda);
    const uint16_t* pb = g.B + (GRP == GRP_ROWS ? (int64_t)t.e * g.b_stride : 0) + (B_OC ? t.n0 : t.n0 * g.ldb);
    const int64_t sa = A_OC ? g.lda : 1, sb = B_OC ? g.ldb : 1;
    constexpr int Q = S / 2;  // register sets of AnyLoads
    std::conditional_t<ANY, AnyLoads<BM, A_OC, Q>, LoadA> da;
    std::conditional_t<ANY, AnyLoads<BN, B_OC, Q>, LoadB> db;
    da.init(wave, lane, g.lda, t.M - t.m0);
    db.init(wave, lane, g.ldb, g.N - t.n0);

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    if (nkt > 0) {
        const int len = (int)(t.kend - t.kbeg);
        pa += t.kbeg * sa, pb += t.kbeg * sb;
        // stages past the end of the reduction read zeros everywhere, so every
        // iteration issues and waits for the same number of loads
        if constexpr (ANY) {
            // stages 0 and 1 go to LDS at once; 2 .. Q + 1 wait in registers
#pragma unroll
            for (int s = 0; s < Q; ++s) {
                da.load(s, pa + s * kBK * sa, len - s * kBK, g.a_end);
                db.load(s, pb + s * kBK * sb, len - s * kBK, g.b_end);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                da.store(s, smem + s * kStageBytes, wave, lane);
                db.store(s, smem + s * kStageBytes + kABytes, wave, lane);
                da.load(s, pa + (s + Q) * kBK * sa, len - (s + Q) * kBK, g.a_end);
                db.load(s, pb + (s + Q) * kBK * sb, len - (s + Q) * kBK, g.b_end);
            }
            waitcnt<63, 0>();
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                char* st = smem + s * kStageBytes;
                da.issue(pa + s * kBK * sa, st, len - s * kBK, wave);
                db.issue(pb + s * kBK * sb, st + kABytes, len - s * kBK, wave);
            }
            waitcnt<(S - 1) * L, 0>();
        }
        __builtin_amdgcn_s_barrier();

        bf16x8 fa0[TM], fb0[TN], fa1[TM], fb1[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) fa0[i] = fragment<BM, A_OC>(smem, wm0 + i * 32, 0, lane);
#pragma unroll
        for (int j = 0; j < TN; ++j) fb0[j] = fragment<BN, B_OC>(smem + kABytes, wn0 + j * 32, 0, lane);

        constexpr int kMfmas = TM * TN, kReads = kMfmas == 4 ? 2 : TM + TN;
        constexpr int kAhead = ANY ? Q + 2 : S;
        const uint16_t* na = pa + kAhead * kBK * sa;
        const uint16_t* nb = pb + kAhead * kBK * sb;
        // (Q stages at a time for the register sets' sake; stages past the end
        // multiply zeros)
        for (int k = 0; k < nkt; k += ANY ? Q : 1)
#pragma unroll
        for (int h = 0; h < (ANY ? Q : 1); ++h) {
            const int kh = k + h;
            char* st = smem + (kh % S) * kStageBytes;
            // MFMAs, LDS reads and loads alternate: a wave waits to issue a
            // read or a load while the other waves' are taken, and its matrix
            // unit works meanwhile (255 tiles over a reduction of 2000, one to a CU:
            // 46.7 us with reads and loads in front of the MFMAs, 36.3 so)
#pragma unroll
            for (int q = 0; q < kMfmas; ++q) {
                acc[q / TN][q % TN] =
                    __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb0[q % TN], fa0[q / TN], acc[q / TN][q % TN], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = q * kReads; r < (q + 1) * kReads && r < TM + TN; ++r)
                    if (r < TM)
                        fa1[r] = fragment<BM, A_OC>(st, wm0 + r * 32, 1, lane);
                    else
                        fb1[r - TM] = fragment<BN, B_OC>(st + kABytes, wn0 + (r - TM) * 32, 1, lane);
                __builtin_amdgcn_sched_barrier(0);
            }
            // this wave has read all of stage k; stage k + 1 must have landed
            waitcnt<ANY ? 63 : (S - 2) * L, 0>();
            __builtin_amdgcn_s_barrier();
            const char* nx = smem + ((kh + 1) % S) * kStageBytes;
            const int left = len - (kh + kAhead) * kBK;
            // ANY: stage k + 2 into a slot that was left before the last
            // barrier, the loads of stage k + 2 + Q into its registers;
            // else the loads of stage k + S into stage k's slot
            constexpr int kSet = Q == 2 ? 0 : 2;
            char* to = ANY ? smem + ((kh + 2) % S) * kStageBytes : st;
#pragma unroll
            for (int q = 0; q < kMfmas; ++q) {
                acc[q / TN][q % TN] =
                    __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb1[q % TN], fa1[q / TN], acc[q / TN][q % TN], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = q * kReads; r < (q + 1) * kReads && r < TM + TN; ++r)
                    if (r < TM)
                        fa0[r] = fragment<BM, A_OC>(nx, wm0 + r * 32, 0, lane);
                    else
                        fb0[r - TM] = fragment<BN, B_OC>(nx + kABytes, wn0 + (r - TM) * 32, 0, lane);
                if (q == (kMfmas > 1 ? kMfmas - 2 : 0)) {
                    if constexpr (ANY) {
                        da.store((h + kSet) % Q, to, wave, lane);
                        da.load((h + kSet) % Q, na, left, g.a_end);
                    } else {
                        da.issue(na, to, left, wave);
                    }
                }
                if (q == kMfmas - 1) {
                    if constexpr (ANY) {
                        db.store((h + kSet) % Q, to + kABytes, wave, lane);
                        db.load((h + kSet) % Q, nb, left, g.b_end);
                    } else {
                        db.issue(nb, to + kABytes, left, wave);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            na += kBK * sa, nb += kBK * sb;
        }
        waitcnt<0, 0>();  // drain the trailing loads
    }
    // the stages become staging space, a wave's rows of WTN fp32 values each:
    // no wave may still read them
    __builtin_amdgcn_s_barrier();
    static_assert(WTM * WTN * 4 * 4 <= (int)sizeof(smem), "staging space");
    char* stage = smem + wave * (WTM * WTN * 4);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) stage_block<32, WTN>(stage, 32 * i, 32 * j, lane, acc[i][j]);
    Epilogue<MODE, WTN> e(g, t, t.n0 + wn0, lane);
    constexpr int kStep = 64 / (WTN / 8);  // rows per access
    e.template walk<WTM / kStep >= 4 ? 4 : WTM / kStep>(stage, t.m0 + wm0, WTM, output_base<GRP>(g, t), t.tn * WC + wave_n,
                                                        (int)((g.N + BN - 1) / BN) * WC);
    e.finish((int64_t)t.tm * WR + wave_m);
}



}  // namespace

}  // namespace fcs
