// What is done with a vocabulary projection's logits besides the cross entropy
// (gfx950): statistics of rows whose logits lie in fp32 planes, log
// probabilities with their entropy and the most likely alternatives, and a
// teacher's listed tokens: their loss and their share of the gradient.
//
// With m a row's largest logit, T the temperature, e_j = exp((z_j - m) / T),
// s = sum_j e_j and w = sum_j e_j (z_j - m) / T:
//   lse = m / T + log s,  log p_j = (z_j - m) / T - log s,  entropy = log s - w / s,
// and a distillation's loss = sum_k p_k (log p_k - log q_k) over the listed
// tokens, q_k as p_j. None of these subtracts large numbers that are nearly
// equal (lse alone has the size of z / T, which is 1e4 and more where T is
// small, and is rounded so). Sets of columns
// (m, s, w) are joined by scaling both to the larger maximum.
//
// The k largest logits without reading all of them again: ordered by value,
// then by lowest index, the k first elements lie in the k first blocks of
// columns, ordered by their maximum, then by lowest index (each of k earlier
// blocks has an element in front of everything in a later one). So a row's
// block maxima are searched first, then the k blocks' columns.
//
// Bound by the latency of a row's few dependent reads, which its neighbours
// hide where there are many (one row: its waves wait in 64 % of their cycles),
// and by the loads of the chosen columns (8192 rows, k = 64: 358 MB at 2.8
// TB/s). 32000 columns (us): 8192 rows, k = 20: 49 and k = 64: 128, beside their
// product's 849; one row, k = 20: 11. Reading all logits again would be 210 for
// 8192 rows. Where a row's block maxima do not fit LDS (16 rows to a block, from
// 114689 columns on) every step of the search reads them from the caches: calls
// of 8192 rows over 2048, without alternatives, with k = 20, with 64: 112000
// columns 2744, 3390, 3417, 128256 columns 3194, 3928, 4086.
#include <algorithm>

#include "fused_common.h"

namespace fcs {
namespace {

struct Stats {
    float mx, sum, mean;  // maximum; sum of e; sum of e (z - mx) / T
};

// An infinite maximum counts as 0 where it is subtracted (see ring_stats).
__device__ __forceinline__ float finite_ref(float mx) { return __builtin_isinf(mx) ? 0.0f : mx; }

__device__ __forceinline__ void join_stats(Stats& a, const Stats& b, float inv_t) {
    const float top = fmaxf(a.mx, b.mx), ref = finite_ref(top);
    // a set that is empty (its maximum says nothing) adds nothing; one whose
    // share underflows leaves nothing of its mean either: a distance past 1e4 is one
    const float da = a.sum != 0.0f ? (finite_ref(a.mx) - ref) * inv_t : 0.0f;
    const float db = b.sum != 0.0f ? (finite_ref(b.mx) - ref) * inv_t : 0.0f;
    const float fa = exp_f32(da), fb = exp_f32(db);
    a.mean = fa * (a.mean + a.sum * fmaxf(da, -1e4f)) + fb * (b.mean + b.sum * fmaxf(db, -1e4f));
    a.sum = a.sum * fa + b.sum * fb;
    a.mx = top;
}
// The planes of a split product, 256 columns of one row to a wave, 4 to a lane: their
// sum, which is left in plane 0, and its statistics.
__global__ __launch_bounds__(256) void row_logits_kernel(FusedArgs g, float* __restrict__ planes, int64_t pld,
                                                         int splits) {
    const int lane = threadIdx.x & 63;
    const int parts = (int)((g.N + kLogitCols - 1) / kLogitCols), part = blockIdx.x % parts;
    const int64_t m = (int64_t)(blockIdx.x / parts) * 4 + (threadIdx.x >> 6);
    if (m >= g.M) return;  // the whole wave
    const int64_t n = (int64_t)part * kLogitCols + lane * 4;
    f32x4 z{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (n < g.N) {
        float* p = planes + m * pld + n;
        z = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 4
        for (int s = 1; s < splits; ++s) z += *reinterpret_cast<const f32x4*>(p + s * g.M * pld);
        *reinterpret_cast<f32x4*>(p) = z;
        const uint64_t hit = g.targets ? (uint64_t)g.targets[m] - (uint64_t)g.v0 - (uint64_t)n : ~(uint64_t)0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            z[q] = n + q < g.N ? z[q] : -INFINITY;
            if (hit == (uint64_t)q && n + q < g.N) g.tlogit[m] = z[q];
        }
    }
    float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    const float ref = finite_ref(mx);
    float sum = 0.0f, mean = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) add_exp(z[q], ref, g.inv_t * kLog2e, sum, mean);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d), mean += __shfl_xor(mean, d);
    if (lane == 0) {
        float* st = g.stat + (int64_t)part * g.M + m;
        const int64_t step = (int64_t)parts * g.M;
        st[0] = mx;
        st[step] = sum;
        st[2 * step] = mean * kLn2;
    }
}

// Between a wave's writes to LDS and its other lanes' reads (or writes of
// another type) there. The LDS takes one wave's accesses in order, so this
// costs no instruction: it keeps the compiler from moving them past each other.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ float wave_min(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = fminf(v, __shfl_xor(v, d));
    return v;
}
// the smaller one, but -inf and NaN do not count
__device__ __forceinline__ float least_number(float low, float v) { return v > -INFINITY && v < low ? v : low; }

// A value and its index as one number that orders by value, then by lowest
// index; never 0, which stands for nothing. NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint64_t order_key(float z, uint32_t index) {
    z = z != z ? -INFINITY : z + 0.0f;
    const uint32_t b = __builtin_bit_cast(uint32_t, z);
    return (uint64_t)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t b = (uint32_t)(key >> 32);
    return __builtin_bit_cast(float, b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return ~(uint32_t)key; }

// The order of values alone: order_key's upper half.
__device__ __forceinline__ uint32_t order_of(float z) { return (uint32_t)(order_key(z, 0) >> 32); }
__device__ __forceinline__ float value_of(uint32_t order) { return key_value((uint64_t)order << 32); }

constexpr int kFinishThreads = 1024;  // at most

// The statistics of the ROWS rows from m0 on, by a block: thread (row, slice)
// joins every so many-th part of its row, so that with 16 rows a wave's reads
// are whole 64-byte pieces (4096 rows of 250 parts: 30 us with the parts of a
// row over the lanes of a wave, 7 so), then pairwise in a fixed order. Rows past the last
// one repeat it. `maxima` (LDS, rows of `stride`, or none) receives the orders of the parts' maxima.
template <int ROWS, int THREADS>
__device__ __forceinline__ void block_stats(const RowLogits& r, int64_t m0, Stats (*s)[ROWS + 1], uint32_t* maxima, int stride) {
    constexpr int S = THREADS / ROWS;
    const int row = threadIdx.x % ROWS, sl = threadIdx.x / ROWS;
    const int64_t m = m0 + row < r.M ? m0 + row : r.M - 1, step = (int64_t)r.parts * r.M;
    Stats a{-INFINITY, 0.0f, 0.0f};
#pragma unroll 4
    for (int p = sl; p < r.parts; p += S) {
        const float* st = r.stat + (int64_t)p * r.M + m;
        const Stats b{st[0], st[step], st[2 * step]};
        if (maxima) maxima[row * stride + p] = order_of(b.mx);
        join_stats(a, b, r.inv_t);
    }
    // 64 slices to LDS at most, the others' through the lanes of a wave first
    constexpr int T = S > 64 ? 64 : S;
    if constexpr (S > T) {
#pragma unroll
        for (int d = ROWS; d < ROWS * (S / T); d <<= 1) {
            const Stats b{__shfl_xor(a.mx, d), __shfl_xor(a.sum, d), __shfl_xor(a.mean, d)};
            join_stats(a, b, r.inv_t);
        }
    }
    static_assert(ROWS * (S / T) <= 64, "within a wave");
    const int at = sl / (S / T);
    if (sl % (S / T) == 0) s[at][row] = a;
    __syncthreads();
#pragma unroll
    for (int d = T / 2; d > 0; d >>= 1) {
        if (sl % (S / T) == 0 && at < d) {
            join_stats(a, s[at + d][row], r.inv_t);
            s[at][row] = a;
        }
        __syncthreads();
    }
}

// ------------------------------------------------- the largest of a row

__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}

// The 64 R largest keys that a wave has seen, largest first: position 64 r +
// lane is v[r] of that lane.
template <int R>
struct TopList {
    uint64_t v[R];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = 0;
    }
    __device__ __forceinline__ uint64_t at(int i) const {
        return R == 1 || i < 64 ? lane_value(v[0], i) : lane_value(v[R - 1], i - 64);
    }
    // key: the same in all lanes
    __device__ __forceinline__ void insert(uint64_t key, int lane) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint64_t prev = __shfl_up(v[r], 1), last = lane_value(v[r], 63);
            v[r] = v[r] >= key ? v[r] : lane == 0 || prev >= key ? key : prev;
            key = last < key ? last : key;  // what moves on
        }
    }
    // every lane's key that belongs among the first k
    __device__ __forceinline__ void offer(uint64_t key, int k, int lane) {
        uint64_t kth = at(k - 1);
        unsigned long long want = __ballot(key > kth);
        while (want) {
            const uint64_t c = lane_value(key, __builtin_ctzll(want));
            want &= want - 1;
            if (c > kth) {
                insert(c, lane);
                kth = at(k - 1);
            }
        }
    }
};

// What a row's SUBS waves have, joined by all of them: a sum, or the smallest,
// of a value that is the same in a wave's lanes. `slot` is LDS for 2 x 16
// values, used in turn, so that one barrier lies between a value's writes and
// the next but one's. All waves of the block call it.
template <int SUBS>
struct RowJoin {
    int (*slot)[16];
    int wave, first, turn;
    __device__ __forceinline__ void put(int v) {
        if constexpr (SUBS > 1) {
            if ((threadIdx.x & 63) == 0) slot[turn][wave] = v;
            __syncthreads();
        }
    }
    __device__ __forceinline__ int sum(int v) {
        if constexpr (SUBS == 1) return v;
        put(v);
        int s = 0;
#pragma unroll
        for (int w = 0; w < SUBS; ++w) s += slot[turn][first + w];
        turn ^= 1;
        return __builtin_amdgcn_readfirstlane(s);
    }
    __device__ __forceinline__ float smallest(float v) {
        if constexpr (SUBS == 1) return v;
        put(__builtin_bit_cast(int, v));
        float s = INFINITY;
#pragma unroll
        for (int w = 0; w < SUBS; ++w) s = fminf(s, __builtin_bit_cast(float, slot[turn][first + w]));
        turn ^= 1;
        return s;
    }
};

// An order v >= least (which at least k of a row's values reach) that at least
// k, and at most `most`, of its values reach; or, where equal values leave no
// such one, the k-th largest value's. n: how many reach it. By halving between
// low (about the smallest value that is a number) and high (the largest), as
// floats first, where values lie close together, then as orders.
// reach(c): the wave's number of values with an order of at least c.
template <int SUBS, class F>
__device__ __forceinline__ uint32_t reached_by(int k, int most, uint32_t least, float low, float high, RowJoin<SUBS>& join,
                                               int& n, F reach) {
    uint32_t lo = least, hi = order_of(high) + 1;  // k values reach lo, fewer reach hi
    n = 0;
    for (int round = 0; !(n >= k && n <= most) && hi - lo > 1; ++round) {
        uint32_t c = order_of(0.5f * low + 0.5f * high);
        if (round >= 8 || c <= lo || c >= hi) c = lo + (hi - lo) / 2;
        const int here = join.sum(reach(c));
        if (here >= k)
            lo = c, n = here, low = value_of(c);
        else
            hi = c, high = value_of(c);
    }
    return lo;
}

// SUBS waves to a row, ROWS rows to a block. TOP: the largest as well, in
// four steps: a value that k blocks' maxima or a few more reach, by halving
// (k = 100 of 126 blocks: 614 us, and 1146 without one where all were read);
// those blocks (of equal maxima the first ones); their columns' values that
// reach it, into LDS; the place of each by counting those in front of it. Where
// more than kCandidates reach it, what k of the first kCandidates reach takes
// its place; if that is no more (equal values), one wave keeps a sorted list
// instead. (A sorted list of all blocks' maxima and then of k blocks' columns,
// kept by one wave to a row, took 74 us where this takes 49: 8192 rows, 32000
// columns, k = 20.)
constexpr int kCandidates = 256, kMostBlocks = kMaxTop + kMaxTop / 4 + 4;
constexpr int64_t kMaximaBytes = 56 << 10;
// a row's words of LDS: its parts' maxima, if they are there, or the candidates
__host__ __device__ inline int row_words(int parts, int in_lds) {
    const int words = (in_lds ? parts : 0) + (in_lds ? parts & 1 : 0);
    return words > 2 * kCandidates ? words : 2 * kCandidates;
}
template <int SUBS, int ROWS, bool TOP>
__global__ __launch_bounds__(64 * SUBS * ROWS) void logprob_finish_kernel(RowLogits in, LogprobOut out, int in_lds) {
    static_assert(64 * SUBS * ROWS <= kFinishThreads, "a block's waves");
    static_assert(SUBS == 1 || ROWS == 1, "rows of several waves each do not share their barriers");
    __shared__ Stats stats[64][ROWS + 1];
    // a row's maxima, where they fit, and then, in their place, the values found; of this row's waves alone
    extern __shared__ uint64_t row_space[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = wave % SUBS, first = wave - sub, row = wave / SUBS;
    const int64_t m0 = (int64_t)blockIdx.x * ROWS;
    const bool there = m0 + row < in.M;
    const int64_t m = there ? m0 + row : in.M - 1;  // (waves past the last row do its work again and store nothing)

    const int stride = row_words(in.parts, in_lds);
    uint32_t* maxima = reinterpret_cast<uint32_t*>(row_space);
    block_stats<ROWS, 64 * SUBS * ROWS>(in, m0, stats, TOP && in_lds ? maxima : nullptr, stride);
    const Stats a = stats[0][row];
    const float ref = finite_ref(a.mx), log_sum = logf(a.sum);
    if (there && sub == 0 && lane == 0) {
        out.lse[m] = ref * in.inv_t + log_sum;
        if (out.entropy) out.entropy[m] = a.sum == 0.0f ? 0.0f : log_sum - a.mean / a.sum;
        if (out.logp) {
            const int64_t t = out.targets[m];
            const uint64_t at = (uint64_t)t - (uint64_t)in.v0;
            out.logp[m] = t == out.ignore ? 0.0f : at >= (uint64_t)in.N || a.sum == 0.0f ? -INFINITY
                                                 : (out.tlogit[m] - ref) * in.inv_t - log_sum;
        }
    }
    if constexpr (TOP) {
        __shared__ int slots[2][16];
        __shared__ int taken[16][2];
        __shared__ uint32_t chosen[ROWS][kMostBlocks];
        __shared__ int found_n[ROWS];
        maxima += row * stride;
        uint64_t* found = reinterpret_cast<uint64_t*>(maxima);
        auto sync = [] {
            if constexpr (SUBS > 1)
                __syncthreads();
            else
                wave_sync();
        };
        RowJoin<SUBS> join{slots, wave, first, 0};
        const int k = out.k, parts = in.parts;
        auto maximum = [&](int p) { return in_lds ? maxima[p] : order_of(in.stat[(int64_t)p * in.M + m]); };

        // the blocks: a wave's share of them is consecutive
        const int per = (parts + SUBS - 1) / SUBS, p0 = sub * per, p1 = p0 + per < parts ? p0 + per : parts;
        const int most = k + k / 4 + 4;
        uint32_t least = 0;
        int count = parts;  // blocks to be read
        if (4 * parts >= 5 * k && parts * in.width > kCandidates) {
            float low = INFINITY;
            for (int p = p0 + lane; p < p1; p += 64) low = least_number(low, value_of(maximum(p)));
            low = join.smallest(wave_min(low));
            least = reached_by<SUBS>(k, parts > most ? most : k + k / 16 + 2, 0, low, a.mx, join, count, [&](uint32_t c) {
                int n = 0;
                for (int p = p0; p < p1; p += 64) n += __popcll(__ballot(p + lane < p1 && maximum(p + lane) >= c));
                return n;
            });
            if (count > most || count < k) count = k;
        }
        // those above it, and of those that are equal the first ones
        int above = 0, equal = 0;
        for (int p = p0; p < p1; p += 64) {
            const uint32_t o = p + lane < p1 ? maximum(p + lane) : 0;
            above += __popcll(__ballot(p + lane < p1 && o > least));
            equal += __popcll(__ballot(p + lane < p1 && o == least));
        }
        if (lane == 0) taken[wave][0] = above, taken[wave][1] = equal;
        sync();
        int at = 0, equal_at = 0, all_above = 0;
#pragma unroll
        for (int w = 0; w < SUBS; ++w) {
            all_above += taken[first + w][0];
            if (w < sub) at += taken[first + w][0], equal_at += taken[first + w][1];
        }
        const int room = count - all_above;       // of them with a maximum of `least`
        at += equal_at < room ? equal_at : room;
        for (int p = p0; p < p1; p += 64) {
            const uint32_t o = p + lane < p1 ? maximum(p + lane) : 0;
            const unsigned long long below = (1ull << lane) - 1, eq = __ballot(p + lane < p1 && o == least);
            const bool take = p + lane < p1 && (o > least || (o == least && equal_at + __popcll(eq & below) < room));
            const unsigned long long t = __ballot(take);
            if (take) chosen[row][at + __popcll(t & below)] = (uint32_t)(p + lane);
            at += __popcll(t);
            equal_at += __popcll(eq);
        }
        if (sub == 0 && lane == 0) found_n[row] = 0;
        sync();

        // their columns, four to a lane, four loads ahead
        const float* z = in.z + m * in.ld;
        const int total = count * in.width, shift = 31 - __builtin_clz(in.width);
        if (least == 0 && total > kCandidates) {
            // (fewer than 1.25 k parts: a value that k of the maxima of 512 groups of columns reach takes their
            // place. 8192 rows of 16032 columns, k = 128, with the product over 2048: 691 us, and 1359 where the
            // candidates alone tell, in five rounds)
            constexpr int R = 8 / SUBS;  // groups to a lane
            float mx[R];
#pragma unroll
            for (int r = 0; r < R; ++r) mx[r] = -INFINITY;
            for (int e0 = 4 * (sub * 64); e0 < total; e0 += 4 * 256 * SUBS) {
                f32x4 v[4];
                int64_t col[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int e = e0 + u * 256 * SUBS + 4 * lane;
                    col[u] = e < total ? ((int64_t)chosen[row][e >> shift] << shift) + (e & (in.width - 1)) : in.N;
                    v[u] = col[u] < in.N ? *reinterpret_cast<const f32x4*>(z + col[u]) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        if (col[u] + h < in.N) mx[(4 * u + h) % R] = fmaxf(mx[(4 * u + h) % R], v[u][h]);
            }
            // (a group without a number counts as -inf, which all columns reach)
            float low = INFINITY;
            uint32_t o[R];
#pragma unroll
            for (int r = 0; r < R; ++r) o[r] = order_of(mx[r]), low = least_number(low, mx[r]);
            low = join.smallest(wave_min(low));
            int reached;
            least = reached_by<SUBS>(k, k + k / 8 + 2, 0, low, a.mx, join, reached, [&](uint32_t c) {
                int r = 0;
#pragma unroll
                for (int i = 0; i < R; ++i) r += __popcll(__ballot(o[i] >= c));
                return r;
            });
        }
        int n;
        bool sorted = false;
        for (;;) {
            // (compared as floats, unless -inf and NaN count too)
            const bool all = least <= order_of(-INFINITY);
            const float over = value_of(least);
            n = 0;
            for (int e0 = 4 * (sub * 64); e0 < total; e0 += 4 * 256 * SUBS) {
                f32x4 v[4];
                int64_t col[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int e = e0 + u * 256 * SUBS + 4 * lane;
                    col[u] = e < total ? ((int64_t)chosen[row][e >> shift] << shift) + (e & (in.width - 1)) : in.N;
                    // (rows are padded to whole vectors)
                    v[u] = col[u] < in.N ? *reinterpret_cast<const f32x4*>(z + col[u]) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const bool take = (all || v[u][h] >= over) && col[u] + h < in.N;
                        const unsigned long long t = __ballot(take);
                        if (t == 0) continue;
                        int base = n;
                        if constexpr (SUBS > 1) {
                            if (lane == 0) base = atomicAdd(&found_n[row], (int)__popcll(t));
                            base = __builtin_amdgcn_readfirstlane(base);
                        }
                        n += (int)__popcll(t);
                        base += (int)__popcll(t & ((1ull << lane) - 1));
                        if (take && base < kCandidates) found[base] = order_key(v[u][h], (uint32_t)(col[u] + h));
                    }
            }
            sync();
            if constexpr (SUBS > 1) n = found_n[row];
            if (n <= kCandidates || sorted) break;
            float low = INFINITY;
            for (int i = sub * 64 + lane; i < kCandidates; i += 64 * SUBS) low = least_number(low, key_value(found[i]));
            low = join.smallest(wave_min(low));
            int reached;
            const uint32_t more = reached_by<SUBS>(k, most, least, low, a.mx, join, reached, [&](uint32_t c) {
                int r = 0;
                for (int i = sub * 64; i < kCandidates; i += 64 * SUBS)
                    r += __popcll(__ballot((uint32_t)(found[i + lane] >> 32) >= c));
                return r;
            });
            sorted = more == least;  // equal values
            least = more;
            sync();
            if (sub == 0 && lane == 0) found_n[row] = 0;
            sync();
        }
        if (n > kCandidates) {
            if (sub != 0) return;  // (no barrier follows)
            TopList<kMaxTop / 64> top;
            top.clear();
            for (int e0 = 0; e0 < total; e0 += 64) {
                const int e = e0 + lane;
                uint64_t key = 0;
                if (e < total) {
                    const int64_t c = ((int64_t)chosen[row][e >> shift] << shift) + (e & (in.width - 1));
                    if (c < in.N) key = order_key(z[c], (uint32_t)c);
                }
                top.offer(key, k, lane);
            }
#pragma unroll
            for (int r = 0; r < kMaxTop / 64; ++r)
                if (there && 64 * r + lane < k) {
                    out.top_ids[m * k + 64 * r + lane] = (int64_t)key_index(top.v[r]) + in.v0;
                    out.top_logp[m * k + 64 * r + lane] =
                        a.sum == 0.0f ? -INFINITY : (key_value(top.v[r]) - ref) * in.inv_t - log_sum;
                }
            return;
        }
        for (int i = sub * 64 + lane; i < n; i += 64 * SUBS) {
            const uint64_t key = found[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) rank += found[j] > key;
            if (there && rank < k) {
                out.top_ids[m * k + rank] = (int64_t)key_index(key) + in.v0;
                out.top_logp[m * k + rank] = a.sum == 0.0f ? -INFINITY : (key_value(key) - ref) * in.inv_t - log_sum;
            }
        }
    }
}

// ------------------------------------------------- a teacher's tokens

// A row's listed tokens, PER of them to a lane (64 r + lane): ids (-1 where
// there is none), probabilities (0 there) and their logarithms. Returns whether
// the row has any. 1 / T scales the distances from the largest logit, not the
// logits: a finite one times 1 / T may be infinite, which would read as absent;
// a distance that becomes infinite has the probability 0 anyway.
template <int PER>
__device__ __forceinline__ bool teacher_row(const Listed& t, float inv_t, int64_t m, int lane, int64_t (&id)[PER],
                                            float (&p)[PER], float (&logp)[PER]) {
    float mx = -INFINITY;
    bool some = false;
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int i = 64 * r + lane;
        id[r] = i < t.n ? t.ids[m * t.n + i] : -1;
        logp[r] = i < t.n && id[r] >= 0 ? t.tlogits[m * t.n + i] : -INFINITY;
        if (logp[r] == -INFINITY) id[r] = -1;
        some = some || id[r] >= 0;
        mx = fmaxf(mx, logp[r]);
    }
    const bool any = __ballot(some) != 0;
    mx = wave_max(mx);
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        logp[r] = id[r] >= 0 ? (logp[r] - mx) * inv_t : 0.0f;
        p[r] = id[r] >= 0 ? exp_f32(logp[r]) : 0.0f;
        s += p[r];
    }
    s = any ? wave_sum(s) : 1.0f;
    const float ls = logf(s);
#pragma unroll
    for (int r = 0; r < PER; ++r) p[r] /= s, logp[r] -= ls;
    return any;
}

// ROWS rows to a block; their teachers' tokens, a wave to a row. Bound by
// memory: 24 us for 8192 rows of 64 tokens, 119 MB at 4.9 TB/s, of which a
// 128-byte line for each token's logit is 67, the statistics of 250 parts a row
// 25, the tokens 6.
template <int ROWS, int PER>
__global__ __launch_bounds__(kFinishThreads) void distill_finish_kernel(RowLogits in, Listed t, float* __restrict__ lse,
                                                                        float* __restrict__ slogits,
                                                                        float* __restrict__ loss) {
    __shared__ Stats stats[64][ROWS + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    block_stats<ROWS, kFinishThreads>(in, (int64_t)blockIdx.x * ROWS, stats, nullptr, 0);
    const int64_t m = (int64_t)blockIdx.x * ROWS + wave;
    if (wave >= ROWS || m >= in.M) return;  // the whole wave
    const Stats a = stats[0][wave];
    const float ref = finite_ref(a.mx), log_sum = logf(a.sum);
    int64_t id[PER];
    float p[PER], logp[PER];
    const bool any = teacher_row(t, in.inv_t, m, lane, id, p, logp);
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int i = 64 * r + lane;
        const uint64_t at = (uint64_t)id[r] - (uint64_t)in.v0;
        const float z = id[r] >= 0 && at < (uint64_t)in.N ? in.z[m * in.ld + (int64_t)at] : 0.0f;
        if (i < t.n) slogits[m * t.n + i] = z;
        // (halves: the distance of two finite logits may be more than the type holds, its quotient by T not)
        if (p[r] != 0.0f) sum += p[r] * (logp[r] + ((0.5f * ref - 0.5f * z) * (2.0f * in.inv_t) + log_sum));
    }
    sum = wave_sum(sum);
    if (lane == 0) {
        lse[m] = ref * in.inv_t + log_sum;
        loss[m] = any ? sum : 0.0f;
    }
}

// Which blocks of columns hold a token that a row lists: the product's epilogue
// stores no others. 8192 rows of 64 tokens over 32000 columns: 5 us, and the
// product takes 834 us for 849.
// A wave to a row, 1024 words of it at a time in LDS.
constexpr int kNeedWords = 1024;
__global__ __launch_bounds__(256) void listed_need_kernel(Listed t, int64_t M, int64_t N, int64_t v0, int shift, int words,
                                                          uint32_t* __restrict__ need) {
    __shared__ uint32_t bits[4][kNeedWords];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * 4 + wave;
    if (m >= M) return;  // the whole wave, which has its own LDS
    for (int w0 = 0; w0 < words; w0 += kNeedWords) {
        const int here = words - w0 < kNeedWords ? words - w0 : kNeedWords;
        for (int w = lane; w < here; w += 64) bits[wave][w] = 0;
        wave_sync();
        for (int i = lane; i < t.n; i += 64) {
            const int64_t id = t.ids[m * t.n + i];
            const uint64_t at = (uint64_t)id - (uint64_t)v0;
            if (id < 0 || at >= (uint64_t)N) continue;
            const int part = (int)(at >> shift), w = (part >> 5) - w0;
            if (w >= 0 && w < here) atomicOr(&bits[wave][w], 1u << (part & 31));
        }
        wave_sync();
        for (int w = lane; w < here; w += 64) need[(int64_t)(w0 + w) * M + m] = bits[wave][w];
    }
}

// One wave to a row (8192 rows of 64 tokens: 14 us, 6.3 MB in, 2.1 MB out, the
// waves wait in 58 % of their cycles; most rows list no token twice).
template <int PER>
__global__ __launch_bounds__(256) void listed_prep_kernel(Listed t, const float* __restrict__ grad, float inv_t,
                                                          int64_t M, float* __restrict__ p_out, float* __restrict__ gw,
                                                          int64_t* __restrict__ targets) {
    __shared__ __attribute__((aligned(16))) int64_t ids[4][64 * PER];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * 4 + wave;
    if (m >= M) return;  // the whole wave, which has its own LDS
    int64_t id[PER];
    float p[PER], logp[PER], total[PER];
    bool firsts[PER];
    const bool any = teacher_row(t, inv_t, m, lane, id, p, logp);
    if (lane == 0) {
        gw[m] = grad[m] * inv_t;
        targets[m] = any ? -1 : INT64_MIN;
    }
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        total[r] = p[r], firsts[r] = id[r] >= 0;
        ids[wave][64 * r + lane] = id[r];
    }
    wave_sync();
    // tokens that are listed several times count together, in order, at their
    // first place; 16 at a time are looked at first, few rows have any
    for (int i0 = 0; i0 < t.n; i0 += 16) {
        bool again = false;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int64_t other = ids[wave][i0 + e];  // (past the last one: -1)
#pragma unroll
            for (int r = 0; r < PER; ++r) again |= other == id[r] && other >= 0 && i0 + e != 64 * r + lane;
        }
        if (!__ballot(again)) continue;
        for (int i = i0; i < i0 + 16; ++i) {
            const int64_t other = ids[wave][i];
            const float q = i < 64 ? __shfl(p[0], i) : __shfl(p[PER - 1], i - 64);
#pragma unroll
            for (int r = 0; r < PER; ++r)
                if (other == id[r] && other >= 0 && i != 64 * r + lane) {
                    total[r] += q;
                    if (i < 64 * r + lane) firsts[r] = false;
                }
        }
    }
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const int i = 64 * r + lane;
        if (i < t.n) p_out[m * t.n + i] = firsts[r] ? total[r] : -1.0f;
    }
}

// One thread to a listed token, whose entry of D the product's epilogue has
// written as if nothing were listed: it is made again from the kept logit, so D
// is rounded once. 2-byte writes anywhere: 10 us for 8192 rows of 64 tokens, 9
// MB in and 8 MB out, the waves wait in 90 % of their cycles.
__global__ __launch_bounds__(256) void listed_grad_kernel(Listed t, const float* __restrict__ lse,
                                                          const float* __restrict__ gw, float inv_t,
                                                          const float* __restrict__ scale, uint16_t* __restrict__ D,
                                                          int64_t ld, int64_t v0, int64_t c, int64_t count) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= count) return;
    const float p = t.p[i];
    const uint64_t at = (uint64_t)t.ids[i] - (uint64_t)v0;
    if (p < 0.0f || at >= (uint64_t)c) return;  // (a NaN goes on)
    const int64_t m = i / t.n;
    const float w = gw[m] * rcp_f32(*scale);
    reinterpret_cast<__bf16*>(D)[m * ld + (int64_t)at] = (__bf16)(w * (exp_f32(t.slogits[i] * inv_t - lse[m]) - p));
}

}  // namespace

hipError_t launch_row_logits(const FusedArgs& g, float* planes, int64_t pld, int splits, hipStream_t s) {
    const int64_t blocks = (g.M + 3) / 4 * ((g.N + kLogitCols - 1) / kLogitCols);
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL(row_logits_kernel, dim3((unsigned)blocks), dim3(256), 0, s, g, planes, pld, splits);
    return hipGetLastError();
}

template <int SUBS, int ROWS>
static hipError_t logprob_finish(const RowLogits& r, const LogprobOut& o, hipStream_t s) {
    // the maxima of the parts in LDS, unless they are more than it holds beside the rest
    const int64_t bytes = (int64_t)ROWS * r.parts * 4;
    const bool in_lds = o.k > 0 && bytes <= kMaximaBytes;
    const unsigned lds = o.k > 0 ? (unsigned)(ROWS * row_words(r.parts, in_lds) * 4) : 0u;
    const auto fn = o.k > 0 ? logprob_finish_kernel<SUBS, ROWS, true> : logprob_finish_kernel<SUBS, ROWS, false>;
    hipLaunchKernelGGL(fn, dim3((unsigned)((r.M + ROWS - 1) / ROWS)), dim3(64 * SUBS * ROWS), lds, s, r, o, in_lds ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_logprob_finish(const RowLogits& r, const LogprobOut& o, hipStream_t s) {
    if (o.k < 0 || o.k > kMaxTop || r.width < 32 || (r.width & (r.width - 1))) return hipErrorInvalidValue;
    // waves to a row x rows to a block, measured with 32000 columns (us, with the
    // product over 64): 8 x 1, 4 x 1, 1 x 16 for k = 20: 300 rows 37, 36, 45, 1200
    // rows 76, 71, 73, 2048 114, 105, 99, 8192 441, 389, 353; for k = 128: 300 rows
    // 43, 45, 86, 2048 135, 126, 141, 8192 528, 478, 467
    if (r.M < 1024) return logprob_finish<8, 1>(r, o, s);
    return r.M < (o.k > 64 ? 4096 : 2048) ? logprob_finish<4, 1>(r, o, s) : logprob_finish<1, 16>(r, o, s);
}

hipError_t launch_distill_finish(const RowLogits& r, const Listed& t, float* lse, float* slogits, float* loss,
                                 hipStream_t s) {
    if (t.n < 1 || t.n > kMaxTop) return hipErrorInvalidValue;
    const int rows = r.M <= 1024 ? 4 : 16;
    const bool few = t.n <= 64;
    hipLaunchKernelGGL(rows == 4 ? (few ? distill_finish_kernel<4, 1> : distill_finish_kernel<4, 2>)
                                 : (few ? distill_finish_kernel<16, 1> : distill_finish_kernel<16, 2>),
                       dim3((unsigned)((r.M + rows - 1) / rows)), dim3(kFinishThreads), 0, s, r, t, lse, slogits, loss);
    return hipGetLastError();
}

hipError_t launch_listed_need(const Listed& t, int64_t M, int64_t N, int64_t v0, int width, int parts, uint32_t* need,
                              hipStream_t s) {
    if (t.n < 1 || t.n > kMaxTop || width < 1 || (width & (width - 1))) return hipErrorInvalidValue;
    hipLaunchKernelGGL(listed_need_kernel, dim3((unsigned)((M + 3) / 4)), dim3(256), 0, s, t, M, N, v0,
                       31 - __builtin_clz((unsigned)width), (parts + 31) / 32, need);
    return hipGetLastError();
}

hipError_t launch_listed_prep(const Listed& t, const float* grad, float inv_t, int64_t M, float* p, float* gw,
                              int64_t* targets, hipStream_t s) {
    if (t.n < 1 || t.n > kMaxTop) return hipErrorInvalidValue;
    hipLaunchKernelGGL(t.n <= 64 ? listed_prep_kernel<1> : listed_prep_kernel<2>, dim3((unsigned)((M + 3) / 4)), dim3(256),
                       0, s, t, grad, inv_t, M, p, gw, targets);
    return hipGetLastError();
}

hipError_t launch_listed_grad(const Listed& t, const float* lse, const float* gw, float inv_t, const float* scale,
                              uint16_t* D, int64_t ld, int64_t v0, int64_t c, int64_t M, hipStream_t s) {
    const int64_t count = M * t.n;  // at most 2^22 x 128
    hipLaunchKernelGGL(listed_grad_kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, s, t, lse, gw, inv_t,
                       scale, D, ld, v0, c, count);
    return hipGetLastError();
}

}  // namespace fcs
