// What is done with a vocabulary projection's logits besides the cross entropy
// (gfx950): statistics of rows whose logits lie in fp32 planes, log
// probabilities with their entropy and the most likely alternatives, and a
// teacher's listed tokens: their loss and their share of the gradient.
//
// With m a row's largest logit, T the temperature, e_j = exp((z_j - m) / T),
// s = sum_j e_j and w = sum_j e_j (z_j - m) / T:
//   lse = m / T + log s,  log p_j = (z_j - m) / T - log s,  entropy = log s - w / s.
// None of these subtracts large numbers that are nearly equal. Sets of columns
// (m, s, w) are joined by scaling both to the larger maximum.
//
// The k largest logits without reading all of them again: ordered by value,
// then by lowest index, the k first elements lie in the k first blocks of
// columns, ordered by their maximum, then by lowest index (each of k earlier
// blocks has an element in front of everything in a later one). So a row's
// block maxima are searched first, then the k blocks' columns.
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
__device__ __forceinline__ Stats shuffled(const Stats& a, int d) {
    return Stats{__shfl_xor(a.mx, d), __shfl_xor(a.sum, d), __shfl_xor(a.mean, d)};
}

// The planes of a product, 256 columns of one row to a wave, 4 to a lane: their
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
        if (splits > 1) *reinterpret_cast<f32x4*>(p) = z;
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
    for (int q = 0; q < 4; ++q) add_exp(z[q], ref, g.inv_t, sum, mean);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d), mean += __shfl_xor(mean, d);
    if (lane == 0) {
        float* st = g.stat + (int64_t)part * g.M + m;
        const int64_t step = (int64_t)parts * g.M;
        st[0] = mx;
        st[step] = sum;
        st[2 * step] = mean;
    }
}

// The statistics of a row from its parts: those of every 64 SUBS-th part from
// 64 sub + lane on, joined over the wave. All lanes get the same.
__device__ __forceinline__ Stats row_stats(const RowLogits& r, int64_t m, int sub, int subs, int lane) {
    Stats a{-INFINITY, 0.0f, 0.0f};
    const int64_t step = (int64_t)r.parts * r.M;
    for (int p = sub * 64 + lane; p < r.parts; p += 64 * subs) {
        const float* st = r.stat + (int64_t)p * r.M + m;
        join_stats(a, Stats{st[0], st[step], st[2 * step]}, r.inv_t);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) join_stats(a, shuffled(a, d), r.inv_t);
    // (a sum of two products may round differently the other way round)
    auto first = [](float v) { return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v))); };
    return Stats{first(a.mx), first(a.sum), first(a.mean)};
}

// ------------------------------------------------- the largest of a row

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
    // every lane's key that belongs among the first k and is over `least`
    __device__ __forceinline__ void offer(uint64_t key, int k, uint64_t least, int lane) {
        uint64_t kth = at(k - 1);
        unsigned long long want = __ballot(key > (kth > least ? kth : least));
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

constexpr int kFinishWaves = 16;

// Rows' lists of SUBS waves each made one, in lists[row's first wave]: all
// waves of the block call it.
template <int SUBS, int R>
__device__ __forceinline__ void join_lists(TopList<R>& top, uint64_t (*lists)[64 * R], int wave, int sub, int k,
                                           int lane) {
    __syncthreads();  // the lists' last readers are done
#pragma unroll
    for (int r = 0; r < R; ++r) lists[wave][64 * r + lane] = top.v[r];
    __syncthreads();
    if (SUBS > 1 && sub == 0) {
        for (int w = 1; w < SUBS; ++w)
#pragma unroll
            for (int r = 0; r < R; ++r) top.offer(lists[wave + w][64 * r + lane], k, 0, lane);
#pragma unroll
        for (int r = 0; r < R; ++r) lists[wave][64 * r + lane] = top.v[r];
    }
    if (SUBS > 1) __syncthreads();
}

// SUBS waves to a row. R = 0: no alternatives.
template <int SUBS, int R>
__global__ __launch_bounds__(64 * kFinishWaves) void logprob_finish_kernel(RowLogits in, LogprobOut out) {
    __shared__ Stats stats[kFinishWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = wave % SUBS, first = wave - sub;
    const int64_t m_ = (int64_t)blockIdx.x * (kFinishWaves / SUBS) + wave / SUBS;
    const bool there = m_ < in.M;
    const int64_t m = there ? m_ : in.M - 1;  // (waves past the last row do its work again and store nothing)

    Stats a = row_stats(in, m, sub, SUBS, lane);
    if (SUBS > 1) {
        if (lane == 0) stats[wave] = a;
        __syncthreads();
        a = stats[first];
        for (int w = 1; w < SUBS; ++w) join_stats(a, stats[first + w], in.inv_t);
    }
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
    if constexpr (R > 0) {
        __shared__ uint64_t lists[kFinishWaves][64 * R];
        const int k = out.k;
        TopList<R> top;
        top.clear();
        // (loops of as many rounds in every wave; nothing beyond the end)
        for (int p0 = 0; p0 < in.parts; p0 += 64 * SUBS) {
            const int p = p0 + sub * 64 + lane;
            top.offer(p < in.parts ? order_key(in.stat[(int64_t)p * in.M + m], p) : 0, k, 0, lane);
        }
        join_lists<SUBS, R>(top, lists, wave, sub, k, lane);
        // the chosen blocks' columns; k of them have maxima that are no less
        // than the last one's, so nothing below that is among the k first
        const uint64_t last = lists[first][k - 1];
        const uint64_t least = last ? (last >> 32 << 32) - 1 : 0;
        const int count = k < in.parts ? k : in.parts, total = count * in.width;
        top.clear();
        const float* z = in.z + m * in.ld;
        for (int e0 = 0; e0 < total; e0 += 64 * SUBS) {
            const int e = e0 + sub * 64 + lane, c = e / in.width;
            uint64_t key = 0;
            if (e < total) {
                const int64_t col = (int64_t)key_index(lists[first][c]) * in.width + e % in.width;
                if (col < in.N) key = order_key(z[col], (uint32_t)col);
            }
            top.offer(key, k, least, lane);
        }
        join_lists<SUBS, R>(top, lists, wave, sub, k, lane);
        if (there && sub == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int i = 64 * r + lane;
                if (i < k) {
                    const uint64_t key = top.v[r];
                    out.top_ids[m * k + i] = (int64_t)key_index(key) + in.v0;
                    out.top_logp[m * k + i] =
                        a.sum == 0.0f ? -INFINITY : (key_value(key) - ref) * in.inv_t - log_sum;
                }
            }
        }
    }
}

// ------------------------------------------------- a teacher's tokens

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

constexpr int kPer = kMaxTop / 64;  // listed tokens to a lane: 64 r + lane

// A row's listed tokens: ids (-1 where there is none), probabilities (0 there)
// and their logarithms. Returns whether the row has any.
__device__ __forceinline__ bool teacher_row(const Listed& t, float inv_t, int64_t m, int lane, int64_t (&id)[kPer],
                                            float (&p)[kPer], float (&logp)[kPer]) {
    float mx = -INFINITY;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
        const int i = 64 * r + lane;
        id[r] = i < t.n ? t.ids[m * t.n + i] : -1;
        logp[r] = id[r] >= 0 ? t.tlogits[m * t.n + i] * inv_t : -INFINITY;
        if (logp[r] == -INFINITY) id[r] = -1;
        mx = fmaxf(mx, logp[r]);
    }
    const bool any = __ballot(id[0] >= 0 || id[kPer - 1] >= 0) != 0;
    mx = wave_max(mx);
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
        logp[r] = id[r] >= 0 ? logp[r] - mx : 0.0f;
        p[r] = id[r] >= 0 ? exp_f32(logp[r]) : 0.0f;
        s += p[r];
    }
    s = any ? wave_sum(s) : 1.0f;
    const float ls = logf(s);
#pragma unroll
    for (int r = 0; r < kPer; ++r) p[r] /= s, logp[r] -= ls;
    return any;
}

// One wave to a row.
__global__ __launch_bounds__(256) void distill_finish_kernel(RowLogits in, Listed t, float* __restrict__ lse,
                                                             float* __restrict__ slogits, float* __restrict__ loss) {
    const int lane = threadIdx.x & 63;
    const int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (m >= in.M) return;  // the whole wave
    const Stats a = row_stats(in, m, 0, 1, lane);
    const float l = finite_ref(a.mx) * in.inv_t + logf(a.sum);
    int64_t id[kPer];
    float p[kPer], logp[kPer];
    const bool any = teacher_row(t, in.inv_t, m, lane, id, p, logp);
    float sum = 0.0f;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
        const int i = 64 * r + lane;
        const uint64_t at = (uint64_t)id[r] - (uint64_t)in.v0;
        const float z = id[r] >= 0 && at < (uint64_t)in.N ? in.z[m * in.ld + (int64_t)at] : 0.0f;
        if (i < t.n) slogits[m * t.n + i] = z;
        if (p[r] != 0.0f) sum += p[r] * (logp[r] + (l - z * in.inv_t));
    }
    sum = wave_sum(sum);
    if (lane == 0) {
        lse[m] = l;
        loss[m] = any ? sum : 0.0f;
    }
}

__global__ __launch_bounds__(256) void listed_prep_kernel(Listed t, const float* __restrict__ grad, float inv_t,
                                                          int64_t M, float* __restrict__ p_out, float* __restrict__ gw,
                                                          int64_t* __restrict__ targets) {
    const int lane = threadIdx.x & 63;
    const int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (m >= M) return;  // the whole wave
    int64_t id[kPer];
    float p[kPer], logp[kPer], total[kPer];
    bool firsts[kPer];
    const bool any = teacher_row(t, inv_t, m, lane, id, p, logp);
#pragma unroll
    for (int r = 0; r < kPer; ++r) total[r] = 0.0f, firsts[r] = id[r] >= 0;
    // tokens that are listed several times count together, at their first place
    for (int i = 0; i < t.n; ++i) {
        const int src = i & 63;
        const int64_t other = i < 64 ? __shfl(id[0], src) : __shfl(id[kPer - 1], src);
        const float q = i < 64 ? __shfl(p[0], src) : __shfl(p[kPer - 1], src);
#pragma unroll
        for (int r = 0; r < kPer; ++r)
            if (other == id[r]) {
                total[r] += q;
                if (i < 64 * r + lane) firsts[r] = false;
            }
    }
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
        const int i = 64 * r + lane;
        if (i < t.n) p_out[m * t.n + i] = firsts[r] ? total[r] : -1.0f;
    }
    if (lane == 0) {
        gw[m] = grad[m] * inv_t;
        targets[m] = any ? -1 : INT64_MIN;
    }
}

// One thread to a listed token.
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

template <int SUBS>
static hipError_t logprob_finish(const RowLogits& r, const LogprobOut& o, hipStream_t s) {
    const int rows = kFinishWaves / SUBS;
    const auto fn = o.k == 0    ? logprob_finish_kernel<SUBS, 0>
                    : o.k <= 64 ? logprob_finish_kernel<SUBS, 1>
                                : logprob_finish_kernel<SUBS, 2>;
    hipLaunchKernelGGL(fn, dim3((unsigned)((r.M + rows - 1) / rows)), dim3(64 * kFinishWaves), 0, s, r, o);
    return hipGetLastError();
}

hipError_t launch_logprob_finish(const RowLogits& r, const LogprobOut& o, hipStream_t s) {
    if (o.k < 0 || o.k > kMaxTop || r.width < 32 || (r.width & (r.width - 1))) return hipErrorInvalidValue;
    return r.M <= 512 ? logprob_finish<16>(r, o, s) : r.M <= 2048 ? logprob_finish<4>(r, o, s) : logprob_finish<1>(r, o, s);
}

hipError_t launch_distill_finish(const RowLogits& r, const Listed& t, float* lse, float* slogits, float* loss,
                                 hipStream_t s) {
    if (t.n < 1 || t.n > kMaxTop) return hipErrorInvalidValue;
    hipLaunchKernelGGL(distill_finish_kernel, dim3((unsigned)((r.M + 3) / 4)), dim3(256), 0, s, r, t, lse, slogits, loss);
    return hipGetLastError();
}

hipError_t launch_listed_prep(const Listed& t, const float* grad, float inv_t, int64_t M, float* p, float* gw,
                              int64_t* targets, hipStream_t s) {
    if (t.n < 1 || t.n > kMaxTop) return hipErrorInvalidValue;
    hipLaunchKernelGGL(listed_prep_kernel, dim3((unsigned)((M + 3) / 4)), dim3(256), 0, s, t, grad, inv_t, M, p, gw,
                       targets);
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
