// Log probabilities of given tokens, entropy and the best alternatives from rows of logits,
// and the gradient.  With m = max L, d = L - m, S = sum exp d, W = sum exp(d) d:
//   logp = d_token - log S,   entropy = log S - W / S
// in one pass with a running maximum: when it grows from m to m', S and W become
//   f S,  f (W + S (m - m')),  f = exp(m - m').
// Everything is relative to the maximum, so that rows at the ends of the type (a mask of its
// lowest value, which all elements may have) keep their digits.
//
// The alternatives ride along.  Once a wave has seen a stretch, its lanes' maxima give a bound
// that n_top elements reach (the want-th largest lane maximum, found bit by bit with ballots);
// elements that reach the bound go to a list in LDS, whose best n_top are taken at the end by
// counting, for each, those before it.  The bound is taken again as the row goes on.  A row that
// overflows the list (ascending logits, thousands of equal ones) is selected by radix passes
// over (value, index) instead.
//
// A workgroup has a row, of 256 threads or, for short rows, of 64; where there are few rows,
// several share one and the last to arrive joins them.  The gradient
//   p ( -w - u (log p + entropy) ) + w [v = token]
// is one pass more, a row's pieces spread over workgroups.
//
// Many rows are bound by memory: 4096 x 49999 bf16 with 5 alternatives 88 us (4.6 TB/s), the gradient, padding
// left unread, 136 us.  A single row is bound by latency: 49999 float32 logits over 13 workgroups
// 6.2 us, with 20 alternatives 9 to 12, two selections of 2 to 3 us each; handing on whole
// sorted lists took twice that.
#include <algorithm>
#include <cmath>

#include "logprobs.h"
#include "row_ops.h"

namespace moe {

namespace {

constexpr int kUnroll = 4;                 // 16-byte pieces a thread and step
constexpr int kList = 1024;                // candidates kept
constexpr int kRankStep = 8;               // candidates compared with at once
constexpr int kKeep = 64;                  // candidates that a workgroup hands on where several share a row
constexpr int kRowCounters = 512, kRowStride = MOE_LOGPROBS_SYNC_INTS / kRowCounters;
constexpr float kLog2e = 1.44269504f;

template <int TYPE> constexpr int kPer = TYPE == MOE_F32 ? 4 : 8;     // elements a piece

template <int TYPE>
__device__ __forceinline__ float element(const void* row, int v) {
    if constexpr (TYPE == MOE_F32) return static_cast<const float*>(row)[v];
    else return bf16_bits_to_f32(static_cast<const uint16_t*>(row)[v]);
}

template <int TYPE>
__device__ __forceinline__ void unpack(const uint4& q, float (&x)[kPer<TYPE>]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == MOE_F32) {
            x[i] = __uint_as_float(w[i]);
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// Whole numbers in the order of the floats (-0 as +0).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kOrderedLow = 0x007FFFFFu;         // of -inf

// A value that `want` of the wave's lanes reach (its upper 16 bits exact), -inf where fewer have any.
__device__ __forceinline__ float lane_bound(float x, int want) {
    const uint32_t key = ordered(x);
    uint32_t t = 0;
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t trial = t | (1u << bit);
        if ((int)__popcll(__ballot(key >= trial)) >= want) t = trial;
    }
    return t <= kOrderedLow ? -INFINITY : unordered(t);
}

// What a workgroup hands on: its sums, its candidates' number, values and indices.
__host__ __device__ constexpr int part_words(int n_top) { return n_top ? 4 + 2 * kKeep : 4; }

struct Sums {
    float m, s, w;
};

// s and w of two sums relative to the larger maximum (-inf: nothing yet).
__device__ __forceinline__ void rebase(Sums& a, float m) {
    const float base = m > -INFINITY ? m : 0.f;
    // (cut off where f is 0 anyway: the difference of two finite maxima may be infinite)
    const float d = a.m > -INFINITY ? fmaxf(a.m - base, -1e4f) : 0.f;
    const float f = a.m > -INFINITY ? __builtin_amdgcn_exp2f(d * kLog2e) : (a.s != a.s ? a.s : 0.f);
    a.w = f * (a.w + a.s * d);
    a.s *= f;
    a.m = m;
}

__device__ __forceinline__ Sums wave_join(Sums a) {
    rebase(a, row_max<64>(a.m));
    a.s = row_sum<64>(a.s);
    a.w = row_sum<64>(a.w);
    return a;
}

struct List {
    __attribute__((aligned(16))) float v[kList + kRankStep];
    __attribute__((aligned(16))) int i[kList + kRankStep];
    int count;
    float bound[4];
};

__device__ __forceinline__ bool before(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

__device__ __forceinline__ void append(List& L, float v, int i) {
    const int at = atomicAdd(&L.count, 1);
    if (at < kList) {
        L.v[at] = v;
        L.i[at] = i;
    }
}

// The bound of all waves together: each has want = ceil(n / waves) lanes that reach its own.
template <int NW>
__device__ __forceinline__ float bound_of(List& L, float lane_max, int n) {
    const float mine = lane_bound(lane_max, (n + NW - 1) / NW);
    if constexpr (NW == 1) return mine;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) L.bound[threadIdx.x >> 6] = mine;
    __syncthreads();
    float b = L.bound[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) b = fminf(b, L.bound[w]);
    return b;
}

// Each entry's place among the list's c (all threads call it, the list complete); out(place, value,
// index) for the best n, (-inf, -1) where there are no more.
template <int NW, typename OUT>
__device__ __forceinline__ void rank_list(List& L, int c, int n, OUT out) {
    constexpr int NT = 64 * NW;
    if ((int)threadIdx.x < kRankStep) {
        L.v[c + threadIdx.x] = -INFINITY;              // (before none)
        L.i[c + threadIdx.x] = 0x7FFFFFFF;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < c; k += NT) {
        const float x = L.v[k];
        const int i = L.i[k];
        int place = 0;
        for (int o = 0; o < c; o += kRankStep) {
            float v[kRankStep];
            int at[kRankStep];
#pragma unroll
            for (int u = 0; u < kRankStep; u += 4) {
                *reinterpret_cast<float4*>(v + u) = *reinterpret_cast<const float4*>(&L.v[o + u]);
                *reinterpret_cast<int4*>(at + u) = *reinterpret_cast<const int4*>(&L.i[o + u]);
            }
#pragma unroll
            for (int u = 0; u < kRankStep; ++u) place += before(v[u], at[u], x, i);
        }
        if (place < n) out(place, x, i);
    }
    for (int k = c + (int)threadIdx.x; k < n; k += NT) out(k, -INFINITY, -1);
}

// The best n of the threads' EACH entries (index -1: none), best first, by way of the list: those that
// reach the bound of all, ranked.
template <int NW, int EACH, typename OUT>
__device__ __forceinline__ void best_of_entries(List& L, const float (&v)[EACH], const int (&at)[EACH], int n, OUT out) {
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < EACH; ++e) top = fmaxf(top, at[e] >= 0 ? v[e] : -INFINITY);
    const float b = bound_of<NW>(L, top, n);
    __syncthreads();
    if (threadIdx.x == 0) L.count = 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < EACH; ++e)
        if (at[e] >= 0 && v[e] >= b) append(L, v[e], at[e]);
    __syncthreads();
    const int c = L.count;
    rank_list<NW>(L, c, n, out);
}

// The best n of the list's entries.
template <int NW, typename OUT>
__device__ __forceinline__ void best_of(List& L, int n, OUT out) {
    constexpr int NT = 64 * NW, EACH = kList / NT;
    __syncthreads();
    const int c = min(L.count, kList);
    if (c <= kKeep) {
        rank_list<NW>(L, c, n, out);
        return;
    }
    float v[EACH];
    int at[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const int k = e * NT + (int)threadIdx.x;
        v[e] = k < c ? L.v[k] : -INFINITY;
        at[e] = k < c ? L.i[k] : -1;
    }
    best_of_entries<NW, EACH>(L, v, at, n, out);
}

// The list overflowed: its entries again, exactly the best n (or all there are) of elements
// [v0, v1), by radix passes over the 52 bits of (value, index).
template <int TYPE, int NW>
__device__ void select_again(List& L, const void* row, int v0, int v1, int n) {
    constexpr int NT = 64 * NW, DIGIT = 10, BINS = 1 << DIGIT, BITS = 60;
    static_assert(BINS <= kList, "the histogram takes the list's place");
    int* hist = L.i;
    uint64_t prefix = 0;
    int left = n;                                      // wanted among those that share the prefix
    for (int shift = BITS - DIGIT; shift >= 0; shift -= DIGIT) {
        __syncthreads();
        for (int k = threadIdx.x; k < BINS; k += NT) hist[k] = 0;
        __syncthreads();
        for (int v = v0 + (int)threadIdx.x; v < v1; v += NT) {
            const float x = element<TYPE>(row, v);
            if (!(x > -INFINITY)) continue;
            const uint64_t key = ((uint64_t)ordered(x) << 20) | (uint32_t)((1 << 20) - 1 - v);
            if ((key >> (shift + DIGIT)) == prefix) atomicAdd(&hist[(int)(key >> shift) & (BINS - 1)], 1);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int bin = BINS - 1, have = 0;
            for (; bin > 0 && have + hist[bin] < left; --bin) have += hist[bin];
            L.count = bin;
            L.bound[0] = __int_as_float(left - have);
        }
        __syncthreads();
        prefix = (prefix << DIGIT) | (uint32_t)L.count;
        left = __float_as_int(L.bound[0]);
    }
    __syncthreads();
    if (threadIdx.x == 0) L.count = 0;
    __syncthreads();
    for (int v = v0 + (int)threadIdx.x; v < v1; v += NT) {
        const float x = element<TYPE>(row, v);
        if (!(x > -INFINITY)) continue;
        const uint64_t key = ((uint64_t)ordered(x) << 20) | (uint32_t)((1 << 20) - 1 - v);
        if (key >= prefix) append(L, x, v);
    }
}

}  // namespace

template <int TYPE, bool TOP, bool ENT, int NW>
__global__ __launch_bounds__(64 * NW) void logprobs_kernel(LogprobArgs a) {
    constexpr int NT = 64 * NW, PER = kPer<TYPE>, WIDE = TYPE == MOE_F32 ? 4 : 2;
    __shared__ List L;
    __shared__ Sums wave_sums[NW];
    __shared__ int flag;
    const int t = blockIdx.x / a.splits, split = blockIdx.x % a.splits, tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, n = a.n_top;
    const char* row = static_cast<const char*>(a.logits) + (int64_t)t * a.ld * WIDE;
    const int token = a.tokens[t];
    const bool scored = (unsigned)token < (unsigned)a.V;
    const float picked = element<TYPE>(row, scored ? token : 0);
    // head elements up to a 16-byte border, whole pieces, and a tail; head and tail one a lane of split 0
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / WIDE, a.V);
    const int pieces = (a.V - head) / PER, tail = a.V - head - pieces * PER;
    const int p0 = min(split * a.pieces, pieces), p1 = min(p0 + a.pieces, pieces);
    const uint4* body = reinterpret_cast<const uint4*>(row + head * WIDE);
    int edge = -1;
    if (split == 0) edge = tid < head ? tid : tid >= 32 && tid < 32 + tail ? head + pieces * PER + tid - 32 : -1;
    const float first = edge >= 0 ? element<TYPE>(row, edge) : -INFINITY;
    Sums sum{fmaxf(-INFINITY, first), first > -INFINITY ? 1.f : first == first ? 0.f : first, 0.f};
    if (first == INFINITY) sum.s = NAN;
    if (TOP && tid == 0) L.count = 0;
    float bound = -INFINITY;
    constexpr uint32_t kNone = TYPE == MOE_F32 ? 0xFF800000u : 0xFF80FF80u;       // -inf
    const int steps = (p1 - p0 + NT * kUnroll - 1) / (NT * kUnroll);
    for (int step = 0; step < max(steps, TOP ? 1 : 0); ++step) {
        uint4 q[kUnroll];
        const int at = p0 + step * NT * kUnroll + tid;
        if (at - tid + NT * kUnroll <= p1) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) q[u] = body[at + u * NT];
        } else {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                q[u] = make_uint4(kNone, kNone, kNone, kNone);
                if (at + u * NT < p1) q[u] = body[at + u * NT];
            }
        }
        float x[kUnroll][PER], most[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            unpack<TYPE>(q[u], x[u]);
            most[u] = x[u][0];
#pragma unroll
            for (int j = 1; j < PER; ++j) most[u] = fmaxf(most[u], x[u][j]);
        }
        float m = sum.m;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) m = fmaxf(m, most[u]);
        rebase(sum, m);
        const float base = m > -INFINITY ? m : 0.f;
        float s[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const float d = x[u][j] - base;
                const float e = __builtin_amdgcn_exp2f(d * kLog2e);
                s[j & 1] += e;
                if constexpr (ENT) w[j & 1] = fmaf(e, fmaxf(d, -1e4f), w[j & 1]);     // (0 where e is 0; a NaN stays in e)
            }
        sum.s += s[0] + s[1];
        if constexpr (ENT) sum.w += w[0] + w[1];
        if constexpr (TOP) {
            // the bound after the 1st, 2nd, 4th, ... stretch
            if ((step & (step + 1)) == 0) bound = fmaxf(bound, bound_of<NW>(L, m, n));
            if (step == 0) {
                if constexpr (NW == 1) __syncthreads();
                if (first > -INFINITY && first >= bound) append(L, first, edge);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (most[u] >= bound && most[u] > -INFINITY) {
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        if (x[u][j] >= bound && x[u][j] > -INFINITY) append(L, x[u][j], head + (at + u * NT) * PER + j);
                }
        }
    }
    sum = wave_join(sum);
    if constexpr (NW > 1) {
        if (lane == 0) wave_sums[wid] = sum;
        __syncthreads();
        sum = wave_sums[min(lane, NW - 1)];
        if (lane >= NW) sum = Sums{-INFINITY, 0.f, 0.f};
        sum = wave_join(sum);
    }
    if constexpr (TOP) {
        __syncthreads();
        if (L.count > kList) {
            // this workgroup's elements again: its pieces, in split 0 the head, and the tail
            const int b0 = split == 0 ? 0 : head + p0 * PER, b1 = a.splits == 1 ? a.V : head + p1 * PER;
            select_again<TYPE, NW>(L, row, b0, b1, n);
            if (a.splits > 1) {
                __syncthreads();
                if (edge >= head && first > -INFINITY) append(L, first, edge);
            }
        }
    }
    float kept[kList / NT];                            // the splits' candidates, where there are several
    int kept_at[kList / NT];
    if (a.splits > 1) {
        const int words = part_words(n);
        float* mine = a.part + ((int64_t)t * a.splits + split) * words;
        int handed = 0;
        if constexpr (TOP) {
            __syncthreads();
            int c = min(L.count, kList);
            if (c > kKeep && c <= NT) {
                // without earlier stretches' entries that the last bound shuts out, so that they need no order yet (64 x 49999
                // with 20 alternatives 19.0 -> 17.6 us, 64 x 150000 26.1 -> 23.6)
                const float v = L.v[min(tid, c - 1)];
                const int i = L.i[min(tid, c - 1)];
                __syncthreads();
                if (tid == 0) L.count = 0;
                __syncthreads();
                if (tid < c && v >= bound) append(L, v, i);
                __syncthreads();
                c = L.count;
            }
            handed = c <= kKeep ? c : n;
            if (c <= kKeep) {
                if (tid < c) {
                    put_device(mine + 4 + tid, L.v[tid]);
                    put_device(mine + 4 + kKeep + tid, __int_as_float(L.i[tid]));
                }
            } else {
                best_of<NW>(L, n, [&](int place, float v, int i) {
                    put_device(mine + 4 + place, v);
                    put_device(mine + 4 + kKeep + place, __int_as_float(i));
                });
            }
        }
        if (tid < 4) put_device(mine + tid, tid == 0 ? sum.m : tid == 1 ? sum.s : tid == 2 ? sum.w : __int_as_float(handed));
        if (!arrive_last(a.sync + t * kRowStride, a.splits, &flag)) return;
        // every load before the first use: the sums by lanes, the candidates a wave a split at a time
        const float* all = a.part + (int64_t)t * a.splits * words;
        const float* from = all + min(lane, a.splits - 1) * words;
        sum = Sums{get_device(from), get_device(from + 1), get_device(from + 2)};
        if constexpr (TOP) {
            const int counts = __float_as_int(get_device(from + 3));
#pragma unroll
            for (int e = 0; e < kList / NT; ++e) {
                const float* entry = all + min(e * NW + wid, a.splits - 1) * words + 4 + lane;
                kept[e] = get_device(entry);
                kept_at[e] = __float_as_int(get_device(entry + kKeep));
            }
#pragma unroll
            for (int e = 0; e < kList / NT; ++e) {
                const int s = e * NW + wid;
                if (s >= a.splits || lane >= __shfl(counts, min(s, a.splits - 1), kWave)) kept_at[e] = -1;
            }
        }
        if (lane >= a.splits) sum = Sums{-INFINITY, 0.f, 0.f};
        sum = wave_join(sum);
    }
    const bool some = sum.m > -INFINITY || sum.s != sum.s;
    const float base = sum.m > -INFINITY ? sum.m : 0.f;
    // (lane 0's sum: the lanes add in different orders, and any of them may have an alternative)
    const float whole = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sum.s)));
    const float log_s = some ? logf(whole) : -INFINITY;
    if (tid == 0) {
        a.stats[2 * (int64_t)t] = sum.m;
        a.stats[2 * (int64_t)t + 1] = log_s;
        a.logp[t] = !scored ? 0.f : some ? picked - base - log_s : -INFINITY;
        if (a.entropy) a.entropy[t] = some ? log_s - sum.w / sum.s : 0.f;
    }
    if constexpr (TOP) {
        auto out = [&](int place, float v, int i) {
            a.top_ids[(int64_t)t * n + place] = i;
            a.top_logp[(int64_t)t * n + place] = i < 0 ? -INFINITY : v - base - log_s;
        };
        if (a.splits > 1) best_of_entries<NW, kList / NT>(L, kept, kept_at, n, out);
        else best_of<NW>(L, n, out);
    }
}

namespace {

constexpr int kGradElements = 32;          // elements a thread

}  // namespace

template <int TYPE, int GTYPE, int NT>
__global__ __launch_bounds__(NT) void logprobs_grad_kernel(LogprobGradArgs a, unsigned blocks) {
    constexpr int WIDE = GTYPE == MOE_F32 ? 4 : 2, IN = TYPE == MOE_F32 ? 4 : 2;
    constexpr int PE = 16 / WIDE, PIECES = kGradElements / PE;     // elements of a 16-byte piece of the gradient, pieces a thread
    const int t = blockIdx.x / blocks, block = blockIdx.x % blocks, tid = threadIdx.x;
    const int token = ld_scalar(a.tokens, t);
    const bool scored = (unsigned)token < (unsigned)a.V;
    const float w = scored && a.dlogp ? ld_scalar(a.dlogp, t) : 0.f, u = a.dentropy ? ld_scalar(a.dentropy, t) : 0.f;
    const float m = ld_scalar(a.stats, 2 * (size_t)t), log_s = ld_scalar(a.stats, 2 * (size_t)t + 1);
    const float H = a.dentropy ? ld_scalar(a.entropy, t) : 0.f;
    const bool none = (w == 0.f && u == 0.f) || (m == -INFINITY && !(log_s != log_s));
    const float base = m > -INFINITY ? m : 0.f;
    const char* row = static_cast<const char*>(a.logits) + (int64_t)t * a.ld * (TYPE == MOE_F32 ? 4 : 2);
    char* out = static_cast<char*>(a.dlogits) + (int64_t)t * a.ldg * WIDE;
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(out) & 15)) & 15) / WIDE, a.V);
    const int pieces = (a.V - head) / PE, tail = a.V - head - pieces * PE;
    auto grad = [&](float x, int v) {
        const float lp = x - base - log_s;
        const float p = exp_down(lp);
        float g = p * fmaf(-u, fmaxf(lp, -1e4f) + H, -w);
        if (v == token) g = fmaf(-u * p, fmaxf(lp, -1e4f) + H, -w * expm1f(lp));     // w (1 - p) without their difference
        return g;
    };
    // head and tail, one a lane of the first workgroup
    if (block == 0) {
        const int v = tid < head ? tid : tid >= 32 && tid < 32 + tail ? head + pieces * PE + tid - 32 : -1;
        if (v >= 0) {
            const float g = none ? 0.f : grad(element<TYPE>(row, v), v);
            if constexpr (GTYPE == MOE_F32) reinterpret_cast<float*>(out)[v] = g;
            else reinterpret_cast<uint16_t*>(out)[v] = (uint16_t)pack_bf16(g, 0.f);
        }
    }
    const int p0 = block * NT * PIECES + tid;
    if (none) {
#pragma unroll
        for (int k = 0; k < PIECES; ++k) {
            const int p = p0 + NT * k;
            if (p >= pieces) break;
            *reinterpret_cast<uint4*>(out + ((int64_t)head + PE * p) * WIDE) = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    uint32_t q[PIECES][PE * IN / 4];
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
        const int p = min(p0 + NT * k, pieces - 1);
        if (pieces > 0) __builtin_memcpy(q[k], row + ((int64_t)head + PE * p) * IN, PE * IN);
    }
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
        const int p = p0 + NT * k;
        if (p >= pieces) break;
        float x[PE], g[PE];
#pragma unroll
        for (int j = 0; j < PE; ++j)
            x[j] = TYPE == MOE_F32 ? __uint_as_float(q[k][j])
                                   : __uint_as_float((j & 1) ? q[k][j >> 1] & 0xFFFF0000u : q[k][j >> 1] << 16);
        const int v = head + PE * p;
#pragma unroll
        for (int j = 0; j < PE; ++j) {
            const float lp = x[j] - base - log_s;
            g[j] = exp_down(lp) * fmaf(-u, fmaxf(lp, -1e4f) + H, -w);
        }
        if (scored && token >= v && token < v + PE)
#pragma unroll
            for (int j = 0; j < PE; ++j)
                if (v + j == token) g[j] = grad(x[j], token);
        uint4* to = reinterpret_cast<uint4*>(out + (int64_t)v * WIDE);
        if constexpr (GTYPE == MOE_F32) {
            __builtin_memcpy(to, g, 16);
        } else {
            uint32_t o[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) o[d] = pack_bf16(g[(2 * d) % PE], g[(2 * d + 1) % PE]);
            *to = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

namespace {

// Rows of up to this many elements have a wave each (us by a wave and by four: 4096 x 2048 float32 9.6 and 12.0, with 5
// alternatives 12.1 and 18.1, 16384 x 1000 14.3 and 30.0; the few rows of 4 x 2048 7.4 and 6.5 with
// alternatives, 5.3 and 5.1 without).
constexpr int kShortRow = 2048;

// Workgroups that share a row: 512 in all, each with a step's pieces at least; their candidates
// fit the list.
int row_splits(int T, int V, int n_top) {
    if (T > kRowCounters || V <= kShortRow) return 1;
    const int steps = (V / 4 + 256 * kUnroll - 1) / (256 * kUnroll);
    int splits = std::min({(512 + T - 1) / T, steps, 64});
    if (n_top) splits = std::min(splits, kList / kKeep);
    return splits;
}

template <int TYPE, bool TOP, bool ENT>
void logprobs_go(const LogprobArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.splits * a.T));
    if (a.V <= kShortRow) hipLaunchKernelGGL((logprobs_kernel<TYPE, TOP, ENT, 1>), grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL((logprobs_kernel<TYPE, TOP, ENT, 4>), grid, dim3(256), 0, s, a);
}

template <int TYPE>
void logprobs_type(const LogprobArgs& a, hipStream_t s) {
    if (a.n_top) a.entropy ? logprobs_go<TYPE, true, true>(a, s) : logprobs_go<TYPE, true, false>(a, s);
    else a.entropy ? logprobs_go<TYPE, false, true>(a, s) : logprobs_go<TYPE, false, false>(a, s);
}

template <int TYPE, int GTYPE>
void grad_threads(const LogprobGradArgs& a, hipStream_t s) {
    const int threads = a.V <= kShortRow ? 64 : 256;
    const unsigned blocks = (unsigned)std::max(1, (a.V + threads * kGradElements - 1) / (threads * kGradElements));
    const dim3 grid(blocks * (unsigned)a.T);
    if (threads == 64) hipLaunchKernelGGL((logprobs_grad_kernel<TYPE, GTYPE, 64>), grid, dim3(64), 0, s, a, blocks);
    else hipLaunchKernelGGL((logprobs_grad_kernel<TYPE, GTYPE, 256>), grid, dim3(256), 0, s, a, blocks);
}

}  // namespace

size_t logprobs_workspace_of(int T, int V, int n_top) {
    const int splits = row_splits(T, V, n_top);
    return splits > 1 ? (size_t)T * splits * part_words(n_top) * 4 : 0;
}

// Calls of fewer tokens may have more workgroups a row: the most that any has.
size_t logprobs_workspace_bytes(int T, int V, int n_top) {
    size_t most = 0;
    for (int t = 1; t <= std::min(T, kRowCounters); ++t) most = std::max(most, logprobs_workspace_of(t, V, n_top));
    return most;
}

int launch_logprobs(LogprobArgs a, hipStream_t s) {
    a.splits = row_splits(a.T, a.V, a.n_top);
    const int per = a.type == MOE_F32 ? 4 : 8;
    const int pieces = a.V / per;
    a.pieces = a.splits == 1 ? pieces : ((pieces + a.splits - 1) / a.splits + 255) / 256 * 256;
    if (a.type == MOE_F32) logprobs_type<MOE_F32>(a, s);
    else logprobs_type<MOE_BF16>(a, s);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_logprobs_grad(const LogprobGradArgs& a, hipStream_t s) {
    if (a.type == MOE_F32) a.grad_type == MOE_F32 ? grad_threads<MOE_F32, MOE_F32>(a, s) : grad_threads<MOE_F32, MOE_BF16>(a, s);
    else a.grad_type == MOE_F32 ? grad_threads<MOE_BF16, MOE_F32>(a, s) : grad_threads<MOE_BF16, MOE_BF16>(a, s);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
