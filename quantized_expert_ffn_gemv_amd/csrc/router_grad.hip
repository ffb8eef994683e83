// The router's losses and its backward pass, over float32 logits [T][E].
//
// Both kernels give a token's row to LPT lanes (4, 16, 32 or 64; the smallest
// that holds the row in at most 4 values a lane, 16 at E = 1024), keep it in
// registers, and need one pass over the logits:
//   m = max L, e = exp(L - m), S = sum e, p = e / S, lse = m + log S,
// m and S by reductions over the lanes.  A row without a logit above -inf has
// p = 0 everywhere.
//
// The gradient is bound by memory: 16384 x 512, 16.3 us (4.2 TB/s); 64 x 64, 2.4 us.  The
// losses by their joins: 32 x 256, 5.4 us; 8191 x 128, 8.5 us; 16384 x 512, 17.1 us.
#include <cmath>

#include "common.h"
#include "row_ops.h"

namespace moe {

namespace {

// Workgroups of the losses: 512 threads (1024: 16384 x 512 15.3 us against 16.8, but 32 x
// 256 and 1024 x 128 slower; both, by the batch, is not built), at most 256 (half as many: 16384 x 512 23.4 us against 16.9,
// 8191 x 128 10.1 and 8.8), 16 joined by one ticket (32: slower at every size).
constexpr int kThreads = 256, kBalThreads = 512;
constexpr int kBalTree = 16;
constexpr int kBalBlocks = 256;
constexpr int kBalSyncStride = 64;                        // counters 256 bytes apart
static_assert(MOE_BALANCE_SYNC_INTS >= kBalSyncStride * (1 + kBalBlocks / kBalTree), "sync buffer layout");

// Expert of slot i of lane `sub`: VEC rows are read 16 bytes a lane.
template <int LPT, bool VEC>
__device__ __forceinline__ int slot_expert(int sub, int i) {
    return VEC ? 4 * (sub + LPT * (i >> 2)) + (i & 3) : sub + LPT * i;
}

// The row's values of this lane; `none` where there is no expert.
template <int LPT, int PER, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int sub, float none, float (&v)[PER]) {
    if constexpr (VEC) {
#pragma unroll
        for (int c = 0; c < PER / 4; ++c) {
            const int e = 4 * (sub + LPT * c);
            float4 q = make_float4(none, none, none, none);
            if (e < E) q = *reinterpret_cast<const float4*>(row + e);
            v[4 * c] = q.x; v[4 * c + 1] = q.y; v[4 * c + 2] = q.z; v[4 * c + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = sub + LPT * i;
            v[i] = e < E ? row[e] : none;
        }
    }
}

// e^d, d <= 0, to 2 ulp: the hardware's power of two of t = d log2 e rounded, times the
// factor 1 + r ln 2 for what the rounding left out, r = d log2 e - t (log2 e in two
// parts).  Without the factor a small p was off by |d| 2^-24.  Below 2^-126 the
// hardware gives 0, and d is cut off there (an infinite one would make r NaN; a NaN stays).
__device__ __forceinline__ float exp_down(float d) {
    constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f;   // log2 e - (float) 1.44269504
    d = d < -128.f ? -128.f : d;
    const float t = d * kLog2e;
    const float r = fmaf(d, kLog2eRest, fmaf(d, kLog2e, -t));
    return __builtin_amdgcn_exp2f(t) * fmaf(r, 0.693147181f, 1.f);
}

// v (logits) -> p in place; returns whether the row has a logit, and lse.  A row without
// one has a sum of 0; NaNs, which fmaxf skips, come back by the sum.
template <int LPT, int PER>
__device__ __forceinline__ bool softmax_row(float (&v)[PER], float& lse) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = fmaxf(m, v[i]);
    m = row_max<LPT>(m);
    const float base = m > -INFINITY ? m : 0.f;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v[i] = exp_down(v[i] - base);
        s += v[i];
    }
    s = row_sum<LPT>(s);
    const bool some = s != 0.f;
    const float r = some ? 1.f / s : 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] *= r;
    lse = some ? base + logf(s) : 0.f;
    return some;
}

struct BalanceArgs {
    const float* logits;
    const int32_t* ids;
    const uint8_t* valid;
    int32_t* counts;
    float* prob_mean;
    int32_t* n_valid;
    float* losses;
    uint64_t* part;           // [blocks + groups of kBalTree][E + 1]: (sum of p, picks) per expert, then (z, tokens)
    int32_t* sync;
    int T, E, k;
};

__device__ __forceinline__ uint64_t pair_of(float x, int n) { return (uint64_t)__float_as_uint(x) | ((uint64_t)(uint32_t)n << 32); }

// The sum of partial rows [first, first + n), n <= N, into the workgroup's LDS, in
// index order.  Every row's load is made (past n the last again), so that they
// overlap; they pass the caches by and cost their number, hence the two sizes.
template <int N>
__device__ __forceinline__ void join_rows(const BalanceArgs& a, int first, int n, float* sp, int* sc) {
    for (int e = threadIdx.x; e <= a.E; e += kBalThreads) {
        uint64_t v[N];
#pragma unroll
        for (int b = 0; b < N; ++b) v[b] = get_device(a.part + (size_t)(first + min(b, n - 1)) * (a.E + 1) + e);
        float p = 0.f;
        int c = 0;
#pragma unroll
        for (int b = 0; b < N; ++b) {
            p += b < n ? __uint_as_float((uint32_t)v[b]) : 0.f;
            c += b < n ? (int)(v[b] >> 32) : 0;
        }
        sp[e] = p;
        sc[e] = c;
    }
    __syncthreads();
}

__device__ __forceinline__ void join_parts(const BalanceArgs& a, int first, int n, float* sp, int* sc) {
    if (n <= 4) join_rows<4>(a, first, n, sp, sc);
    else join_rows<kBalTree>(a, first, n, sp, sc);
}

__device__ __forceinline__ void put_part(const BalanceArgs& a, int slot, const float* sp, const int* sc) {
    for (int e = threadIdx.x; e <= a.E; e += kBalThreads) put_device(a.part + (size_t)slot * (a.E + 1) + e, pair_of(sp[e], sc[e]));
}

}  // namespace

// Sums of p, picks, lse^2 and tokens per workgroup, joined by a tree of arrival
// tickets: the last of each 16 workgroups sums their partial rows, the last
// of those sums the groups' rows and writes the results, all in index order.
// Eight waves a workgroup, one token per LPT lanes at a time with the next one's
// logits in flight.
template <int LPT, int PER, bool VEC>
__global__ __launch_bounds__(kBalThreads) void balance_kernel(BalanceArgs a) {
    constexpr int TPW = kWave / LPT, WAVES = kBalThreads / kWave;  // tokens per wave at once
    constexpr int ROW = LPT * PER;                        // experts a row of LDS holds
    __shared__ float sp[ROW + 1];                         // [E]: z, tokens
    __shared__ int sc[ROW + 1];
    __shared__ float wp[WAVES][ROW];
    __shared__ float wz[WAVES];
    __shared__ int wn[WAVES], flag;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, sub = lane % LPT;
    for (int e = tid; e <= a.E; e += kBalThreads) sc[e] = 0;
    __syncthreads();
    float acc[PER], z = 0.f, next[PER];
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    const int step = (int)gridDim.x * WAVES * TPW, first_t = ((int)blockIdx.x * WAVES + wid) * TPW + lane / LPT;
    bool live = false;
    auto load = [&](int t) {
        live = t < a.T && (a.valid == nullptr || a.valid[t] != 0);
        load_row<LPT, PER, VEC>(a.logits + (size_t)(t < a.T ? t : 0) * a.E, a.T > 0 ? a.E : 0, sub, -INFINITY, next);
    };
    if (first_t - lane / LPT < a.T) load(first_t);
    for (int t = first_t; t - lane / LPT < a.T; t += step) {
        float v[PER], lse;
        const bool mine = live;
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = mine ? next[i] : -INFINITY;
        if (t - lane / LPT + step < a.T) load(t + step);
        const bool part = softmax_row<LPT, PER>(v, lse);
        if (part) {
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] += v[i];
            if (sub == 0) { z = fmaf(lse, lse, z); ++n; }
            for (int j = sub; j < a.k; j += LPT) {
                const int e = a.ids[(size_t)t * a.k + j];
                if (e >= 0 && e < a.E) atomicAdd(&sc[e], 1);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int off = LPT; off < kWave; off <<= 1) acc[i] += __shfl_xor(acc[i], off, kWave);
    z = wave_sum_xor(z, kWave);
    for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off, kWave);
    if (lane < LPT) {
#pragma unroll
        for (int i = 0; i < PER; ++i) wp[wid][slot_expert<LPT, VEC>(sub, i)] = acc[i];
    }
    if (lane == 0) { wz[wid] = z; wn[wid] = n; }
    __syncthreads();
    for (int e = tid; e < a.E; e += kBalThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += wp[w][e];
        sp[e] = s;
    }
    if (tid == 0) {
        float s = 0.f;
        int c = 0;
        for (int w = 0; w < WAVES; ++w) { s += wz[w]; c += wn[w]; }
        sp[a.E] = s;
        sc[a.E] = c;
    }
    __syncthreads();

    const int blocks = (int)gridDim.x;
    if (blocks > 1) {
        const int group = (int)blockIdx.x / kBalTree, first = group * kBalTree;
        const int members = min(kBalTree, blocks - first), groups = (blocks + kBalTree - 1) / kBalTree;
        put_part(a, (int)blockIdx.x, sp, sc);
        if (!arrive_last(a.sync + kBalSyncStride * (1 + group), members, &flag)) return;
        join_parts(a, first, members, sp, sc);
        if (groups > 1) {
            put_part(a, blocks + group, sp, sc);
            if (!arrive_last(a.sync, groups, &flag)) return;
            join_parts(a, blocks, groups, sp, sc);
        }
    }
    // results: |V| tokens take part
    const int nv = sc[a.E];
    float bal = 0.f;
    for (int e = tid; e < a.E; e += kBalThreads) {
        const float P = nv > 0 ? sp[e] / (float)nv : 0.f;
        a.counts[e] = sc[e];
        a.prob_mean[e] = P;
        bal = fmaf((float)sc[e], P, bal);
    }
    bal = wave_sum_xor(bal, kWave);
    __syncthreads();
    if (lane == 0) wz[wid] = bal;
    __syncthreads();
    if (tid == 0) {
        float s = 0.f;
        for (int w = 0; w < WAVES; ++w) s += wz[w];
        *a.n_valid = nv;
        a.losses[0] = nv > 0 ? s * ((float)a.E / (float)a.k) / (float)nv : 0.f;
        a.losses[1] = nv > 0 ? sp[a.E] / (float)nv : 0.f;
    }
}

struct RouteGradArgs {
    const float* logits;
    const int32_t* ids;
    const float* gates;
    const float* dgates;          // NULL: no gates' part
    const float* dlosses;         // NULL: no losses' part
    const int32_t* counts;
    const int32_t* n_valid;
    const uint8_t* valid;
    float* dlogits;
    int T, E, k, renorm;
};

// A token per LPT lanes.  The experts' f (from the counts) stand in LDS; a token's
// picks are read once, pick p by lane p % LPT, and handed round by lane reads.
template <int LPT, int PER, bool VEC>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteGradArgs a) {
    constexpr int TPW = kWave / LPT, KP = LPT >= 32 ? 1 : LPT == 16 ? 2 : 4;   // picks a lane (k <= min(E, 32))
    __shared__ float fs[LPT * PER];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, sub = lane % LPT, base = lane - sub;
    float ca = 0.f, cz = 0.f;
    if (a.dlosses) {
        const int nv = *a.n_valid;
        const float V = (float)(nv > 1 ? nv : 1);
        ca = a.dlosses[0] * (float)a.E / V;
        cz = a.dlosses[1] * 2.f / V;
        for (int e = tid; e < LPT * PER; e += kThreads) fs[e] = e < a.E ? (float)a.counts[e] / (V * (float)a.k) : 0.f;
        __syncthreads();
    }
    const bool soft = a.dlosses != nullptr || (a.dgates != nullptr && !a.renorm);
    const int step = (int)gridDim.x * 4 * TPW;
    for (int t = ((int)blockIdx.x * 4 + wid) * TPW + lane / LPT; t - lane / LPT < a.T; t += step) {
        const bool in = t < a.T;
        const size_t row = (size_t)(in ? t : 0);
        float v[PER], g[KP], dg[KP];
        int id[KP];
        if (soft) load_row<LPT, PER, VEC>(a.logits + row * a.E, a.E, sub, -INFINITY, v);
        if (a.dgates) {
#pragma unroll
            for (int p = 0; p < KP; ++p) {
                const int j = sub + p * LPT;
                const size_t at = row * a.k + (j < a.k ? j : 0);
                id[p] = a.ids[at];
                g[p] = j < a.k ? a.gates[at] : 0.f;
                dg[p] = j < a.k ? a.dgates[at] : 0.f;
            }
        }
        const bool losses = a.dlosses && in && (a.valid == nullptr || a.valid[t] != 0);
        float inner = 0.f;
        if (a.dgates) {
#pragma unroll
            for (int p = 0; p < KP; ++p) inner = fmaf(g[p], dg[p], inner);
            inner = row_sum<LPT>(inner);
        }
        typedef float row_t __attribute__((ext_vector_type(PER)));
        row_t d = 0.f;
        if (soft) {
            float lse;
            const bool some = softmax_row<LPT, PER>(v, lse);
            float f[PER], pf = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                f[i] = a.dlosses ? fs[slot_expert<LPT, VEC>(sub, i)] : 0.f;
                pf = fmaf(v[i], f[i], pf);
            }
            pf = row_sum<LPT>(pf);
            const float zl = cz * lse, all = a.renorm ? 0.f : inner;
            // (a token without either part stays 0 whatever its logits hold: a padded one's p may be NaN)
            if (some && (losses || (a.dgates && !a.renorm))) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const float loss = losses ? fmaf(ca, f[i] - pf, zl) : 0.f;
                    d[i] = v[i] * (loss - all);
                }
            }
        }
        if (a.dgates) {
#pragma unroll
            for (int p = 0; p < KP; ++p) {
                const float mine = g[p] * (a.renorm ? dg[p] - inner : dg[p]);
                for (int j = 0; j < min(LPT, a.k - p * LPT); ++j) {
                    int e;
                    float add;
                    if constexpr (LPT == kWave) {
                        e = __builtin_amdgcn_readlane(id[p], j);
                        add = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), j));
                    } else {
                        e = __shfl(id[p], base + j, kWave);
                        add = __shfl(mine, base + j, kWave);
                    }
                    if constexpr (LPT == kWave && PER > 4) {               // e is uniform: its slot by register index
                        if (e < 0 || e >= a.E) continue;
                        const int i = VEC ? 4 * (e / (4 * LPT)) + (e & 3) : e / LPT;
                        d[i] += (VEC ? (e >> 2) % LPT : e % LPT) == sub ? add : 0.f;
                    } else {
#pragma unroll
                        for (int i = 0; i < PER; ++i) d[i] += slot_expert<LPT, VEC>(sub, i) == e ? add : 0.f;
                    }
                }
            }
        }
        if (!in) continue;
        float* out = a.dlogits + row * a.E;
        if constexpr (VEC) {
#pragma unroll
            for (int c = 0; c < PER / 4; ++c) {
                const int e = 4 * (sub + LPT * c);
                if (e < a.E) *reinterpret_cast<float4*>(out + e) = make_float4(d[4 * c], d[4 * c + 1], d[4 * c + 2], d[4 * c + 3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = sub + LPT * i;
                if (e < a.E) out[e] = d[i];
            }
        }
    }
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Calls go(LPT, PER) with the lanes per token and values per lane for E experts.
template <typename GO>
void by_experts(int E, GO go) {
    if (E <= 16) go(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
    else if (E <= 64) go(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
    else if (E <= 128) go(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
    else if (E <= 256) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    else if (E <= 512) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
    else go(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

}  // namespace

size_t balance_workspace_bytes(const moe_dims& d) {
    return (size_t)(kBalBlocks + kBalBlocks / kBalTree) * ((size_t)d.E + 1) * sizeof(uint64_t);
}

int launch_balance_loss(const moe_dims& d, const float* logits, const int32_t* ids, const uint8_t* valid,
                        int32_t* counts, float* prob_mean, int32_t* n_valid, float* losses, void* ws, int32_t* sync,
                        hipStream_t s) {
    const BalanceArgs a{logits, ids, valid, counts, prob_mean, n_valid, losses, static_cast<uint64_t*>(ws), sync,
                        d.T, d.E, d.k};
    const bool vec = d.E % 4 == 0 && aligned16(logits);
    by_experts(d.E, [&](auto lpt, auto per) {
        constexpr int L = lpt.value, P = per.value;
        const long tpb = kBalThreads / L;                 // tokens per workgroup and step
        long blocks = ((long)d.T + tpb - 1) / tpb;
        // up to two tokens in a row a lane group rather than a second level of joins (256 tokens
        // x 1024: 9.4 us against 10.7, 512 x 128: 6.6 and 7.3; four in a row for 1024 x 128: 7.8 and 7.3)
        blocks = blocks < 1 ? 1 : blocks;
        if (blocks > kBalTree && blocks <= 2 * kBalTree) blocks = kBalTree;
        if (blocks > kBalBlocks) blocks = kBalBlocks;
        if (vec) hipLaunchKernelGGL((balance_kernel<L, P, true>), dim3((unsigned)blocks), dim3(kBalThreads), 0, s, a);
        else hipLaunchKernelGGL((balance_kernel<L, P, false>), dim3((unsigned)blocks), dim3(kBalThreads), 0, s, a);
    });
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_route_backward(const moe_dims& d, const float* logits, const int32_t* ids, const float* gates, int renorm,
                          const float* dgates, const float* dlosses, const int32_t* counts, const int32_t* n_valid,
                          const uint8_t* valid, float* dlogits, hipStream_t s) {
    if (d.T == 0) return MOE_OK;
    const RouteGradArgs a{logits, ids, gates, dgates, dlosses, counts, n_valid, valid, dlogits, d.T, d.E, d.k,
                          renorm != 0};
    const bool vec = d.E % 4 == 0 && aligned16(logits) && aligned16(dlogits);
    by_experts(d.E, [&](auto lpt, auto per) {
        constexpr int L = lpt.value, P = per.value;
        const long tpb = 4 * (kWave / L);
        long blocks = ((long)d.T + tpb - 1) / tpb;
        blocks = blocks > 2048 ? 2048 : blocks;           // (16384 x 512: 17.8 us; 1024 19.4, 4096 18.6, 8192 18.3)
        if (vec) hipLaunchKernelGGL((route_backward_kernel<L, P, true>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
        else hipLaunchKernelGGL((route_backward_kernel<L, P, false>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    });
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
