// The router's losses and its backward pass, over float32 logits [T][E].
//
// Both kernels give a token's row to LPT lanes (4, 16, 32 or 64; the smallest
// that holds the row in at most 4 values a lane, 16 at E = 1024), keep it in
// registers, and need one pass over the logits:
//   m = max L, e = exp(L - m), S = sum e, p = e / S, lse = m + log S,
// m and S by reductions over the lanes.  A row without a logit above -inf has
// p = 0 everywhere.
#include <cmath>

#include "common.h"
#include "row_ops.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kBalTree = 16;                              // workgroups joined by one ticket
constexpr int kBalBlocks = kBalTree * kBalTree;           // at most this many workgroups
constexpr int kBalSyncStride = 64;                        // counters 256 bytes apart
static_assert(MOE_BALANCE_SYNC_INTS == kBalSyncStride * (1 + kBalTree), "sync buffer layout");

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

// v (logits) -> p in place; returns whether the row has a logit, and lse.
template <int LPT, int PER>
__device__ __forceinline__ bool softmax_row(float (&v)[PER], float& lse) {
    float m = v[0];
    bool nan = v[0] != v[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) {
        m = fmaxf(m, v[i]);
        nan |= v[i] != v[i];
    }
    m = row_max<LPT>(m);                                  // fmaxf skips NaNs: the sum below brings them back
    const bool some = m > -INFINITY || row_max<LPT>(nan ? 1.f : 0.f) > 0.f;
    const float base = m > -INFINITY ? m : 0.f;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v[i] = expf(v[i] - base);
        s += v[i];
    }
    s = row_sum<LPT>(s);
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
    float* part;              // [blocks + kBalTree][stride]: E sums of p, E counts, z, n
    int32_t* sync;
    int T, E, k, stride;
};

// Sum of partial rows [first, first + n) of `part` into the workgroup's LDS.
__device__ __forceinline__ void join_parts(const BalanceArgs& a, int first, int n, float* sp, int* sc, float* sz, int* sn) {
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        float p = 0.f;
        int c = 0;
#pragma unroll 4
        for (int b = 0; b < n; ++b) {
            const float* row = a.part + (size_t)(first + b) * a.stride;
            p += get_device(row + e);
            c += get_device(reinterpret_cast<const int*>(row) + a.E + e);
        }
        sp[e] = p;
        sc[e] = c;
    }
    if (threadIdx.x == 0) {
        float z = 0.f;
        int cnt = 0;
        for (int b = 0; b < n; ++b) {
            const float* row = a.part + (size_t)(first + b) * a.stride + 2 * a.E;
            z += get_device(row);
            cnt += get_device(reinterpret_cast<const int*>(row) + 1);
        }
        *sz = z;
        *sn = cnt;
    }
    __syncthreads();
}

__device__ __forceinline__ void put_part(const BalanceArgs& a, int slot, const float* sp, const int* sc, float z, int n) {
    float* row = a.part + (size_t)slot * a.stride;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        put_device(row + e, sp[e]);
        put_device(reinterpret_cast<int*>(row) + a.E + e, sc[e]);
    }
    if (threadIdx.x == 0) {
        put_device(row + 2 * a.E, z);
        put_device(reinterpret_cast<int*>(row) + 2 * a.E + 1, n);
    }
}

}  // namespace

// Sums of p, picks, lse^2 and tokens per workgroup, joined by a tree of arrival
// tickets: the last of each 16 workgroups sums their 16 partial rows, the last
// of those sums the groups' rows and writes the results, all in index order.
template <int LPT, int PER, bool VEC>
__global__ __launch_bounds__(kThreads) void balance_kernel(BalanceArgs a) {
    constexpr int TPW = kWave / LPT;                      // tokens per wave at once
    __shared__ float sp[1024];
    __shared__ int sc[1024];
    __shared__ float wp[4][1024];
    __shared__ float sz;
    __shared__ int sn;
    __shared__ float wz[4];
    __shared__ int wn[4], flag;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, sub = lane % LPT;
    for (int e = tid; e < a.E; e += kThreads) sc[e] = 0;
    __syncthreads();
    float acc[PER], z = 0.f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    const int step = (int)gridDim.x * 4 * TPW;
    for (int t = ((int)blockIdx.x * 4 + wid) * TPW + lane / LPT; t - lane / LPT < a.T; t += step) {
        const bool live = t < a.T && (a.valid == nullptr || a.valid[t] != 0);
        float v[PER], lse;
        load_row<LPT, PER, VEC>(a.logits + (size_t)(live ? t : 0) * a.E, live ? a.E : 0, sub, -INFINITY, v);
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
        for (int i = 0; i < PER; ++i) {
            const int e = slot_expert<LPT, VEC>(sub, i);
            if (e < a.E) wp[wid][e] = acc[i];
        }
    }
    if (lane == 0) { wz[wid] = z; wn[wid] = n; }
    __syncthreads();
    for (int e = tid; e < a.E; e += kThreads) sp[e] = (wp[0][e] + wp[1][e]) + (wp[2][e] + wp[3][e]);
    if (tid == 0) {
        sz = (wz[0] + wz[1]) + (wz[2] + wz[3]);
        sn = (wn[0] + wn[1]) + (wn[2] + wn[3]);
    }
    __syncthreads();

    const int blocks = (int)gridDim.x;
    if (blocks > 1) {
        const int group = (int)blockIdx.x / kBalTree, first = group * kBalTree;
        const int members = min(kBalTree, blocks - first), groups = (blocks + kBalTree - 1) / kBalTree;
        put_part(a, (int)blockIdx.x, sp, sc, sz, sn);
        if (!arrive_last(a.sync + kBalSyncStride * (1 + group), members, &flag)) return;
        join_parts(a, first, members, sp, sc, &sz, &sn);
        if (groups > 1) {
            put_part(a, blocks + group, sp, sc, sz, sn);
            if (!arrive_last(a.sync, groups, &flag)) return;
            join_parts(a, blocks, groups, sp, sc, &sz, &sn);
        }
    }
    // results: |V| tokens take part
    const float inv = sn > 0 ? 1.f / (float)sn : 0.f;
    float bal = 0.f;
    for (int e = tid; e < a.E; e += kThreads) {
        const float P = sn > 0 ? sp[e] / (float)sn : 0.f;
        a.counts[e] = sc[e];
        a.prob_mean[e] = P;
        bal = fmaf((float)sc[e], P, bal);
    }
    bal = wave_sum_xor(bal, kWave);
    __syncthreads();
    if (lane == 0) wz[wid] = bal;
    __syncthreads();
    if (tid == 0) {
        *a.n_valid = sn;
        a.losses[0] = ((wz[0] + wz[1]) + (wz[2] + wz[3])) * ((float)a.E / (float)a.k) * inv;
        a.losses[1] = sn > 0 ? sz / (float)sn : 0.f;
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

// One wave walks its tokens; the experts' f (from the counts) stay in registers.
template <int LPT, int PER, bool VEC>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteGradArgs a) {
    constexpr int TPW = kWave / LPT;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, sub = lane % LPT;
    float f[PER], ca = 0.f, cz = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) f[i] = 0.f;
    if (a.dlosses) {
        const int nv = *a.n_valid;
        const float V = (float)(nv > 1 ? nv : 1);
        ca = a.dlosses[0] * (float)a.E / V;
        cz = a.dlosses[1] * 2.f / V;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = slot_expert<LPT, VEC>(sub, i);
            if (e < a.E) f[i] = (float)a.counts[e] / (V * (float)a.k);
        }
    }
    const bool soft = a.dlosses != nullptr || (a.dgates != nullptr && !a.renorm);
    const int step = (int)gridDim.x * 4 * TPW;
    for (int t = ((int)blockIdx.x * 4 + wid) * TPW + lane / LPT; t - lane / LPT < a.T; t += step) {
        const bool in = t < a.T;
        const size_t row = (size_t)(in ? t : 0);
        float d[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) d[i] = 0.f;
        const float* g = a.gates + row * a.k;
        const float* dg = a.dgates + row * a.k;
        float inner = 0.f;
        if (a.dgates && in)
            for (int j = 0; j < a.k; ++j) inner = fmaf(g[j], dg[j], inner);
        if (soft) {
            float v[PER], lse;
            load_row<LPT, PER, VEC>(a.logits + row * a.E, in ? a.E : 0, sub, -INFINITY, v);
            const bool some = softmax_row<LPT, PER>(v, lse);
            const bool part = some && a.dlosses && in && (a.valid == nullptr || a.valid[t] != 0);
            float pf = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) pf = fmaf(v[i], f[i], pf);
            pf = row_sum<LPT>(pf);
            const float zl = cz * lse, all = a.renorm ? 0.f : inner;
            if (some) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const float loss = part ? fmaf(ca, f[i] - pf, zl) : 0.f;
                    d[i] = v[i] * (loss - all);
                }
            }
        }
        if (!in) continue;
        if (a.dgates) {
            const int32_t* id = a.ids + row * a.k;
            for (int j = 0; j < a.k; ++j) {
                const int e = id[j];
                const float add = g[j] * (a.renorm ? dg[j] - inner : dg[j]);
#pragma unroll
                for (int i = 0; i < PER; ++i) d[i] += slot_expert<LPT, VEC>(sub, i) == e ? add : 0.f;
            }
        }
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
    return (size_t)(kBalBlocks + kBalTree) * (2 * (size_t)d.E + 2) * sizeof(float);
}

int launch_balance_loss(const moe_dims& d, const float* logits, const int32_t* ids, const uint8_t* valid,
                        int32_t* counts, float* prob_mean, int32_t* n_valid, float* losses, void* ws, int32_t* sync,
                        hipStream_t s) {
    const BalanceArgs a{logits, ids, valid, counts, prob_mean, n_valid, losses, static_cast<float*>(ws), sync,
                        d.T, d.E, d.k, 2 * d.E + 2};
    const bool vec = d.E % 4 == 0 && aligned16(logits);
    by_experts(d.E, [&](auto lpt, auto per) {
        constexpr int L = lpt.value, P = per.value;
        const long tpb = 4 * (kWave / L);                 // tokens per workgroup and step
        long blocks = ((long)d.T + tpb - 1) / tpb;
        blocks = blocks < 1 ? 1 : blocks > kBalBlocks ? kBalBlocks : blocks;
        if (vec) hipLaunchKernelGGL((balance_kernel<L, P, true>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
        else hipLaunchKernelGGL((balance_kernel<L, P, false>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
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
        blocks = blocks > 2048 ? 2048 : blocks;
        if (vec) hipLaunchKernelGGL((route_backward_kernel<L, P, true>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
        else hipLaunchKernelGGL((route_backward_kernel<L, P, false>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    });
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
