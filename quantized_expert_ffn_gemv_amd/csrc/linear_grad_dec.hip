// dx = dy W for few tokens (the weight stream sets the pace), on the matrix cores
// with exact code operands (mfma_ops.h).  With d = dy s the scaled gradient of a
// scale group,
//   dx[t][k] = sum_n d[t][n] q[n][k] + sum_n dy[t][n] b[n]
//            = (1/L) sum_n (128 + L q) d  +  sum_n dy (b - (128/L) s),
// L the codes' lever.  d is carried as three bf16 parts, which hold a float32's 24
// bits (with two, 2^-16 of d was left out, and of 16 + q of it at a weight of zero: outputs
// changed where terms cancel), the codes are exact, the second sum and all accumulation are
// float32.
//
// The sum runs over weight rows, which the codes are not packed along.  A lane
// takes one word (eight columns k) of eight rows; v_perm_b32 pairs the words of
// rows i and i + 4, and each of the eight columns then costs a shift and an
// and-or per pair, as in the forward direction: the B operand (columns = k) of
// column j of every lane's word, for one v_mfma_f32_16x16x32_bf16 per j and part.
// A operand: rows = tokens, the same weight rows in the same pairs.
// Finer scale groups (SPG = 2 or 4 in a 128-run) have one d each: every group's d
// is multiplied with all columns and a lane keeps the sums of its own group.
//
// A workgroup owns one 128-run of K and a share of the weight rows, its waves 32
// rows at a time in turn; their sums meet in LDS, those of several workgroups in
// the workspace, where the last to arrive adds them in order.
//
// Bound by latency where a wave has few rounds (1 token, 4096 x 4096 at 4 bits: 7.1 us;
// 37 tokens, 5111 x 2048 at 2 bits, groups of 64: 12), by the code stream past that
// (8 tokens, 49999 x 4096: 37 us, 3.0 TB/s of the bytes that have to move; float32 dy 36;
// groups of 32 73, by their matrix instructions).
#include <algorithm>
#include <type_traits>

#include "launch_util.h"
#include "linear.h"
#include "mfma_ops.h"
#include "row_ops.h"

namespace moe {

namespace {

constexpr int kGradWaves = 8;
constexpr int kUnit = 32;                              // weight rows per wave and step
constexpr int kRound = kGradWaves * kUnit;             // per workgroup
constexpr int kTok = 16;                               // tokens per workgroup
constexpr int kCounters = 256, kCounterStride = MOE_LINEAR_SYNC_INTS / kCounters;   // ints

struct GradArgs {
    LinearGradArgs l;
    int splits, rows;        // workgroups that share a run's weight rows, rows each (a multiple of kRound)
    float* part;             // [token block][run][split][16][128]
};

template <int SPG, bool F32>
struct GradFrag {
    uint32_t c[8];                                     // this lane's word of rows 8 h + i
    uint32_t dy[F32 ? 8 : 4];                          // token l % 16, rows 8 h ..
    uint32_t sb[(SPG + 1) / 2];                        // scales (lanes 0-31) or biases (32-63) of row l % 32
};

}  // namespace

template <int BITS, int SPG, bool F32>
__global__ __launch_bounds__(64 * kGradWaves) void linear_grad_dec_kernel(GradArgs ga) {
    using Frag = GradFrag<SPG, F32>;
    constexpr int SW = (SPG + 1) / 2, STEP = 2 * 64 * kGradWaves;
    const LinearGradArgs& a = ga.l;
    __shared__ __attribute__((aligned(16))) float sums[kGradWaves][kTok][128];
    __shared__ float zs[kGradWaves][SPG][kTok];
    __shared__ __attribute__((aligned(16))) float srow[kGradWaves][SPG][64];   // scales, biases of a unit's rows
    __shared__ int flag;
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, h = lane >> 4, N = a.w.N;
    const int runs = a.w.K / 128, ngs = runs * SPG;
    // workgroups on one XCD share weight rows: the token blocks of a run their codes, its
    // runs the lines of their scales (one grid for all three: with the blocks on a second axis, of
    // eight, a single run's met on one XCD, 4000 tokens, 417 x 128: 24.5 us against 9.3)
    const int blocks = (a.T + kTok - 1) / kTok, all = runs * ga.splits * blocks, per = (all + 7) / 8;
    const int id = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
    if (id >= all) return;
    const int block = id % blocks, run = id / blocks % runs, split = id / blocks / runs;
    const int t0 = block * kTok;
    const int first = split * ga.rows, last = min(first + ga.rows, N);

    const gbytes_t codes = uniform_gptr(a.w.q + (size_t)run * N * (16 * BITS));
    const int64_t dyrow = (int64_t)min(t0 + c, a.T - 1) * a.lddy;
    // Rows n0 .. n0 + 31; with TAIL some of them past N: their dy reads as 0 and they count
    // nothing.  (dy rows have any alignment.)
    auto load = [&](Frag& f, int n0, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = TAIL ? min(n0 + 8 * h + i, N - 1) : n0 + 8 * h + i;
            const uint32_t at = (uint32_t)n * (16 * BITS) + BITS * c;
            f.c[i] = BITS == 4 ? *reinterpret_cast<const __attribute__((address_space(1))) uint32_t*>(codes + at)
                               : *reinterpret_cast<const __attribute__((address_space(1))) uint16_t*>(codes + at);
        }
        const int nr = TAIL ? min(n0 + (lane & 31), N - 1) : n0 + (lane & 31);
        const uint16_t* sb = (lane < 32 ? a.w.scale : a.w.bias) + (size_t)nr * ngs + run * SPG;
        if constexpr (SPG == 1) {
            f.sb[0] = *sb;
        } else if constexpr (SPG == 2) {
            f.sb[0] = *reinterpret_cast<const uint32_t*>(sb);
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(sb);
            f.sb[0] = v.x;
            f.sb[SW - 1] = v.y;
        }
        const int64_t at = dyrow + n0 + 8 * h;
        if constexpr (!TAIL) {
            if constexpr (F32) __builtin_memcpy(f.dy, static_cast<const float*>(a.dy) + at, 32);
            else __builtin_memcpy(f.dy, static_cast<const uint16_t*>(a.dy) + at, 16);
        } else {
#pragma unroll
            for (int i = 0; i < (F32 ? 8 : 4); ++i) f.dy[i] = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (n0 + 8 * h + i >= N) continue;
                if constexpr (F32) f.dy[i] = static_cast<const uint32_t*>(a.dy)[at + i];
                else f.dy[i >> 1] |= (uint32_t)static_cast<const uint16_t*>(a.dy)[at + i] << (16 * (i & 1));
            }
        }
    };

    floatx4_t acc[SPG][8];
    float z[SPG];
#pragma unroll
    for (int u = 0; u < SPG; ++u) {
        z[u] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[u][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    }
    auto compute = [&](const Frag& f) {
#pragma unroll
        for (int u = 0; u < SPG; ++u) srow[wid][u][lane] = f16_bits_to_f32((f.sb[u >> 1] >> (16 * (u & 1))) & 0xFFFFu);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        const uint32_t base = vreg_const(0x43004300u), mask = vreg_const(BITS == 4 ? 0x00780078u : 0x00300030u);
        uint32_t B[8][4];
#pragma unroll
        for (int half = 0; half < (BITS == 4 ? 2 : 1); ++half)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t p = __builtin_amdgcn_perm(f.c[i + 4], f.c[i], half ? 0x07060302u : 0x05040100u);
#pragma unroll
                for (int jj = 0; jj < (BITS == 4 ? 4 : 8); ++jj)
                    B[4 * half + jj][i] = and_or(shift_to(p, BITS == 4 ? 4 * jj - 3 : 2 * jj - 4), mask, base);
            }
#pragma unroll
        for (int u = 0; u < SPG; ++u) {
            float s[8], be[8];
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const floatx4_t vs = *reinterpret_cast<const floatx4_t*>(&srow[wid][u][8 * h + i]);
                const floatx4_t vb = *reinterpret_cast<const floatx4_t*>(&srow[wid][u][32 + 8 * h + i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[i + e] = vs[e];
                    be[i + e] = fmaf(-kOffset<BITS>, vs[e], vb[e]);
                }
            }
            uint32_t parts[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float d[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = i + 4 * x;
                    float g;
                    if constexpr (F32) g = __uint_as_float(f.dy[r]);
                    else g = (r & 1) ? __uint_as_float(f.dy[r >> 1] & 0xFFFF0000u) : __uint_as_float(f.dy[r >> 1] << 16);
                    d[x] = g * s[r];
                    z[u] = fmaf(g, be[r], z[u]);
                }
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    parts[x][i] = pack_bf16(d[0], d[1]);
                    d[0] -= __uint_as_float(parts[x][i] << 16);
                    d[1] -= __uint_as_float(parts[x][i] & 0xFFFF0000u);
                }
            }
#pragma unroll
            for (int x = 0; x < 3; ++x)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[u][j] = mfma16(parts[x], B[j], acc[u][j]);
            // one scale group's products after another: together their operands would not fit the registers
            if (SPG > 1) __builtin_amdgcn_sched_barrier(0);
        }
    };
    {
        // this wave's whole units: unit wid + 8 i of the share; the next one's loads are always
        // made (the last again at the end), so that no branch waits for them
        const int whole = (last - first) / kUnit, mine = whole > wid ? (whole - wid + kGradWaves - 1) / kGradWaves : 0;
        const std::false_type full{};
        Frag f0, f1;
        if (mine > 0) {
            auto at = [&](int i) { return first + kUnit * (wid + kGradWaves * min(i, mine - 1)); };
            load(f0, at(0), full);
            for (int i = 0; i < mine; i += 2) {
                load(f1, at(i + 1), full);
                compute(f0);
                if (i + 1 >= mine) break;
                load(f0, at(i + 2), full);
                compute(f1);
            }
        }
        if (whole * kUnit < last - first && whole % kGradWaves == wid) {
            load(f0, first + kUnit * whole, std::true_type{});
            compute(f0);
        }
    }
    // second sums: over the quarters here, over the waves below
#pragma unroll
    for (int u = 0; u < SPG; ++u) {
        float v = z[u];
        v += __shfl_xor(v, 16, kWave);
        v += __shfl_xor(v, 32, kWave);
        if (h == 0) zs[wid][u][c] = v;
    }
    const int end = min(kTok, a.T - t0) * 128;                     // results
    float* part = ga.part + (((size_t)block * runs + run) * ga.splits + split) * (kTok * 128);
    // this lane's columns 8 c .. 8 c + 7, of its own scale group
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = acc[0][j][i];
#pragma unroll
            for (int u = 1; u < SPG; ++u) v[j] = c / (16 / SPG) == u ? acc[u][j][i] : v[j];
        }
        floatx4_t* dst = reinterpret_cast<floatx4_t*>(&sums[wid][4 * h + i][8 * c]);
        dst[0] = floatx4_t{v[0], v[1], v[2], v[3]};
        dst[1] = floatx4_t{v[4], v[5], v[6], v[7]};
    }
    __syncthreads();
    for (int o = 2 * tid; o < end; o += STEP) {
        const int tt = o >> 7, k = o & 127;
        float2v_t v = {0.f, 0.f};
        float zz = 0.f;
#pragma unroll
        for (int w = 0; w < kGradWaves; ++w) {
            v += *reinterpret_cast<const float2v_t*>(&sums[w][tt][k]);
            zz += zs[w][k / (128 / SPG)][tt];
        }
        v = v * kInvLever<BITS> + zz;
        if (ga.splits == 1) *reinterpret_cast<uint32_t*>(a.dx + (size_t)(t0 + tt) * a.lddx + 128 * run + k) = pack_bf16(v[0], v[1]);
        else put_device(reinterpret_cast<uint64_t*>(part + o), __builtin_bit_cast(uint64_t, v));
    }
    if (ga.splits == 1) return;
    if (!arrive_last(a.sync + kCounterStride * (block * runs + run), ga.splits, &flag)) return;
    // pairs of results, AT a thread side by side and several splits at once, so that the
    // loads overlap (every one is made, past the tokens the last pair's again: none waits
    // behind a branch)
    const float* from = ga.part + ((size_t)block * runs + run) * ga.splits * (kTok * 128);
    constexpr int AT = 2;
    static_assert(AT * STEP == kTok * 128, "all of them at once");
    float2v_t v[AT];
#pragma unroll
    for (int x = 0; x < AT; ++x) v[x] = float2v_t{0.f, 0.f};
    auto add = [&](auto n) {
#pragma unroll 4
        for (int s = 0; s < ga.splits; ++s)
#pragma unroll
            for (int x = 0; x < decltype(n)::value; ++x) {
                const int o = min(2 * tid + x * STEP, end - 2);
                v[x] += __builtin_bit_cast(float2v_t, get_device(reinterpret_cast<const uint64_t*>(from + (size_t)s * (kTok * 128) + o)));
            }
    };
    if (end <= STEP) add(std::integral_constant<int, 1>{});
    else add(std::integral_constant<int, AT>{});
#pragma unroll
    for (int x = 0; x < AT; ++x) {
        const int o = 2 * tid + x * STEP;
        if (o < end)
            *reinterpret_cast<uint32_t*>(a.dx + (size_t)(t0 + (o >> 7)) * a.lddx + 128 * run + (o & 127)) = pack_bf16(v[x][0], v[x][1]);
    }
}

// Splits of the weight rows, whole rounds of rows each: one workgroup a CU (4096 x
// 4096, 1 token: 7.1 us; half as many 8.1, twice 7.8; 49999 x 4096, 8 tokens: 37, 60,
// 39), rounded up where a CU holds two (SPG = 1), else down (twice as many, 37 x 5111 x 2048 at
// groups of 64: 16.7 us against 12.3); and partial sums, written and read, of at most
// twice the codes' bytes.
int grad_splits(const moe_qmatrix& w, int T) {
    // (more than one split only where runs times token blocks are fewer than the counters)
    const int runs = w.K / 128, blocks = (T + kTok - 1) / kTok, cus = device_cus() < kCounters ? device_cus() : kCounters;
    const int rounds = (w.N + kRound - 1) / kRound;
    const int fill = (cus + (w.group_size == 128 ? runs * blocks - 1 : 0)) / (runs * blocks);
    const long bytes = (long)w.N * 16 * w.bits * 2 / (512 * 2 * (T < kTok ? T : kTok));
    int s = fill < rounds ? fill : rounds;
    s = s < bytes ? s : (int)bytes;
    s = s < 1 ? 1 : s;
    const int per = (rounds + s - 1) / s;                      // rounds a split
    return (rounds + per - 1) / per;
}

// A CU's rounds of weight rows, and its workgroups' starts and ends.
double linear_grad_dec_us(const moe_qmatrix& w, int T) {
    static const double c[3][3] = {{4.7, 1.3, 0.4}, {4.5, 1.95, 0.9}, {4.4, 3.3, 0.45}};   // groups of 128, 64, 32
    const double* f = c[w.group_size == 128 ? 0 : w.group_size == 64 ? 1 : 2];
    const double per_cu = (double)(w.K / 128) * ((T + kTok - 1) / kTok) / device_cus(), rounds = (w.N + kRound - 1) / kRound;
    return f[0] + f[1] * std::max(1.0, per_cu * rounds) + f[2] * per_cu;
}

size_t linear_grad_dec_workspace_bytes(const moe_qmatrix& w, int T) {
    const int s = grad_splits(w, T);
    return s == 1 ? 0 : (size_t)((T + kTok - 1) / kTok) * (w.K / 128) * s * kTok * 128 * sizeof(float);
}

// The most of any call of up to T tokens: splits go by the tokens of one block, then by the
// blocks, and past a block for every CU there is one.
size_t linear_grad_dec_most_bytes(const moe_qmatrix& w, int T) {
    size_t most = 0;
    for (int t = 1; t <= T && t <= kTok * (kCounters + 1); t += t < kTok ? 1 : kTok) most = std::max(most, linear_grad_dec_workspace_bytes(w, t));
    return std::max(most, linear_grad_dec_workspace_bytes(w, T));
}

namespace {

template <int BITS, int SPG>
void grad_go(const GradArgs& g, hipStream_t s) {
    const long all = (long)(g.l.w.K / 128) * g.splits * ((g.l.T + kTok - 1) / kTok);
    const dim3 grid((unsigned)((all + 7) / 8 * 8));
    if (g.l.dy_type == MOE_F32)
        hipLaunchKernelGGL((linear_grad_dec_kernel<BITS, SPG, true>), grid, dim3(64 * kGradWaves), 0, s, g);
    else
        hipLaunchKernelGGL((linear_grad_dec_kernel<BITS, SPG, false>), grid, dim3(64 * kGradWaves), 0, s, g);
}

template <int BITS>
void grad_groups(const GradArgs& g, hipStream_t s) {
    const int spg = 128 / g.l.w.group_size;
    if (spg == 1) grad_go<BITS, 1>(g, s);
    else if (spg == 2) grad_go<BITS, 2>(g, s);
    else grad_go<BITS, 4>(g, s);
}

}  // namespace

int launch_linear_grad_dec(const LinearGradArgs& a, hipStream_t s) {
    GradArgs g{a, grad_splits(a.w, a.T), 0, static_cast<float*>(a.ws)};
    const int rounds = (a.w.N + kRound - 1) / kRound;
    g.rows = (rounds + g.splits - 1) / g.splits * kRound;
    if (a.w.bits == 4) grad_groups<4>(g, s);
    else grad_groups<2>(g, s);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
