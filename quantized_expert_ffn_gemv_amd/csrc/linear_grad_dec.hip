// dx = dy W for few tokens (the weight stream sets the pace), on the matrix cores
// with exact code operands (mfma_ops.h).  With d = dy s the scaled gradient of a
// scale group,
//   dx[t][k] = sum_n d[t][n] q[n][k] + sum_n dy[t][n] b[n]
//            = (1/L) sum_n (128 + L q) d  +  sum_n dy (b - (128/L) s),
// L the codes' lever.  d is carried as two bf16 parts (together 2^-16 of it left
// out; dx is rounded to bf16's 2^-8), the codes are exact, the second sum and all
// accumulation are float32.
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
#include "launch_util.h"
#include "linear.h"
#include "mfma_ops.h"
#include "row_ops.h"

namespace moe {

namespace {

constexpr int kGradWaves = 8;
constexpr int kUnit = 32;                              // weight rows per wave and step
constexpr int kRound = kGradWaves * kUnit;             // per workgroup
constexpr int kCounterStride = 2;                      // ints

struct GradArgs {
    LinearGradArgs l;
    int splits, rows;        // workgroups that share a run's weight rows, rows each (a multiple of kRound)
    float* part;             // [token block][run][split][16 NT][128]
};

template <int BITS, int SPG, int NT, bool F32>
struct GradFrag {
    uint32_t c[8];                                     // this lane's word of rows 8 h + i
    uint32_t dy[NT][F32 ? 8 : 4];                      // token l % 16 of each tile, rows 8 h ..
    uint32_t sb[(SPG + 1) / 2];                        // scales (lanes 0-31) or biases (32-63) of row l % 32
};

}  // namespace

template <int BITS, int SPG, int NT, bool F32>
__global__ __launch_bounds__(64 * kGradWaves) void linear_grad_dec_kernel(GradArgs ga) {
    using Frag = GradFrag<BITS, SPG, NT, F32>;
    constexpr int TOK = 16 * NT, SW = (SPG + 1) / 2;
    const LinearGradArgs& a = ga.l;
    __shared__ __attribute__((aligned(16))) float sums[kGradWaves][16][128];
    __shared__ float zs[kGradWaves][SPG][TOK];
    __shared__ __attribute__((aligned(16))) float srow[kGradWaves][SPG][64];   // scales, biases of a unit's rows
    __shared__ int flag;
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, h = lane >> 4, N = a.w.N;
    const int runs = a.w.K / 128, ngs = runs * SPG;
    // workgroups on one XCD share weight rows (and the lines of their scales)
    const int all = runs * ga.splits, per = (all + 7) / 8;
    const int id = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
    if (((int)blockIdx.x >> 3) >= per || id >= all) return;
    const int split = id / runs, run = id % runs;
    const int t0 = (int)blockIdx.y * TOK;
    const int first = split * ga.rows, last = min(first + ga.rows, N);

    const uint8_t* codes = a.w.q + (size_t)run * N * (16 * BITS);
    auto load = [&](Frag& f, int n0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint8_t* row = codes + (size_t)min(n0 + 8 * h + i, N - 1) * (16 * BITS);
            f.c[i] = BITS == 4 ? reinterpret_cast<const uint32_t*>(row)[c] : reinterpret_cast<const uint16_t*>(row)[c];
        }
        const uint16_t* sb = (lane < 32 ? a.w.scale : a.w.bias) + (size_t)min(n0 + (lane & 31), N - 1) * ngs + run * SPG;
        if constexpr (SPG == 1) {
            f.sb[0] = *sb;
        } else if constexpr (SPG == 2) {
            f.sb[0] = *reinterpret_cast<const uint32_t*>(sb);
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(sb);
            f.sb[0] = v.x;
            f.sb[SW - 1] = v.y;
        }
        // dy rows have any alignment; the last rows' unit stops at N
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t at = (int64_t)min(t0 + 16 * t + c, a.T - 1) * a.lddy + n0 + 8 * h;
            constexpr int W = F32 ? 8 : 4;
            if (n0 + kUnit <= N) {
                if constexpr (F32) __builtin_memcpy(f.dy[t], static_cast<const float*>(a.dy) + at, 32);
                else __builtin_memcpy(f.dy[t], static_cast<const uint16_t*>(a.dy) + at, 16);
            } else {
                for (int i = 0; i < W; ++i) f.dy[t][i] = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (n0 + 8 * h + i >= N) continue;
                    if constexpr (F32) f.dy[t][i] = static_cast<const uint32_t*>(a.dy)[at + i];
                    else f.dy[t][i >> 1] |= (uint32_t)static_cast<const uint16_t*>(a.dy)[at + i] << (16 * (i & 1));
                }
            }
        }
    };

    floatx4_t acc[SPG][NT][8];
    float z[SPG][NT];
#pragma unroll
    for (int u = 0; u < SPG; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            z[u][t] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[u][t][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
        }
    auto compute = [&](const Frag& f, int n0) {
        // rows past N have dy = 0 and count nothing
#pragma unroll
        for (int u = 0; u < SPG; ++u) srow[wid][u][lane] = f16_bits_to_f32((f.sb[u >> 1] >> (16 * (u & 1))) & 0xFFFFu);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        uint32_t hi[SPG][NT][4], lo[SPG][NT][4];
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
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float d[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float g;
                    if constexpr (F32) g = __uint_as_float(f.dy[t][i]);
                    else g = (i & 1) ? __uint_as_float(f.dy[t][i >> 1] & 0xFFFF0000u) : __uint_as_float(f.dy[t][i >> 1] << 16);
                    d[i] = g * s[i];
                    z[u][t] = fmaf(g, be[i], z[u][t]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    hi[u][t][i] = pack_bf16(d[i], d[i + 4]);
                    lo[u][t][i] = pack_bf16(d[i] - __uint_as_float(hi[u][t][i] << 16),
                                            d[i + 4] - __uint_as_float(hi[u][t][i] & 0xFFFF0000u));
                }
            }
        }
        const uint32_t base = vreg_const(0x43004300u), mask = vreg_const(BITS == 4 ? 0x00780078u : 0x00300030u);
#pragma unroll
        for (int half = 0; half < (BITS == 4 ? 2 : 1); ++half) {
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                p[i] = __builtin_amdgcn_perm(f.c[i + 4], f.c[i], half ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int jj = 0; jj < (BITS == 4 ? 4 : 8); ++jj) {
                const int j = 4 * half + jj;
                uint32_t B[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) B[i] = and_or(shift_to(p[i], BITS == 4 ? 4 * jj - 3 : 2 * jj - 4), mask, base);
#pragma unroll
                for (int u = 0; u < SPG; ++u)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        acc[u][t][j] = mfma16(hi[u][t], B, acc[u][t][j]);
                        acc[u][t][j] = mfma16(lo[u][t], B, acc[u][t][j]);
                    }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    };
    {
        Frag f0, f1;
        int n = first + kUnit * wid;
        if (n < last) load(f0, n);
        while (n < last) {
            if (n + kRound < last) load(f1, n + kRound);
            compute(f0, n);
            n += kRound;
            if (n >= last) break;
            if (n + kRound < last) load(f0, n + kRound);
            compute(f1, n);
            n += kRound;
        }
    }
    // second sums: over the quarters here, over the waves below
#pragma unroll
    for (int u = 0; u < SPG; ++u)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float v = z[u][t];
            v += __shfl_xor(v, 16, kWave);
            v += __shfl_xor(v, 32, kWave);
            if (h == 0) zs[wid][u][16 * t + c] = v;
        }
    const int tokens = min(TOK, a.T - t0);
    float* part = ga.part + (((size_t)blockIdx.y * runs + run) * ga.splits + split) * (TOK * 128);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (t > 0) __syncthreads();
        // this lane's columns 8 c .. 8 c + 7, of its own scale group
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = acc[0][t][j][i];
#pragma unroll
                for (int u = 1; u < SPG; ++u) v[j] = c / (16 / SPG) == u ? acc[u][t][j][i] : v[j];
            }
            floatx4_t* dst = reinterpret_cast<floatx4_t*>(&sums[wid][4 * h + i][8 * c]);
            dst[0] = floatx4_t{v[0], v[1], v[2], v[3]};
            dst[1] = floatx4_t{v[4], v[5], v[6], v[7]};
        }
        __syncthreads();
        for (int o = tid; o < min(16, tokens - 16 * t) * 128; o += 64 * kGradWaves) {
            const int tt = o >> 7, k = o & 127;
            float v = 0.f, zz = 0.f;
#pragma unroll
            for (int w = 0; w < kGradWaves; ++w) {
                v += sums[w][tt][k];
                zz += zs[w][k / (128 / SPG)][16 * t + tt];
            }
            v = fmaf(v, kInvLever<BITS>, zz);
            if (ga.splits == 1)
                a.dx[(size_t)(t0 + 16 * t + tt) * a.lddx + 128 * run + k] = (uint16_t)(pack_bf16(v, 0.f) & 0xFFFFu);
            else
                put_device(part + (16 * t + tt) * 128 + k, v);
        }
    }
    if (ga.splits == 1) return;
    if (!arrive_last(a.sync + kCounterStride * ((int)blockIdx.y * runs + run), ga.splits, &flag)) return;
    const float* from = ga.part + ((size_t)blockIdx.y * runs + run) * ga.splits * (TOK * 128);
    for (int o = tid; o < tokens * 128; o += 64 * kGradWaves) {
        float v = 0.f;
#pragma unroll 8
        for (int s = 0; s < ga.splits; ++s) v += get_device(from + (size_t)s * (TOK * 128) + o);
        a.dx[(size_t)(t0 + (o >> 7)) * a.lddx + 128 * run + (o & 127)] = (uint16_t)(pack_bf16(v, 0.f) & 0xFFFFu);
    }
}

namespace {

// Token tiles per workgroup: two where the sums fit the registers.
inline int grad_tiles(const moe_qmatrix& w, int T) { return T > 16 && w.group_size >= 64 ? 2 : 1; }

// Splits of the weight rows: enough workgroups for two on every CU, whole rounds
// of rows each, and partial sums of at most half the codes' bytes.
int grad_splits(const moe_qmatrix& w, int T) {
    const int runs = w.K / 128, tok = 16 * grad_tiles(w, T), blocks = (T + tok - 1) / tok;
    const int rounds = (w.N + kRound - 1) / kRound;
    const int fill = (2 * device_cus() + runs * blocks - 1) / (runs * blocks);
    const int bytes = w.N * 16 * w.bits / (2 * 512 * 2 * (T < tok ? T : tok));
    int s = fill < rounds ? fill : rounds;
    s = s < bytes ? s : bytes;
    s = s < 1 ? 1 : s;
    const int per = (rounds + s - 1) / s;                      // rounds a split
    return (rounds + per - 1) / per;
}

}  // namespace

size_t linear_grad_dec_workspace_bytes(const moe_qmatrix& w, int T) {
    const int tok = 16 * grad_tiles(w, T), blocks = (T + tok - 1) / tok, s = grad_splits(w, T);
    return s == 1 ? 0 : (size_t)blocks * (w.K / 128) * s * tok * 128 * sizeof(float);
}

namespace {

template <int BITS, int SPG, int NT>
void grad_go(const GradArgs& g, hipStream_t s) {
    const int all = g.l.w.K / 128 * g.splits;
    const dim3 grid((unsigned)((all + 7) / 8 * 8), (unsigned)((g.l.T + 16 * NT - 1) / (16 * NT)));
    if (g.l.dy_type == MOE_F32)
        hipLaunchKernelGGL((linear_grad_dec_kernel<BITS, SPG, NT, true>), grid, dim3(64 * kGradWaves), 0, s, g);
    else
        hipLaunchKernelGGL((linear_grad_dec_kernel<BITS, SPG, NT, false>), grid, dim3(64 * kGradWaves), 0, s, g);
}

template <int BITS>
void grad_groups(const GradArgs& g, hipStream_t s) {
    const int spg = 128 / g.l.w.group_size;
    if (grad_tiles(g.l.w, g.l.T) == 2) {
        if (spg == 1) grad_go<BITS, 1, 2>(g, s);
        else grad_go<BITS, 2, 2>(g, s);
    } else {
        if (spg == 1) grad_go<BITS, 1, 1>(g, s);
        else if (spg == 2) grad_go<BITS, 2, 1>(g, s);
        else grad_go<BITS, 4, 1>(g, s);
    }
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
