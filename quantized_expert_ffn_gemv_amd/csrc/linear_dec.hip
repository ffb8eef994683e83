// y = x W^T for few tokens (the weight stream sets the pace), on the matrix
// cores with exact code operands (mfma_ops.h):
//   y[t][n] = sum_g (s/L) C_g + (b - (128/L) s) X_g,
//   C_g = sum_{k in g} (128 + L q) x,  X_g = sum_{k in g} x,
// L the codes' lever; C and X come from v_mfma_f32_16x16x32_bf16 (X from an
// operand of ones), so the only roundings are float32's and y's own.
//
// Activations are the A operand (rows = tokens) and codes the B operand (columns
// = weight rows), so a lane's four sums share one weight row's scale.
//
// Bound by the weight stream: 8 tokens x 49999 x 4096 at 4 bits, float32 out, take 26 us
// (4.2 TB/s of the bytes that have to move), 28672 x 8192 32 us (3.9 TB/s); 4096 x 4096,
// one or two tiles a CU, 6.8 us, most of it launch, start and the last tile.
#include <algorithm>

#include "launch_util.h"
#include "linear.h"
#include "mfma_ops.h"
#include "row_ops.h"

namespace moe {

namespace {

constexpr int kStreamMaxWaves = 8;
constexpr int kStreamGroups = 64;      // groups of K per launch: at most 8 a wave

// Words c of the lane quarters transposed: out[st] of quarter q = word q of
// quarter st (the tr order of mfma_ops.h, from 16-byte loads in natural order;
// 2-bit codes have two words a quarter, each standing for two).
template <int BITS>
__device__ __forceinline__ void quarter_transpose(const uint32_t* c, uint32_t (&out)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = BITS == 4 ? c[i] : c[i >> 1];
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);   // quarters 0 1 | 2 3
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    out[0] = lo[0];
    out[1] = lo[1];
    out[2] = hi[0];
    out[3] = hi[1];
}

// LDS row of a tile's n scales: whole 16-byte pieces and one more, so that 16 rows
// read at one group hit distinct banks.
__host__ __device__ inline int scale_pitch(int n) { return 8 * ((n + 7) / 8) + 8; }

// Kernels of which two workgroups fit a CU's registers (128 a lane; with twice the
// operands the bound made them spill: 8 tokens, 28672 x 4096, groups of 32 27 us against 23).
constexpr bool two_fit(int nt, int gpw) { return nt * gpw <= 2; }

struct StreamArgs {
    LinearArgs l;
    int g0, ng;              // the launch's groups of K: [g0, g0 + ng)
    const float* add;        // sums of earlier launches over other groups [T][N], or NULL
};

// SPG consecutive values in one LDS read (a group's start is a multiple of SPG values).
template <int SPG, int SW>
__device__ __forceinline__ void load_scales_of(const uint16_t* p, uint32_t (&w)[SW]) {
    if constexpr (SPG == 1) {
        w[0] = *p;
    } else if constexpr (SPG == 2) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[SW - 1] = v.y;
    }
}

// 16 bytes from a 2-byte aligned address (global memory takes any alignment).
__device__ __forceinline__ uint4 load16_any(const uint16_t* p) {
    uint4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

}  // namespace

// The activations stay in registers: wave w of a workgroup owns groups GPW w ..
// GPW w + GPW - 1 for the whole launch, keeps their activation operands, and
// streams only weights, tile after tile of 16 RT rows.  Units (tile, group) pass
// through a ring of RBU * GPW register slots; a slot's next unit is requested as
// soon as its codes are used, so the stream does not stop at tile borders.  A
// tile's scales and biases are read by the workgroup's threads 16 bytes each and
// passed on through LDS (read by each lane where it needs them they took eight
// times the codes' cache cycles: 16 rows' cache lines for two bytes each; 49999 x
// 4096 38 us against 28).  The waves' sums meet in LDS, one barrier a tile.
template <int BITS, int SPG, int NT, int RT, int GPW, int RBU>
__global__ __launch_bounds__(64 * kStreamMaxWaves, (two_fit(NT, GPW) ? 4 : 2)) void linear_stream_kernel(StreamArgs sa) {
    const LinearArgs& a = sa.l;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int RB = 16 * RT, STEPS = 4 / SPG, SW = (SPG + 1) / 2;
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6, m = lane & 15, q = lane >> 4;
    const int t0 = (int)blockIdx.y * 16 * NT, tokens = min(16 * NT, a.T - t0);
    const int NG = sa.ng, ngs = a.w.K / 128 * SPG, g0 = wid * GPW;   // groups are counted from sa.g0 here
    const int tiles = (a.w.N + RB - 1) / RB, stride = gridDim.x;
    // LDS: scale slots [2][scales, biases][RB][pitch], X of every wave, the waves' sums [2][rows4][tokens][RB]
    const int pitch = scale_pitch(NG * SPG);                   // of a row of scales in LDS
    uint16_t* slots = reinterpret_cast<uint16_t*>(lds);
    float* xs = reinterpret_cast<float*>(lds + 8 * RB * (size_t)pitch) + (size_t)wid * GPW * NT * SPG * 16;
    float* red = reinterpret_cast<float*>(lds + 8 * RB * (size_t)pitch) + (size_t)waves * GPW * NT * SPG * 16;
    const int rows4 = (waves + 3) & ~3;                        // the sums are added four waves at a time

    uint32_t code[RBU][GPW][RT][BITS];
    const size_t code_step = (size_t)a.w.N * (16 * BITS);
    auto load = [&](int i, int j, int tile) {
        const gbytes_t base = uniform_gptr(a.w.q + (size_t)(sa.g0 + min(g0 + j, NG - 1)) * code_step);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const uint32_t at = (uint32_t)min(tile * RB + 16 * r + m, a.w.N - 1) * (16 * BITS);
            if constexpr (BITS == 4) {
                const u32x4_t v = *reinterpret_cast<gu32x4_t>(base + (at + 16u * q));
                code[i][j][r][0] = v.x; code[i][j][r][1] = v.y; code[i][j][r][2] = v.z; code[i][j][r][3] = v.w;
            } else {
                const u32x2_t v = *reinterpret_cast<gu32x2_t>(base + (at + 8u * q));
                code[i][j][r][0] = v.x; code[i][j][r][1] = v.y;
            }
        }
    };
    // this thread's pieces (8 values of a row) of a tile's scales and biases: 2 RB PPR in
    // all, PPR a row, PP a thread (the launch has enough threads); a row's last piece may
    // run into the next row, the matrix' last one is read by value
    constexpr int PP = (RT * GPW * SPG + 15) / 16;
    const int PPR = (NG * SPG + 7) / 8, threads = blockDim.x;
    const size_t all_values = (size_t)a.w.N * ngs;
    const uint16_t* from[PP];
    int prow[PP], pcol[PP];
    bool mine[PP];
    uint16_t* to[PP];
#pragma unroll
    for (int p = 0; p < PP; ++p) {
        const int id = tid + p * threads, row = id / PPR % RB, c = id % PPR;
        mine[p] = id < 2 * RB * PPR;
        from[p] = id < RB * PPR ? a.w.scale : a.w.bias;
        prow[p] = row;
        pcol[p] = sa.g0 * SPG + 8 * c;
        to[p] = slots + (id < RB * PPR ? 0 : RB * pitch) + row * pitch + 8 * c;
    }
    auto load_scales = [&](int p, int tile) {
        const size_t at = (size_t)min(tile * RB + prow[p], a.w.N - 1) * ngs + pcol[p];
        if (at + 8 <= all_values) return load16_any(from[p] + at);
        uint64_t lo = 0, hi = 0;
#pragma unroll 1
        for (int i = 0; i < (int)(all_values - at); ++i) {
            const uint64_t v = (uint64_t)from[p][at + i] << (16 * (i & 3));
            lo |= i < 4 ? v : 0;
            hi |= i < 4 ? 0 : v;
        }
        return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
    };

#pragma unroll
    for (int i = 0; i < RBU; ++i)
#pragma unroll
        for (int j = 0; j < GPW; ++j) load(i, j, (int)blockIdx.x + i * stride);
    uint4 sreg[PP];
#pragma unroll
    for (int p = 0; p < PP; ++p) sreg[p] = load_scales(p, blockIdx.x);

    // activation operands A[j][t][st] and group sums X[j][t][scale group], once;
    // zeros for groups past K
    const uint32_t ones[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    const floatx4_t zero = {0.f, 0.f, 0.f, 0.f};
    uint32_t A[GPW][NT][4][4];
#pragma unroll
    for (int j = 0; j < GPW; ++j) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int g = sa.g0 + min(g0 + j, NG - 1);
            const uint16_t* p = a.x + (size_t)min(t0 + 16 * t + m, a.T - 1) * a.ldx + (size_t)g * 128;
            uint32_t xw[16];
#pragma unroll
            for (int st = 0; st < 4; ++st) {
                if constexpr (SPG > 1 && BITS == 2) {          // elements e .. e+3 and e+8 .. e+11
                    const uint16_t* pe = p + 32 * st + 16 * (q >> 1) + 4 * (q & 1);
                    const uint2 lo = *reinterpret_cast<const uint2*>(pe), hi = *reinterpret_cast<const uint2*>(pe + 8);
                    xw[4 * st] = lo.x; xw[4 * st + 1] = lo.y; xw[4 * st + 2] = hi.x; xw[4 * st + 3] = hi.y;
                } else {
                    const uint4 v = *reinterpret_cast<const uint4*>(p + (SPG > 1 ? 32 * st + 8 * q : 32 * q + 8 * st));
                    xw[4 * st] = v.x; xw[4 * st + 1] = v.y; xw[4 * st + 2] = v.z; xw[4 * st + 3] = v.w;
                }
            }
            if (g0 + j >= NG)
#pragma unroll
                for (int i = 0; i < 16; ++i) xw[i] = 0u;
            floatx4_t X;
#pragma unroll
            for (int st = 0; st < 4; ++st) {
                if constexpr (SPG == 1) act_operand<BITS>(xw, st, A[j][t][st]);
                else act_operand<4>(xw, st, A[j][t][st]);      // the tr order's eight elements, paired (i, i + 4)
                X = mfma16(A[j][t][st], ones, st % STEPS == 0 ? zero : X);
                if (st % STEPS == STEPS - 1 && m == 0)         // every column holds the sums: one lane a quarter stores
                    *reinterpret_cast<floatx4_t*>(xs + ((j * NT + t) * SPG + st / STEPS) * 16 + 4 * q) = X;
            }
        }
    }
#pragma unroll
    for (int p = 0; p < PP; ++p) {
        if (mine[p]) *reinterpret_cast<uint4*>(to[p]) = sreg[p];
        sreg[p] = load_scales(p, (int)blockIdx.x + stride);
    }
    for (int p = 0; p < 2; ++p)
        for (int o = tid; o < (rows4 - waves) * tokens * RB; o += blockDim.x) red[(size_t)(p * rows4 + waves) * tokens * RB + o] = 0.f;
    lds_barrier();

    int parity = 0, turn = 0;
    for (int tile0 = blockIdx.x; tile0 < tiles; tile0 += RBU * stride) {
#pragma unroll
        for (int i = 0; i < RBU; ++i) {
            const int tile = tile0 + i * stride;
            if (tile >= tiles) break;
            // the thread's output of this tile (waves take turns), its row bias and residual
            // requested ahead of the next units
            int o = tid - 64 * turn;
            o += o < 0 ? (int)blockDim.x : 0;
            const int on = min(tile * RB + o % RB, a.w.N - 1);
            const size_t ot = (size_t)(t0 + min(o / RB, tokens - 1));
            // (without one: any valid address, the value unused, so that no branch waits on the load)
            const float rb = *(a.row_bias ? a.row_bias + on : reinterpret_cast<const float*>(a.x));
            const uint16_t res = *(a.residual ? a.residual + ot * a.ldr + on : a.x);
            const float add = *(sa.add ? sa.add + ot * a.w.N + on : reinterpret_cast<const float*>(a.x));
            floatx4_t acc[NT][RT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[t][r] = zero;
            const uint16_t* slot = slots + parity * 2 * RB * pitch;
#pragma unroll
            for (int j = 0; j < GPW; ++j) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint16_t* ps = slot + (16 * r + m) * pitch + min(g0 + j, NG - 1) * SPG;
                    uint32_t sw[SW], bw[SW];
                    load_scales_of<SPG>(ps, sw);
                    load_scales_of<SPG>(ps + RB * pitch, bw);
                    uint32_t tr[4];
                    if constexpr (SPG > 1) quarter_transpose<BITS>(code[i][j][r], tr);
#pragma unroll
                    for (int u = 0; u < SPG; ++u) {
                        floatx4_t C[NT];
#pragma unroll
                        for (int k = 0; k < STEPS; ++k) {
                            const int st = u * STEPS + k;
                            uint32_t B[4];
                            if constexpr (SPG == 1) code_operand<BITS>(code[i][j][r], st, B);
                            else code_operand_tr<BITS>(tr, st, q, B);
#pragma unroll
                            for (int t = 0; t < NT; ++t) C[t] = mfma16(A[j][t][st], B, k == 0 ? zero : C[t]);
                        }
                        const float s = f16_bits_to_f32((sw[u >> 1] >> (16 * (u & 1))) & 0xFFFFu);
                        const float b = f16_bits_to_f32((bw[u >> 1] >> (16 * (u & 1))) & 0xFFFFu);
                        const float sl = s * kInvLever<BITS>, be = fmaf(-kOffset<BITS>, s, b);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const floatx4_t X = *reinterpret_cast<const floatx4_t*>(xs + ((j * NT + t) * SPG + u) * 16 + 4 * q);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[t][r][e] = fmaf(sl, C[t][e], fmaf(be, X[e], acc[t][r][e]));
                        }
                    }
                }
                // the sums are taken here: left to the conditional stores below, every unit's matrix-core
                // results would stay in registers until then
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < RT; ++r) asm volatile("" : "+v"(acc[t][r]));
                load(i, j, tile + RBU * stride);
            }
            // the waves' sums, [token][row] each, and the next tile's scales; one barrier per tile
            float* sums = red + (size_t)(parity * rows4 + wid) * tokens * RB;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int tt = 16 * t + 4 * q + e;
                    if (tt < tokens)
#pragma unroll
                        for (int r = 0; r < RT; ++r) sums[tt * RB + 16 * r + m] = acc[t][r][e];
                }
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                if (mine[p]) *reinterpret_cast<uint4*>(to[p] + (parity ^ 1) * 2 * RB * pitch) = sreg[p];
                sreg[p] = load_scales(p, tile + 2 * stride);
            }
            lds_barrier();
            const float* all = red + (size_t)parity * rows4 * tokens * RB;
            bool first = true;
            for (; o < tokens * RB; o += blockDim.x) {
                float v = 0.f;
                for (int k = 0; k < rows4; k += 4) {
                    const float* p = all + k * tokens * RB + o;
                    v += (p[0] + p[tokens * RB]) + (p[2 * tokens * RB] + p[3 * tokens * RB]);
                }
                const int n = tile * RB + o % RB;
                const size_t t = (size_t)(t0 + o / RB);
                if (n < a.w.N) {
                    if (first) {
                        v += sa.add ? add : 0.f;
                        v += a.row_bias ? rb : 0.f;
                        v += a.residual ? bf16_bits_to_f32(res) : 0.f;
                    } else {
                        if (sa.add) v += sa.add[t * a.w.N + n];
                        if (a.row_bias) v += a.row_bias[n];
                        if (a.residual) v += bf16_bits_to_f32(a.residual[t * a.ldr + n]);
                    }
                    if (a.y_type == MOE_F32) static_cast<float*>(a.y)[t * a.ldy + n] = v;
                    else static_cast<uint16_t*>(a.y)[t * a.ldy + n] = (uint16_t)(pack_bf16(v, 0.f) & 0xFFFFu);
                }
                first = false;
            }
            parity ^= 1;
            turn = turn + 2 < waves ? turn + 2 : 0;
        }
    }
}

// Two token tiles where their operands fit the registers (K <= 4096) and every CU has
// more than two weight tiles to share its start among; with one and with two, us: 32 tokens, K =
// 4096: 4096 outputs 9.8, 12.2; 8192 13.0, 15.4; 16384 18.8, 19.4; 49999 45.3, 38.6; K = 2048: 6.3,
// 7.4; 8.9, 9.1; 13.4, 12.9; 26.7, 25.3; 64 tokens, 28672 x 4096 46.5, 37.2.
// A second ring entry per slot where a slot is one group and a workgroup has a second tile to
// request ahead: without and with, 8 tokens, 400000 x 1024 69.0, 64.0; 49999 x 1024 11.9, 12.0; 28672 x
// 1024 9.5, 9.2; 2 bits 8.1, 8.5.
// Tiles of 32 weight rows (units of 1 KB) for 2-bit codes of groups of 128 where they
// still give every CU one; with 16 rows and with 32, 8 tokens, K = 4096: 4096 outputs 6.1, 7.0; 8192
// 7.6, 7.4; 49999 22.8, 20.9; K = 1024: 4096 3.8, 4.0; 8192 4.7, 4.1; 28672 9.3, 7.3.  (4-bit codes
// and finer groups gained nothing when they were built, and are not.)
// Two workgroups a CU, one multiplying while the other's waves meet, where each still has
// four tiles of 16 rows; with one and with two, 8 tokens, 4 bits: 49999 x 1024 15.4, 11.8; 49999 x
// 2048 17.7, 15.5; 16384 x 1024 6.6, 6.3; with fewer tiles 8192 x 2048 5.6, 6.4; 16384 x 512 5.7, 6.4.
StreamForm stream_form(const moe_qmatrix& w, int T, int runs) {
    const int cus = device_cus(), spg = 128 / w.group_size;
    StreamForm f{};
    f.rt = w.bits == 2 && spg == 1 && (w.N + 31) / 32 >= cus ? 2 : 1;
    const int tiles = (w.N + 16 * f.rt - 1) / (16 * f.rt);
    f.nt = T > 16 && runs <= 32 && (long)tiles * ((T + 31) / 32) > 2 * cus ? 2 : 1;
    f.gpw = runs <= 8 ? 1 : runs <= 16 ? 2 : runs <= 32 ? 4 : runs <= 48 ? 6 : 8;
    // waves for the groups, and threads for the pieces of a tile's scales (pp each)
    const int pp = (f.rt * f.gpw * spg + 15) / 16, pieces = 2 * 16 * f.rt * ((runs * spg + 7) / 8);
    f.waves = std::max((runs + f.gpw - 1) / f.gpw, (pieces + 64 * pp - 1) / (64 * pp));
    const int blocks = (T + 16 * f.nt - 1) / (16 * f.nt);      // of tokens
    const bool two = two_fit(f.nt, f.gpw) && (long)tiles * f.rt * blocks >= 8L * cus;
    const int all = cus * ((two ? 2 : 1) * kStreamMaxWaves / f.waves);
    f.resident = all > blocks ? all / blocks : 1;
    f.rbu = f.gpw == 1 && tiles > f.resident ? 2 : 1;
    return f;
}

// A CU's units (16 weight rows, a token tile) by the form that takes them, and the starts.
double linear_dec_us(const moe_qmatrix& w, int T) {
    static const double start[3] = {6.2, 6.2, 5.9}, run[3] = {0.112, 0.147, 0.148};          // groups of 128, 64, 32
    static const double wave[3] = {0.096, 0.105, 0.115};                                     // one run a wave, one token tile
    static const double two[2][3] = {{0.48, 0.48, 0.58}, {0.82, 0.98, 1.12}};                // two, up to four waves and more
    static const double unit[2][4][3] = {{{0.89, 1.03, 0.95}, {1.55, 2.3, 2.3}, {2.19, 2.64, 3.0}, {2.78, 3.4, 3.7}},
                                         {{1.55, 1.75, 2.1}, {2.36, 2.7, 3.4}, {}, {}}};     // 2, 4, 6, 8 runs a wave
    const int fine = w.group_size == 128 ? 0 : w.group_size == 64 ? 1 : 2;
    double us = 0.;
    for (int g0 = 0, all = w.K / 128; g0 < all; g0 += kStreamGroups) {
        const int runs = std::min(all - g0, kStreamGroups);
        const StreamForm f = stream_form(w, T, runs);
        const double units = (double)((w.N + 15) / 16) * ((T + 16 * f.nt - 1) / (16 * f.nt)) / device_cus();
        us += start[fine] + (f.nt == 2 && f.gpw == 1 ? 1.8 : 0.) + run[fine] * runs;
        if (f.gpw == 1) us += units * (f.nt == 1 ? wave[fine] * runs : two[runs > 4][fine]);
        else us += units * unit[f.nt - 1][f.gpw / 2 - 1][fine];
    }
    return us;
}

namespace {

template <int BITS, int SPG, int NT, int RT, int GPW, int RBU>
void stream_go(const StreamArgs& sa, const StreamForm& f, hipStream_t s) {
    const LinearArgs& a = sa.l;
    const int tiles = (a.w.N + 16 * RT - 1) / (16 * RT), blocks = (a.T + 16 * NT - 1) / (16 * NT);
    const int tokens = a.T < 16 * NT ? a.T : 16 * NT;
    const dim3 grid((unsigned)(tiles < f.resident ? tiles : f.resident), (unsigned)blocks);
    const size_t lds = (size_t)8 * 16 * RT * scale_pitch(sa.ng * SPG) +
                       (size_t)(f.waves * GPW * NT * SPG * 16 + 2 * ((f.waves + 3) & ~3) * tokens * 16 * RT) * sizeof(float);
    hipLaunchKernelGGL((linear_stream_kernel<BITS, SPG, NT, RT, GPW, RBU>), grid, dim3(64 * f.waves), lds, s, sa);
}

template <int BITS, int SPG, int RT>
void stream_rows(const StreamArgs& sa, const StreamForm& f, hipStream_t s) {
    if (f.nt == 2) {
        if (f.gpw == 1 && f.rbu == 2) stream_go<BITS, SPG, 2, RT, 1, 2>(sa, f, s);
        else if (f.gpw == 1) stream_go<BITS, SPG, 2, RT, 1, 1>(sa, f, s);
        else if (f.gpw == 2) stream_go<BITS, SPG, 2, RT, 2, 1>(sa, f, s);
        else stream_go<BITS, SPG, 2, RT, 4, 1>(sa, f, s);
    } else if (f.gpw == 1) {
        if (f.rbu == 2) stream_go<BITS, SPG, 1, RT, 1, 2>(sa, f, s);
        else stream_go<BITS, SPG, 1, RT, 1, 1>(sa, f, s);
    } else if (f.gpw == 2) {
        stream_go<BITS, SPG, 1, RT, 2, 1>(sa, f, s);
    } else if (f.gpw == 4) {
        stream_go<BITS, SPG, 1, RT, 4, 1>(sa, f, s);
    } else if (f.gpw == 6) {
        stream_go<BITS, SPG, 1, RT, 6, 1>(sa, f, s);
    } else {
        stream_go<BITS, SPG, 1, RT, 8, 1>(sa, f, s);
    }
}

template <int BITS, int SPG>
void stream_launch(const StreamArgs& sa, hipStream_t s) {
    const StreamForm f = stream_form(sa.l.w, sa.l.T, sa.ng);
    if constexpr (BITS == 2 && SPG == 1) {
        if (f.rt == 2) return stream_rows<BITS, SPG, 2>(sa, f, s);
    }
    stream_rows<BITS, SPG, 1>(sa, f, s);
}

}  // namespace

// Tokens at once: all, or where K takes several launches as many as have 1 GB of sums (a tile
// of tokens reads the whole matrix either way).
static int tokens_at_once(const moe_qmatrix& w, int T) {
    if (w.K / 128 <= kStreamGroups) return T;
    const long most = ((1L << 30) / (4L * w.N)) / 32 * 32;         // (N is at most 2^20)
    return T < most ? T : (int)most;
}

size_t linear_dec_workspace_bytes(const moe_qmatrix& w, int T) {
    return w.K / 128 > kStreamGroups ? (size_t)tokens_at_once(w, T) * w.N * sizeof(float) : 0;
}

void linear_dec_kernels(const moe_qmatrix& w, int T, int32_t* kernels) {
    const int runs = w.K / 128;
    const StreamForm f = stream_form(w, tokens_at_once(w, T), std::min(runs, kStreamGroups));
    kernels[1] = f.nt;
    kernels[2] = f.rt;
    kernels[3] = f.gpw;
    kernels[4] = f.rbu;
    kernels[5] = (runs + kStreamGroups - 1) / kStreamGroups;
}

// K beyond what a workgroup's registers hold is taken in several launches, each
// adding to the sums that the last one left in the workspace.
static void launch_turn(const LinearArgs& a, hipStream_t s) {
    const int NG = a.w.K / 128, spg = 128 / a.w.group_size;
    for (int g0 = 0; g0 < NG; g0 += kStreamGroups) {
        StreamArgs sa{a, g0, NG - g0 < kStreamGroups ? NG - g0 : kStreamGroups, nullptr};
        if (g0 > 0) sa.add = static_cast<const float*>(a.ws);
        if (g0 + sa.ng < NG) {
            sa.l.y = a.ws;
            sa.l.ldy = a.w.N;
            sa.l.y_type = MOE_F32;
            sa.l.row_bias = nullptr;
            sa.l.residual = nullptr;
        }
        if (a.w.bits == 4) {
            if (spg == 1) stream_launch<4, 1>(sa, s);
            else if (spg == 2) stream_launch<4, 2>(sa, s);
            else stream_launch<4, 4>(sa, s);
        } else {
            if (spg == 1) stream_launch<2, 1>(sa, s);
            else if (spg == 2) stream_launch<2, 2>(sa, s);
            else stream_launch<2, 4>(sa, s);
        }
    }
}

int launch_linear_dec(const LinearArgs& a, hipStream_t s) {
    const int at_once = tokens_at_once(a.w, a.T);
    const size_t e = a.y_type == MOE_F32 ? 4 : 2;
    for (int t0 = 0; t0 < a.T; t0 += at_once) {
        LinearArgs b = a;
        b.T = std::min(at_once, a.T - t0);
        b.x = a.x + (int64_t)t0 * a.ldx;
        b.residual = a.residual ? a.residual + (int64_t)t0 * a.ldr : nullptr;
        b.y = static_cast<uint8_t*>(a.y) + (int64_t)t0 * a.ldy * e;
        launch_turn(b, s);
    }
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
