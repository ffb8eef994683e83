// Gradients of a matrix that tokens share: for set i of tokens (an adapter's, or all of them)
//   d[i][r][c] = s_i sum_{t in i} g[t][r] x[t][c]      (float32)
// with g float32 and x bf16, float32, or a checkpoint's int8 codes with one scale for 128 columns.
// The adapters' factors (r a rank, x the layer's input or dy) and the router's weight (r an
// expert, x the router's input) are of this form.
//
// The sum runs over tokens, across the rows of both operands.  A wave has 128 columns: a lane
// takes 8 columns of 8 tokens and turns the block by v_perm_b32; column j of every lane's 8 is
// one v_mfma_f32_16x16x32_bf16 over 32 tokens and 16 r, so that a lane ends with 8 neighbouring
// columns of 4 r.  g goes as three bf16 parts (all 24 bits); bf16 x and codes are exact, a
// code's scale goes into g (128 columns have one); a float32 x goes as three parts too, of whose
// nine products the six largest are taken (2^-24 of the product left out).
//
// A workgroup's waves share its tokens and meet in LDS (many tokens), or have 128 columns each
// (few).  Where columns and r give too few workgroups, tokens are split in chunks, whose sums a
// second kernel adds in order.  No atomics: equal calls give equal bits.
//
// What it costs: both factors of 4 adapters, 4096 tokens, 2048 (codes) and 8192 (bf16) columns at rank 16
// 18.6 us, 4.1 TB/s of x and dy, and 4.7 for the join; the router's weight, 8192 tokens x 128 x 2048 from codes,
// 21.7 us and 6.  There the vector ALUs are the bound, 300 instructions a step to prepare the operands of 48 products,
// at 1.65 us a step and SIMD (bf16 x: 1.4), beside 8 us for the launch, the first loads and the sums' way out.
// 64 r a wave would halve the turning of x for twice the accumulators (20.5 us and 6.1; no gain), loads two
// steps ahead changed nothing.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "adapters.h"
#include "token_tiles.h"

namespace moe {

namespace {

constexpr int kGradWaves = 8;
constexpr int kStep = 32;                 // tokens a product
enum ListKind { kAll = 0, kScan = 1, kPlan = 2 };
// Waves a SIMD that the registers are held to: four with 16 r (128 VGPRs, two workgroups of eight waves a CU, which
// hide each other's loads), three with 32 (168, three workgroups of four), two with float32 x (up to 202).
template <int RTW, int WT, bool F32> constexpr int kGradResident = F32 ? 2 : RTW > 1 ? 3 : WT > 1 ? 4 : 3;

struct GradArgs {
    TokenSets who;
    TokenPlan plan;
    const float* scale;       // [n] or NULL
    WeightGradCall w[2];      // a launch has one or two matrices
    int groups0;              // workgroups (first grid axis) of the first
    int chunk;                // kAll: tokens an entry
    float* part[2];           // [slots][R C (+ R)]
    int64_t slot_floats[2];
};

template <int XT>
struct XFrag {
    uint4 v[XT == MOE_F32 ? 16 : XT == kCodes ? 4 : 8];
    float s;                  // codes: the scale of token lane % 32
};

// A set's tokens in LDS, padded with the last to whole steps: numbers, and bytes to their rows of x.
template <int LIST>
struct Listed {
    static constexpr int N = LIST == kAll ? 8 : LIST == kScan ? kScanTokens : kMostChunk;
    __attribute__((aligned(16))) int token[N];
    __attribute__((aligned(16))) int64_t row[N];
};

// One workgroup's block of 128 columns, XT the kind of x.
template <int XT, int RTW, int LIST, int WT>
__device__ __forceinline__ void weight_grad_block(const GradArgs& a, const WeightGradCall& w, int block, float* part, int64_t slot_floats,
                                                  int set, int first, int cnt, int slot, const Listed<LIST>& list,
                                                  float (*sums)[16][132]) {
    constexpr int ES = XT == MOE_F32 ? 4 : XT == kCodes ? 1 : 2;
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int R = a.who.R, C = w.C;
    const int rank = a.who.rank ? min(max(ld_scalar(a.who.rank, set), 0), R) : R;
    const int r0 = 16 * RTW * (int)blockIdx.y;
    const int own = 128 * block + 8 * c, col = first_of_8(own, C), shift = own - col;    // 8 or more: none are this lane's

    floatx4_t acc[RTW][8];
    float bsum[RTW];
#pragma unroll
    for (int rt = 0; rt < RTW; ++rt) {
        bsum[rt] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[rt][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    }
    const bool biased = LIST == kAll && w.bias != nullptr && block == 0;
    // product rt has the r's r_at(row) + rt: a lane's g of all RTW products are neighbours
    auto r_at = [&](int row) { return min(r0 + RTW * row, R - RTW); };
    const uint32_t gcol = r_at(c);
    const char* x = static_cast<const char*>(w.x);
    const int64_t xlane = ((int64_t)(8 * q) * w.ldx + col) * ES;            // (kAll: rows are a constant stride apart)
    const uint32_t ldg = (uint32_t)w.ldg, glane = 4 * (8 * q * ldg + gcol), ngs = (uint32_t)C / 128;
    // 32 tokens; with TAIL (kAll) some of them past the end: the last again, their g 0
    auto load_x = [&](XFrag<XT>& f, int step, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        const int k0 = kStep * step;
        const char* row[8];
        if constexpr (LIST == kAll) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (TAIL) row[i] = x + ((int64_t)(first + min(k0 + 8 * q + i, cnt - 1)) * w.ldx + col) * ES;
                else row[i] = x + (int64_t)(first + k0 + i) * w.ldx * ES + xlane;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) row[i] = x + list.row[k0 + 8 * q + i] + (int64_t)col * ES;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (XT == MOE_BF16) {
                __builtin_memcpy(&f.v[i], row[i], 16);
            } else if constexpr (XT == MOE_F32) {
                __builtin_memcpy(&f.v[2 * i], row[i], 32);
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(row[i]);
                (i & 1) ? (f.v[i >> 1].z = v.x, f.v[i >> 1].w = v.y) : (f.v[i >> 1].x = v.x, f.v[i >> 1].y = v.y);
            }
        }
        if constexpr (XT == kCodes) {
            uint32_t t;
            if constexpr (LIST == kAll) t = first + (TAIL ? min(k0 + (lane & 31), cnt - 1) : k0 + (lane & 31));
            else t = list.token[k0 + (lane & 31)];
            f.s = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(w.xscale) + (uint64_t)(4 * (__umul24(t, ngs) + block)));
        }
    };
    auto load_g = [&](float (&g)[RTW][8], int step, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        const int k0 = kStep * step;
        if constexpr (LIST == kAll && !TAIL) {
            const float* row = w.g + (int64_t)(first + k0) * w.ldg;            // (rows by scalars)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float gv[RTW];
                __builtin_memcpy(gv, reinterpret_cast<const char*>(row + (int64_t)i * w.ldg) + glane, 4 * RTW);
#pragma unroll
                for (int rt = 0; rt < RTW; ++rt) g[rt][i] = gv[rt];
            }
            return;
        }
        uint32_t tok[8];
        if constexpr (LIST == kAll) {
#pragma unroll
            for (int i = 0; i < 8; ++i) tok[i] = first + min(k0 + 8 * q + i, cnt - 1);
        } else {
            *reinterpret_cast<uint4*>(tok) = *reinterpret_cast<const uint4*>(&list.token[k0 + 8 * q]);
            *reinterpret_cast<uint4*>(tok + 4) = *reinterpret_cast<const uint4*>(&list.token[k0 + 8 * q + 4]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float gv[RTW];
            __builtin_memcpy(gv, reinterpret_cast<const char*>(w.g) + (uint64_t)(4 * (__umul24(tok[i], ldg) + gcol)), 4 * RTW);
#pragma unroll
            for (int rt = 0; rt < RTW; ++rt) g[rt][i] = gv[rt];
        }
    };
    // g's operands: times the codes' scales, 0 past the end, as three bf16 parts
    auto prepare_g = [&](const XFrag<XT>& f, float (&g)[RTW][8], uint32_t (&gp)[RTW][3][4], int step, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        float xs[8];
        if constexpr (XT == kCodes)
#pragma unroll
            for (int i = 0; i < 8; ++i) xs[i] = __shfl(f.s, 8 * q + i, kWave);
#pragma unroll
        for (int rt = 0; rt < RTW; ++rt) {
            if constexpr (LIST != kAll || TAIL)
#pragma unroll
                for (int i = 0; i < 8; ++i) g[rt][i] = kStep * step + 8 * q + i < cnt ? g[rt][i] : 0.f;
            if (biased)
#pragma unroll
                for (int i = 0; i < 8; ++i) bsum[rt] += g[rt][i];
            if constexpr (XT == kCodes)
#pragma unroll
                for (int i = 0; i < 8; ++i) g[rt][i] *= xs[i];
            bf16_parts(g[rt], gp[rt]);
        }
    };
    // columns 4 half .. 4 half + 3 of the block, turned
    auto prepare_x = [&](const XFrag<XT>& f, int half, uint32_t (&b)[4][4]) {
        if constexpr (XT == kCodes) {
            // byte j of tokens 2 p and 2 p + 1: small integers, whose float32 has its bits in the upper half
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t lo4 = half ? f.v[p].y : f.v[p].x, hi4 = half ? f.v[p].w : f.v[p].z;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float lo = (float)(int8_t)(lo4 >> (8 * j)), hi = (float)(int8_t)(hi4 >> (8 * j));
                    b[j][p] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
                }
            }
        } else if constexpr (XT == MOE_BF16) {
            turn4(f.v, half, b);
        }
    };
    auto multiply = [&](const uint32_t (&gp)[RTW][3][4], int half, const uint32_t (&b)[4][4], int parts) {
#pragma unroll
        for (int rt = 0; rt < RTW; ++rt)
#pragma unroll
            for (int p = 0; p < 3; ++p)
                if (p < parts)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[rt][4 * half + j] = mfma16(gp[rt][p], b[j], acc[rt][4 * half + j]);
    };
    // float32 x: its upper 8 bits with all of g's parts, the next 8 with two, the rest with one
    auto multiply_f32 = [&](const XFrag<XT>& f, const uint32_t (&gp)[RTW][3][4]) {
        float v[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) __builtin_memcpy(v[i], &f.v[(2 * i) % (sizeof(f.v) / 16)], 32);
#pragma unroll
        for (int px = 0; px < 3; ++px) {
            uint4 rowv[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t o[4];
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    o[d] = __builtin_amdgcn_perm(__float_as_uint(v[i][2 * d + 1]), __float_as_uint(v[i][2 * d]), 0x07060302u);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] -= __uint_as_float(__float_as_uint(v[i][j]) & 0xFFFF0000u);
                rowv[i] = make_uint4(o[0], o[1], o[2], o[3]);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t b[4][4];
                turn4(rowv, half, b);
                multiply(gp, half, b, 3 - px);
            }
        }
    };
    if (r0 < rank) {
        const int steps = LIST == kAll ? cnt / kStep : (cnt + kStep - 1) / kStep, w0 = WT == 1 ? 0 : wid;
        const std::false_type full{};
        XFrag<XT> f;
        float g[RTW][8];
        uint32_t gp[RTW][3][4], b[4][4];
        if (w0 < steps) {
            load_g(g, w0, full);
            load_x(f, w0, full);
        }
        for (int k = w0; k < steps; k += WT) {
            // the next step's loads go out as their registers come free, before the products (always: the last
            // step's again at the end)
            const int next = min(k + WT, steps - 1);
            prepare_g(f, g, gp, k, full);
            load_g(g, next, full);
            if constexpr (XT == MOE_F32) {
                multiply_f32(f, gp);
                load_x(f, next, full);
            } else {
                __builtin_amdgcn_sched_barrier(0);
                prepare_x(f, 0, b);
                multiply(gp, 0, b, 3);
                __builtin_amdgcn_sched_barrier(0);
                prepare_x(f, 1, b);
                load_x(f, next, full);
                __builtin_amdgcn_sched_barrier(0);
                multiply(gp, 1, b, 3);
            }
        }
        if (LIST == kAll && cnt % kStep && wid == steps % WT) {
            const std::true_type tail{};
            load_g(g, steps, tail);
            load_x(f, steps, tail);
            prepare_g(f, g, gp, steps, tail);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                prepare_x(f, half, b);
                if constexpr (XT != MOE_F32) multiply(gp, half, b, 3);
            }
        }
    }
    const float s = slot < 0 && a.scale && cnt > 0 ? ld_scalar(a.scale, set) : 1.f;      // (a set without a token: 0, whatever its scale)
    float* out = slot < 0 ? w.out + (int64_t)set * R * C : part + (int64_t)slot * slot_floats;
    float* bias = slot < 0 ? w.bias : part + (int64_t)slot * slot_floats + (int64_t)R * C;
    // By way of LDS, so that a store has whole rows of 512 bytes (from the products' layout, 8 columns a
    // lane, every other 16 bytes: 256 adapters 4096 x 4096 50.8 us, most of them zeros); with one
    // token wave each has a part of its own and no barrier.
    {
        constexpr bool ONE = WT == 1;
        auto meet = [&] {
            if constexpr (ONE) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
            else __syncthreads();
        };
        const int at = ONE ? lane : tid, c4 = 4 * (at & 31), wide = min(C - 128 * block - c4, 4);
#pragma unroll
        for (int rt = 0; rt < RTW; ++rt) {
            if (rt) meet();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float* to = &sums[wid][4 * q + i][8 * c];
                if (shift == 0) {
                    *reinterpret_cast<floatx4_t*>(to) = floatx4_t{acc[rt][0][i], acc[rt][1][i], acc[rt][2][i], acc[rt][3][i]};
                    *reinterpret_cast<floatx4_t*>(to + 4) = floatx4_t{acc[rt][4][i], acc[rt][5][i], acc[rt][6][i], acc[rt][7][i]};
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j >= shift) to[j - shift] = acc[rt][j][i];
                }
            }
            meet();
#pragma unroll
            for (int row = at >> 5; row < 16; row += 2 * WT) {
                const int r = r_at(row) + rt;
                if (r < r0 + RTW * row || wide <= 0) continue;             // (another row's)
                floatx4_t v = *reinterpret_cast<const floatx4_t*>(&sums[ONE ? wid : 0][row][c4]);
#pragma unroll
                for (int k = 1; k < WT; ++k) v += *reinterpret_cast<const floatx4_t*>(&sums[k][row][c4]);
                v = r < rank ? v * s : floatx4_t{0.f, 0.f, 0.f, 0.f};
                float* to = out + (int64_t)r * C + 128 * block + c4;
                if (wide >= 4) __builtin_memcpy(to, &v, 16);
                else
                    for (int j = 0; j < wide; ++j) to[j] = v[j];
            }
        }
        if constexpr (LIST == kAll) {
            if (!biased) return;
            __syncthreads();
#pragma unroll
            for (int rt = 0; rt < RTW; ++rt) {
                float v = bsum[rt];
                v += __shfl_xor(v, 16, kWave);
                v += __shfl_xor(v, 32, kWave);
                if (q == 0) sums[wid][rt][c] = v;
            }
            __syncthreads();
            if (tid < 16 * RTW) {
                const int r = r_at(tid & 15) + (tid >> 4);
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < WT; ++k) v += sums[k][tid >> 4][tid & 15];
                if (r >= r0 + RTW * (tid & 15)) bias[r] = v;
            }
        }
    }
}

}  // namespace

// F32: the second matrix' x may be float32.
// WT == 1: kFewWaves waves, each with all of the set's tokens and 128 columns.
constexpr int kFewWaves = 4;
template <int RTW, int LIST, int WT, bool F32>
__global__ __launch_bounds__(64 * (WT > 1 ? WT : kFewWaves), (kGradResident<RTW, WT, F32>)) void weight_grad_kernel(GradArgs a) {
    constexpr int THREADS = 64 * (WT > 1 ? WT : kFewWaves);
    __shared__ Listed<LIST> list;
    __shared__ int found;
    __shared__ __attribute__((aligned(16))) float sums[THREADS / 64][16][132];
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool second = (int)blockIdx.x >= a.groups0;
    const WeightGradCall& w = a.w[second];
    int set = 0, first = 0, cnt, slot = -1;
    if constexpr (LIST == kAll) {
        first = (int)blockIdx.z * a.chunk;
        cnt = min(a.chunk, a.who.T - first);
        slot = gridDim.z > 1 ? (int)blockIdx.z : -1;
    } else {
        const int64_t bytes = w.ldx * (w.x_type == MOE_F32 ? 4 : w.x_type == kCodes ? 1 : 2);
        if constexpr (LIST == kScan) {
            set = blockIdx.z;
            if (wid == 0) {
                int id[kScanTokens / 64], n = 0;
#pragma unroll
                for (int k = 0; k < kScanTokens / 64; ++k) {
                    if (k * 64 >= a.who.T) break;
                    id[k] = a.who.ids[min(k * 64 + lane, a.who.T - 1)];
                }
#pragma unroll
                for (int k = 0; k < kScanTokens / 64; ++k) {
                    if (k * 64 >= a.who.T) break;
                    const int t = k * 64 + lane;
                    const bool mine = t < a.who.T && id[k] == set;
                    const uint64_t mask = __ballot(mine);
                    if (mine) {
                        const int at = n + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
                        list.token[at] = t;
                        list.row[at] = t * bytes;
                    }
                    n += __popcll(mask);
                }
                if (lane == 0) found = n;
            }
            __syncthreads();
            cnt = __builtin_amdgcn_readfirstlane(found);
        } else {
            const int4 e = a.plan.chunks[blockIdx.z];
            set = __builtin_amdgcn_readfirstlane(e.x);
            if (set < 0) return;
            cnt = __builtin_amdgcn_readfirstlane(e.z);
            slot = __builtin_amdgcn_readfirstlane(e.w);
            for (int k = tid; k < cnt; k += THREADS) {
                const int t = a.plan.order[e.y + k];
                list.token[k] = t;
                list.row[k] = t * bytes;
            }
            __syncthreads();
        }
        // (cnt up to a multiple of 32: the lists hold whole steps)
        if (tid < kStep && cnt > 0 && cnt % kStep && tid >= cnt % kStep) {
            list.token[cnt - cnt % kStep + tid] = list.token[cnt - 1];
            list.row[cnt - cnt % kStep + tid] = list.row[cnt - 1];
        }
        __syncthreads();
    }
    int block = (int)blockIdx.x - (second ? a.groups0 : 0);
    if constexpr (WT == 1) {
        block = block * kFewWaves + wid;
        if (128 * block >= w.C) return;
    }
    float* part = a.part[second];
    const int64_t floats = a.slot_floats[second];
    if (w.x_type == kCodes) weight_grad_block<kCodes, RTW, LIST, WT>(a, w, block, part, floats, set, first, cnt, slot, list, sums);
    else if (!F32 || w.x_type == MOE_BF16) weight_grad_block<MOE_BF16, RTW, LIST, WT>(a, w, block, part, floats, set, first, cnt, slot, list, sums);
    else weight_grad_block<F32 ? MOE_F32 : MOE_BF16, RTW, LIST, WT>(a, w, block, part, floats, set, first, cnt, slot, list, sums);
}

// The chunks' sums of a set that has several, in order.  joins NULL: one set of `number` chunks.
__global__ __launch_bounds__(256) void weight_grad_join_kernel(GradArgs a, int number) {
    const int set = blockIdx.y;
    int2 j = make_int2(0, number);
    if (a.plan.joins) j = a.plan.joins[set];
    if (j.y == 0) return;
    const bool second = (int)blockIdx.x >= a.groups0;
    const WeightGradCall& w = a.w[second];
    const int64_t size = (int64_t)a.who.R * w.C, all = a.slot_floats[second];
    const int64_t e = 4 * ((int64_t)(blockIdx.x - (second ? a.groups0 : 0)) * 256 + threadIdx.x);
    if (e >= all) return;
    const float* p = a.part[second] + (int64_t)j.x * all + e;
    const float s = a.scale ? a.scale[set] : 1.f;
    float* out = w.out + (int64_t)set * size + e;
    if (e + 4 <= size) {
        floatx4_t v{0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < j.y; k += 4) {
            floatx4_t o[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) __builtin_memcpy(&o[u], p + min(k + u, j.y - 1) * all, 16);
#pragma unroll
            for (int u = 0; u < 4; ++u) v += k + u < j.y ? o[u] : floatx4_t{0.f, 0.f, 0.f, 0.f};
        }
        v *= s;
        __builtin_memcpy(out, &v, 16);
        return;
    }
    for (int i = 0; i < 4 && e + i < all; ++i) {
        float v = 0.f;
        for (int k = 0; k < j.y; ++k) v += p[k * all + i];
        if (e + i < size) out[i] = v * s;
        else w.bias[e + i - size] = v;
    }
}

namespace {

// Products of 16 r a wave.  (Rows past R take the last r's again and store nothing: of R = 33 the second group has one.)
int products_of(int R) { return R <= 16 ? 1 : 2; }
int groups_of(int R) { return (R + 16 * products_of(R) - 1) / (16 * products_of(R)); }

template <int RTW, bool F32>
void grad_go(const GradArgs& a, int kind, int blocks, unsigned entries, bool few, hipStream_t s) {
    constexpr int WT = RTW == 2 ? 4 : kGradWaves;
    const dim3 grid((unsigned)blocks, (unsigned)((a.who.R + 16 * RTW - 1) / (16 * RTW)), entries), many(64 * WT), one(64 * kFewWaves);
    if (kind == kAll) hipLaunchKernelGGL((weight_grad_kernel<RTW, kAll, WT, false>), grid, many, 0, s, a);
    else if (kind == kScan && few) hipLaunchKernelGGL((weight_grad_kernel<RTW, kScan, 1, F32>), grid, one, 0, s, a);
    else if (kind == kScan) hipLaunchKernelGGL((weight_grad_kernel<RTW, kScan, WT, F32>), grid, many, 0, s, a);
    else if (few) hipLaunchKernelGGL((weight_grad_kernel<RTW, kPlan, 1, F32>), grid, one, 0, s, a);
    else hipLaunchKernelGGL((weight_grad_kernel<RTW, kPlan, WT, F32>), grid, many, 0, s, a);
}

}  // namespace

// ids: tokens up to kScanTokens are one chunk (every workgroup finds its own).
//
// How many tokens a chunk has: as many workgroups as the card holds at once, 256 of eight waves (R <= 16) or 512 of
// four.  us so, with twice the workgroups and with half: the factors of 4 adapters, 4096 tokens, 2048 and 8192 columns at rank
// 16 60.9, 60.9 and 61.2 (whole calls); rank 64, 2048 x 2048 52.5, 58.0, 50.9; the router's weight, 8192 tokens x 128 x
// 2048 26.7, 31.7, 28.9; 4096 x 256 x 4096 38.4, 41.1, 43.7.
// At most kMostChunk where the tokens are listed in LDS (the first of these 65.2 with 256, 62.3 with 512, 60.9 with 1024).
// At least kLeastChunk (1024 tokens, one adapter of 1024 x 1024 at rank 16 22.8 us, with 512 23.7; 600 x 32 x 512 9.3, with 512
// 11.0).  Over all tokens the chunks' sums are joined one after the other, so that a narrow matrix wants chunks that grow with
// the root of the tokens (chunks of 256, 512, 1024, 2048: 4096 x 32 x 512 13.7, 13.0, 16.0, 23.6; 16384 x 32 x 512
// 36.0, 26.1, 23.9, 29.9; 65536 x 8 x 128 128.7, 59.8, 36.3, 28.5).  Adapters' chunks of 256 cost
// 6 % at most there (65536 tokens of one, 128 x 128 108.7, with 1024 102.3).
static WeightGradPlan plan_of(int T, int n, int R, int C0, int C1, bool ids) {
    WeightGradPlan p{};
    if (ids && T <= kScanTokens) {
        p.chunk = T > 0 ? T : 1;
        return p;
    }
    const int wgs = groups_of(R) * ((C0 + 127) / 128 + (C1 + 127) / 128);
    auto up = [](double v) { return (int)std::ceil(v / kLeastChunk) * kLeastChunk; };
    const int want = ((R > 16 ? 512 : 256) + wgs - 1) / wgs;
    const int even = up((T + want - 1) / want), least = ids ? kLeastChunk : up(8 * std::sqrt((double)T));
    p.chunk = std::max(least, ids ? std::min(even, kMostChunk) : even);
    // a set in several chunks has more than `chunk` tokens, and one chunk at most is not full
    if (T > p.chunk) p.slots = n == 1 ? (T + p.chunk - 1) / p.chunk : 2 * T / p.chunk;
    const size_t most = T <= kLeastChunk ? 0 : ids ? 2 * std::max<size_t>(want, (T + kMostChunk - 1) / kMostChunk) : want;
    p.most_floats = most * (size_t)R * ((size_t)C0 + C1 + 1);
    return p;
}

WeightGradPlan weight_grad_plan(int T, int n, int R, int C0, int C1) { return plan_of(T, n, R, C0, C1, true); }

static int weight_grad(const TokenSets& who, int kind, const TokenPlan* plan, const float* scale, const WeightGradPlan& p,
                       const WeightGradCall* calls, int n_calls, float* part, hipStream_t s) {
    const unsigned chunks = who.T > p.chunk ? (unsigned)((who.T + p.chunk - 1) / p.chunk) : 1u;
    // Few tokens a set: a wave has them all, where workgroups that share them would be more than the card has at
    // once (us of all gradients by waves and by workgroups, 4096 x 4096 at rank 16: 64 tokens of 16 adapters 14.2 and
    // 17.3, 512 of 16 27.6 and 28.9; 2048 x 2048, 1024 of 64 32.7 and 37.8; but 4096 x 4096, 128 of 4 15.2
    // and 14.0, and 64 of one 2048 x 2048 at rank 32 15.7 and 13.9).
    int all_blocks = 0;
    for (int i = 0; i < n_calls; ++i) all_blocks += (calls[i].C + 127) / 128;
    const bool few = kind != kAll && who.T <= 64 * who.n && all_blocks * groups_of(who.R) * who.n > 512;
    GradArgs a{};
    a.who = who;
    if (plan) a.plan = *plan;
    a.scale = scale; a.chunk = p.chunk;
    int blocks = 0, joins = 0, joins0 = 0;
    for (int i = 0; i < n_calls; ++i) {
        a.w[i] = calls[i];
        a.slot_floats[i] = (int64_t)who.R * calls[i].C + (calls[i].bias ? who.R : 0);
        a.part[i] = part;
        part += p.slots * a.slot_floats[i];
        const int mine = (calls[i].C + 127) / 128, groups = few ? (mine + kFewWaves - 1) / kFewWaves : mine;
        if (i == 0) a.groups0 = groups;
        blocks += groups;
        joins += (int)((a.slot_floats[i] + 1023) / 1024);
        if (i == 0) joins0 = joins;
    }
    const unsigned entries = kind == kAll ? chunks : kind == kScan ? (unsigned)who.n : (unsigned)(who.T / p.chunk + who.n);
    const bool f32 = calls[n_calls - 1].x_type == MOE_F32;
    if (products_of(who.R) == 1) f32 ? grad_go<1, true>(a, kind, blocks, entries, few, s) : grad_go<1, false>(a, kind, blocks, entries, few, s);
    else f32 ? grad_go<2, true>(a, kind, blocks, entries, few, s) : grad_go<2, false>(a, kind, blocks, entries, few, s);
    if (p.slots) {
        a.groups0 = joins0;
        hipLaunchKernelGGL(weight_grad_join_kernel, dim3((unsigned)joins, (unsigned)who.n), dim3(256), 0, s, a, (int)chunks);
    }
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_weight_grad(const TokenSets& who, const TokenPlan* plan, const float* scale, const WeightGradPlan& p,
                       const WeightGradCall* calls, int n_calls, float* part, hipStream_t s) {
    return weight_grad(who, plan ? kPlan : kScan, plan, scale, p, calls, n_calls, part, s);
}

size_t router_weight_workspace_bytes(int T, int E, int H) { return plan_of(T, 1, E, H, 0, false).most_floats * 4; }

int launch_router_weight_grad(int T, int E, int H, const float* dlogits, const void* x, int64_t ldx, const float* xscale,
                              float* dw, float* dbias, void* ws, hipStream_t s) {
    const TokenSets who{nullptr, nullptr, T, 1, E};
    const WeightGradCall call{dlogits, E, x, ldx, xscale, xscale ? kCodes : MOE_BF16, H, dw, dbias};
    return weight_grad(who, kAll, nullptr, nullptr, plan_of(T, 1, E, H, 0, false), &call, 1, static_cast<float*>(ws), s);
}

}  // namespace moe
