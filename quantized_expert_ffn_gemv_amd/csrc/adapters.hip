// Low-rank adapters of many requests beside a shared projection.  With i = ids[t], both
// factors stored by rank (A [R][K], B [R][N]),
//   h[t][r] = sum_k x[t][k] A_i[r][k],     y[t][n] = base[t][n] + s_i sum_r h[t][r] B_i[r][n];
// backwards with dy for x and the factors changed over:
//   g[t][r] = sum_n dy[t][n] B_i[r][n],    dx[t][k] = base[t][k] + s_i sum_r g[t][r] A_i[r][k],
// so two kernels serve both directions: `shrink` (sums along the rows) and `expand` (sums over
// the ranks).  The factors' gradients are weight_grad.hip's.
//
// A workgroup has up to 16 tokens of one adapter, or 64 (expand: 32) where tokens are planned, so that
// an adapter's rows are read once for them.  Few tokens (decode): a workgroup finds its tile by
// looking through the ids; more: a first kernel puts the tokens in order.  Sums along the rows are
// split over workgroups where tiles are few; expand adds the parts.
//
// Operands of v_mfma_f32_16x16x32_bf16 straight from memory.  shrink: both run along the sum,
// 16 bytes a lane.  expand: the factor's rows run across the sum; a lane takes 8 columns of 8
// ranks (4 where R <= 16) and turns the block by v_perm_b32; column j of every lane's 8 is
// one product, so that a lane ends with 8 neighbouring columns of y for 4 tokens (a float32 y:
// two groups of 4): 16-byte loads and stores.  x and the factors are exact operands, h and a float32 dy go as three bf16
// parts (all 24 bits); sums are float32, y is rounded once.
#include <algorithm>
#include <type_traits>

#include "adapters.h"
#include "token_tiles.h"

namespace moe {

namespace {

constexpr int kWaves = 4;
constexpr int kMostSplits = 16;           // workgroups that share a tile's columns in shrink
constexpr int kUnitCols = 128;            // columns of a wave's step in shrink, of a wave in expand

struct ShrinkArgs {
    TokenSets who;
    TokenPlan plan;
    const uint16_t* w;        // [n][R][ldw]
    int64_t ldw;
    const void* x;
    int64_t ldx;
    int C, splits, units;     // units of 128 columns a split (a multiple of kWaves, but for the last)
    float* part;              // [splits][T][16 RT]
};

struct ExpandArgs {
    TokenSets who;
    TokenPlan plan;
    const uint16_t* w;
    int64_t ldw;
    const float* scale;
    const float* part;
    int splits, C;
    const void* base;
    int64_t ldbase;
    void* y;
    int64_t ldy;
    float* h;                 // [T][R] or NULL
    // instead of parts: the sums are taken here, x (bf16) times w1
    const uint16_t* w1;       // [n][R][K]
    const uint16_t* x;
    int64_t ldx;
    int K, blocks;            // workgroups a tile
};

// This workgroup's tokens, into `list` (padded with the last one): their number and adapter (-1: none).
template <bool PLAN, int NW = kWaves, int SUBS = 1>
__device__ __forceinline__ int my_tile(const TokenSets& who, const TokenPlan& plan, int idx, int& set, int* list) {
    constexpr int TOK = PLAN ? kPlanTile / SUBS : kScanTile;
    const int tid = threadIdx.x;
    if constexpr (PLAN) {
        const PlanTileEntry& e = plan.tiles[idx / SUBS];
        const int sub = idx % SUBS * TOK;
        const int token = e.token[sub + min(tid, TOK - 1)];
        const int2 head = *reinterpret_cast<const int2*>(&e);
        set = __builtin_amdgcn_readfirstlane(head.x);
        const int rows = min(__builtin_amdgcn_readfirstlane(head.y) - sub, TOK);
        if (rows <= 0) return 0;
        const int last = __shfl(token, rows - 1, kWave);               // (of the first wave, which has them all)
        if (tid < TOK) list[tid] = tid < rows ? token : last;
        __syncthreads();
        return rows;
    } else {
        __shared__ int own[NW][TOK];
        const int wid = tid >> 6;
        const int rows = scan_tile(who, idx, set, own[wid]);
        if (rows == 0) return 0;
        if (tid < TOK) list[tid] = own[0][min(tid, rows - 1)];
        __syncthreads();
        return rows;
    }
}

}  // namespace

// Bound by latency and memory: a wave has 16 rows (64 planned) of 128 columns in flight at a time and no more
// than a few turns.  48 tokens of 32 adapters, 4096 columns at rank 16: 4.3 us, of which the ids and the tile's
// rows are two round trips; 4096 tokens x 2048 at rank 32: 11.1 us, x 8192 at rank 16 20.7 us (3.3 TB/s).
// Twice the workgroups take 1.2 us less there and expand, which adds their sums, 1.1 more.
template <int RT, bool F32, bool PLAN>
__global__ __launch_bounds__(64 * kWaves) void adapter_shrink_kernel(ShrinkArgs a) {
    constexpr int NT = PLAN ? kPlanTile / 16 : 1, PARTS = F32 ? 3 : 1;
    __shared__ int list[16 * NT];
    constexpr int AT_ONCE = RT <= 2 ? NT : 1;              // groups of 16 tokens whose sums meet at once
    __shared__ __attribute__((aligned(16))) float sums[kWaves][16 * AT_ONCE][16 * RT + 4];
    int set;
    const int rows = my_tile<PLAN>(a.who, a.plan, (int)blockIdx.y, set, list);
    if (rows == 0 || set < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int rank = a.who.rank ? min(max(ld_scalar(a.who.rank, set), 0), a.who.R) : a.who.R;
    const int all = (a.C + kUnitCols - 1) / kUnitCols;
    const int u0 = (int)blockIdx.x * a.units, u1 = min(u0 + a.units, all);
    const uint16_t* w[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
        w[rt] = a.w + ((int64_t)set * a.who.R + min(16 * rt + c, max(rank - 1, 0))) * a.ldw;
    int64_t xrow[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xrow[nt] = (int64_t)list[16 * nt + c] * a.ldx;
    floatx4_t acc[NT][RT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[nt][rt] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    // 32 columns; with TAIL some of them do not exist (both operands read as 0 there)
    auto step = [&](int col, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        uint32_t wf[RT][4], xf[NT][PARTS][4], m[4];
        const int at = TAIL ? first_of_8(col, a.C) : col;
        if constexpr (TAIL) mask_first(col - at, m);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const uint4 v = load_bf16x8(w[rt] + at);
            wf[rt][0] = v.x; wf[rt][1] = v.y; wf[rt][2] = v.z; wf[rt][3] = v.w;
            if constexpr (TAIL)
#pragma unroll
                for (int d = 0; d < 4; ++d) wf[rt][d] &= m[d];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if constexpr (F32) {
                float v[8];
                __builtin_memcpy(v, static_cast<const float*>(a.x) + xrow[nt] + at, 32);
                if constexpr (TAIL)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = j >= col - at ? v[j] : 0.f;
                bf16_parts(v, xf[nt]);
            } else {
                const uint4 v = load_bf16x8(static_cast<const uint16_t*>(a.x) + xrow[nt] + at);
                xf[nt][0][0] = v.x; xf[nt][0][1] = v.y; xf[nt][0][2] = v.z; xf[nt][0][3] = v.w;
                if constexpr (TAIL)
#pragma unroll
                    for (int d = 0; d < 4; ++d) xf[nt][0][d] &= m[d];
            }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int p = 0; p < PARTS; ++p) acc[nt][rt] = mfma16(wf[rt], xf[nt][p], acc[nt][rt]);
    };
    for (int u = u0 + wid; u < u1; u += kWaves) {
        const int c0 = u * kUnitCols + 8 * q;
        if ((u + 1) * kUnitCols <= a.C) {
#pragma unroll
            for (int p = 0; p < 4; ++p) step(c0 + 32 * p, std::false_type{});
        } else {
            for (int p = 0; p < 4; ++p) step(c0 + 32 * p, std::true_type{});
        }
    }
    // the waves' sums; ranks past the adapter's are 0
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += AT_ONCE) {
        if (16 * n0 >= rows) break;
        if (n0) __syncthreads();
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) *reinterpret_cast<floatx4_t*>(&sums[wid][16 * k + c][16 * rt + 4 * q]) = acc[n0 + k][rt];
        __syncthreads();
        for (int e = tid; e < 16 * AT_ONCE * 4 * RT; e += 64 * kWaves) {
            const int row = e / (4 * RT), r = 4 * (e % (4 * RT));
            if (16 * n0 + row >= rows) break;
            floatx4_t v = *reinterpret_cast<const floatx4_t*>(&sums[0][row][r]);
#pragma unroll
            for (int k = 1; k < kWaves; ++k) v += *reinterpret_cast<const floatx4_t*>(&sums[k][row][r]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = r + i < rank ? v[i] : 0.f;
            *reinterpret_cast<floatx4_t*>(a.part + ((int64_t)blockIdx.x * a.who.T + list[16 * n0 + row]) * (16 * RT) + r) = v;
        }
    }
}

// Bound by memory where there are many tokens: base in, y out (4096 tokens x 8192 at rank 32: 30.5 us, 4.7 TB/s with
// the factors and sums; x 2048 at rank 16 11.4), by latency where there are few (48 tokens x 4096: 4.4 us).  That the
// loads of factor and base go out before the sums are there took 1.5 us off the few.
// RT = 1: products over 16 ranks (v_mfma_f32_16x16x16_bf16); else over 32 at a time.
// SELF: the workgroup takes the tile's sums itself, all of K over its eight waves, instead of reading
// shrink's: one launch, for few tokens with small factors; the workgroups of a tile sit on one XCD, so that
// they share a's rows in its L2.
constexpr int kSelfWaves = 8;
// A planned tile is two workgroups here (4096 tokens, 2048 -> 8192, rank 32: 35.6 us by one of 64 tokens,
// which filled the card one and a half times, 32.2 by two).
constexpr int kExpandSubs = 2;
template <int RT, bool F32, bool PLAN, bool SELF>
__global__ __launch_bounds__(64 * (SELF ? kSelfWaves : kWaves)) void adapter_expand_kernel(ExpandArgs a) {
    constexpr int NW = SELF ? kSelfWaves : kWaves;
    constexpr int NT = PLAN ? kPlanTile / kExpandSubs / 16 : 1, TOK = 16 * NT, RP = 16 * RT, KS = RT == 1 ? 1 : RT / 2;
    constexpr int HS = RP + 4, PARTS = 3, PER = RT == 1 ? 4 : 8;      // ranks a lane holds of a step
    __shared__ int list[TOK];
    __shared__ __attribute__((aligned(16))) float hs[TOK][HS];
    __shared__ __attribute__((aligned(16))) float sums[SELF ? NW : 1][SELF ? 16 : 1][HS];
    int set, xblock = blockIdx.x, tile = blockIdx.y;
    if constexpr (SELF) {
        tile = (int)(blockIdx.x & 7) + 8 * ((int)(blockIdx.x >> 3) / a.blocks);
        xblock = (int)(blockIdx.x >> 3) % a.blocks;
        if (tile >= a.who.T) return;
    }
    const int rows = my_tile<PLAN, NW, kExpandSubs>(a.who, a.plan, tile, set, list);
    if (rows == 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int R = a.who.R;
    const int rank = set < 0 ? 0 : a.who.rank ? min(max(ld_scalar(a.who.rank, set), 0), R) : R;
    // the lane's columns: 8 neighbours, or of a float32 y twice 4, 64 apart, so that a store of 16 bytes a lane
    // is whole lines (8 neighbours, every other 16 bytes: 4096 tokens, 2048 -> 8192 75.7 us, so 69.9)
    constexpr int G = F32 ? 2 : 1, GW = 8 / G;
    int col[G], shift[G];                                              // shift GW or more: no column is this lane's
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int own = (xblock * NW + wid) * kUnitCols + 64 * g + GW * c;
        col[g] = min(own, a.C - GW);
        shift[g] = own - col[g];
    }

    // every load that needs only the list goes out first: the factor's rows, the base's of the first 16
    // tokens (rows 4 q + i; the list is padded with its last token)
    uint4 rowv[KS][8], bb[2][4][F32 ? 2 : 1];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int i = 0; i < 8; ++i)
        {
            rowv[ks][i] = make_uint4(0, 0, 0, 0);
            if (i >= PER) continue;
            const uint16_t* row = a.w + ((int64_t)max(set, 0) * R + min(32 * ks + PER * q + i, max(rank - 1, 0))) * a.ldw;
#pragma unroll
            for (int g = 0; g < G; ++g) __builtin_memcpy(reinterpret_cast<char*>(&rowv[ks][i]) + 2 * GW * g, row + col[g], 2 * GW);
        }
    auto load_base = [&](int nt) {
        if (a.base) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const char* row = static_cast<const char*>(a.base) + (int64_t)list[16 * nt + 4 * q + i] * a.ldbase * (F32 ? 4 : 2);
#pragma unroll
                for (int g = 0; g < G; ++g) __builtin_memcpy(&bb[nt & 1][i][g], row + col[g] * (F32 ? 4 : 2), 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < (F32 ? 2 : 1); ++d) bb[nt & 1][i][d] = make_uint4(0, 0, 0, 0);
        }
    };
    if (a.y) load_base(0);

    const float s = set < 0 ? 0.f : ld_scalar(a.scale, set);
    if constexpr (SELF) {
        const uint16_t* w[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) w[rt] = a.w1 + ((int64_t)max(set, 0) * R + min(16 * rt + c, max(rank - 1, 0))) * a.K;
        const uint16_t* x = a.x + (int64_t)list[c] * a.ldx;
        floatx4_t acc[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[rt] = floatx4_t{0.f, 0.f, 0.f, 0.f};
        for (int u = rank > 0 ? wid : a.K; u < a.K / kUnitCols; u += NW)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int at = u * kUnitCols + 32 * p + 8 * q;
                const uint4 xv = load_bf16x8(x + at);
                const uint32_t xf[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const uint4 v = load_bf16x8(w[rt] + at);
                    const uint32_t wf[4] = {v.x, v.y, v.z, v.w};
                    acc[rt] = mfma16(wf, xf, acc[rt]);
                }
            }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) *reinterpret_cast<floatx4_t*>(&sums[wid][c][16 * rt + 4 * q]) = acc[rt];
        __syncthreads();
    }
    // the sums of the tile's tokens: the splits' parts, four at a time or (few tokens) all at once, or the waves'
    for (int e = tid; e < TOK * (RP / 4); e += 64 * NW) {
        const int row = e / (RP / 4), r = 4 * (e % (RP / 4));
        floatx4_t v{0.f, 0.f, 0.f, 0.f};
        if (row < rows && set >= 0) {
            if constexpr (SELF) {
#pragma unroll
                for (int k = 0; k < NW; ++k) v += *reinterpret_cast<const floatx4_t*>(&sums[k][row][r]);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = r + i < rank ? v[i] : 0.f;
            } else {
                const float* p = a.part + (int64_t)list[row] * RP + r;
                auto add = [&](int k, auto number) {
                    constexpr int N = decltype(number)::value;
                    floatx4_t o[N];
#pragma unroll
                    for (int u = 0; u < N; ++u)
                        o[u] = *reinterpret_cast<const floatx4_t*>(p + (int64_t)min(k + u, a.splits - 1) * a.who.T * RP);
#pragma unroll
                    for (int u = 0; u < N; ++u) v += k + u < a.splits ? o[u] : floatx4_t{0.f, 0.f, 0.f, 0.f};
                };
                if (!PLAN && RT <= 2 && a.splits > 4) add(0, std::integral_constant<int, kMostSplits>{});
                else for (int k = 0; k < a.splits; k += 4) add(k, std::integral_constant<int, 4>{});
            }
        }
        if (a.h && xblock == 0 && row < rows)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r + i < R) a.h[(int64_t)list[row] * R + r + i] = v[i];
        *reinterpret_cast<floatx4_t*>(&hs[row][r]) = v * s;
    }
    __syncthreads();
    if (a.y == nullptr || (xblock * NW + wid) * kUnitCols >= a.C) return;
    if (set < 0 && a.y == a.base) return;

    // the factor's block, turned: column j of the lane's 8, its ranks in order
    uint32_t wf[KS][8][PER / 2];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
        for (int i = 0; i < PER; ++i)                                  // (what lies past the rank may be no number)
            if (32 * ks + PER * q + i >= rank) rowv[ks][i] = make_uint4(0, 0, 0, 0);
        uint32_t t[8][4];
        turn8(rowv[ks], t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int d = 0; d < PER / 2; ++d) wf[ks][j][d] = t[j][d];
    }
    const bool some = rank > 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        if (16 * nt >= rows) break;
        floatx4_t acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
        if (16 * (nt + 1) < rows) load_base(nt + 1);
        if (some) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float v[8];
                uint32_t hp[PARTS][4];
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const floatx4_t f = i < PER ? *reinterpret_cast<const floatx4_t*>(&hs[16 * nt + c][32 * ks + PER * q + i])
                                                : floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i + e] = f[e];
                }
                bf16_parts(v, hp);
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if constexpr (RT == 1) {
                            typedef short s16x4_t __attribute__((ext_vector_type(4)));
                            const uint2 A = make_uint2(hp[p][0], hp[p][1]), B = make_uint2(wf[0][j][0], wf[0][j][1]);
                            acc[j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4_t, A),
                                                                              __builtin_bit_cast(s16x4_t, B), acc[j], 0, 0, 0);
                        } else {
                            acc[j] = mfma16(hp[p], wf[ks][j], acc[j]);
                        }
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (16 * nt + 4 * q + i >= rows) continue;
            const int64_t row = (int64_t)list[16 * nt + 4 * q + i] * a.ldy;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (shift[g] >= GW) continue;
                const uint4 base = bb[nt & 1][i][g];
                const uint32_t b[4] = {base.x, base.y, base.z, base.w};
                if constexpr (F32) {
                    float v[4], *out = static_cast<float*>(a.y) + row + col[g];
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(b[j]) + acc[4 * g + j][i];
                    if (shift[g] == 0) {
                        __builtin_memcpy(out, v, 16);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j >= shift[g]) out[j] = v[j];
                    }
                } else {
                    uint32_t o[4];
                    uint16_t* out = static_cast<uint16_t*>(a.y) + row + col[g];
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        o[d] = pack_bf16(__uint_as_float(b[d] << 16) + acc[2 * d][i], __uint_as_float(b[d] & 0xFFFF0000u) + acc[2 * d + 1][i]);
                    if (shift[g] == 0) {
                        __builtin_memcpy(out, o, 16);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j >= shift[g]) out[j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
                    }
                }
            }
        }
    }
}

// Tokens in order of their adapters (equal ones in token order), and the tiles and chunks made of
// them: a workgroup for each adapter, and one for the tokens without.  It counts the tokens of
// smaller numbers, which is where its own begin, and puts its own there.  Entries of the lists
// stand where no other set's can: a set's tiles from (tokens before it) / kPlanTile + set on, what
// is left up to the next set's first empty; chunks likewise, and partial sums from
// 2 (tokens before it) / chunk on (a set in c > 1 chunks has more than (c - 1) chunk tokens, so
// it ends before the next one's).  (One workgroup for all sets took 8.4 us of 4096 tokens, its steps one
// after the other.)
constexpr int kPlanWaves = 16, kPlanPer = 4;           // tokens a thread and round
__global__ __launch_bounds__(64 * kPlanWaves) void adapter_plan_kernel(TokenSets who, TokenPlan plan) {
    constexpr int ROUND = 64 * kPlanWaves * kPlanPer;
    __shared__ int2 waves[kPlanWaves];
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, set = blockIdx.x, n = who.n;
    auto below = [](uint64_t mask) { return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0)); };
    auto load = [&](int base, int (&v)[kPlanPer]) {
#pragma unroll
        for (int j = 0; j < kPlanPer; ++j) {
            const int t = base + kPlanPer * tid + j, id = who.ids[min(t, who.T - 1)];
            v[j] = t >= who.T ? n + 1 : (unsigned)id < (unsigned)n ? id : n;
        }
    };
    int held[kPlanPer];
    load(0, held);
    int less = 0, mine = 0;
    for (int base = 0; base < who.T; base += ROUND) {
        int v[kPlanPer];
        if (base == 0) {
#pragma unroll
            for (int j = 0; j < kPlanPer; ++j) v[j] = held[j];
        } else {
            load(base, v);
        }
#pragma unroll
        for (int j = 0; j < kPlanPer; ++j) {
            less += __popcll(__ballot(v[j] < set));
            mine += __popcll(__ballot(v[j] == set));
        }
    }
    if (lane == 0) waves[wid] = make_int2(less, mine);
    __syncthreads();
    less = mine = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
        less += waves[w].x;
        mine += waves[w].y;
    }
    // the lists' entries
    const int tile0 = less / kPlanTile + set, tile1 = (less + mine) / kPlanTile + set + 1;
    for (int k = tid; k < tile1 - tile0; k += 64 * kPlanWaves)
        *reinterpret_cast<int2*>(&plan.tiles[tile0 + k]) = make_int2(set < n ? set : -1, max(min(kPlanTile, mine - k * kPlanTile), 0));
    const int chunks = set < n ? max(1, (mine + plan.chunk - 1) / plan.chunk) : 0, slot0 = 2 * less / plan.chunk;
    const int chunk0 = less / plan.chunk + set, chunk1 = set < n ? (less + mine) / plan.chunk + set + 1 : who.T / plan.chunk + n;
    for (int k = tid; k < chunk1 - chunk0; k += 64 * kPlanWaves)
        plan.chunks[chunk0 + k] = k < chunks ? make_int4(set, less + k * plan.chunk, max(min(plan.chunk, mine - k * plan.chunk), 0),
                                                         chunks > 1 ? slot0 + k : -1)
                                             : make_int4(-1, 0, 0, -1);
    if (tid == 0 && set < n) plan.joins[set] = make_int2(slot0, chunks > 1 ? chunks : 0);
    // its tokens, in order
    int next = less;
    for (int base = 0; base < who.T; base += ROUND) {
        int v[kPlanPer];
        if (base == 0) {
#pragma unroll
            for (int j = 0; j < kPlanPer; ++j) v[j] = held[j];
        } else {
            load(base, v);
        }
        int place = 0, count = 0;
#pragma unroll
        for (int j = 0; j < kPlanPer; ++j) {
            const uint64_t mask = __ballot(v[j] == set);
            place += below(mask);
            count += __popcll(mask);
        }
        __syncthreads();
        if (lane == 0) waves[wid].x = count;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = waves[w].x;
            place += w < wid ? c : 0;
            all += c;
        }
#pragma unroll
        for (int j = 0; j < kPlanPer; ++j)
            if (v[j] == set) {
                const int token = base + kPlanPer * tid + j, at = next + place++ - less;      // its place among the set's
                plan.order[less + at] = token;
                plan.tiles[tile0 + at / kPlanTile].token[at % kPlanTile] = token;
            }
        next += all;
    }
}

namespace {

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
bool planned(int T) { return T > kScanTokens; }

// Workgroups' worth of tiles, and how the columns of a shrink are split: workgroups twice the
// CUs where there are columns for it, four waves each with a unit at least.
// (Whole calls with 256, 512 and 1024 workgroups wanted, 8 adapters, 2048 and 8192 columns: gradients of 4096 tokens at rank 16 65.8,
// 60.9 and 58.7 us, rank 64 91.5, 90.5 and 93.8, rank 128, where the registers leave a wave a SIMD, 164, 156 and 167;
// of 1024 at rank 128 75.2, 77.5 and 77.3.  Forwards 2048 columns have no more than 4 splits: no difference.)
constexpr int kShrinkBlocks = 512;
int shrink_splits(int T, int n, int C) {
    const int sets = std::max(1, std::min(n, T));
    const int tiles = planned(T) ? (T + kPlanTile - 1) / kPlanTile + sets / 2 : sets;
    const int units = (C + kUnitCols - 1) / kUnitCols, most = (units + kWaves - 1) / kWaves;
    return std::min({(kShrinkBlocks + tiles - 1) / tiles, most, kMostSplits});
}

// Rows of partial sums that calls of up to T tokens need at most: no more splits than kMostSplits,
// and past kScanTokens no more than (kShrinkBlocks + tiles) / tiles with T / kPlanTile tiles or more.
int64_t part_rows(int T) { return std::min((int64_t)kMostSplits * T, (int64_t)kShrinkBlocks * kPlanTile + T); }

struct Space {
    float* part;
    float* g;
    TokenPlan plan;
    float* grad_part;
    size_t bytes;
};

Space space(const moe_adapters& m, int T, bool grad, const WeightGradPlan& p, void* ws) {
    char* at = static_cast<char*>(ws);
    auto take = [&](size_t n) { char* r = at; at += up256(n); return r; };
    Space sp{};
    sp.part = reinterpret_cast<float*>(take((size_t)part_rows(T) * 16 * rank_tiles(m.R) * 4));
    if (grad) {
        sp.g = reinterpret_cast<float*>(take((size_t)T * m.R * 4));
        sp.grad_part = reinterpret_cast<float*>(take(p.most_floats * 4));
    }
    if (planned(T)) {
        const int tiles = T / kPlanTile + m.n + 1, chunk = grad ? p.chunk : T;
        sp.plan.order = reinterpret_cast<int32_t*>(take((size_t)T * 4));
        sp.plan.tiles = reinterpret_cast<PlanTileEntry*>(take((size_t)tiles * sizeof(PlanTileEntry)));
        sp.plan.chunks = reinterpret_cast<int4*>(take((size_t)(T / kLeastChunk + m.n) * 16));
        sp.plan.joins = reinterpret_cast<int2*>(take((size_t)m.n * 8));
        sp.plan.chunk = chunk;
    }
    sp.bytes = (size_t)(at - static_cast<char*>(ws));
    return sp;
}

template <bool F32, bool PLAN>
void shrink_go(const ShrinkArgs& a, dim3 grid, hipStream_t s) {
    switch (rank_tiles(a.who.R)) {
        case 1: hipLaunchKernelGGL((adapter_shrink_kernel<1, F32, PLAN>), grid, dim3(64 * kWaves), 0, s, a); break;
        case 2: hipLaunchKernelGGL((adapter_shrink_kernel<2, F32, PLAN>), grid, dim3(64 * kWaves), 0, s, a); break;
        case 4: hipLaunchKernelGGL((adapter_shrink_kernel<4, F32, PLAN>), grid, dim3(64 * kWaves), 0, s, a); break;
        default: hipLaunchKernelGGL((adapter_shrink_kernel<8, F32, PLAN>), grid, dim3(64 * kWaves), 0, s, a);
    }
}

template <bool F32, bool PLAN>
void expand_go(const ExpandArgs& a, dim3 grid, hipStream_t s) {
    switch (rank_tiles(a.who.R)) {
        case 1: hipLaunchKernelGGL((adapter_expand_kernel<1, F32, PLAN, false>), grid, dim3(64 * kWaves), 0, s, a); break;
        case 2: hipLaunchKernelGGL((adapter_expand_kernel<2, F32, PLAN, false>), grid, dim3(64 * kWaves), 0, s, a); break;
        case 4: hipLaunchKernelGGL((adapter_expand_kernel<4, F32, PLAN, false>), grid, dim3(64 * kWaves), 0, s, a); break;
        default: hipLaunchKernelGGL((adapter_expand_kernel<8, F32, PLAN, false>), grid, dim3(64 * kWaves), 0, s, a);
    }
}

template <bool F32>
void self_go(const ExpandArgs& a, dim3 grid, hipStream_t s) {
    if (a.who.R <= 16) hipLaunchKernelGGL((adapter_expand_kernel<1, F32, false, true>), grid, dim3(64 * kSelfWaves), 0, s, a);
    else hipLaunchKernelGGL((adapter_expand_kernel<2, F32, false, true>), grid, dim3(64 * kSelfWaves), 0, s, a);
}

unsigned tile_blocks(const TokenSets& who) {
    return planned(who.T) ? (unsigned)(who.T / kPlanTile + who.n + 1) : (unsigned)who.T;
}

void shrink(const TokenSets& who, const Space& sp, const uint16_t* w, int64_t ldw, int C, const void* x, int64_t ldx, bool f32,
            hipStream_t s) {
    ShrinkArgs a{};
    a.who = who; a.plan = sp.plan; a.w = w; a.ldw = ldw; a.C = C; a.x = x; a.ldx = ldx; a.part = sp.part;
    a.splits = shrink_splits(who.T, who.n, C);
    const int units = (C + kUnitCols - 1) / kUnitCols;
    a.units = ((units + a.splits - 1) / a.splits + kWaves - 1) / kWaves * kWaves;
    const dim3 grid((unsigned)a.splits, tile_blocks(who));
    if (planned(who.T)) f32 ? shrink_go<true, true>(a, grid, s) : shrink_go<false, true>(a, grid, s);
    else f32 ? shrink_go<true, false>(a, grid, s) : shrink_go<false, false>(a, grid, s);
}

void expand(const TokenSets& who, const Space& sp, int splits, const float* scale, const uint16_t* w, int64_t ldw, int C,
            const void* base, int64_t ldbase, void* y, int64_t ldy, bool f32, float* h, hipStream_t s) {
    ExpandArgs a{};
    a.who = who; a.plan = sp.plan; a.w = w; a.ldw = ldw; a.scale = scale; a.part = sp.part; a.splits = splits; a.C = C;
    a.base = base; a.ldbase = ldbase; a.y = y; a.ldy = ldy; a.h = h;
    const unsigned blocks = y ? (unsigned)((C + kWaves * kUnitCols - 1) / (kWaves * kUnitCols)) : 1u;
    const dim3 grid(blocks, tile_blocks(who) * (planned(who.T) ? kExpandSubs : 1));
    if (planned(who.T)) f32 ? expand_go<true, true>(a, grid, s) : expand_go<false, true>(a, grid, s);
    else f32 ? expand_go<true, false>(a, grid, s) : expand_go<false, false>(a, grid, s);
}

// Few tokens in one launch, every workgroup with all of its tile's sums: where a's rows are 64 KB at most, K is 2048 at
// most (less than 4096 with no more tokens than adapters), and the workgroups of an XCD find room at once: all of a tile's
// sit on one, and each takes the sums anew (K columns each, and what 512 more would take, up to 64 x 2048).  us by two
// launches and by one:
//   rank 8, K 2048, N 4096:   1 token 6.2 and 5.3, 40 of 40 adapters 6.7 and 5.6, 128 of 64 8.1 and 8.7
//   rank 16, K 1024:          1 token x N 16384 6.1 and 4.9, x 100000 6.1 and 12.3; 128 of 64 x 4096 9.0 and 8.4,
//                             x 16384 15.7 and 21.9, x 100000 66 and 119
//   rank 16, K 2048, N 4096:  64 tokens of 4 7.2 and 7.8; rank 32: 1 token 7.1 and 8.1 (a's rows 128 KB)
//   rank 4, K 3200, N 4096:   40 tokens of 40 7.2 and 6.0; K 4096: 1 token 6.3 and 6.2, 64 of 4, whose tiles have 16 rows
//                             of x, 7.4 and 9.3; K 8192: 1 token 6.3 and 8.6.
// Over 1344 sizes (K 256 to 4096, rank 4 to 32, N 1024 to 49152, 1 to 512 tokens) the choice costs 1 % beside
// the better side, the limit on a's rows alone 10 %, two launches throughout 8 %.
constexpr int kSelfColumns = 64 * 2048;
int self_blocks(const moe_adapters& m) { return (m.N + kSelfWaves * kUnitCols - 1) / (kSelfWaves * kUnitCols); }
bool one_launch(const moe_adapters& m, int T) {
    if (planned(T) || m.R > 32 || m.R * m.K > 32768 || m.K >= (T > m.n ? 2176 : 4096)) return false;
    const int tiles = std::min(T, std::min(m.n, T) + T / kScanTile), an_xcd = (tiles + 7) / 8 * self_blocks(m);
    return (int64_t)an_xcd * (m.K + 512) <= kSelfColumns;
}

void make_plan(const TokenSets& who, const TokenPlan& plan, hipStream_t s) {
    hipLaunchKernelGGL(adapter_plan_kernel, dim3((unsigned)who.n + 1), dim3(64 * kPlanWaves), 0, s, who, plan);
}

}  // namespace

size_t adapter_workspace_bytes(const moe_adapters& m, int T, bool grad) {
    const WeightGradPlan p = grad ? weight_grad_plan(T, m.n, m.R, m.K, m.N) : WeightGradPlan{};
    return space(m, T, grad, p, nullptr).bytes;
}

int launch_adapter(const moe_adapters& m, int T, const int32_t* ids, const uint16_t* x, int64_t ldx, const void* base,
                   int64_t ldbase, void* y, int64_t ldy, int y_type, float* h, void* ws, hipStream_t s) {
    const TokenSets who{ids, m.rank, T, m.n, m.R};
    const Space sp = space(m, T, false, WeightGradPlan{}, ws);
    if (one_launch(m, T)) {
        ExpandArgs a{};
        a.who = who; a.w = m.b; a.ldw = m.ldb; a.scale = m.scale; a.C = m.N; a.base = base; a.ldbase = ldbase; a.y = y; a.ldy = ldy;
        a.h = h; a.w1 = m.a; a.x = x; a.ldx = ldx; a.K = m.K; a.blocks = self_blocks(m);
        const dim3 grid(8u * (unsigned)((T + 7) / 8 * a.blocks));
        y_type == MOE_F32 ? self_go<true>(a, grid, s) : self_go<false>(a, grid, s);
        return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
    }
    if (planned(T)) make_plan(who, sp.plan, s);
    shrink(who, sp, m.a, m.K, m.K, x, ldx, false, s);
    expand(who, sp, shrink_splits(T, m.n, m.K), m.scale, m.b, m.ldb, m.N, base, ldbase, y, ldy, y_type == MOE_F32, h, s);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_adapter_grad(const AdapterGradArgs& a, hipStream_t s) {
    const moe_adapters& m = a.m;
    const TokenSets who{a.ids, m.rank, a.T, m.n, m.R};
    const WeightGradPlan p = weight_grad_plan(a.T, m.n, m.R, m.K, m.N);
    const Space sp = space(m, a.T, true, p, a.ws);
    const bool f32 = a.dy_type == MOE_F32;
    if (planned(a.T)) make_plan(who, sp.plan, s);
    if (a.T > 0 && (a.dx || a.da)) {
        shrink(who, sp, m.b, m.ldb, m.N, a.dy, a.lddy, f32, s);
        expand(who, sp, shrink_splits(a.T, m.n, m.N), m.scale, m.a, m.K, m.K, a.dx_base, a.lddx_base, a.dx, a.lddx, false, sp.g, s);
    }
    WeightGradCall calls[2];
    int n = 0;
    if (a.da) calls[n++] = WeightGradCall{sp.g, m.R, a.x, a.ldx, a.xscale, a.xscale ? kCodes : MOE_BF16, m.K, a.da, nullptr};
    if (a.db) calls[n++] = WeightGradCall{a.h, m.R, a.dy, a.lddy, nullptr, a.dy_type, m.N, a.db, nullptr};
    if (n) return launch_weight_grad(who, planned(a.T) ? &sp.plan : nullptr, m.scale, p, calls, n, sp.grad_part, s);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
