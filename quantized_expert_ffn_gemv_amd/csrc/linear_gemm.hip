// Products of many tokens with one quantised matrix, forward and input gradient,
// as a dense half-precision GEMM on the matrix cores:
//   forward    y[t][n]  = sum_k x[t][k]  w[n][k]
//   gradient   dx[t][k] = sum_n dy[t][n] w[n][k]
// Both operands are laid out once per call in blocks of 32 along the summed index,
// [block][part][row][32], so that a stage of a tile is one contiguous run a part (rows a
// power of two apart met in one L2 channel: 4096 x 8192 x 2048 took 1.08 times as long with
// 256-wide tiles, 1.27 times with 128-wide ones):
//   B  the weights as two fp16 parts, the second what the first leaves out (2^-22 of a
//      weight and less), rows n forward and, transposed, rows k for the gradient, each weight
//      row n scaled by a power of two 2^en so that its largest possible |w| lies in
//      [2^14, 2^15): no overflow, and 39 binades down to the parts' last bit;
//   A  the activations (or dy, which also takes the weight rows' 2^-en) as fp16,
//      each token's row scaled by 2^et into the same range.  bf16 values keep all
//      their bits there; a float32 dy takes two parts like the weights, laid out one
//      behind the other, and its second is multiplied with the weights' first only.
// Powers of two leave the significands alone, so what is rounded is 2^-22 of an operand,
// the sums in float32, and the result.  (One part of the weights, 2^-11, took 123 us where two
// take 199, but terms that cancel showed it, and bf16 results differed by 8e-4 from those of
// float32 operands, now 6e-5.)
// Laying the weights out costs one pass over the codes and 4 bytes a weight written and
// read; a matrix is taken in chunks of output columns, which bound the workspace.
#include <algorithm>
#include <type_traits>

#include "launch_util.h"
#include "linear.h"
#include "mfma_ops.h"
#include "row_ops.h"

namespace moe {

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef float floatx16_t __attribute__((ext_vector_type(16)));

constexpr int kTop = 14;                               // scaled rows' largest exponent
constexpr int kMid = 16;                               // en of weights below 1/4: dy takes 2^(kMid - en), near 1
constexpr int kNone = 400;                             // exponent of zero rows: 2^-400 leaves no finite dy above 0
constexpr int kStep = 32;                              // summed elements per block
constexpr int kBlocks = 4;                             // rows are whole runs of this many blocks (zeros behind)
constexpr int kParts = 2;                              // fp16 parts of a weight
constexpr int kKeep = 4;                               // pieces of a row of A a thread keeps
constexpr int kPrepGroups = 8;                         // 128-runs of K a workgroup lays out
// Laid-out weights per chunk, at most: past the 256 MB cache, for enough tiles in a chunk's
// GEMM.  The chunks of a matrix are of like size.  Laid-out rows of x or dy, the same: calls of
// more tokens take them in turns, the weights of a chunk laid out once.
constexpr size_t kChunkBytes = (size_t)1 << 30;
constexpr int kLeastTokens = 256;

__host__ __device__ inline int round_up(int v, int to) { return (v + to - 1) / to * to; }

// Exponent that brings a row whose largest magnitude is `top` into [2^14, 2^15):
// kNone for zero rows (dy at such a weight row must not set the scale of its
// token); infinities and NaNs count as the largest exponent.
__device__ __forceinline__ int scale_exponent(float top) {
    if (top == 0.f) return kNone;
    const uint32_t u = __float_as_uint(top) & 0x7FFFFFFFu;
    const int e = u >= 0x7F800000u ? 128 : __builtin_amdgcn_frexp_expf(top) - 1;
    return kTop - e;
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const half2_t v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// a and b as fp16 in hi, and what that leaves out in lo.
__device__ __forceinline__ void split_half(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_half(a, b);
    const half2_t h = __builtin_bit_cast(half2_t, hi);
    lo = pack_half(a - (float)h[0], b - (float)h[1]);
}

// |w|'s bound over a row's groups, taken by `lanes` threads that start at `first`.
template <int BITS>
__device__ __forceinline__ float row_bound(const moe_qmatrix& w, size_t n, int first, int lanes) {
    const int ngs = w.K / w.group_size;
    float top = 0.f;
    for (int g = first; g < ngs; g += lanes) {
        const float s = f16_bits_to_f32(w.scale[n * ngs + g]), b = f16_bits_to_f32(w.bias[n * ngs + g]);
        top = fmaxf(top, fmaxf(fabsf(b), fabsf(fmaf((float)((1 << BITS) - 1), s, b))));
    }
    return top;
}

// Word wi (0 .. 15) of a row's piece of a 128-run: eight codes, k = 8 wi ..
template <int BITS>
__device__ __forceinline__ uint32_t code_word(const uint8_t* piece, int wi) {
    return BITS == 4 ? reinterpret_cast<const uint32_t*>(piece)[wi] : reinterpret_cast<const uint16_t*>(piece)[wi];
}

template <int BITS>
__device__ __forceinline__ float word_code(uint32_t w, int j) {
    return (float)((w >> (BITS * j)) & ((1u << BITS) - 1));
}

struct PrepArgs {
    moe_qmatrix w;
    const void* a;            // activations or dy
    int64_t lda;
    int a_type;
    int T, len, kd;           // rows; elements of a row; kd: len rounded up (zeros behind)
    uint16_t* ah;             // fp16 [a_parts][kd / 32][T][32]
    int32_t* et;              // [T]
    int16_t* en;              // [N]
    uint16_t* wh;             // fp16 [K / 32][kParts][rows][32], gradient [kd / 32][kParts][columns][32]
    int c0, cn;               // this chunk's weight rows (forward) or 128-runs of K (gradient)
    int a_blocks;             // workgroups that lay out A (the first ones); 0 in later chunks
    int a_rows;               // rows each: 1, or 4 (rows of at most 64 kKeep pieces: 3769 x 2240
                              // x 256, one part, 24.6 us against 28.1, 4096 x 2048 x 2048 53.8 and 56.1)
};

// One row of A by LANES threads, a workgroup of 256 or a wave, in pieces of eight values:
// the first LANES kKeep pieces stay in registers between the maximum and the rounding, the rest is read
// twice.  dy's values take 2^(kMid - en) of their weight row.  Every thread's kKeep
// loads are made whatever the row's length (past its whole pieces the last one again):
// behind a branch each waited for the one before (4096 x 8192 of dy with its weights in one part: 54
// us against 46).
template <bool GRAD, bool F32, int LANES>
__device__ __forceinline__ void prep_a_row(const PrepArgs& p, int t) {
    constexpr int KEEP = kKeep, GROUP = LANES * KEEP, SIZE = F32 ? 4 : 2;
    __shared__ float tops[4];
    const int tid = threadIdx.x % LANES;
    const uint8_t* src = static_cast<const uint8_t*>(p.a) + (size_t)t * p.lda * SIZE;
    const int whole = p.len / 8, rest = p.len % 8, pieces = p.kd / 8, groups = (pieces + GROUP - 1) / GROUP;
    float v[KEEP][8], tail[8], top = 0.f;
    bool bad = false;
    auto get = [&](int first) {                                    // pieces first + tid + LANES c (zeros past the whole ones)
        uint32_t x[KEEP][F32 ? 8 : 4];
        uint4 e[KEEP];
        if (whole > 0) {
#pragma unroll
            for (int c = 0; c < KEEP; ++c) {
                const int i = min(first + tid + LANES * c, whole - 1);
                __builtin_memcpy(x[c], src + (size_t)i * (8 * SIZE), 8 * SIZE);   // (rows of dy have any alignment)
                if constexpr (GRAD) e[c] = *reinterpret_cast<const uint4*>(p.en + 8 * i);
            }
        }
#pragma unroll
        for (int c = 0; c < KEEP; ++c) {
            const bool in = first + tid + LANES * c < whole;
            const uint32_t ew[4] = {e[c].x, e[c].y, e[c].z, e[c].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float f;
                if constexpr (F32) f = __uint_as_float(x[c][j]);
                else f = __uint_as_float((j & 1) ? x[c][j >> 1] & 0xFFFF0000u : x[c][j >> 1] << 16);
                if constexpr (GRAD) f = ldexpf(f, kMid - (int)(int16_t)(ew[j >> 1] >> (16 * (j & 1))));
                v[c][j] = in ? f : 0.f;
            }
        }
    };
    auto look = [&](const float (&x)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            top = fmaxf(top, fabsf(x[j]));
            bad |= x[j] != x[j];
        }
    };
    if (rest != 0 && tid == 0) {                                   // the piece that the row ends in
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = 8 * whole + j;
            tail[j] = 0.f;
            if (j < rest) {
                if constexpr (F32) tail[j] = reinterpret_cast<const float*>(src)[i];
                else tail[j] = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(src)[i]);
                if constexpr (GRAD) tail[j] = ldexpf(tail[j], kMid - p.en[i]);
            }
        }
        look(tail);
    }
    for (int g = groups - 1; g >= 0; --g) {
        get(g * GROUP);
#pragma unroll
        for (int c = 0; c < KEEP; ++c) look(v[c]);
    }
    top = row_max<kWave>(bad ? INFINITY : top);
    if constexpr (LANES > kWave) {
        if ((tid & 63) == 0) tops[tid >> 6] = top;
        __syncthreads();
        top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    }
    const int e = scale_exponent(top);
    if (tid == 0) p.et[t] = GRAD ? e + kMid : e;
    auto put = [&](const float (&x)[8], int i) {
        uint32_t o[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) split_half(ldexpf(x[2 * j], e), ldexpf(x[2 * j + 1], e), o[j], lo[j]);
        uint16_t* dst = p.ah + ((size_t)(8 * i / kStep) * p.T + t) * kStep + (8 * i & (kStep - 1));
        *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        if constexpr (F32) *reinterpret_cast<uint4*>(dst + (size_t)p.T * p.kd) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    };
    if (rest != 0 && tid == 0) put(tail, whole);
    for (int g = 0; g < groups; ++g) {
        if (g > 0) get(g * GROUP);
#pragma unroll
        for (int c = 0; c < KEEP; ++c) {
            const int i = g * GROUP + tid + LANES * c;
            if (i < pieces && !(rest != 0 && i == whole)) put(v[c], i);
        }
    }
}

// Rows of A of workgroup `blk`: one, or one a wave.
template <bool GRAD, bool F32>
__device__ __forceinline__ void prep_a(const PrepArgs& p, int blk) {
    if (p.a_rows == 1) {
        prep_a_row<GRAD, F32, 256>(p, blk);
    } else {
        const int t = __builtin_amdgcn_readfirstlane(blk * 4 + (int)(threadIdx.x >> 6));
        if (t < p.T) prep_a_row<GRAD, F32, kWave>(p, t);
    }
}

}  // namespace

// Forward: workgroups [0, a_blocks) lay out rows of x, the others 16 weight rows times
// kPrepGroups 128-runs of K each.
template <int BITS>
__global__ __launch_bounds__(256) void linear_prep_kernel(PrepArgs p) {
    if ((int)blockIdx.x < p.a_blocks) {
        prep_a<false, false>(p, blockIdx.x);
        return;
    }
    __shared__ int ens[16];
    const int tid = threadIdx.x;
    const int NG = p.w.K / 128, parts = (NG + kPrepGroups - 1) / kPrepGroups;
    const int blk = (int)blockIdx.x - p.a_blocks, part = blk % parts;
    const int r0 = blk / parts * 16;                               // within the chunk
    const int ngs = p.w.K / p.w.group_size, gshift = __builtin_ctz(p.w.group_size);
    {
        const int r = r0 + (tid >> 4);
        const float top = row_max<16>(r < p.cn ? row_bound<BITS>(p.w, (size_t)(p.c0 + r), tid & 15, 16) : 0.f);
        if ((tid & 15) == 0) {
            ens[tid >> 4] = scale_exponent(top);
            if (r < p.cn && part == 0) p.en[p.c0 + r] = (int16_t)ens[tid >> 4];
        }
    }
    __syncthreads();
    // 16 threads a row and group, each one word of eight codes: four neighbours fill the 64
    // bytes of a row in a block
    const int rr = tid >> 4, wi = tid & 15, r = r0 + rr;
    if (r >= p.cn) return;
    const size_t n = (size_t)(p.c0 + r);
    const int e = ens[rr];
    const uint8_t* src = p.w.q + n * (16 * BITS);
    const size_t step = (size_t)p.w.N * (16 * BITS);
#pragma unroll 4
    for (int g = part * kPrepGroups; g < min(NG, (part + 1) * kPrepGroups); ++g) {
        const uint32_t c = code_word<BITS>(src + g * step, wi);
        const int k0 = 128 * g + 8 * wi;
        const size_t at = n * ngs + (k0 >> gshift);
        const float s = ldexpf(f16_bits_to_f32(p.w.scale[at]), e), b = ldexpf(f16_bits_to_f32(p.w.bias[at]), e);
        uint16_t* dst = p.wh + ((size_t)(k0 / kStep) * (kParts * p.cn) + r) * kStep + (k0 & (kStep - 1));
        uint32_t o[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            split_half(fmaf(word_code<BITS>(c, 2 * j), s, b), fmaf(word_code<BITS>(c, 2 * j + 1), s, b), o[j], lo[j]);
        *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + (size_t)p.cn * kStep) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// Gradient, first: the weight rows' exponents.  16 threads a row.
template <int BITS>
__global__ __launch_bounds__(256) void linear_rows_kernel(PrepArgs p) {
    const int n = (int)blockIdx.x * 16 + (int)(threadIdx.x >> 4);
    const float top = row_max<16>(n < p.w.N ? row_bound<BITS>(p.w, (size_t)n, threadIdx.x & 15, 16) : 0.f);
    if (n < p.w.N && (threadIdx.x & 15) == 0) p.en[n] = (int16_t)scale_exponent(top);
}

// Gradient: workgroups [0, a_blocks) lay out rows of dy, the others one 128-run of
// K times 128 weight rows each.  A thread takes one word of eight rows: its 8 x 8
// codes are eight 16-byte pieces of the transposed matrix, and four neighbours
// (32 weight rows) fill the 64 bytes of a row in a block.
template <int BITS>
__global__ __launch_bounds__(256) void linear_grad_prep_kernel(PrepArgs p) {
    if ((int)blockIdx.x < p.a_blocks) {
        if (p.a_type == MOE_F32) prep_a<true, true>(p, blockIdx.x);
        else prep_a<true, false>(p, blockIdx.x);
        return;
    }
    const int tid = threadIdx.x, blk = (int)blockIdx.x - p.a_blocks;
    const int nblocks = (p.kd + 127) / 128;
    const int gl = blk / nblocks, g = p.c0 + gl;
    const int n0 = (blk % nblocks) * 128 + 32 * (tid >> 6) + 8 * (tid & 3), wi = (tid >> 2) & 15;
    if (n0 >= p.kd) return;
    const int ngs = p.w.K / p.w.group_size, gshift = __builtin_ctz(p.w.group_size);
    uint32_t c[8];
    float s[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = min(n0 + i, p.w.N - 1);
        c[i] = code_word<BITS>(p.w.q + ((size_t)g * p.w.N + n) * (16 * BITS), wi);
        const size_t at = (size_t)n * ngs + ((128 * g + 8 * wi) >> gshift);
        const int e = p.en[n];
        const bool in = n0 + i < p.w.N;
        s[i] = in ? ldexpf(f16_bits_to_f32(p.w.scale[at]), e) : 0.f;
        b[i] = in ? ldexpf(f16_bits_to_f32(p.w.bias[at]), e) : 0.f;
    }
    uint16_t* dst = p.wh + ((size_t)(n0 / kStep) * (kParts * 128 * p.cn) + 128 * gl + 8 * wi) * kStep + (n0 & (kStep - 1));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t o[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            split_half(fmaf(word_code<BITS>(c[2 * i], j), s[2 * i], b[2 * i]),
                       fmaf(word_code<BITS>(c[2 * i + 1], j), s[2 * i + 1], b[2 * i + 1]), o[i], lo[i]);
        *reinterpret_cast<uint4*>(dst + j * kStep) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + (j + 128 * (size_t)p.cn) * kStep) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

namespace {

struct GemmArgs {
    const uint16_t* A;        // fp16 [a_parts][kd / 32][M][32]
    const uint16_t* B;        // fp16 [kd / 32][kParts][N][32]
    int M, N, kd, a_parts;
    const int32_t* et;        // [M]
    const int16_t* en;        // [N], or NULL (folded into A)
    const float* row_bias;    // [N] or NULL
    const uint16_t* residual; // or NULL
    int64_t ldr;
    void* y;
    int64_t ldy;
    int y_type;
    int splits;               // of the sum; more than one: unscaled sums to part
    float* part;              // float32 [splits][M][N]
};

// Results [t][n .. n + 7] from scaled sums: the row bias, the residual, the rounding.
__device__ __forceinline__ void put_results(const GemmArgs& p, int t, int n, float (&v)[8]) {
    if (n + 8 <= p.N) {                                            // (16 bytes at any alignment)
        if (p.residual) {
            uint32_t w[4];
            __builtin_memcpy(w, p.residual + (size_t)t * p.ldr + n, 16);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                v[2 * x] += __uint_as_float(w[x] << 16);
                v[2 * x + 1] += __uint_as_float(w[x] & 0xFFFF0000u);
            }
        }
        if (p.y_type == MOE_F32) {
            __builtin_memcpy(static_cast<float*>(p.y) + (size_t)t * p.ldy + n, v, 32);
        } else {
            const uint32_t w[4] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
            __builtin_memcpy(static_cast<uint16_t*>(p.y) + (size_t)t * p.ldy + n, w, 16);
        }
    } else {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            if (n + x >= p.N) continue;
            float u = v[x];
            if (p.residual) u += bf16_bits_to_f32(p.residual[(size_t)t * p.ldr + n + x]);
            if (p.y_type == MOE_F32) static_cast<float*>(p.y)[(size_t)t * p.ldy + n + x] = u;
            else static_cast<uint16_t*>(p.y)[(size_t)t * p.ldy + n + x] = (uint16_t)(pack_bf16(u, 0.f) & 0xFFFFu);
        }
    }
}

}  // namespace

// C = A (B1 + B2)^T in tiles of 32 WM WR x 32 WN WC by WR x WC waves (each 32 WM x 32 WN on
// v_mfma_f32_32x32x16_f16: A lane l holds row l % 32 and k = 8 (l / 32) + i, B the
// same of a column; accumulator 4 j + i is row 8 j + 4 (l / 32) + i of column
// l % 32).  Stages of KB blocks of 32 summed elements, A's rows and both parts of B's, pass
// through a ring of STAGES LDS slots by direct-to-LDS loads waited for by count; one barrier
// a stage.  A's operands are read once for both parts.
// A row's 64 bytes of a block are four 16-byte pieces, piece c of row r at place
// c ^ ((r >> 2) & 3): 16 rows read at one piece hit all banks once.  Workgroups
// on one XCD take neighbouring tiles (8 rows of tiles at a time), which share
// their operands in its L2.  4096 x 8192 x 2048 takes 199 us for both parts (1.38 PF, what a
// large library product of halves reaches here).  Tiles taken in turn by one workgroup, the
// loads running on into the next, were slower (131 us against 123 with one part).
template <int WM, int WN, int WR, int WC, int STAGES, int KB>
__global__ __launch_bounds__(64 * WR * WC) __attribute__((amdgpu_waves_per_eu(2, 2))) void linear_gemm_kernel(GemmArgs p) {
    constexpr int BM = 32 * WM * WR, BN = 32 * WN * WC, WAVES = WR * WC;
    constexpr int BLOCK = (BM + kParts * BN) * 2 * kStep, SLOT = KB * BLOCK;   // bytes
    constexpr int LOADS = BLOCK / kDma / WAVES;                         // a wave's loads per block
    static_assert(LOADS * kDma * WAVES == BLOCK, "whole loads");
    extern __shared__ __attribute__((aligned(16))) uint8_t slots[];
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN, tiles = tm * tn;
    // tile of this workgroup
    int tile = blockIdx.x;
    {
        const int per = (tiles + 7) / 8;
        tile = (tile & 7) * per + (tile >> 3);
        if (tile >= tiles) return;
    }
    const int band = tile / (8 * tn), rows = min(8, tm - 8 * band), in = tile - band * 8 * tn;
    const int m0 = (8 * band + in % rows) * BM, n0 = (in / rows) * BN;

    // this wave's loads of a block: LOADS chunks of 1 KB (16 rows) of A's rows, then B's
    uint32_t off[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int chunk = LOADS * wid + i, row = 16 * chunk + (lane >> 2);
        const int part = row < BM + BN ? 0 : 1;
        const int r = 16 * chunk < BM ? min(m0 + row, p.M - 1) - m0
                                      : min(n0 + row - BM - part * BN, p.N - 1) - n0 + part * p.N;
        off[i] = (uint32_t)r * (2 * kStep) + 16u * ((lane & 3) ^ ((row >> 2) & 3));
    }
    // blocks [first, last) of the sum, of blocks1 a part of A, in whole stages (kd is whole stages)
    const int blocks1 = p.kd / kStep, stages = blocks1 * p.a_parts / KB, each = (stages + p.splits - 1) / p.splits;
    const int steps = min(each, stages - (int)blockIdx.y * each), first = (int)blockIdx.y * each * KB, last = first + steps * KB;
    const int both = max(0, min(steps, (blocks1 - first) / KB));   // stages of A's first part: with both of B's
    const size_t strideA = (size_t)p.M * (2 * kStep), strideB = (size_t)p.N * (kParts * 2 * kStep);   // bytes from block to block
    const uint8_t* firstB = reinterpret_cast<const uint8_t*>(p.B + (size_t)n0 * kStep);
    const uint8_t* srcA = reinterpret_cast<const uint8_t*>(p.A + (size_t)m0 * kStep) + (size_t)first * strideA;
    const uint8_t* srcB = firstB + (size_t)(first < blocks1 ? first : first - blocks1) * strideB;
    // The loads of a stage are made in its HALVES = 2 KB halves of a block, half of a block's
    // LOADS each (the first the odd one too); the sources then move on to the next block (past
    // the end: the last again).
    constexpr int HALVES = 2 * KB, ODD = LOADS / 2, EVEN = LOADS - ODD;
    int staged = first, slot_in = 0;                               // next block, slot it goes to
    auto put = [&](int half, int i) {                              // load i of a half
        uint8_t* slot = slots + slot_in * SLOT + (half >> 1) * BLOCK + LOADS * wid * kDma;
        const int c = EVEN * (half & 1) + i;
        dma16_sv(16 * (LOADS * wid + c) < BM ? srcA : srcB, off[c], slot + c * kDma);
    };
    auto put_done = [&](int half) {
        if (half & 1) {
            ++staged;
            if (staged < last) {
                srcA += strideA;
                srcB = staged == blocks1 ? firstB : srcB + strideB;
            }
        }
        if (half == HALVES - 1) slot_in = slot_in + 1 < STAGES ? slot_in + 1 : 0;
    };
    floatx16_t acc[WM][WN];
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int j = 0; j < WN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    const int wm = wid / WC, wn = wid % WC, m = lane & 31, h = lane >> 5;
    const int arow = 32 * WM * wm + m, brow = BM + 32 * WN * wn + m;
    half8_t a[2][WM], b[2][kParts][WN];
    auto read = [&](int half, int at) {                            // half a block of the stage in slot `at`
        const uint8_t* slot = slots + at * SLOT + (half >> 1) * BLOCK;
        const int kk = half & 1;
        // rows r, r + 32, ... swap pieces alike: (r >> 2) & 3 is the same
        const int place = 16 * ((2 * kk + h) ^ ((m >> 2) & 3));
#pragma unroll
        for (int i = 0; i < WM; ++i) a[kk][i] = *reinterpret_cast<const half8_t*>(slot + (arow + 32 * i) * 64 + place);
#pragma unroll
        for (int x = 0; x < kParts; ++x)
#pragma unroll
            for (int j = 0; j < WN; ++j) b[kk][x][j] = *reinterpret_cast<const half8_t*>(slot + (brow + BN * x + 32 * j) * 64 + place);
        asm volatile("" ::: "memory");                             // the reads stay here, ahead of the products
        __builtin_amdgcn_sched_barrier(0);
    };
    // Half a block's products, a load of a later stage after every few of them: the loads issue
    // while the matrix cores work (made together behind the barrier, they left them idle).
    auto multiply = [&](int half, auto parts) {
        constexpr int P = decltype(parts)::value, N = WM * WN * P;
        const int kk = half & 1, each = kk ? ODD : EVEN;
#pragma unroll
        for (int x = 0; x < P; ++x)
#pragma unroll
            for (int i = 0; i < WM; ++i)
#pragma unroll
                for (int j = 0; j < WN; ++j) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[kk][i], b[kk][x][j], acc[i][j], 0, 0, 0);
                    const int n = (x * WM + i) * WN + j;
#pragma unroll
                    for (int c = 0; c < each; ++c)
                        if (n == (N * c + N / 2) / each) {
                            __builtin_amdgcn_sched_barrier(0);
                            put(half, c);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                }
        put_done(half);
    };
    // During stage s the loads of stage s + STAGES - 1 are made, into the slot that stage
    // s - 1 left at the barrier; one half of a block is read from LDS while the other is
    // multiplied: read together behind the barrier, the waves' reads left the matrix cores idle.
    static_assert(STAGES >= 3, "a stage in flight behind the next one");
    for (int s = 0; s + 1 < STAGES; ++s)
#pragma unroll
        for (int half = 0; half < HALVES; ++half) {
#pragma unroll
            for (int c = 0; c < ((half & 1) ? ODD : EVEN); ++c) put(half, c);
            put_done(half);
        }
    wait_vmem<(STAGES - 2) * KB * LOADS>();
    lds_barrier();
    int at = 0;
    read(0, 0);
    auto stage = [&](auto parts) {
#pragma unroll
        for (int half = 0; half + 1 < HALVES; ++half) {
            read(half + 1, at);
            multiply(half, parts);
        }
        // this wave's part of the next stage has arrived; then every wave's, and this one is read
        wait_vmem<(STAGES - 2) * KB * LOADS - ODD>();
        lds_barrier();
        at = at + 1 < STAGES ? at + 1 : 0;
        read(0, at);                                               // (past the end: a stage never used)
        multiply(HALVES - 1, parts);
    };
    for (int s = 0; s < both; ++s) stage(std::integral_constant<int, kParts>{});
    for (int s = both; s < steps; ++s) stage(std::integral_constant<int, 1>{});
    wait_vmem<0>();                                                // loads past the last stage, before their LDS is used again
    lds_barrier();
    // each wave turns its sums around in LDS, 32 rows at a time: rows of 32 WN results
    constexpr int COLS = 32 * WN, PITCH = COLS + 4;
    static_assert(WAVES * 32 * PITCH * 4 <= STAGES * SLOT, "the results fit the slots");
    float* turn = reinterpret_cast<float*>(slots) + wid * 32 * PITCH;
    const int c0 = n0 + COLS * wn;
    constexpr int PER_ROW = COLS / 8, PASS = 64 / PER_ROW;         // lanes a row, eight results each; rows at once
    const int cc = 8 * (lane % PER_ROW), n = c0 + cc;
    int en[8], et[WM][32 / PASS];
    float rb[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        en[x] = p.en && p.splits == 1 ? p.en[min(n + x, p.N - 1)] : 0;
        rb[x] = p.row_bias && p.splits == 1 ? p.row_bias[min(n + x, p.N - 1)] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int rr = 0; rr < 32 / PASS; ++rr)
            et[i][rr] = p.splits == 1 ? p.et[min(m0 + 32 * (WM * wm + i) + PASS * rr + lane / PER_ROW, p.M - 1)] : 0;
#pragma unroll
    for (int i = 0; i < WM; ++i) {
        const int r0 = m0 + 32 * (WM * wm + i);
#pragma unroll
        for (int e = 0; e < 16; ++e)
#pragma unroll
            for (int j = 0; j < WN; ++j) turn[(8 * (e >> 2) + 4 * h + (e & 3)) * PITCH + 32 * j + m] = acc[i][j][e];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#pragma unroll
        for (int rr = 0; rr < 32 / PASS; ++rr) {
            const int r = PASS * rr + lane / PER_ROW, t = r0 + r;
            if (t >= p.M || n >= p.N) continue;
            float v[8];
#pragma unroll
            for (int x = 0; x < 8; x += 4) {
                const floatx4_t f = *reinterpret_cast<const floatx4_t*>(turn + r * PITCH + cc + x);
#pragma unroll
                for (int u = 0; u < 4; ++u) v[x + u] = ldexpf(f[u], -(et[i][rr] + en[x + u])) + rb[x + u];
            }
            if (p.splits == 1) {
                put_results(p, t, n, v);
            } else {
                float* part = p.part + ((size_t)blockIdx.y * p.M + t) * p.N + n;
                if (n + 8 <= p.N) __builtin_memcpy(part, v, 32);
                else
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (n + x < p.N) part[x] = v[x];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    }
}

// The splits' sums joined in order, scaled back and finished; a thread eight results.
__global__ __launch_bounds__(256) void linear_join_kernel(GemmArgs p) {
    const int cols = (p.N + 7) / 8;
    const long id = (long)blockIdx.x * 256 + threadIdx.x;
    if (id >= (long)cols * p.M) return;
    const int t = (int)(id / cols), n = (int)(id % cols) * 8;
    const size_t step = (size_t)p.M * p.N;
    const float* src = p.part + (size_t)t * p.N + n;
    float v[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) v[x] = 0.f;
    if (n + 8 <= p.N) {
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            float u[8];
            __builtin_memcpy(u, src + s * step, 32);
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] += u[x];
        }
    } else {
        for (int s = 0; s < p.splits; ++s)
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] += n + x < p.N ? src[s * step + x] : 0.f;
    }
    const int et = p.et[t];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const int c = min(n + x, p.N - 1);
        v[x] = ldexpf(v[x], -(et + (p.en ? p.en[c] : 0))) + (p.row_bias ? p.row_bias[c] : 0.f);
    }
    put_results(p, t, n, v);
}

namespace {

template <int WM, int WN, int WR, int WC, int STAGES, int KB>
void gemm_go(const GemmArgs& p, hipStream_t s) {
    constexpr int BM = 32 * WM * WR, BN = 32 * WN * WC;
    static_assert(kBlocks % KB == 0, "stages are whole");
    const int tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
    const int blocks = ((tm * tn + 7) / 8) * 8;
    const size_t lds = (size_t)STAGES * KB * (BM + kParts * BN) * 2 * kStep;
    hipLaunchKernelGGL((linear_gemm_kernel<WM, WN, WR, WC, STAGES, KB>), dim3((unsigned)blocks, (unsigned)p.splits),
                       dim3(64 * WR * WC), lds, s, p);
}

enum Tile { k256x256, k256x128, k128, k64, k64One };

constexpr int kMaxSplits = 16;

// The splits' sums are at most what fills the card with the largest tiles.
long split_results() { return 65536L * device_cus(); }

struct Choice {
    Tile tile;
    int splits;               // of the sum
    double us;                // estimated
};

// Tiles and splits by estimated time, fitted to 391 products (T 64 .. 8192, N 16 .. 60000, K 128
// .. 12800, both directions) with every tile and up to eight numbers of splits each; taking
// the least estimate costs 1.6 % over taking the fastest, 44 % at most.  A round of tiles
// over the CUs takes, for a sum of 4096,
//   256 x 256  168 us, one a CU;                   256 x 128  90, one a CU;
//   128 x 128  107, two a CU, 55 with one;         64 x 64    41, two a CU, 17 with one,
//   whose ring takes all of the LDS (200 x 2048 x 4096: 33 us against 37 with half of it);
// a last round with few tiles up to a quarter less.  Whole calls with each of the four, us:
//   4096 x 8192 x 2048  218 265 242 338    3000 x 4096 x 4096  184 217 186 245
//   4096 x 5120 x 2048  183 176 153 209    4096 x 2048 x 8192  327 254 256 333
//   1500 x 4096 x 4096  156 114 113 130     700 x 4096 x 4096  151 108  80  81
//   1024 x 2048 x 2048   84  61  46  38     512 x 4096 x 4096  151 106  79  57
//   6000 x 6000 x 1024  163 173 144 209     300 x 30000 x 1024  78  89  74  81
// Long sums over few tiles are split, where the shorter sums gain more than the join takes
// (a launch, and the partial sums written and read).  Without and with two, three and six: 489 x
// 18984 x 8960 627 586 529 542, gradient 649 x 27100 x 2944 (256 x 256) 1848 1113 843 521.
Choice gemm_choice(int M, int N, int kd, int a_parts) {
    const long cus = device_cus();
    const int sum = kd * a_parts;
    auto tiles = [&](int rows, int cols) { return (long)((M + rows - 1) / rows) * ((N + cols - 1) / cols); };
    auto one_a_cu = [&](long t, double start, double round, double less) {
        const long rest = t % cus;
        return t / cus * (start + round) + (rest ? start + round * (1 - less * (1 - (double)rest / cus)) : 0.);
    };
    auto two_a_cu = [&](long t, double one, double two) {
        const long rest = t % (2 * cus);
        return t / (2 * cus) * two + (rest == 0 ? 0. : rest <= cus ? one : one + (two - one) * (double)(rest - cus) / cus);
    };
    const long t[4] = {tiles(256, 256), tiles(256, 128), tiles(128, 128), tiles(64, 64)};
    const int stage[4] = {1, 1, 1, 2};                             // blocks
    Choice best{k256x256, 1, 0.};
    for (int s = 1; s == 1 || (s <= kMaxSplits && s * 512 <= sum && t[2] < 2 * cus && (long)s * M * N <= split_results()); ++s) {
        // (A's second part meets one of B's two)
        const double join = s == 1 ? 0. : 5 + 1.2e-6 * s * M * N, k = kd / 4096. * (a_parts == 2 ? 1.5 : 1.) / s;
        const double cost[4] = {one_a_cu(t[0] * s, 3.4, 168 * k, 0.26), one_a_cu(t[1] * s, 4.3, 90 * k, 0.19),
                                two_a_cu(t[2] * s, 1.3 + 55 * k, 107 * k), two_a_cu(t[3] * s, 17 * k, 41 * k)};
        for (int i = 0; i < 4; ++i) {
            const double us = cost[i] + join;
            if ((s > 1 || i > 0) && us >= best.us) continue;
            const bool one = i == 3 && t[3] * s <= cus;
            const int stages = sum / kStep / (one ? 4 : stage[i]), each = (stages + s - 1) / s;
            best = Choice{one ? k64One : (Tile)i, (stages + each - 1) / each, us};   // (no split without a stage)
        }
    }
    return best;
}

void gemm(GemmArgs p, hipStream_t s) {
    const Choice c = gemm_choice(p.M, p.N, p.kd, p.a_parts);
    p.splits = c.splits;
    switch (c.tile) {
    case k256x256: gemm_go<4, 2, 2, 4, 3, 1>(p, s); break;
    case k256x128: gemm_go<4, 2, 2, 2, 4, 1>(p, s); break;
    case k128: gemm_go<2, 2, 2, 2, 3, 1>(p, s); break;
    case k64: gemm_go<1, 1, 2, 2, 3, 2>(p, s); break;
    case k64One: gemm_go<1, 1, 2, 2, 3, 4>(p, s); break;
    }
    if (p.splits > 1) {
        const long threads = (long)p.M * ((p.N + 7) / 8);
        hipLaunchKernelGGL(linear_join_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, p);
    }
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// Workspace: A, et, en, the chunk's weights, then the splits' sums.
struct Plan {
    int tokens;                            // per GEMM
    int kd, a_parts, chunk, total;         // chunk: weight rows (forward) or 128-runs (gradient) per GEMM
    size_t et, en, wh, part, bytes;
};

Plan plan_of(const moe_qmatrix& w, int T, int type, bool grad) {
    Plan p{};
    p.kd = grad ? round_up(w.N, kStep * kBlocks) : w.K;
    p.a_parts = grad && type == MOE_F32 ? 2 : 1;
    p.total = grad ? w.K / 128 : w.N;
    const size_t row = (size_t)2 * p.kd * p.a_parts;                                   // bytes of a row of A
    const int at_once = std::max(kLeastTokens, (int)(kChunkBytes / row) / kLeastTokens * kLeastTokens);
    const int turns = (T + at_once - 1) / at_once;
    p.tokens = std::min(round_up((T + turns - 1) / turns, kLeastTokens), T);
    const size_t unit = (size_t)2 * kParts * p.kd * (grad ? 128 : 1);                  // bytes
    size_t c = kChunkBytes / unit;
    const int tile = grad ? 2 : 256;                                                 // a tile's worth
    const int most = c < (size_t)tile ? tile : c > (size_t)p.total ? p.total : (int)c / tile * tile;
    const int chunks = (p.total + most - 1) / most;
    p.chunk = std::min(round_up((p.total + chunks - 1) / chunks, tile), p.total);
    const int most_tokens = std::min(T, at_once);                  // (the turns' even share may fall as T grows)
    p.et = align256(row * most_tokens);
    p.en = p.et + align256((size_t)most_tokens * 4);
    p.wh = p.en + align256((size_t)w.N * 2);
    p.part = p.wh + align256(unit * p.chunk);
    // (for any number of splits, so that more tokens never need less)
    const long results = (long)most_tokens * (grad ? 128 * p.chunk : p.chunk);
    p.bytes = p.part + (p.kd * p.a_parts < 1024 ? 0 : align256(std::min(kMaxSplits * results, split_results()) * sizeof(float)));
    return p;
}

}  // namespace

size_t linear_gemm_workspace_bytes(const moe_qmatrix& w, int T, int type, bool grad) {
    return plan_of(w, T, type, grad).bytes;
}

// The layouts' bytes, then the products.
double linear_gemm_us(const moe_qmatrix& w, int T, int type, bool grad, double limit) {
    const double N = w.N, K = w.K, wide = type == MOE_F32 ? 4 : 2, matrix = N * K * (2 * kParts + w.bits / 8.);   // bytes
    double us = grad ? 11.9 + 0.351e-6 * matrix + 0.363e-6 * T * N * (wide + wide) + 0.414e-6 * T * K * 2
                     : 8.8 + 0.4e-3 * K + 0.305e-6 * matrix + 0.278e-6 * T * K * 4 + 0.289e-6 * T * N * wide;
    if (us >= limit) return us;
    const Plan p = plan_of(w, T, type, grad);
    // whole chunks and turns alike, then the last ones
    const int wide_c = grad ? 128 : 1, last_c = p.total % p.chunk, last_t = T % p.tokens;
    auto products = [&](int tokens, int chunk, double times) {
        if (tokens > 0 && chunk > 0 && us < limit) us += times * gemm_choice(tokens, chunk * wide_c, p.kd, p.a_parts).us;
    };
    products(p.tokens, p.chunk, (double)(T / p.tokens) * (p.total / p.chunk));
    products(last_t, p.chunk, p.total / p.chunk);
    products(p.tokens, last_c, T / p.tokens);
    products(last_t, last_c, 1);
    return us;
}

void linear_gemm_kernels(const moe_qmatrix& w, int T, int type, bool grad, int32_t* kernels) {
    static const int32_t shape[][3] = {{256, 256, 1}, {256, 128, 1}, {128, 128, 1}, {64, 64, 2}, {64, 64, 4}};   // by Tile
    const Plan p = plan_of(w, T, type, grad);
    const Choice c = gemm_choice(p.tokens, p.chunk * (grad ? 128 : 1), p.kd, p.a_parts);
    kernels[1] = shape[c.tile][0];
    kernels[2] = shape[c.tile][1];
    kernels[3] = c.splits;
    kernels[4] = shape[c.tile][2];
    kernels[5] = (p.total + p.chunk - 1) / p.chunk;
    kernels[6] = p.a_parts;
    kernels[7] = (T + p.tokens - 1) / p.tokens;
}

namespace {

PrepArgs prep_of(const moe_qmatrix& w, const Plan& pl, uint8_t* ws) {
    PrepArgs p{};
    p.w = w;
    p.kd = pl.kd;
    p.ah = reinterpret_cast<uint16_t*>(ws);
    p.et = reinterpret_cast<int32_t*>(ws + pl.et);
    p.en = reinterpret_cast<int16_t*>(ws + pl.en);
    p.wh = reinterpret_cast<uint16_t*>(ws + pl.wh);
    p.a_rows = pl.kd <= 8 * kWave * kKeep ? 4 : 1;
    return p;
}

// Every chunk of the matrix with every turn of tokens: the chunk is laid out in the first
// turn's launch, the tokens in the first chunk's, or in each one's where there are several
// turns (they share their place).  prep(p, w) lays out p's tokens and, with w, the chunk;
// product(t0, p) multiplies.
template <typename PREP, typename PRODUCT>
void by_chunks(const Plan& pl, PrepArgs p, int T, const uint8_t* a, int64_t row, PREP prep, PRODUCT product) {
    for (p.c0 = 0; p.c0 < pl.total; p.c0 += pl.chunk) {
        p.cn = std::min(pl.chunk, pl.total - p.c0);
        for (int t0 = 0; t0 < T; t0 += pl.tokens) {
            p.T = std::min(pl.tokens, T - t0);
            p.a = a + (int64_t)t0 * row;
            p.a_blocks = p.c0 == 0 || pl.tokens < T ? (p.T + p.a_rows - 1) / p.a_rows : 0;
            prep(p, t0 == 0);
            product(t0, p);
        }
    }
}

}  // namespace

int launch_linear_gemm(const LinearArgs& a, hipStream_t s) {
    const Plan pl = plan_of(a.w, a.T, a.y_type, false);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    PrepArgs p = prep_of(a.w, pl, ws);
    p.lda = a.ldx; p.a_type = MOE_BF16; p.len = a.w.K;
    const int parts = (a.w.K / 128 + kPrepGroups - 1) / kPrepGroups, e = a.y_type == MOE_F32 ? 4 : 2;
    by_chunks(pl, p, a.T, reinterpret_cast<const uint8_t*>(a.x), 2 * a.ldx,
        [&](const PrepArgs& q, bool w) {
            const dim3 grid((unsigned)(q.a_blocks + (w ? (q.cn + 15) / 16 * parts : 0)));
            if (a.w.bits == 4) hipLaunchKernelGGL(linear_prep_kernel<4>, grid, dim3(256), 0, s, q);
            else hipLaunchKernelGGL(linear_prep_kernel<2>, grid, dim3(256), 0, s, q);
        },
        [&](int t0, const PrepArgs& q) {
            GemmArgs g{};
            g.part = reinterpret_cast<float*>(ws + pl.part);
            g.A = q.ah; g.B = q.wh; g.M = q.T; g.N = q.cn; g.kd = pl.kd; g.a_parts = 1; g.et = q.et; g.en = q.en + q.c0;
            g.row_bias = a.row_bias ? a.row_bias + q.c0 : nullptr;
            g.residual = a.residual ? a.residual + (int64_t)t0 * a.ldr + q.c0 : nullptr;
            g.ldr = a.ldr; g.ldy = a.ldy; g.y_type = a.y_type;
            g.y = static_cast<uint8_t*>(a.y) + ((int64_t)t0 * a.ldy + q.c0) * e;
            gemm(g, s);
        });
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_linear_grad_gemm(const LinearGradArgs& a, hipStream_t s) {
    const Plan pl = plan_of(a.w, a.T, a.dy_type, true);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    PrepArgs p = prep_of(a.w, pl, ws);
    p.lda = a.lddy; p.a_type = a.dy_type; p.len = a.w.N;
    const dim3 rows((unsigned)((a.w.N + 15) / 16));
    if (a.w.bits == 4) hipLaunchKernelGGL(linear_rows_kernel<4>, rows, dim3(256), 0, s, p);
    else hipLaunchKernelGGL(linear_rows_kernel<2>, rows, dim3(256), 0, s, p);
    by_chunks(pl, p, a.T, static_cast<const uint8_t*>(a.dy), (a.dy_type == MOE_F32 ? 4 : 2) * a.lddy,
        [&](const PrepArgs& q, bool w) {
            const dim3 grid((unsigned)(q.a_blocks + (w ? q.cn * ((pl.kd + 127) / 128) : 0)));
            if (a.w.bits == 4) hipLaunchKernelGGL(linear_grad_prep_kernel<4>, grid, dim3(256), 0, s, q);
            else hipLaunchKernelGGL(linear_grad_prep_kernel<2>, grid, dim3(256), 0, s, q);
        },
        [&](int t0, const PrepArgs& q) {
            GemmArgs g{};
            g.part = reinterpret_cast<float*>(ws + pl.part);
            g.A = q.ah; g.B = q.wh; g.M = q.T; g.N = 128 * q.cn; g.kd = pl.kd; g.a_parts = pl.a_parts; g.et = q.et;
            g.ldy = a.lddx; g.y_type = MOE_BF16; g.y = a.dx + (int64_t)t0 * a.lddx + 128 * (size_t)q.c0;
            gemm(g, s);
        });
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
