// Products of many tokens with one quantised matrix, forward and input gradient,
// as a dense half-precision GEMM on the matrix cores:
//   forward    y[t][n]  = sum_k x[t][k]  w[n][k]
//   gradient   dx[t][k] = sum_n dy[t][n] w[n][k]
// Both operands are laid out once per call with the summed index contiguous:
//   B  the weights as fp16, [n][k] forward and transposed [k][n] for the gradient,
//      each weight row n scaled by a power of two 2^en so that its largest possible
//      |w| lies in [2^14, 2^15): no overflow, and 29 binades of full fp16 precision
//      below a row's largest weight;
//   A  the activations (or dy, which also takes the weight rows' 2^-en) as fp16,
//      each token's row scaled by 2^et into the same range.  bf16 values keep all
//      their bits there.
// Powers of two leave the significands alone, so the roundings are fp16's of the
// weights (2^-11 of each, an eighth of the bf16 result's own step; fp32 results
// take the weights as two fp16 parts, 2^-22), float32's in the sums, and the
// result's.  Laying the weights out costs one pass over the codes and 2 bytes a
// weight; a matrix is taken in chunks of output columns that stay in the 256 MB
// cache between the two kernels.
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
constexpr int kStep = 32;                              // summed elements per LDS stage
constexpr int kStages = 4;
constexpr size_t kChunkBytes = (size_t)128 << 20;      // laid-out weights per chunk

__host__ __device__ inline int round_up(int v, int to) { return (v + to - 1) / to * to; }

// Exponent that brings a row whose largest magnitude is `top` into [2^14, 2^15):
// 0 for zero rows; infinities and NaNs count as the largest exponent.
__device__ __forceinline__ int scale_exponent(float top) {
    if (top == 0.f) return 0;
    const uint32_t u = __float_as_uint(top) & 0x7FFFFFFFu;
    const int e = u >= 0x7F800000u ? 128 : __builtin_amdgcn_frexp_expf(top) - 1;
    return kTop - e;
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const half2_t v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
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

// Code k (0 .. 31 of a quarter of a 128-run) from the quarter's words.
template <int BITS>
__device__ __forceinline__ float quarter_code(const uint32_t (&c)[BITS], int k) {
    constexpr int PER = 32 / BITS;
    return (float)((c[k / PER] >> (BITS * (k % PER))) & ((1u << BITS) - 1));
}

struct PrepArgs {
    moe_qmatrix w;
    const void* a;            // activations or dy
    int64_t lda;
    int a_type;
    int T, len, kd;           // rows; elements of a row; kd: len rounded up (zeros behind)
    uint16_t* ah;             // fp16 [T][kd]
    int32_t* et;              // [T]
    int32_t* en;              // [N]
    uint16_t* wh;             // fp16: forward [planes][rows][K], gradient [columns][kd]
    int c0, cn;               // this chunk's weight rows (forward) or 128-runs of K (gradient)
    int planes;
    int a_blocks;             // workgroups that lay out A (the first ones); 0 in later chunks
};

// One row of A by a workgroup of 256.
__device__ __forceinline__ void prep_a_row(const PrepArgs& p, int t, bool grad) {
    __shared__ float tops[4];
    const int tid = threadIdx.x;
    const int64_t row = (int64_t)t * p.lda;
    const uint16_t* ab = static_cast<const uint16_t*>(p.a) + row;
    const float* af = static_cast<const float*>(p.a) + row;
    auto value = [&](int i) {
        const float v = p.a_type == MOE_F32 ? af[i] : bf16_bits_to_f32(ab[i]);
        return grad ? ldexpf(v, kMid - p.en[i]) : v;
    };
    float top = 0.f;
    bool bad = false;
    for (int i = tid; i < p.len; i += 256) {
        const float v = value(i);
        top = fmaxf(top, fabsf(v));
        bad |= v != v;
    }
    top = row_max<kWave>(bad ? INFINITY : top);
    if ((tid & 63) == 0) tops[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    const int e = scale_exponent(top);
    if (tid == 0) p.et[t] = grad ? e + kMid : e;
    uint32_t* out = reinterpret_cast<uint32_t*>(p.ah + (size_t)t * p.kd);
    for (int i = 2 * tid; i < p.kd; i += 512) {
        const float v0 = i < p.len ? ldexpf(value(i), e) : 0.f, v1 = i + 1 < p.len ? ldexpf(value(i + 1), e) : 0.f;
        out[i >> 1] = pack_half(v0, v1);
    }
}

}  // namespace

// Forward: workgroups [0, a_blocks) lay out rows of x, the others 16 weight rows each.
template <int BITS>
__global__ __launch_bounds__(256) void linear_prep_kernel(PrepArgs p) {
    if ((int)blockIdx.x < p.a_blocks) {
        prep_a_row(p, blockIdx.x, false);
        return;
    }
    __shared__ int ens[16];
    const int tid = threadIdx.x;
    const int r0 = ((int)blockIdx.x - p.a_blocks) * 16;            // within the chunk
    const int ngs = p.w.K / p.w.group_size, gshift = __builtin_ctz(p.w.group_size), NG = p.w.K / 128;
    {
        const int r = r0 + (tid >> 4);
        const float top = row_max<16>(r < p.cn ? row_bound<BITS>(p.w, (size_t)(p.c0 + r), tid & 15, 16) : 0.f);
        if ((tid & 15) == 0) {
            ens[tid >> 4] = scale_exponent(top);
            if (r < p.cn) p.en[p.c0 + r] = ens[tid >> 4];
        }
    }
    __syncthreads();
    const int rr = (tid >> 2) & 15, q = tid & 3, r = r0 + rr;      // 4 threads a row and group, 4 groups at once
    if (r >= p.cn) return;
    const size_t n = (size_t)(p.c0 + r);
    const int e = ens[rr];
    const size_t plane = (size_t)p.cn * p.w.K;
    for (int g = tid >> 6; g < NG; g += 4) {
        uint32_t c[BITS];
        const uint8_t* src = p.w.q + ((size_t)g * p.w.N + n) * (16 * BITS) + 4 * BITS * q;
#pragma unroll
        for (int i = 0; i < BITS; ++i) c[i] = reinterpret_cast<const uint32_t*>(src)[i];
        const int k0 = 128 * g + 32 * q;                           // 32 consecutive k share a scale group
        const size_t at = n * ngs + (k0 >> gshift);
        const float s = ldexpf(f16_bits_to_f32(p.w.scale[at]), e), b = ldexpf(f16_bits_to_f32(p.w.bias[at]), e);
        uint16_t* dst = p.wh + (size_t)r * p.w.K + k0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w0 = fmaf(quarter_code<BITS>(c, 8 * i + 2 * j), s, b);
                const float w1 = fmaf(quarter_code<BITS>(c, 8 * i + 2 * j + 1), s, b);
                o[j] = pack_half(w0, w1);
                const half2_t h = __builtin_bit_cast(half2_t, o[j]);
                lo[j] = pack_half(w0 - (float)h[0], w1 - (float)h[1]);
            }
            reinterpret_cast<uint4*>(dst)[i] = make_uint4(o[0], o[1], o[2], o[3]);
            if (p.planes == 2) reinterpret_cast<uint4*>(dst + plane)[i] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// Gradient, first: the weight rows' exponents.  16 threads a row.
template <int BITS>
__global__ __launch_bounds__(256) void linear_rows_kernel(PrepArgs p) {
    const int n = (int)blockIdx.x * 16 + (int)(threadIdx.x >> 4);
    const float top = row_max<16>(n < p.w.N ? row_bound<BITS>(p.w, (size_t)n, threadIdx.x & 15, 16) : 0.f);
    if (n < p.w.N && (threadIdx.x & 15) == 0) p.en[n] = scale_exponent(top);
}

// Gradient: workgroups [0, a_blocks) lay out rows of dy, the others one 128-run of
// K times 64 weight rows each, transposed through LDS.
template <int BITS>
__global__ __launch_bounds__(256) void linear_grad_prep_kernel(PrepArgs p) {
    if ((int)blockIdx.x < p.a_blocks) {
        prep_a_row(p, blockIdx.x, true);
        return;
    }
    constexpr int PITCH = 64 + 8;                                  // halves a k row in LDS
    __shared__ __attribute__((aligned(16))) uint16_t tile[128 * PITCH];
    const int tid = threadIdx.x, blk = (int)blockIdx.x - p.a_blocks;
    const int nblocks = (p.kd + 63) / 64;
    const int gl = blk / nblocks, n0 = (blk % nblocks) * 64, g = p.c0 + gl;
    const int ngs = p.w.K / p.w.group_size, gshift = __builtin_ctz(p.w.group_size);
    {
        const int rr = tid >> 2, q = tid & 3, n = n0 + rr;
        const bool in = n < p.w.N;
        const size_t nn = in ? n : 0;
        uint32_t c[BITS];
        const uint8_t* src = p.w.q + ((size_t)g * p.w.N + nn) * (16 * BITS) + 4 * BITS * q;
#pragma unroll
        for (int i = 0; i < BITS; ++i) c[i] = reinterpret_cast<const uint32_t*>(src)[i];
        const int k0 = 128 * g + 32 * q;
        const size_t at = nn * ngs + (k0 >> gshift);
        const int e = p.en[nn];
        const float s = in ? ldexpf(f16_bits_to_f32(p.w.scale[at]), e) : 0.f;
        const float b = in ? ldexpf(f16_bits_to_f32(p.w.bias[at]), e) : 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            tile[(32 * q + i) * PITCH + rr] = (uint16_t)(pack_half(fmaf(quarter_code<BITS>(c, i), s, b), 0.f) & 0xFFFFu);
    }
    __syncthreads();
    for (int o = tid; o < 128 * 8; o += 256) {                     // 16-byte pieces, 8 a k row
        const int k = o >> 3, piece = o & 7;
        if (n0 + 8 * piece < p.kd)
            *reinterpret_cast<uint4*>(p.wh + ((size_t)gl * 128 + k) * p.kd + n0 + 8 * piece) =
                *reinterpret_cast<const uint4*>(tile + k * PITCH + 8 * piece);
    }
}

namespace {

struct GemmArgs {
    const uint16_t* A;        // fp16 [M][kd]
    const uint16_t* B;        // fp16 [planes][N][kd]
    int M, N, kd, planes;
    const int32_t* et;        // [M]
    const int32_t* en;        // [N], or NULL (folded into A)
    const float* row_bias;    // [N] or NULL
    const uint16_t* residual; // or NULL
    int64_t ldr;
    void* y;
    int64_t ldy;
    int y_type;
};

}  // namespace

// C = A B^T in tiles of 64 WM x 64 WN by four waves (2 x 2, each 32 WM x 32 WN on
// v_mfma_f32_32x32x16_f16: A lane l holds row l % 32 and k = 8 (l / 32) + i, B the
// same of a column; accumulator 4 j + i is row 8 j + 4 (l / 32) + i of column
// l % 32).  Stages of 32 summed elements pass through a ring of four LDS slots,
// three ahead, by direct-to-LDS loads waited for by count; one barrier a stage.
// A row's 64 bytes of a stage are four 16-byte pieces, piece c of row r at place
// c ^ ((r >> 2) & 3): 16 rows read at one piece hit all banks once.  Workgroups
// on one XCD take neighbouring tiles (8 rows of tiles at a time), which share
// their operands in its L2.
template <int WM, int WN>
__global__ __launch_bounds__(256) void linear_gemm_kernel(GemmArgs p) {
    constexpr int BM = 64 * WM, BN = 64 * WN;
    constexpr int SLOT = (BM + BN) * 2 * kStep;                    // bytes
    constexpr int LOADS = SLOT / kDma / 4;                         // a wave's loads per stage
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

    // this lane's part of the wave's loads: chunk i (1 KB, 16 rows of A's or B's tile)
    uint32_t off[LOADS];
    const uint8_t* base[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int row = 16 * (LOADS * wid + i) + (lane >> 2);      // of the slot: A's rows, then B's
        const bool isA = 16 * (LOADS * wid + i) < BM;
        const int r = isA ? min(m0 + row, p.M - 1) - m0 : min(n0 + row - BM, p.N - 1) - n0;
        const int piece = (lane & 3) ^ ((row >> 2) & 3);
        base[i] = reinterpret_cast<const uint8_t*>(isA ? p.A + (size_t)m0 * p.kd : p.B + (size_t)n0 * p.kd);
        off[i] = (uint32_t)r * (uint32_t)(2 * p.kd) + 16u * piece;
    }
    const int steps1 = p.kd / kStep, steps = steps1 * p.planes;
    const size_t plane = (size_t)p.N * p.kd * 2;
    auto stage = [&](int s) {
        const int sc = min(s, steps - 1);
        const int pl = sc >= steps1 ? 1 : 0, ks = sc - pl * steps1;
        uint8_t* slot = slots + (s & (kStages - 1)) * SLOT;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const bool isA = 16 * (LOADS * wid + i) < BM;
            const uint8_t* b = base[i] + (size_t)ks * (2 * kStep) + (isA ? 0 : pl * plane);
            dma16_sv(b, off[i], slot + (LOADS * wid + i) * kDma);
        }
    };
    floatx16_t acc[WM][WN];
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int j = 0; j < WN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    for (int s = 0; s < kStages - 1; ++s) stage(s);

    const int wm = wid >> 1, wn = wid & 1, m = lane & 31, h = lane >> 5;
    const int arow = 32 * WM * wm + m, brow = BM + 32 * WN * wn + m;
    for (int s = 0; s < steps; ++s) {
        wait_vmem<(kStages - 2) * LOADS>();                        // stage s has arrived
        lds_barrier();                                             // for every wave; stage s - 1 is used up
        stage(s + kStages - 1);
        const uint8_t* slot = slots + (s & (kStages - 1)) * SLOT;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            half8_t a[WM], b[WN];
            // rows r, r + 32, ... swap pieces alike: (r >> 2) & 3 is the same
            const int place = 16 * ((2 * kk + h) ^ ((m >> 2) & 3));
#pragma unroll
            for (int i = 0; i < WM; ++i) a[i] = *reinterpret_cast<const half8_t*>(slot + (arow + 32 * i) * 64 + place);
#pragma unroll
            for (int j = 0; j < WN; ++j) b[j] = *reinterpret_cast<const half8_t*>(slot + (brow + 32 * j) * 64 + place);
#pragma unroll
            for (int i = 0; i < WM; ++i)
#pragma unroll
                for (int j = 0; j < WN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    }
    wait_vmem<0>();                                                // loads past the last stage, before the LDS is given up
#pragma unroll
    for (int j = 0; j < WN; ++j) {
        const int n = n0 + 32 * WN * wn + 32 * j + m;
        if (n >= p.N) continue;
        const int en = p.en ? p.en[n] : 0;
        const float rb = p.row_bias ? p.row_bias[n] : 0.f;
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = m0 + 32 * WM * wm + 32 * i + 8 * (e >> 2) + 4 * h + (e & 3);
                if (t >= p.M) continue;
                float v = ldexpf(acc[i][j][e], -(p.et[t] + en)) + rb;
                if (p.residual) v += bf16_bits_to_f32(p.residual[(size_t)t * p.ldr + n]);
                if (p.y_type == MOE_F32) static_cast<float*>(p.y)[(size_t)t * p.ldy + n] = v;
                else static_cast<uint16_t*>(p.y)[(size_t)t * p.ldy + n] = (uint16_t)(pack_bf16(v, 0.f) & 0xFFFFu);
            }
    }
}

namespace {

template <int WM, int WN>
void gemm_go(const GemmArgs& p, hipStream_t s) {
    const int tm = (p.M + 64 * WM - 1) / (64 * WM), tn = (p.N + 64 * WN - 1) / (64 * WN);
    const int blocks = ((tm * tn + 7) / 8) * 8;
    const size_t lds = (size_t)kStages * (64 * WM + 64 * WN) * 2 * kStep;
    hipLaunchKernelGGL((linear_gemm_kernel<WM, WN>), dim3((unsigned)blocks), dim3(256), lds, s, p);
}

void gemm(const GemmArgs& p, hipStream_t s) {
    const int cus = device_cus();
    auto tiles = [&](int b) { return (long)((p.M + b - 1) / b) * ((p.N + b - 1) / b); };
    if (tiles(256) >= cus) gemm_go<4, 4>(p, s);
    else if (tiles(128) >= cus) gemm_go<2, 2>(p, s);
    else gemm_go<1, 1>(p, s);
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// Workspace: A, et, en, then the chunk's weights.
struct Plan {
    int kd, planes, chunk, total;          // chunk: weight rows (forward) or 128-runs (gradient) per GEMM
    size_t et, en, wh, bytes;
};

Plan plan_of(const moe_qmatrix& w, int T, int type, bool grad) {
    Plan p{};
    p.kd = grad ? round_up(w.N, kStep) : w.K;
    p.planes = !grad && type == MOE_F32 ? 2 : 1;
    p.total = grad ? w.K / 128 : w.N;
    const size_t unit = grad ? (size_t)256 * p.kd : (size_t)2 * p.kd * p.planes;       // bytes
    size_t c = kChunkBytes / unit;
    const size_t least = grad ? 2 : 256;                                             // a tile's worth
    c = c < least ? least : c;
    p.chunk = (size_t)p.total < c ? p.total : (int)c;
    p.et = align256((size_t)T * p.kd * 2);
    p.en = p.et + align256((size_t)T * 4);
    p.wh = p.en + align256((size_t)w.N * 4);
    p.bytes = p.wh + align256(unit * p.chunk);
    return p;
}

}  // namespace

size_t linear_gemm_workspace_bytes(const moe_qmatrix& w, int T, int type, bool grad) {
    return plan_of(w, T, type, grad).bytes;
}

int launch_linear_gemm(const LinearArgs& a, hipStream_t s) {
    const Plan pl = plan_of(a.w, a.T, a.y_type, false);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    PrepArgs p{};
    p.w = a.w; p.a = a.x; p.lda = a.ldx; p.a_type = MOE_BF16; p.T = a.T; p.len = a.w.K; p.kd = pl.kd;
    p.ah = reinterpret_cast<uint16_t*>(ws);
    p.et = reinterpret_cast<int32_t*>(ws + pl.et);
    p.en = reinterpret_cast<int32_t*>(ws + pl.en);
    p.wh = reinterpret_cast<uint16_t*>(ws + pl.wh);
    p.planes = pl.planes;
    for (int c0 = 0; c0 < pl.total; c0 += pl.chunk) {
        p.c0 = c0;
        p.cn = pl.total - c0 < pl.chunk ? pl.total - c0 : pl.chunk;
        p.a_blocks = c0 == 0 ? a.T : 0;
        const dim3 grid((unsigned)(p.a_blocks + (p.cn + 15) / 16));
        if (a.w.bits == 4) hipLaunchKernelGGL(linear_prep_kernel<4>, grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL(linear_prep_kernel<2>, grid, dim3(256), 0, s, p);
        GemmArgs g{};
        g.A = p.ah; g.B = p.wh; g.M = a.T; g.N = p.cn; g.kd = pl.kd; g.planes = pl.planes; g.et = p.et; g.en = p.en + c0;
        g.row_bias = a.row_bias ? a.row_bias + c0 : nullptr;
        g.residual = a.residual ? a.residual + c0 : nullptr;
        g.ldr = a.ldr; g.ldy = a.ldy; g.y_type = a.y_type;
        g.y = a.y_type == MOE_F32 ? static_cast<void*>(static_cast<float*>(a.y) + c0)
                                  : static_cast<void*>(static_cast<uint16_t*>(a.y) + c0);
        gemm(g, s);
    }
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_linear_grad_gemm(const LinearGradArgs& a, hipStream_t s) {
    const Plan pl = plan_of(a.w, a.T, a.dy_type, true);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    PrepArgs p{};
    p.w = a.w; p.a = a.dy; p.lda = a.lddy; p.a_type = a.dy_type; p.T = a.T; p.len = a.w.N; p.kd = pl.kd;
    p.ah = reinterpret_cast<uint16_t*>(ws);
    p.et = reinterpret_cast<int32_t*>(ws + pl.et);
    p.en = reinterpret_cast<int32_t*>(ws + pl.en);
    p.wh = reinterpret_cast<uint16_t*>(ws + pl.wh);
    p.planes = 1;
    const dim3 rows((unsigned)((a.w.N + 15) / 16));
    if (a.w.bits == 4) hipLaunchKernelGGL(linear_rows_kernel<4>, rows, dim3(256), 0, s, p);
    else hipLaunchKernelGGL(linear_rows_kernel<2>, rows, dim3(256), 0, s, p);
    for (int c0 = 0; c0 < pl.total; c0 += pl.chunk) {
        p.c0 = c0;
        p.cn = pl.total - c0 < pl.chunk ? pl.total - c0 : pl.chunk;
        p.a_blocks = c0 == 0 ? a.T : 0;
        const dim3 grid((unsigned)(p.a_blocks + p.cn * ((pl.kd + 63) / 64)));
        if (a.w.bits == 4) hipLaunchKernelGGL(linear_grad_prep_kernel<4>, grid, dim3(256), 0, s, p);
        else hipLaunchKernelGGL(linear_grad_prep_kernel<2>, grid, dim3(256), 0, s, p);
        GemmArgs g{};
        g.A = p.ah; g.B = p.wh; g.M = a.T; g.N = 128 * p.cn; g.kd = pl.kd; g.planes = 1; g.et = p.et;
        g.ldy = a.lddx; g.y_type = MOE_BF16; g.y = a.dx + 128 * (size_t)c0;
        gemm(g, s);
    }
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
