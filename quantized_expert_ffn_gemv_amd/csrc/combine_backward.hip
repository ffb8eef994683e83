// The combine in reverse (Flash-MoE page, sec. 3, differentiated): with r the
// row of pair (t, j),
//   dg[t][j] = sum_n dout[t][n] Y[r][n]      (float32)
//   dY[r][n] = bf16(g[t][j] dout[t][n]).
// Bound by memory: Y is read and dY written once, dout once per token (its k
// readers share a workgroup's L1 where they can).  No atomics: a pair's dot
// product belongs to one wave (or one workgroup), summed in a fixed order.
// Measured: 4096 tokens x 2048, 8 picks 59.9 us (4.8 TB/s of 285 MB), 2048 x 8192, 4
// picks 64.3 us (4.7 TB/s), 8 x 5120, 2 picks 2.9 us.
#include "common.h"
#include "row_ops.h"

namespace moe {

namespace {

// Calls of at most this many pairs give each pair a workgroup (8 tokens x 5120, 2 picks:
// 2.9 us against 3.8; 512 x 2048, 8 picks: 10.0 us against 7.9 by waves, 4096 x 2048: 70
// and 60).
constexpr int kCombineFewPairs = 512;

struct CombineGradArgs {
    const uint16_t* dout;     // bf16 [T][H]
    const uint16_t* y;        // bf16 [P][H]
    const int32_t* p2r;       // [P]
    const float* gates;       // [P]
    float* dgates;            // [P]
    uint16_t* dy;             // bf16 [P][H]
    int P, H, k;
};

// The pair's 16-byte pieces c0, c0 + step, ... of its row: returns this lane's
// part of the dot product and, with DY, stores g * dout.
template <bool DY>
__device__ __forceinline__ float combine_grad_row(const uint16_t* dout, const uint16_t* y, uint16_t* dy, float g,
                                                  int pieces, int c0, int step) {
    float dot0 = 0.f, dot1 = 0.f;
    constexpr int U = 4;                       // pieces in flight per lane
    for (int c = c0; c < pieces; c += U * step) {
        uint4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cc = c + u * step;
            const int cl = cc < pieces ? cc : c;
            a[u] = reinterpret_cast<const uint4*>(dout)[cl];
            b[u] = reinterpret_cast<const uint4*>(y)[cl];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cc = c + u * step;
            if (cc >= pieces) break;
            const uint32_t aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
            const uint32_t bw[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a0 = __uint_as_float(aw[i] << 16), a1 = __uint_as_float(aw[i] & 0xFFFF0000u);
                dot0 = fmaf(a0, __uint_as_float(bw[i] << 16), dot0);
                dot1 = fmaf(a1, __uint_as_float(bw[i] & 0xFFFF0000u), dot1);
                if constexpr (DY) o[i] = pack_bf16(g * a0, g * a1);
            }
            if constexpr (DY) reinterpret_cast<uint4*>(dy)[cc] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    return dot0 + dot1;
}

}  // namespace

// LP lanes per pair, a workgroup's 256 / LP pairs consecutive.
template <bool DY, int LP>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineGradArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)blockIdx.x * 4 + (int)(threadIdx.x >> 6));
    const int p = LP == kWave ? wave : wave * (kWave / LP) + lane / LP;
    const bool in = p < a.P;
    const size_t pc = in ? p : a.P - 1;
    const int t = (int)pc / a.k;
    const int row = LP == kWave ? ld_scalar(a.p2r, pc) : a.p2r[pc];
    float dot = 0.f;
    if (in && row >= 0 && row < a.P) {
        const float g = !DY ? 0.f : LP == kWave ? ld_scalar(a.gates, pc) : a.gates[pc];
        dot = combine_grad_row<DY>(a.dout + (size_t)t * a.H, a.y + (size_t)row * a.H,
                                   DY ? a.dy + (size_t)row * a.H : nullptr, g, a.H / 8, lane % LP, LP);
    }
    dot = row_sum<LP>(dot);
    if (in && lane % LP == 0) a.dgates[p] = dot;
}

// One workgroup per pair: for calls with few pairs, whose time is one row's latency.
template <bool DY>
__global__ __launch_bounds__(256) void combine_backward_few_kernel(CombineGradArgs a) {
    __shared__ float part[4];
    const int p = blockIdx.x, t = p / a.k;
    const int row = ld_scalar(a.p2r, (size_t)p);
    const bool ok = row >= 0 && row < a.P;
    float dot = 0.f;
    if (ok) {
        const float g = DY ? ld_scalar(a.gates, (size_t)p) : 0.f;
        dot = combine_grad_row<DY>(a.dout + (size_t)t * a.H, a.y + (size_t)row * a.H,
                                   DY ? a.dy + (size_t)row * a.H : nullptr, g, a.H / 8, (int)threadIdx.x, 256);
    }
    dot = wave_sum_xor(dot, kWave);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
    __syncthreads();
    if (threadIdx.x == 0) a.dgates[p] = (part[0] + part[1]) + (part[2] + part[3]);
}

namespace {

template <int LP>
void combine_go(const CombineGradArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.P + 256 / LP - 1) / (256 / LP)));
    if (a.dy) hipLaunchKernelGGL((combine_backward_kernel<true, LP>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((combine_backward_kernel<false, LP>), grid, dim3(256), 0, s, a);
}

}  // namespace

int launch_combine_backward(const moe_dims& d, const uint16_t* dout, const uint16_t* y, const int32_t* p2r,
                            const float* gates, float* dgates, uint16_t* dy, hipStream_t s) {
    const CombineGradArgs a{dout, y, p2r, gates, dgates, dy, d.T * d.k, d.H, d.k};
    if (a.P == 0) return MOE_OK;
    if (a.P <= kCombineFewPairs) {
        if (dy) hipLaunchKernelGGL(combine_backward_few_kernel<true>, dim3((unsigned)a.P), dim3(256), 0, s, a);
        else hipLaunchKernelGGL(combine_backward_few_kernel<false>, dim3((unsigned)a.P), dim3(256), 0, s, a);
    } else {
        // a wave per pair, or half or a quarter of one where a row has no more 16-byte pieces (H =
        // 128: 5652 tokens, 9 picks 8.4 us against 17.4 by waves; H = 256: 8000 tokens, 8
        // picks 15.2 and 21.4)
        if (a.H <= 128) combine_go<16>(a, s);
        else if (a.H <= 256) combine_go<32>(a, s);
        else combine_go<kWave>(a, s);
    }
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
