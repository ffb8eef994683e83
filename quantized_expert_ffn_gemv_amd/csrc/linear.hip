// Dense products with one quantised matrix: y = x W^T and its input gradient
// dx = dy W, w[n][k] = q[n][k] s[n][g] + b[n][g] (the FMA form of the Flash-MoE
// page, sec. 2, with the group-major codes of moe_qweights).
#include "linear.h"
#include "row_ops.h"

namespace moe {

namespace {

constexpr int kTok = 8;            // tokens per pass
constexpr int kDecTokens = 128;
constexpr int kGradDecTokens = 64;

// Code k (0..127) of row n's piece of a 128-wide run.
template <int BITS>
__device__ __forceinline__ float code_at(const uint8_t* piece, int k) {
    if constexpr (BITS == 4) return (float)((piece[k >> 1] >> (4 * (k & 1))) & 15);
    else return (float)((piece[k >> 2] >> (2 * (k & 3))) & 3);
}

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int type) {
    return type == MOE_F32 ? static_cast<const float*>(p)[i]
                           : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

}  // namespace

template <int BITS>
__global__ __launch_bounds__(128) void linear_grad_simple_kernel(LinearGradArgs a) {
    const int k = (int)blockIdx.x * 128 + (int)threadIdx.x, t0 = (int)blockIdx.y * kTok;
    const int ngs = a.w.K / a.w.group_size;
    float acc[kTok] = {};
    for (int n = 0; n < a.w.N; ++n) {
        const uint8_t* piece = a.w.q + ((size_t)blockIdx.x * a.w.N + n) * (16 * BITS);
        const size_t gi = (size_t)n * ngs + k / a.w.group_size;
        const float w = fmaf(code_at<BITS>(piece, (int)threadIdx.x), f16_bits_to_f32(a.w.scale[gi]), f16_bits_to_f32(a.w.bias[gi]));
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int t = min(t0 + i, a.T - 1);
            acc[i] = fmaf(load_elem(a.dy, (int64_t)t * a.lddy + n, a.dy_type), w, acc[i]);
        }
    }
    for (int i = 0; i < kTok; ++i)
        if (t0 + i < a.T) a.dx[(size_t)(t0 + i) * a.lddx + k] = (uint16_t)f32_to_bf16_bits(acc[i]);
}

size_t linear_workspace_bytes(const moe_qmatrix& w, int T, int type, bool grad) {
    if (T > (grad ? kGradDecTokens : kDecTokens)) return linear_gemm_workspace_bytes(w, T, type, grad);
    return grad ? 0 : linear_dec_workspace_bytes(w, T);
}

int launch_linear(const LinearArgs& a, hipStream_t s) {
    return a.T > kDecTokens ? launch_linear_gemm(a, s) : launch_linear_dec(a, s);
}

int launch_linear_grad(const LinearGradArgs& a, hipStream_t s) {
    if (a.T > kGradDecTokens) return launch_linear_grad_gemm(a, s);
    const dim3 grid((unsigned)(a.w.K / 128), (unsigned)((a.T + kTok - 1) / kTok));
    if (a.w.bits == 4) hipLaunchKernelGGL(linear_grad_simple_kernel<4>, grid, dim3(128), 0, s, a);
    else hipLaunchKernelGGL(linear_grad_simple_kernel<2>, grid, dim3(128), 0, s, a);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
