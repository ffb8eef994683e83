// Dense products with one quantised matrix: which kernels a call takes.  The
// streaming kernels read the codes once per 16 or 32 tokens and multiply them as they
// are (linear_dec.hip, linear_grad_dec.hip); the others lay both operands out for a
// dense GEMM first (linear_gemm.hip).
#include <algorithm>

#include "launch_util.h"
#include "linear.h"

namespace moe {

namespace {

// By the estimated times of both kinds, fitted to 3500 calls of each (T 8 .. 65536, N 1 ..
// 983599, K 128 .. 32768, both directions, widths, groups and types), of which they are off by
// 13 to 22 %.  Taking the smaller one costs 0.6 % over taking the faster kernels each time, 50 to
// 70 % at most (streaming always: 9 % forward, 15 % gradient; laying out always: 54 and 68 %).
// Streaming against laying out, us (bf16, 4 bits, groups of 128 unless said):
//   forward  512 x 4096 x 4096 45, 58    700 x 4096 x 4096 59, 80   1500 x 4096 x 4096 111, 113
//            1024 x 2048 x 2048 34, 38   4096 x 4096 x 1024 101, 71   100 x 325 x 9216  20, 31
//            1000 x 2500 x 640 (groups of 64) 32, 28; float32 result 32, 29
//            float32 results: 1024 x 8192 x 2048 93, 78   4096 x 8192 x 2048 396, 236   1024 x 49999 x 4096 755, 1011
//   gradient 1749 x 388 x 640 (groups of 32) 27, 18   304 x 6 x 16768 18, 24
//            1000 x 2500 x 640 (groups of 64) 36, 34   148 x 25955 x 10880 (groups of 32) 991, 1146
//            253 x 24471 x 4736 270, 372; float32 dy: 1024 x 49999 x 4096 1656, 1493   4096 x 8192 x 2048 528, 410
bool streams(const moe_qmatrix& w, int T, int type, bool grad) {
    const double us = grad ? linear_grad_dec_us(w, T) : linear_dec_us(w, T);
    return us <= linear_gemm_us(w, T, type, grad, us);
}

}  // namespace

size_t linear_workspace_bytes(const moe_qmatrix& w, int T, int type, bool grad) {
    if (!streams(w, T, type, grad)) return linear_gemm_workspace_bytes(w, T, type, grad);
    return grad ? linear_grad_dec_workspace_bytes(w, T) : linear_dec_workspace_bytes(w, T);
}

// Laid-out products never need less for more tokens, so the first number of tokens from above
// that takes them says whether their need counts; the streamed ones' does not grow with T alone
// (the gradient's splits fall).
size_t linear_workspace_bytes_up_to(const moe_qmatrix& w, int T, int type, bool grad) {
    size_t most = grad ? linear_grad_dec_most_bytes(w, T) : linear_dec_workspace_bytes(w, T);
    for (int t = T; t >= 1; --t)
        if (!streams(w, t, type, grad)) return std::max(most, linear_gemm_workspace_bytes(w, T, type, grad));
    return most;
}

void linear_kernels(const moe_qmatrix& w, int T, int type, bool grad, int32_t* kernels) {
    if (!streams(w, T, type, grad)) {
        kernels[0] = MOE_LINEAR_LAID_OUT;
        linear_gemm_kernels(w, T, type, grad, kernels);
        return;
    }
    kernels[0] = MOE_LINEAR_STREAMED;
    if (grad) kernels[1] = grad_splits(w, T);
    else linear_dec_kernels(w, T, kernels);
}

int launch_linear(const LinearArgs& a, hipStream_t s) {
    return streams(a.w, a.T, a.y_type, false) ? launch_linear_dec(a, s) : launch_linear_gemm(a, s);
}

int launch_linear_grad(const LinearGradArgs& a, hipStream_t s) {
    return streams(a.w, a.T, a.dy_type, true) ? launch_linear_grad_dec(a, s) : launch_linear_grad_gemm(a, s);
}

}  // namespace moe
