// Dense products with one quantised matrix: which kernels a call takes.  With few
// tokens the codes are streamed once per 16 or 32 tokens and multiplied as they
// are (linear_dec.hip, linear_grad_dec.hip); with many, both operands are laid out
// for a dense GEMM first (linear_gemm.hip).
#include "linear.h"

namespace moe {

namespace {

constexpr int kDecTokens = 128;
constexpr int kGradDecTokens = 128;

}  // namespace

size_t linear_workspace_bytes(const moe_qmatrix& w, int T, int type, bool grad) {
    if (T > (grad ? kGradDecTokens : kDecTokens)) return linear_gemm_workspace_bytes(w, T, type, grad);
    return grad ? linear_grad_dec_workspace_bytes(w, T) : linear_dec_workspace_bytes(w, T);
}

int launch_linear(const LinearArgs& a, hipStream_t s) {
    return a.T > kDecTokens ? launch_linear_gemm(a, s) : launch_linear_dec(a, s);
}

int launch_linear_grad(const LinearGradArgs& a, hipStream_t s) {
    return a.T > kGradDecTokens ? launch_linear_grad_gemm(a, s) : launch_linear_grad_dec(a, s);
}

}  // namespace moe
