// Dense products with one quantised matrix: which kernels a call takes.  With few
// tokens the codes are streamed once per 16 or 32 tokens and multiplied as they
// are (linear_dec.hip, linear_grad_dec.hip); with many, both operands are laid out
// for a dense GEMM first (linear_gemm.hip).
#include "linear.h"

namespace moe {

namespace {

// Most tokens that the streaming kernels take, measured at 4096 x 4096 (us, streaming
// against GEMM) and alike from 2048 x 2048 to 20000 x 4096:
//   forward, groups of 128 and 64: 320 tokens 32 against 37 and 36 against 37, 448
//   tokens of groups of 64 43 against 38; groups of 32 (four folds a run): 192 tokens
//   30 against 33, 256 33 against 31; float32 results cost the GEMM a second pass over
//   the weights: 640 tokens 52 against 104;
//   gradient, groups of 128: 256 tokens 28 against 37, 448 48 against 42; finer groups
//   (every group's dy times scale meets all columns): 128 tokens 25 (64) and 35 (32)
//   against 38, 192 tokens 42 and 63 against 37.
int most_streamed(const moe_qmatrix& w, int type, bool grad) {
    if (grad) return w.group_size == 128 ? 256 : 128;
    if (w.group_size == 32) return 224;
    return type == MOE_F32 ? 640 : 320;
}

}  // namespace

size_t linear_workspace_bytes(const moe_qmatrix& w, int T, int type, bool grad) {
    if (T > most_streamed(w, type, grad)) return linear_gemm_workspace_bytes(w, T, type, grad);
    return grad ? linear_grad_dec_workspace_bytes(w, T) : linear_dec_workspace_bytes(w, T);
}

// The streaming kernels' needs do not grow with T alone: the splits of the summed
// axis fall as tokens rise.  (The GEMM's do.)
size_t linear_workspace_bytes_up_to(const moe_qmatrix& w, int T, int type, bool grad) {
    const int streamed = most_streamed(w, type, grad);
    size_t most = linear_workspace_bytes(w, T, type, grad);
    for (int t = 1; t <= streamed && t < T; ++t) {
        const size_t n = linear_workspace_bytes(w, t, type, grad);
        most = n > most ? n : most;
    }
    return most;
}

int launch_linear(const LinearArgs& a, hipStream_t s) {
    return a.T > most_streamed(a.w, a.y_type, false) ? launch_linear_gemm(a, s) : launch_linear_dec(a, s);
}

int launch_linear_grad(const LinearGradArgs& a, hipStream_t s) {
    return a.T > most_streamed(a.w, a.dy_type, true) ? launch_linear_grad_gemm(a, s) : launch_linear_grad_dec(a, s);
}

}  // namespace moe
