// Dense products with one quantised matrix: which kernels a call takes.  The
// streaming kernels read the codes once per 16 or 32 tokens and multiply them as they
// are (linear_dec.hip, linear_grad_dec.hip); the others lay both operands out for a
// dense GEMM first (linear_gemm.hip).
#include <algorithm>

#include "launch_util.h"
#include "linear.h"

namespace moe {

namespace {

// Estimated times of a call (us): fitted to 410 calls of both kinds each way, N = 16 ..
// 30000, K = 128 .. 8192, T = 64 .. 4000, groups of 128 and 32 (64: halfway between), of
// which they are off by 10 to 20 %.  Taking the smaller one costs 0.7 % over taking the
// better kernels each time (a limit on the tokens alone cost 18 %).  Streaming against GEMM:
//   forward  320 x 4096 x 4096 32, 37   448 x 4096 x 4096 43, 39   320 x 8192 x 1152  39, 29
//            64 x 30000 x 1152 30, 47   640 x 512 x 8192  28, 39   4000 x 128 x 8192 33, 53
//   gradient 256 x 4096 x 4096 28, 37   640 x 30000 x 256 48, 109  4000 x 417 x 128   9, 21
//            640 x 2048 x 2048 23, 30  1280 x 8192 x 1152 72, 65   4000 x 512 x 8192 183, 67
double stream_us(const moe_qmatrix& w, int T, bool grad) {
    const double cus = device_cus(), runs = w.K / 128;
    const int fine = w.group_size == 128 ? 0 : w.group_size == 64 ? 1 : 2;
    if (grad) {
        static const double c[3][3] = {{4.9, 0.99, 0.27}, {4.7, 1.7, 0.64}, {4.5, 2.46, 1.0}};
        const double per_cu = runs * ((T + 15) / 16) / cus, rounds = (w.N + 255) / 256;
        return c[fine][0] + c[fine][1] * std::max(1.0, per_cu * rounds) + c[fine][2] * per_cu;
    }
    static const double c[3][4] = {{5.3, 0.105, 0.42, 0.077}, {4.9, 0.12, 0.40, 0.10}, {4.5, 0.134, 0.38, 0.125}};
    const double units = (double)((w.N + 15) / 16) * ((T + 31) / 32) / cus, launches = (w.K + 8191) / 8192;
    return c[fine][0] * launches + c[fine][1] * runs + units * (c[fine][2] + c[fine][3] * runs);
}

double gemm_us(const moe_qmatrix& w, int T, int type, bool grad) {
    const double N = w.N, K = w.K, wide = type == MOE_F32 ? 4 : 2;              // bytes of y or dy
    if (grad)
        return 11.0 + 2.7e-3 * N + 0.22e-6 * 2.5 * N * K + 0.13e-6 * T * N * (wide + 2) + 0.5e-6 * T * K * 2 + 0.81e-9 * 2 * T * N * K;
    const double planes = wide / 2;
    return 8.1 + 3.0e-3 * K * planes + 0.29e-6 * (0.5 + 2 * planes) * N * K + 0.19e-6 * T * K * 4 + 0.51e-6 * T * N * wide +
           0.64e-9 * 2 * planes * T * N * K;
}

bool streams(const moe_qmatrix& w, int T, int type, bool grad) {
    return stream_us(w, T, grad) <= gemm_us(w, T, type, grad);
}

}  // namespace

size_t linear_workspace_bytes(const moe_qmatrix& w, int T, int type, bool grad) {
    if (!streams(w, T, type, grad)) return linear_gemm_workspace_bytes(w, T, type, grad);
    return grad ? linear_grad_dec_workspace_bytes(w, T) : linear_dec_workspace_bytes(w, T);
}

// The needs do not grow with T alone: the gradient's splits fall as tokens rise, and more
// tokens may take kernels that need less.
size_t linear_workspace_bytes_up_to(const moe_qmatrix& w, int T, int type, bool grad) {
    size_t most = 0;
    for (int t = 1; t <= T; ++t) most = std::max(most, linear_workspace_bytes(w, t, type, grad));
    return most;
}

int launch_linear(const LinearArgs& a, hipStream_t s) {
    return streams(a.w, a.T, a.y_type, false) ? launch_linear_dec(a, s) : launch_linear_gemm(a, s);
}

int launch_linear_grad(const LinearGradArgs& a, hipStream_t s) {
    return streams(a.w, a.T, a.dy_type, true) ? launch_linear_grad_dec(a, s) : launch_linear_grad_gemm(a, s);
}

}  // namespace moe
