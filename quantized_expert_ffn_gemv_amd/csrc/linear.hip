// Dense products with one quantised matrix: which kernels a call takes.  The
// streaming kernels read the codes once per 16 or 32 tokens and multiply them as they
// are (linear_dec.hip, linear_grad_dec.hip); the others lay both operands out for a
// dense GEMM first (linear_gemm.hip).
#include <algorithm>

#include "launch_util.h"
#include "linear.h"

namespace moe {

namespace {

// Estimated times of a call (us): fitted to 410 calls of both kinds, N = 16 .. 30000, K =
// 128 .. 8192, T = 64 .. 4000, groups of 128 and 32 (64: halfway between), of which they
// are off by 13 to 20 %.  Taking the smaller one costs 1 % over taking the better kernels
// each time (a limit on the tokens alone cost 15 %).  Streaming against GEMM:
//   forward  320 x 4096 x 4096 32, 37   448 x 4096 x 4096 43, 39   320 x 8192 x 1152 39, 29
//            64 x 30000 x 1152 30, 47   640 x 512 x 8192  27, 32   4000 x 128 x 8192 33, 48
//   gradient 256 x 4096 x 4096 28, 37   640 x 30000 x 256 47, 61   4000 x 417 x 128   9, 21
//            640 x 2048 x 2048 23, 31  1280 x 8192 x 1152 70, 62   4000 x 512 x 8192 180, 68
double stream_us(const moe_qmatrix& w, int T, bool grad) {
    const double cus = device_cus();
    const int runs = w.K / 128, fine = w.group_size == 128 ? 0 : w.group_size == 64 ? 1 : 2;
    if (grad) {
        static const double c[3][3] = {{4.9, 0.965, 0.28}, {4.7, 1.69, 0.66}, {4.55, 2.41, 1.04}};
        const double per_cu = (double)runs * ((T + 15) / 16) / cus, rounds = (w.N + 255) / 256;
        return c[fine][0] + c[fine][1] * std::max(1.0, per_cu * rounds) + c[fine][2] * per_cu;
    }
    static const double c[3][4] = {{5.7, 0.087, 0.22, 0.060}, {5.3, 0.103, 0.21, 0.0725}, {4.9, 0.119, 0.19, 0.085}};
    // a tile's time goes with the busiest SIMD's groups (whole waves of linear_dec.hip's groups a wave)
    const int groups = runs <= 8 ? 1 : runs <= 16 ? 2 : runs <= 32 ? 4 : runs <= 48 ? 6 : 8;
    const int waves = (std::min(runs, 64) + groups - 1) / groups, load = groups * 4 * ((waves + 3) / 4) * (runs > 32 ? 2 : 1);
    const double units = (double)((w.N + 15) / 16) * ((T + 31) / 32) / cus, launches = (runs + 63) / 64;
    return launches * (c[fine][0] + units * (c[fine][2] + c[fine][3] * load)) + c[fine][1] * runs;
}

double gemm_us(const moe_qmatrix& w, int T, int type, bool grad) {
    const double N = w.N, K = w.K, wide = type == MOE_F32 ? 4 : 2;              // bytes of y or dy
    if (grad)
        return 11.7 + 0.39e-3 * N + 0.46e-6 * 2.5 * N * K + 0.31e-6 * T * N * (wide + 2) + 0.48e-6 * T * K * 2 + 0.84e-9 * 2 * T * N * K;
    const double planes = wide / 2;
    return 9.3 + 1.05e-3 * K * planes + 0.35e-6 * (0.5 + 2 * planes) * N * K + 0.25e-6 * T * K * 4 + 0.46e-6 * T * N * wide +
           0.82e-9 * 2 * planes * T * N * K;
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
