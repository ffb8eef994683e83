// Arguments and launchers of the dense quantised products.
#pragma once

#include "common.h"

namespace moe {

struct LinearArgs {
    moe_qmatrix w;
    int T;
    const uint16_t* x;
    int64_t ldx;
    const float* row_bias;        // or NULL
    const uint16_t* residual;     // or NULL
    int64_t ldr;
    void* y;
    int64_t ldy;
    int y_type;                   // MOE_BF16, MOE_F32
    void* ws;
};

struct LinearGradArgs {
    moe_qmatrix w;
    int T;
    const void* dy;
    int64_t lddy;
    int dy_type;
    uint16_t* dx;
    int64_t lddx;
    void* ws;
    int32_t* sync;
};

// Workspace of a call of T tokens, and of all calls of 1 .. T tokens.
size_t linear_workspace_bytes(const moe_qmatrix& w, int T, int type, bool grad);
size_t linear_workspace_bytes_up_to(const moe_qmatrix& w, int T, int type, bool grad);
// moe_linear_kernels' answer, for T > 0.
void linear_kernels(const moe_qmatrix& w, int T, int type, bool grad, int32_t* kernels);
int launch_linear(const LinearArgs& a, hipStream_t s);
int launch_linear_grad(const LinearGradArgs& a, hipStream_t s);
// The codes streamed (linear_dec.hip): any T, the matrix read once per 16 or 32 tokens.
struct StreamForm {
    int nt, rt;               // tiles of 16 tokens and of 16 weight rows a workgroup multiplies at once
    int gpw, waves;           // 128-runs of K a wave, waves a workgroup
    int rbu;                  // tiles requested ahead
    int resident;             // workgroups per token block, at most
};
StreamForm stream_form(const moe_qmatrix& w, int T, int runs);
size_t linear_dec_workspace_bytes(const moe_qmatrix& w, int T);
void linear_dec_kernels(const moe_qmatrix& w, int T, int32_t* kernels);
int launch_linear_dec(const LinearArgs& a, hipStream_t s);
// Input gradient, the codes streamed (linear_grad_dec.hip).
int grad_splits(const moe_qmatrix& w, int T);
size_t linear_grad_dec_workspace_bytes(const moe_qmatrix& w, int T);
size_t linear_grad_dec_most_bytes(const moe_qmatrix& w, int T);
int launch_linear_grad_dec(const LinearGradArgs& a, hipStream_t s);
// Both operands laid out for a dense product (linear_gemm.hip).
size_t linear_gemm_workspace_bytes(const moe_qmatrix& w, int T, int type, bool grad);
void linear_gemm_kernels(const moe_qmatrix& w, int T, int type, bool grad, int32_t* kernels);
int launch_linear_gemm(const LinearArgs& a, hipStream_t s);
int launch_linear_grad_gemm(const LinearGradArgs& a, hipStream_t s);

// Estimated times of a call (us); linear_gemm_us stops at the first part past `limit`.
double linear_dec_us(const moe_qmatrix& w, int T);
double linear_grad_dec_us(const moe_qmatrix& w, int T);
double linear_gemm_us(const moe_qmatrix& w, int T, int type, bool grad, double limit);

}  // namespace moe
