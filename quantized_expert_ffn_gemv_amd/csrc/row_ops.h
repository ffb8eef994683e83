// Row-wise helpers of the gradient and loss kernels: packed bf16 rounding,
// the exponential of softmax rows, reductions over the lanes that share a row, and the arrival ticket by which
// the last workgroup of a group joins the others' partial sums.
#pragma once

#include "common.h"

namespace moe {

typedef float float2v_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Two floats rounded to bf16 (nearest even; NaN stays NaN), lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const float2v_t v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

template <int CTRL>
__device__ __forceinline__ float dpp_mov(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xF, 0xF, true));
}

// op over the LANES lanes (a power of two, 4 .. 64) that share a row, in every
// one of them.  Within 16 lanes by DPP: quad xor 1, quad xor 2, then the mirror
// of 8 and of 16 lanes, whose partner groups hold equal values by then.
template <int LANES, typename OP>
__device__ __forceinline__ float row_reduce(float v, OP op) {
    v = op(v, dpp_mov<0xB1>(v));
    v = op(v, dpp_mov<0x4E>(v));
    if constexpr (LANES >= 8) v = op(v, dpp_mov<0x141>(v));
    if constexpr (LANES >= 16) v = op(v, dpp_mov<0x140>(v));
    if constexpr (LANES >= 32) v = op(v, __shfl_xor(v, 16, kWave));
    if constexpr (LANES >= 64) v = op(v, __shfl_xor(v, 32, kWave));
    return v;
}

template <int LANES>
__device__ __forceinline__ float row_max(float v) {
    return row_reduce<LANES>(v, [](float a, float b) { return fmaxf(a, b); });
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
    return row_reduce<LANES>(v, [](float a, float b) { return a + b; });
}

// e^d, d <= 0, to 2 ulp: the hardware's power of two of t = d log2 e rounded, times the
// factor 1 + r ln 2 for what the rounding left out, r = d log2 e - t (log2 e in two
// parts).  Without the factor a small p was off by |d| 2^-24.  Below 2^-126 the
// hardware gives 0, and d is cut off there (an infinite one would make r NaN; a NaN stays).
__device__ __forceinline__ float exp_down(float d) {
    constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f;   // log2 e - (float) 1.44269504
    d = d < -128.f ? -128.f : d;
    const float t = d * kLog2e;
    const float r = fmaf(d, kLog2eRest, fmaf(d, kLog2e, -t));
    return __builtin_amdgcn_exp2f(t) * fmaf(r, 0.693147181f, 1.f);
}

// Device-scope accesses for data handed between workgroups of one launch: they
// bypass the caches that are not coherent between compute dies.
template <typename T>
__device__ __forceinline__ void put_device(T* p, T v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <typename T>
__device__ __forceinline__ T get_device(const T* p) {
    return __hip_atomic_load(const_cast<T*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Arrive at `counter`, n arrivals in all; true in every thread of the last
// workgroup to arrive, which leaves the counter at zero.  The workgroup's
// device-scope stores have completed before its arrival counts (the full wait),
// so the last one reads every other's with device-scope loads.
__device__ __forceinline__ bool arrive_last(int32_t* counter, int n, int* flag) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
        if (last) put_device(counter, (int32_t)0);
        *flag = last;
    }
    __syncthreads();
    return *flag != 0;
}

}  // namespace moe
