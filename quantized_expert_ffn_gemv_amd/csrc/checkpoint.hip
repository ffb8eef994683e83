// Activations kept in 8 bits: 128 columns share a scale,
//   scale = max |x| / 127,   q = round(127 x / max |x|), ties to even,   x^ = q scale,
// and the gates' gradient of the combine from such rows.
//
// q is the rounding of the exact quotient 127 x / max |x|.  With 8-bit significands X and A
// that is 127 X 2^-k / A; off a tie (n + 1/2) it is off by 2^-k / (2 A) at least, 1 / 32385 of
// itself, and a tie has 8 bits.  A float32 quotient (2^-23 of itself off) rounded to 18 bits
// therefore lies on a tie where the exact one does, and on its side where not.
//
// All three kernels are bound by memory: 3 bytes an element saving or restoring, 1 (and
// dout, once a token) for the gates' gradient.  32768 x 2048 saved and restored: 82 us, 5.0 TB/s,
// a large copy's rate; the gates of 4096 tokens x 8 picks x 2048: 18.1 us, 4.8 TB/s.  Groups go four to
// 16 lanes, so that a lane has 64 bytes in flight; a token's picks are neighbouring waves, which
// share its dout through the caches.
#include "common.h"
#include "row_ops.h"

namespace moe {

namespace {

constexpr int kGroups = 4;                 // groups of 128 columns that 16 lanes have in flight

__device__ __forceinline__ uint32_t code_of(float x, float pre, float inv) {
    const float q = __uint_as_float((__float_as_uint(x * pre * inv) + 0x20u) & ~0x3Fu);
    return (uint32_t)(int)rintf(q) & 0xFFu;
}

}  // namespace

// 16 lanes a group of 128, 8 columns each.
__global__ __launch_bounds__(256) void checkpoint_save_kernel(const uint16_t* x, int64_t ldx, int8_t* q, float* scale,
                                                              int64_t groups, int per_row) {
    const int c = threadIdx.x & 15;
    const int64_t g0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 16;
    const int64_t stride = (int64_t)gridDim.x * 16;
    uint4 v[kGroups];
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
        const int64_t g = min(g0 + u * stride, groups - 1), row = g / per_row;
        __builtin_memcpy(&v[u], x + row * ldx + (g - row * per_row) * 128 + 8 * c, 16);
    }
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
        const int64_t g = g0 + u * stride;
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        // the largest magnitude, as whole numbers: an infinity and a NaN are above all others
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) most = max(most, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t o = k == 0 ? __builtin_amdgcn_update_dpp(0, most, 0xB1, 0xF, 0xF, true)
                               : k == 1 ? __builtin_amdgcn_update_dpp(0, most, 0x4E, 0xF, 0xF, true)
                               : k == 2 ? __builtin_amdgcn_update_dpp(0, most, 0x141, 0xF, 0xF, true)
                                        : __builtin_amdgcn_update_dpp(0, most, 0x140, 0xF, 0xF, true);
            most = max(most, o);
        }
        const float top = __uint_as_float(most);
        const bool number = most < 0x7F800000u;
        // a tiny maximum is brought up first (127 / max would overflow)
        const float pre = top < 0x1p-100f ? 0x1p100f : 1.f;
        const float inv = number && most ? 127.f / (top * pre) : 0.f;
        uint32_t o[2] = {0, 0};
        if (number)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i >> 1] |= (code_of(__uint_as_float(w[i] << 16), pre, inv) | code_of(__uint_as_float(w[i] & 0xFFFF0000u), pre, inv) << 8) << (16 * (i & 1));
        if (g >= groups) break;
        *reinterpret_cast<uint2*>(q + g * 128 + 8 * c) = make_uint2(o[0], o[1]);
        if (c == 0) scale[g] = number ? top / 127.f : NAN;
    }
}

// 8 columns a lane.
__global__ __launch_bounds__(256) void checkpoint_restore_kernel(uint16_t* x, int64_t ldx, const int8_t* q, const float* scale,
                                                                 int64_t groups, int per_row) {
    const int c = threadIdx.x & 15;
    const int64_t g0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 16;
    const int64_t stride = (int64_t)gridDim.x * 16;
    uint2 v[kGroups];
    float s[kGroups];
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
        const int64_t g = min(g0 + u * stride, groups - 1);
        v[u] = *reinterpret_cast<const uint2*>(q + g * 128 + 8 * c);
        s[u] = scale[g];
    }
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
        const int64_t g = g0 + u * stride, row = g / per_row;
        if (g >= groups) break;
        const uint32_t w[2] = {v[u].x, v[u].y};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t pair = w[i >> 1] >> (16 * (i & 1));
            o[i] = pack_bf16((float)(int8_t)pair * s[u], (float)(int8_t)(pair >> 8) * s[u]);
        }
        __builtin_memcpy(x + row * ldx + (g - row * per_row) * 128 + 8 * c, o, 16);
    }
}

namespace {

struct GatesSavedArgs {
    const uint16_t* dout;     // bf16 [T][H]
    const int8_t* q;          // [rows][H]
    const float* scale;       // [rows][H / 128]
    const int32_t* p2r;       // [P]
    const float* gates;       // [P]
    float* dgates;            // [P]
    uint16_t* dy;             // bf16 [P][H] or NULL
    int P, H, k;
};

// Pieces of 8 columns c0, c0 + step, ... of the pair's row: this lane's part of the dot product;
// with DY also g * dout.
template <bool DY>
__device__ __forceinline__ float gates_row(const uint16_t* dout, const int8_t* y, const float* scale, uint16_t* dy, float g,
                                           int pieces, int c0, int step) {
    float dot = 0.f;
    constexpr int U = 4;
    for (int c = c0; c < pieces; c += U * step) {
        uint4 a[U];
        uint2 b[U];
        float s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cc = c + u * step;
            const int cl = cc < pieces ? cc : c;
            a[u] = reinterpret_cast<const uint4*>(dout)[cl];
            b[u] = reinterpret_cast<const uint2*>(y)[cl];
            s[u] = scale[cl >> 4];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int cc = c + u * step;
            if (cc >= pieces) break;
            const uint32_t aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
            const uint32_t bw[2] = {b[u].x, b[u].y};
            uint32_t o[4];
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t pair = bw[i >> 1] >> (16 * (i & 1));
                const float a0 = __uint_as_float(aw[i] << 16), a1 = __uint_as_float(aw[i] & 0xFFFF0000u);
                part = fmaf(a0, (float)(int8_t)pair, part);
                part = fmaf(a1, (float)(int8_t)(pair >> 8), part);
                if constexpr (DY) o[i] = pack_bf16(g * a0, g * a1);
            }
            dot = fmaf(part, s[u], dot);
            if constexpr (DY) reinterpret_cast<uint4*>(dy)[cc] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    return dot;
}

}  // namespace

// LP lanes a pair, as many as have a piece.  (Few pairs by a workgroup each were no faster: 8 tokens x 8 picks x
// 2048 4.7 to 5.9 us both, 64 x 5120 5.2 to 5.5, 16 x 8192 4.9 to 5.3 against 5.8.)
template <bool DY, int LP>
__global__ __launch_bounds__(256) void gates_saved_kernel(GatesSavedArgs a) {
    const int p = ((int)blockIdx.x * 256 + (int)threadIdx.x) / LP, sub = threadIdx.x % LP;
    const bool in = p < a.P;
    const int pc = in ? p : a.P - 1, t = pc / a.k, row = a.p2r[pc];
    float dot = 0.f;
    if (in && row >= 0 && row < a.P)
        dot = gates_row<DY>(a.dout + (size_t)t * a.H, a.q + (size_t)row * a.H, a.scale + (size_t)row * (a.H / 128),
                            DY ? a.dy + (size_t)row * a.H : nullptr, DY ? a.gates[pc] : 0.f, a.H / 8, sub, LP);
    dot = row_sum<LP>(dot);
    if (in && sub == 0) a.dgates[p] = dot;
}

namespace {

template <int LP>
void gates_go(const GatesSavedArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.P + 256 / LP - 1) / (256 / LP)));
    if (a.dy) hipLaunchKernelGGL((gates_saved_kernel<true, LP>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((gates_saved_kernel<false, LP>), grid, dim3(256), 0, s, a);
}

unsigned save_blocks(int64_t groups) { return (unsigned)((groups + 16 * kGroups - 1) / (16 * kGroups)); }

}  // namespace

int launch_checkpoint_save(const moe_checkpoint& c, const uint16_t* x, int64_t ldx, hipStream_t s) {
    const int64_t groups = (int64_t)c.rows * (c.K / 128);
    hipLaunchKernelGGL(checkpoint_save_kernel, dim3(save_blocks(groups)), dim3(256), 0, s, x, ldx, c.q, c.scale, groups, c.K / 128);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_checkpoint_restore(const moe_checkpoint& c, uint16_t* x, int64_t ldx, hipStream_t s) {
    const int64_t groups = (int64_t)c.rows * (c.K / 128);
    hipLaunchKernelGGL(checkpoint_restore_kernel, dim3(save_blocks(groups)), dim3(256), 0, s, x, ldx, c.q, c.scale, groups, c.K / 128);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_combine_backward_saved(const moe_dims& d, const uint16_t* dout, const moe_checkpoint& y, const int32_t* p2r,
                                  const float* gates, float* dgates, uint16_t* dy, hipStream_t s) {
    const GatesSavedArgs a{dout, y.q, y.scale, p2r, gates, dgates, dy, d.T * d.k, d.H, d.k};
    if (a.P == 0) return MOE_OK;
    if (a.H <= 128) gates_go<16>(a, s);
    else if (a.H <= 256) gates_go<32>(a, s);
    else gates_go<64>(a, s);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
