// Device helpers of the adapters' kernels: which tokens a workgroup has, float32
// operands as bf16 parts, and 8 x 8 blocks of bf16 turned in registers.
#pragma once

#include "adapters.h"
#include "mfma_ops.h"
#include "row_ops.h"

namespace moe {

__device__ __forceinline__ int set_of(const int32_t* ids, int t, int n) {
    const int i = ids[t];
    return (unsigned)i < (unsigned)n ? i : -1;
}

// Tokens of the tile that token `leader` leads, into `list` (this wave's own, kScanTile ints):
// the tokens of its set from it on, where its place among them is a multiple of kScanTile.
// Returns their number, 0 where it leads none.  Every wave looks through all ids: T up to kScanTokens.
__device__ __forceinline__ int scan_tile(const TokenSets& who, int leader, int& set, int* list) {
    const int lane = threadIdx.x & 63;
    set = __builtin_amdgcn_readfirstlane(set_of(who.ids, leader, who.n));
    int id[kScanTokens / 64];
#pragma unroll
    for (int c = 0; c < kScanTokens / 64; ++c) {
        if (c * 64 >= who.T) break;
        id[c] = who.ids[min(c * 64 + lane, who.T - 1)];
    }
    int count = 0, first = 0;
#pragma unroll
    for (int c = 0; c < kScanTokens / 64; ++c) {
        if (c * 64 >= who.T) break;
        const int t = c * 64 + lane;
        const int mine = (unsigned)id[c] < (unsigned)who.n ? id[c] : -1;
        const bool same = t < who.T && mine == set;
        const uint64_t mask = __ballot(same);
        const int place = count + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
        if (c == leader >> 6) {
            first = __builtin_amdgcn_readlane(place, leader & 63);
            if (first % kScanTile) return 0;
        }
        const int at = place - first;
        if (same && t >= leader && at < kScanTile) list[at] = t;
        count += __popcll(mask);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    return min(count - first, kScanTile);
}

// 8 floats as three bf16 operands of 4 words that add up to them: the upper 8 bits of each, the next 8
// of what is left, and the rest, cut and not rounded, which leaves nothing of a float32's 24 bits.  (An
// infinity's rest is a NaN.)
__device__ __forceinline__ void bf16_parts(const float (&v)[8], uint32_t (&out)[3][4]) {
    constexpr uint32_t HI = 0x07060302u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
        out[0][i] = __builtin_amdgcn_perm(b, a, HI);
#pragma unroll
        for (int p = 1; p < 3; ++p) {
            a = __float_as_uint(__uint_as_float(a) - __uint_as_float(a & 0xFFFF0000u));
            b = __float_as_uint(__uint_as_float(b) - __uint_as_float(b & 0xFFFF0000u));
            out[p][i] = __builtin_amdgcn_perm(b, a, HI);
        }
    }
}

// rows[i]: 8 bf16 columns of row i -> out[j]: column 4 half + j of the 8 rows, in row order.
__device__ __forceinline__ void turn4(const uint4* rows, int half, uint32_t (&out)[4][4]) {
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint32_t a = reinterpret_cast<const uint32_t*>(&rows[2 * p])[2 * half + d];
            const uint32_t b = reinterpret_cast<const uint32_t*>(&rows[2 * p + 1])[2 * half + d];
            out[2 * d][p] = __builtin_amdgcn_perm(b, a, 0x05040100u);
            out[2 * d + 1][p] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        }
}

__device__ __forceinline__ void turn8(const uint4 (&rows)[8], uint32_t (&out)[8][4]) {
    turn4(rows, 0, reinterpret_cast<uint32_t (&)[4][4]>(out[0]));
    turn4(rows, 1, reinterpret_cast<uint32_t (&)[4][4]>(out[4]));
}

// Columns come 8 to a lane.  Where fewer are left (C no multiple of 8; C is 8 or more) the
// lane takes the last 8 of the row, of which the first `shift` are its neighbour's (8: all): loads
// stay whole and behind no branch.
__device__ __forceinline__ int first_of_8(int col, int C) { return min(col, C - 8); }

// Masks for the words of 8 bf16, of which the first `shift` are to read as 0.
__device__ __forceinline__ void mask_first(int shift, uint32_t (&m)[4]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) m[d] = (2 * d >= shift ? 0xFFFFu : 0u) | (2 * d + 1 >= shift ? 0xFFFF0000u : 0u);
}

__device__ __forceinline__ uint4 load_bf16x8(const uint16_t* p) {     // any alignment of 2
    uint4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

}  // namespace moe
