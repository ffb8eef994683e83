// Arguments and launchers of the low-rank adapters and of the gradients of matrices
// that many tokens share (adapters' factors, the router's weight).
#pragma once

#include "common.h"

namespace moe {

// Which tokens go with which adapter.
struct TokenSets {
    const int32_t* ids;       // [T]: token t's adapter; out of [0, n): none
    const int32_t* rank;      // [n] or NULL: all R
    int T, n, R;
};

// The tokens in order of their adapters, made once a call where there are too many for every
// workgroup to look through the ids itself; tokens without an adapter come last, as set -1.
constexpr int kPlanTile = 64;
struct PlanTileEntry {
    int32_t set, rows;        // rows 0: an empty entry
    int32_t pad[2];
    int32_t token[kPlanTile]; // (past the rows: anything)
};
struct TokenPlan {
    int32_t* order;           // [T]
    PlanTileEntry* tiles;     // [T / kPlanTile + n + 1]
    int4* chunks;             // [T / chunk + n]: (set or -1 for an empty entry, first place, tokens, slot), each adapter's
                              // tokens by up to `chunk`, one entry where it has none; slot: where an adapter with
                              // several has its partial sums, else -1
    int2* joins;              // [n]: an adapter's first slot and their number (0: it has none)
    int chunk;
};
constexpr int kScanTile = 16;

// Up to this many tokens every workgroup looks through the ids itself (4096 x 4096, rank 16, us by
// scans and by the plan: 128 tokens of 4 adapters 8.8 and 14.0, 384 13.6 and 15.0, 512 16.8 and 16.0; 512 of
// 256 adapters 27.3 and 33.3).
constexpr int kScanTokens = 512;

inline int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// The factors' gradients: d[i][r][c] = scale[i] sum over adapter i's tokens of g[t][r] x[t][c].
struct WeightGradCall {
    const float* g;           // [T][ldg]
    int64_t ldg;
    const void* x;            // rows of C: bf16, float32, or int8 codes
    int64_t ldx;
    const float* xscale;      // [T][C / 128] with codes
    int x_type;               // MOE_BF16, MOE_F32, or kCodes
    int C;
    float* out;               // [n][R][C]
    float* bias;              // [R] or NULL: sums of g (one set of tokens)
};
constexpr int kCodes = 2;

// Workspace of a call of T tokens; a smaller call's is no larger.
size_t adapter_workspace_bytes(const moe_adapters& m, int T, bool grad);
int launch_adapter(const moe_adapters& m, int T, const int32_t* ids, const uint16_t* x, int64_t ldx, const void* base,
                   int64_t ldbase, void* y, int64_t ldy, int y_type, float* h, void* ws, hipStream_t s);
struct AdapterGradArgs {
    moe_adapters m;
    int T;
    const int32_t* ids;
    const void* dy;
    int64_t lddy;
    int dy_type;
    const void* x;            // bf16 rows, or a checkpoint's codes with xscale
    int64_t ldx;
    const float* xscale;
    const float* h;
    const uint16_t* dx_base;
    int64_t lddx_base;
    uint16_t* dx;
    int64_t lddx;
    float* da;
    float* db;
    void* ws;
};
int launch_adapter_grad(const AdapterGradArgs& a, hipStream_t s);

size_t router_weight_workspace_bytes(int T, int E, int H);
int launch_router_weight_grad(int T, int E, int H, const float* dlogits, const void* x, int64_t ldx, const float* xscale,
                              float* dw, float* dbias, void* ws, hipStream_t s);

// weight_grad.hip: one launch for up to two matrices over the same tokens, and one more
// where sums were split.
struct WeightGradPlan {
    int chunk;                // tokens a workgroup, at most
    int slots;                // partial sums at most (0: none are split)
    size_t most_floats;       // of the partial sums of any call of up to T tokens
};
constexpr int kLeastChunk = 256, kMostChunk = 1024;
WeightGradPlan weight_grad_plan(int T, int n, int R, int C0, int C1);
int launch_weight_grad(const TokenSets& who, const TokenPlan* plan, const float* scale, const WeightGradPlan& p,
                       const WeightGradCall* calls, int n_calls, float* part, hipStream_t s);

}  // namespace moe
