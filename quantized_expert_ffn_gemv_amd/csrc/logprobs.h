// Arguments and launchers of the token probabilities.
#pragma once

#include "common.h"

namespace moe {

struct LogprobArgs {
    int T, V;
    const void* logits;
    int64_t ld;
    int type;
    const int32_t* tokens;
    float* logp;
    float* stats;
    float* entropy;           // or NULL
    int n_top;
    int32_t* top_ids;
    float* top_logp;
    float* part;              // [T][splits][part_words]
    int32_t* sync;
    int splits, pieces;       // workgroups a row; 16-byte pieces of a row each
};

struct LogprobGradArgs {
    int T, V;
    const void* logits;
    int64_t ld;
    int type;
    const int32_t* tokens;
    const float* stats;
    const float* dlogp;       // or NULL
    const float* entropy;
    const float* dentropy;    // or NULL
    void* dlogits;
    int64_t ldg;
    int grad_type;
};

// Workspace of a call of T tokens, and of all calls of 1 .. T tokens.
size_t logprobs_workspace_of(int T, int V, int n_top);
size_t logprobs_workspace_bytes(int T, int V, int n_top);
int launch_logprobs(LogprobArgs a, hipStream_t s);
int launch_logprobs_grad(const LogprobGradArgs& a, hipStream_t s);

}  // namespace moe
