// Internal declarations of the operators around the products and the logits:
// layer norm (layernorm.hip), rotary positions (rotary.hip) and the router of
// a mixture-of-experts layer (router.hip).  The entry points are in
// api_block.hip.  Nothing here is part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon_internal.h"

namespace muon {

// ---- layer norm --------------------------------------------------------------
constexpr int kNormMaxCols = 16384;  // a row lies in the registers of one workgroup

// One call as the kernels see it.  Row r is head r % heads of token r / heads.
struct NormCall {
    const void* x;
    const void* dy;   // gradient only
    void* out;        // y, or dx (null: not wanted)
    int64_t x_token, x_head, dy_token, dy_head, out_token, out_head;
    const void* weight;  // null: ones
    const void* bias;    // forward only; null: zeros
    float* mean;         // forward: written, gradient: read; null: not wanted, zero
    float* rstd;
    int32_t rows, heads, cols;
    int32_t bf16, weight_bf16, center;
    int32_t nontemporal;  // set by the launch
    float eps;
    // gradient only
    void* dweight;  // null: not wanted
    void* dbias;
    float* partials;  // [weight, bias][block][cols]
    int32_t grad_bf16, accumulate;
};

hipError_t launch_norm_forward(const NormCall& c, int cus, hipStream_t st);
// Workgroups of the gradient's first pass, and with them its partial sums: from
// the sizes alone.
int norm_grad_blocks(int32_t rows, int32_t cols, bool bf16, int cus);
hipError_t launch_norm_grad(const NormCall& c, int cus, hipStream_t st);

// ---- rotary positions ----------------------------------------------------------
constexpr int kRotaryTensors = 4;
constexpr int kRotaryPairs = 2048;  // the sines and cosines of one token, at least, lie in LDS

struct RotaryTensor {
    const void* x;
    void* y;
    int64_t x_token, x_head, y_token, y_head;
    int32_t heads;
};
struct RotaryCall {
    RotaryTensor t[kRotaryTensors];
    int32_t count;
    const int32_t* positions;
    const double* frequencies;
    int32_t tokens, head_dim, first, pairs;
    int32_t interleaved, transpose, bf16;
    float scale;
};
// whether every workgroup of the call can be numbered
bool rotary_fits(const RotaryCall& c);
hipError_t launch_rotary(const RotaryCall& c, hipStream_t st);

// ---- router ----------------------------------------------------------------------
constexpr int kRouterMaxExperts = 1024;  // as many as the products take
constexpr int kRouterMaxChoices = 32;
constexpr int64_t kRouterMaxTokens = (int64_t)1 << 28;  // 2^22 workgroups of 512 threads
constexpr int kRouterTokens = 64;  // of a workgroup: one bit each in an expert's mask

struct RouterCall {
    const void* logits;
    int64_t ld;
    int32_t tokens, experts, top_k;
    int32_t bf16, renormalize;
    int32_t* chosen;
    float* gates;
    int32_t* rows;    // null: not wanted
    int32_t* order;   // null: not wanted
    int32_t* counts;
    int32_t* offsets;
    int32_t* live;    // null: not wanted
    float* losses;    // null: not wanted
};
// What the launches of one call hand on, in its workspace; `blocks` workgroups
// of kRouterTokens tokens.
struct RouterSpace {
    uint8_t* hist;    // [block][expert]: choices
    float* probs;     // [block][expert]: sum of probabilities
    int32_t* base;    // [block][expert]: choices in the blocks before
    double* total;    // [expert]: sum of probabilities
    double* lse;      // [block]: sum of squared logarithms
    int32_t* live;    // [block]: tokens with a logit
    int32_t blocks;
};
hipError_t launch_router(const RouterCall& c, const RouterSpace& s, hipStream_t st);

struct RouterGradCall {
    const void* logits;
    int64_t ld;
    int32_t tokens, experts, top_k;
    int32_t bf16, renormalize;
    const int32_t* chosen;
    const int32_t* counts;
    const int32_t* live;
    const float* dgates;  // null: zeros
    void* dlogits;
    int64_t ld_out;
    float balance, z;
};
hipError_t launch_router_grad(const RouterGradCall& c, int cus, hipStream_t st);

}  // namespace muon
