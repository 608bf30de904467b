// Internal declarations of the operators on what the optimizer step consumes:
// the global gradient norm and the clip (grads.hip), the products grouped by
// expert (experts.hip) and the largest attention logits (qk_smax.hip).  The
// entry points are in api_inputs.hip.  Nothing here is part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon_internal.h"

namespace muon {

// ---- gradient norm and clip ----------------------------------------------
// Tensors travel in kernel arguments, at most kGradGroup per launch (14 KB).
constexpr int kGradGroup = 256;
constexpr int kGradGroupSmall = 16;  // lists up to this length: 1 KB of arguments
// A chunk is kGradUnits units of 16 bytes of one tensor (the last chunk of a
// tensor may hold fewer); a row of a tensor starts a new unit.
constexpr int kGradUnits = 1024;
// Workgroups of the sum-of-squares launches of one call together, and with
// them the partial sums the second pass adds up (one more per launch at most).
constexpr int kGradBlocks = 2048;
// Lists of at most this many chunks (one each for its four teams of 256
// threads) go through one workgroup in one launch: 5 us, against 3 + 4 us and
// the gap between two launches.
constexpr int kGradSingle = 4;

template <int CAP>
struct GradGroup {
    const void* g[CAP];
    void* out[CAP];
    int64_t rows[CAP], cols[CAP];
    int64_t ld_g[CAP], ld_out[CAP];
    int32_t chunk_prefix[CAP + 1];
    uint8_t bf16[CAP], out_bf16[CAP];
    int32_t count;
};
static_assert(sizeof(GradGroup<kGradGroup>) <= 16384, "a group must fit a 16 KB argument block");

// Partial sums of squares of one group: block b of `blocks` adds up the chunks
// b, b + blocks, ... in order and writes partials[b].
template <int CAP>
hipError_t launch_grad_sumsq(const GradGroup<CAP>& g, int blocks, double* partials, hipStream_t st);
// norm and clip scale from `nparts` partial sums
hipError_t launch_grad_finalize(const double* partials, int nparts, float max_norm, float* norm_out,
                                float* scale_out, hipStream_t st);
// out = g * scale for one group, the scale formed from the partial sums by
// every block; norm_out and scale_out (null: not written) from block 0
template <int CAP>
hipError_t launch_grad_scale(const GradGroup<CAP>& g, int blocks, const double* partials, int nparts,
                             float max_norm, float* norm_out, float* scale_out, hipStream_t st);
// everything in one workgroup: the norm, and with clip the outputs
template <int CAP>
hipError_t launch_grad_single(const GradGroup<CAP>& g, int clip, float max_norm, float* norm_out,
                              float* scale_out, hipStream_t st);

// ---- products grouped by expert --------------------------------------------
// Weight (or weight gradient) pointers travel in kernel arguments.
constexpr int kMaxExperts = 1024;
constexpr int kExpertsSmall = 128;

enum ExpertOp { kExpertForward = 0, kExpertGradInput = 1, kExpertGradWeight = 2 };

// One call as the kernels see it.  Forward and input gradient:
//   C[t][j] = sum_k A[t][k] W_e[j][k]  (forward: j < rows, k < cols)
//   C[t][j] = sum_k A[t][k] W_e[k][j]  (input gradient: j < cols, k < rows)
// for the rows t of group e.  Weight gradient: W_e[n][k] (+)= sum over the
// rows t of group e of B[t][n] A[t][k] (A: the inputs, B: the output's
// gradients).
struct ExpertCall {
    const int32_t* offsets;  // experts + 1
    const void* a;
    const void* b;           // weight gradient only
    void* c;                 // forward, input gradient
    int64_t ld_a, ld_b, ld_c, ld_w;
    int64_t tokens;          // rows of a, b and c; < 2^31
    int32_t experts;
    int32_t rows, cols;      // of each weight
    int32_t bf16;            // type of a, b, c and the weights
    int32_t out_bf16;        // weight gradient: its type
    int32_t accumulate;
};
template <int CAP>
struct ExpertPtrs {
    void* w[CAP];
};

hipError_t launch_expert(ExpertOp op, const ExpertCall& call, const void* const* w, hipStream_t st);

// ---- largest attention logits ----------------------------------------------
struct SmaxCall {
    const void* q;
    const void* k;
    int64_t tq, tk;                          // tokens
    int64_t q_token, q_head, k_token, k_head;  // strides in elements
    const int32_t* cu_q;
    const int32_t* cu_k;
    int32_t sequences, heads_q, heads_k, head_dim;
    int32_t bf16, causal;
    float scale;
    int32_t tile;            // queries of a tile
    int32_t qtiles, splits;  // bound of query tiles over all sequences, key parts of each
    int32_t tile_major;      // order of the workgroups: a tile's heads together
};
constexpr int kSmaxTile = 64;   // queries (and keys) per tile of the kernel for any type
constexpr int kSmaxLong = 512;  // mean queries of a sequence from which tiles hold 256
// whether the bf16 kernels take the call (the one for any type takes all)
bool smax_chunked(const SmaxCall& c);
// fills tile, qtiles and splits from the sizes, for the bf16 kernels or
// for the other one; returns the number of partial maxima
int64_t smax_plan(SmaxCall& c, int cus, bool chunked);
hipError_t launch_smax(const SmaxCall& c, float* partials, float* smax_q, float* smax_k,
                       int accumulate, hipStream_t st);

}  // namespace muon
