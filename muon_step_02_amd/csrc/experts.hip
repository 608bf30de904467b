// Products of a mixture-of-experts layer grouped by expert (gfx950).  Rows of
// group e are offsets[e] ... offsets[e + 1] - 1, weights W_e are (rows, cols) =
// (fan-out, fan-in):
//
//   forward          y_t  = W_e x_t         for the rows t of group e
//   input gradient   dx_t = W_e^T dy_t
//   weight gradient  dW_e (+)= sum_t dy_t x_t^T
//
// The group sizes are device data (a router's result), so the host sizes a
// launch by what they can be at most and every workgroup finds its group and
// tile itself.  Offsets are clamped into [0, tokens] and to ascending order
// where they are read: whatever they hold, no access leaves the tensors.
#include <string.h>

#include "inputs.h"
#include "tile_any.h"

namespace muon {

namespace {

struct Group {
    int e;
    int row0, row1;  // rows of the group
    int tile;        // row tile within it
};

__device__ __forceinline__ void group_rows(const ExpertCall& c, int e, int& r0, int& r1) {
    const int T = (int)c.tokens;
    r0 = min(max(gld(c.offsets + e), 0), T);
    r1 = min(max(gld(c.offsets + e + 1), r0), T);
}

// The group that holds row tile `mt` (tiles of BM rows, each group's last one
// ragged), or false: none.  Every wave searches for itself: 64 groups at a
// time, one per lane, with a prefix sum of their tiles.
template <int BM>
__device__ __forceinline__ bool find_group(const ExpertCall& c, int mt, Group& g) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 < c.experts; e0 += 64) {
        const int e = e0 + lane;
        int r0 = 0, r1 = 0;
        if (e < c.experts) group_rows(c, e, r0, r1);
        const int tiles = (r1 - r0 + BM - 1) / BM;
        int sum = tiles;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int up = __shfl_up(sum, off, 64);
            if (lane >= off) sum += up;
        }
        const unsigned long long hit = __ballot(before + sum > mt);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            g.e = __builtin_amdgcn_readfirstlane(e0 + l);
            g.row0 = __builtin_amdgcn_readfirstlane(__shfl(r0, l, 64));
            g.row1 = __builtin_amdgcn_readfirstlane(__shfl(r1, l, 64));
            g.tile = __builtin_amdgcn_readfirstlane(mt - before - __shfl(sum - tiles, l, 64));
            return true;
        }
        before += __shfl(sum, 63, 64);
    }
    return false;
}

__device__ __forceinline__ const void* at(const void* base, int bf16, int64_t off) {
    return reinterpret_cast<const char*>(base) + off * (bf16 ? 2 : 4);
}

// ---- any type, alignment and size: 64 x 64 tiles in fp32 -------------------

// One value of the result: rounded once, from the fp32 sum.
__device__ __forceinline__ void put_value(void* base, int bf16, int64_t off, float v, int accumulate) {
    if (bf16) {
        uint16_t* p = reinterpret_cast<uint16_t*>(base) + off;
        if (accumulate) v += bf16_bits_to_f32(gld(p));
        gst(p, f32_to_bf16_bits(v));
    } else {
        float* p = reinterpret_cast<float*>(base) + off;
        if (accumulate) v += gld(p);
        gst(p, v);
    }
}

__device__ __forceinline__ void put_tile(const any::f32x16& acc, void* base, int bf16, int64_t ld,
                                         int rows, int cols, int accumulate) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int j = 32 * (wave & 1) + (lane & 31);
    if (j >= cols) return;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int i = 32 * (wave >> 1) + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (i < rows) put_value(base, bf16, (int64_t)i * ld + j, acc[r], accumulate);
    }
}

// Forward and input gradient: block -> (row tile, column tile), column tiles
// fastest.
template <ExpertOp OP, int CAP>
__global__ __launch_bounds__(256) void expert_rows_any_kernel(ExpertCall c, ExpertPtrs<CAP> w, int ntiles) {
    __shared__ any::Lds lds;
    const int mt = blockIdx.x / ntiles, nt = blockIdx.x - mt * ntiles;
    Group g;
    if (!find_group<any::kTile>(c, mt, g)) return;
    const int i0 = g.row0 + g.tile * any::kTile, j0 = nt * any::kTile;
    const int N = OP == kExpertForward ? c.rows : c.cols;
    const int K = OP == kExpertForward ? c.cols : c.rows;
    const int nrows = min(any::kTile, g.row1 - i0), ncols = min(any::kTile, N - j0);
    const any::Operand p{at(c.a, c.bf16, (int64_t)i0 * c.ld_a), c.ld_a, nrows};
    const void* we = w.w[g.e];
    const any::Operand q{at(we, c.bf16, OP == kExpertForward ? (int64_t)j0 * c.ld_w : j0), c.ld_w, ncols};
    const any::f32x16 acc = any::product<false, OP == kExpertGradInput>(p, q, c.bf16, K, lds);
    void* out = const_cast<void*>(at(c.c, c.bf16, (int64_t)i0 * c.ld_c + j0));
    put_tile(acc, out, c.bf16, c.ld_c, nrows, ncols, 0);
}

// Weight gradient: block -> (expert, row tile, column tile) of dW.
template <int CAP>
__global__ __launch_bounds__(256) void expert_weight_any_kernel(ExpertCall c, ExpertPtrs<CAP> w, int mtiles,
                                                                int ntiles) {
    __shared__ any::Lds lds;
    const int per = mtiles * ntiles;
    const int e = blockIdx.x / per, rest = blockIdx.x - e * per;
    const int mt = rest / ntiles, nt = rest - mt * ntiles;
    int r0, r1;
    group_rows(c, e, r0, r1);
    if (c.accumulate && r1 == r0) return;
    const int i0 = mt * any::kTile, j0 = nt * any::kTile;
    const int nrows = min(any::kTile, c.rows - i0), ncols = min(any::kTile, c.cols - j0);
    const any::Operand p{at(c.b, c.bf16, (int64_t)r0 * c.ld_b + i0), c.ld_b, nrows};
    const any::Operand q{at(c.a, c.bf16, (int64_t)r0 * c.ld_a + j0), c.ld_a, ncols};
    const any::f32x16 acc = any::product<true, true>(p, q, c.bf16, r1 - r0, lds);
    void* out = const_cast<void*>(at(w.w[e], c.out_bf16, (int64_t)i0 * c.ld_w + j0));
    put_tile(acc, out, c.out_bf16, c.ld_w, nrows, ncols, c.accumulate);
}

template <int CAP>
hipError_t launch_any(ExpertOp op, const ExpertCall& c, const ExpertPtrs<CAP>& w, hipStream_t st) {
    const int T = any::kTile;
    const int64_t nr = (c.rows + T - 1) / T, nc = (c.cols + T - 1) / T;
    if (op == kExpertGradWeight) {
        expert_weight_any_kernel<CAP><<<(unsigned)(c.experts * nr * nc), 256, 0, st>>>(c, w, (int)nr, (int)nc);
    } else {
        // at most this many row tiles: every group may end in a ragged one
        const int64_t mt = c.tokens / T + (c.tokens < c.experts ? c.tokens : c.experts);
        if (op == kExpertForward)
            expert_rows_any_kernel<kExpertForward, CAP><<<(unsigned)(mt * nr), 256, 0, st>>>(c, w, (int)nr);
        else
            expert_rows_any_kernel<kExpertGradInput, CAP><<<(unsigned)(mt * nc), 256, 0, st>>>(c, w, (int)nc);
    }
    return hipGetLastError();
}

template <int CAP>
hipError_t launch_cap(ExpertOp op, const ExpertCall& c, const void* const* ptrs, hipStream_t st) {
    ExpertPtrs<CAP> w;
    memset(&w, 0, sizeof(w));
    for (int e = 0; e < c.experts; ++e) w.w[e] = const_cast<void*>(ptrs[e]);
    return launch_any<CAP>(op, c, w, st);
}

}  // namespace

hipError_t launch_expert(ExpertOp op, const ExpertCall& c, const void* const* w, hipStream_t st) {
    return c.experts <= kExpertsSmall ? launch_cap<kExpertsSmall>(op, c, w, st)
                                      : launch_cap<kMaxExperts>(op, c, w, st);
}

}  // namespace muon
