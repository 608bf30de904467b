// The largest attention logit of every head, which QK-Clip reads (gfx950):
//
//   S_h = max over sequences and unmasked pairs (i, j) of
//         scale * <q[i][h], k[j][h / (heads_q / heads_k)]>
//
// with j <= i + (Lk - Lq) where the attention is causal (the queries are the
// last Lq of Lk positions).  ("The Optimizer Wars: How Muon Is Replacing Adam
// in Frontier AI Training", ai.info, section "What is MuonClip?": the clip
// scales a head's query and key weights by sqrt(min(1, tau / S_max)).)
//
// No logit is stored: a workgroup holds a tile of queries of one head, runs
// over the keys, and keeps a running maximum in registers.  A maximum does
// not depend on the order it is taken in, so any split over workgroups gives
// the same bits.  A NaN logit makes the head's maximum NaN; a pair that the
// mask excludes never counts, whatever its values.  A head without any pair
// gets -inf, which clips nothing.
#include "inputs.h"
#include "tile_any.h"

namespace muon {

namespace {

// the larger one, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    return (a > b || a != a) ? a : b;
}

struct Query {
    int q0, q1, k0, k1;  // tokens of the sequence
    int tile;
};

__device__ __forceinline__ void clamp_range(const int32_t* cu, int i, int T, int& a, int& b) {
    a = min(max(gld(cu + i), 0), T);
    b = min(max(gld(cu + i + 1), a), T);
}

// The sequence that holds query tile `t`, or false: none.
template <int BM>
__device__ __forceinline__ bool find_query(const SmaxCall& c, int t, Query& g) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int s0 = 0; s0 < c.sequences; s0 += 64) {
        const int s = s0 + lane;
        int a = 0, b = 0;
        if (s < c.sequences) clamp_range(c.cu_q, s, (int)c.tq, a, b);
        const int tiles = (b - a + BM - 1) / BM;
        int sum = tiles;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int up = __shfl_up(sum, off, 64);
            if (lane >= off) sum += up;
        }
        const unsigned long long hit = __ballot(before + sum > t);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            g.q0 = __builtin_amdgcn_readfirstlane(__shfl(a, l, 64));
            g.q1 = __builtin_amdgcn_readfirstlane(__shfl(b, l, 64));
            g.tile = __builtin_amdgcn_readfirstlane(t - before - __shfl(sum - tiles, l, 64));
            int ka, kb;
            clamp_range(c.cu_k, s0 + l, (int)c.tk, ka, kb);
            g.k0 = __builtin_amdgcn_readfirstlane(ka);
            g.k1 = __builtin_amdgcn_readfirstlane(kb);
            return true;
        }
        before += __shfl(sum, 63, 64);
    }
    return false;
}

__device__ __forceinline__ const void* at(const void* base, int bf16, int64_t off) {
    return reinterpret_cast<const char*>(base) + off * (bf16 ? 2 : 4);
}

__device__ __forceinline__ float block_max(float m, float* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = max_nan(m, __shfl_xor(m, off, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = red[0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) m = max_nan(m, red[w]);
    return m;
}

// Any type, alignment and head size: 64 x 64 tiles in fp32.  Block -> (query
// tile, key split, head); split s takes the key tiles s, s + splits, ...
__global__ __launch_bounds__(256) void smax_any_kernel(SmaxCall c, float* partials) {
    __shared__ any::Lds lds;
    __shared__ float red[4];
    const int per = c.splits * c.heads_q;
    const int t = blockIdx.x / per, rest = blockIdx.x - t * per;
    const int split = rest / c.heads_q, h = rest - split * c.heads_q;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float m = -INFINITY;
    Query g;
    if (find_query<kSmaxTile>(c, t, g)) {
        const int hk = h / (c.heads_q / c.heads_k);
        const int i0 = g.tile * kSmaxTile;  // within the sequence
        const int nq = min(kSmaxTile, g.q1 - g.q0 - i0);
        const int Lk = g.k1 - g.k0;
        const int shift = Lk - (g.q1 - g.q0);
        // keys that any query of the tile sees
        const int end = c.causal ? min(Lk, i0 + nq + shift) : Lk;
        const any::Operand q{at(c.q, c.bf16, (int64_t)(g.q0 + i0) * c.q_token + (int64_t)h * c.q_head),
                             c.q_token, nq};
        for (int j0 = split * kSmaxTile; j0 < end; j0 += c.splits * kSmaxTile) {
            const int nk = min(kSmaxTile, Lk - j0);
            const any::Operand k{at(c.k, c.bf16, (int64_t)(g.k0 + j0) * c.k_token + (int64_t)hk * c.k_head),
                                 c.k_token, nk};
            const any::f32x16 acc = any::product<false, false>(q, k, c.bf16, c.head_dim, lds);
            const int j = 32 * (wave & 1) + (lane & 31);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int i = 32 * (wave >> 1) + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                const bool in = i < nq && j < nk && (!c.causal || j0 + j <= i0 + i + shift);
                m = max_nan(m, in ? acc[r] : -INFINITY);
            }
        }
    }
    m = block_max(m, red);
    // the scale is positive: it may follow the maximum
    if (threadIdx.x == 0) gst(partials + (int64_t)h * c.qtiles * c.splits + t * c.splits + split, m * c.scale);
}

// Partials of a head to its maximum; block: one key head and its query heads.
__global__ __launch_bounds__(256) void smax_finalize_kernel(const float* partials, int per_head, int group,
                                                            int accumulate, float* smax_q, float* smax_k) {
    __shared__ float red[4];
    float all = -INFINITY;
    for (int u = 0; u < group; ++u) {
        const int h = blockIdx.x * group + u;
        float m = -INFINITY;
        for (int i = threadIdx.x; i < per_head; i += 256) m = max_nan(m, gld(partials + (int64_t)h * per_head + i));
        __syncthreads();
        m = block_max(m, red);
        if (threadIdx.x == 0 && smax_q) gst(smax_q + h, accumulate ? max_nan(m, gld(smax_q + h)) : m);
        all = max_nan(all, m);
    }
    if (threadIdx.x == 0 && smax_k)
        gst(smax_k + blockIdx.x, accumulate ? max_nan(all, gld(smax_k + blockIdx.x)) : all);
}

}  // namespace

void smax_plan(SmaxCall& c, int cus) {
    const int64_t seq = c.sequences < c.tq ? c.sequences : c.tq;
    c.qtiles = (int)(c.tq / kSmaxTile + seq);
    // few query tiles: the keys are split too, up to four workgroups a compute unit
    const int64_t have = (int64_t)c.qtiles * c.heads_q, want = 4 * (int64_t)cus;
    const int64_t ktiles = (c.tk + kSmaxTile - 1) / kSmaxTile;
    int64_t s = have > 0 ? want / have : 1;
    if (s > ktiles) s = ktiles;
    c.splits = s < 1 ? 1 : (int)s;
}

hipError_t launch_smax(const SmaxCall& c, float* partials, float* smax_q, float* smax_k, int accumulate,
                       hipStream_t st) {
    const int per_head = c.qtiles * c.splits;
    if (per_head > 0) {
        smax_any_kernel<<<(unsigned)(per_head * (int64_t)c.heads_q), 256, 0, st>>>(c, partials);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    smax_finalize_kernel<<<c.heads_k, 256, 0, st>>>(partials, per_head, c.heads_q / c.heads_k, accumulate,
                                                    smax_q, smax_k);
    return hipGetLastError();
}

}  // namespace muon
