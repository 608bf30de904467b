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
#include <algorithm>

#include "inputs.h"
#include "tile_any.h"
#include "tile_bf16.h"

namespace muon {

namespace {

// the larger one, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    return __builtin_elementwise_maximum(a, b);  // v_maximum3_f32
}

struct Query {
    int q0, q1, k0, k1;  // tokens of the sequence
    int tile;
};

__device__ __forceinline__ void clamp_range(const int32_t* cu, int i, int T, int& a, int& b) {
    a = min(max(gld(cu + i), 0), T);
    b = min(max(gld(cu + i + 1), a), T);
}

// The sequence that holds query tile `t`, or false: none.  Tiles are numbered
// through the sequences of more than twice the mean keys first, then through
// the others: a long one that came last would be waited for (16 packed
// sequences, the last one a third of all tokens: 32.8 -> 31.2 us).
template <int BM>
__device__ __forceinline__ bool find_query(const SmaxCall& c, int t, Query& g) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int others = 0; others < 2; ++others) {
        for (int s0 = 0; s0 < c.sequences; s0 += 64) {
            const int s = s0 + lane;
            int a = 0, b = 0, ka = 0, kb = 0;
            if (s < c.sequences) {
                clamp_range(c.cu_q, s, (int)c.tq, a, b);
                clamp_range(c.cu_k, s, (int)c.tk, ka, kb);
            }
            const bool is_long = (int64_t)(kb - ka) * c.sequences > 2 * c.tk;
            const int tiles = is_long != (others != 0) ? (b - a + BM - 1) / BM : 0;
            int sum = tiles;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int up = __shfl_up(sum, off, 64);
                if (lane >= off) sum += up;
            }
            const unsigned long long hit = __ballot(before + sum > t);
            if (hit) {
                const int l = __builtin_ctzll(hit);
                auto of = [&](int v) { return __builtin_amdgcn_readfirstlane(__shfl(v, l, 64)); };
                g.q0 = of(a);
                g.q1 = of(b);
                g.k0 = of(ka);
                g.k1 = of(kb);
                g.tile = of(t - before - (sum - tiles));
                return true;
            }
            before += __builtin_amdgcn_readfirstlane(__shfl(sum, 63, 64));
        }
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
// tile, key part, head).  One accumulator block a wave, and the queries are read
// again for every key tile: 4096 causal tokens of 8 heads of 128 in fp32 take 275
// us (62 TFLOP/s of unmasked pairs), of 129 in bf16 408.
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
        const int tiles = (max(end, 0) + kSmaxTile - 1) / kSmaxTile;
        const int j1 = min(end, (int)((int64_t)tiles * (split + 1) / c.splits) * kSmaxTile);
        for (int j0 = (int)((int64_t)tiles * split / c.splits) * kSmaxTile; j0 < j1; j0 += kSmaxTile) {
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

// bf16, head sizes up to 256: four waves of 32 RB queries each (RB row blocks
// of 32), the queries in registers for the whole run over the keys.  Keys
// come in tiles of 64 through three LDS stages, copied two tiles ahead: rows
// of 64-wide sub-slabs (tile_bf16.h), one barrier a tile.  Each key fragment
// read from LDS feeds RB MFMAs.  Query rows behind the last one repeat it and
// keys behind the last one repeat it too: a repeated logit changes no
// maximum, so only the tiles on the causal diagonal need a mask.
//
// Block -> (head, query tile, key part): the keys that a tile sees are cut into
// c.splits equal parts.  Late query tiles, which see the most keys, come first;
// where the heads divide by 8, each XCD takes a run of heads.  They come one
// after the other, so that the keys of those at work stay in its L2, unless the
// keys of all fit it: then a tile's heads come together, and the longest tiles
// of all heads first (16 packed sequences: 31.2 -> 29.0 us).  (Workgroups that
// stay and take the tasks in turn: 8192 tokens of 64 heads 445 -> 586 us; the
// causal tasks differ too much in length.)
//
// The matrix cores bound it: 8192 causal tokens of 64 heads of 128 take 432-514
// us by box, 1.07-1.27 PFLOP/s of unmasked pairs, 739 us without the mask (1.49
// PFLOP/s); head sizes 64, 96, 192 and 256 239, 364, 645 and 1012 us (1.15, 1.13,
// 1.28 and 1.09 PFLOP/s; 80 runs as 96: 348 us); counters: matrix cores busy 60% of the cycles with the mask, no LDS
// bank conflict, 0.48 GB fetched for 0.27 GB of queries and keys.  Short
// sequences are bound by a workgroup's start: 5.4 us for one that has a single
// key tile.  Fragments read one k-step ahead cost 590 us against 567 for two;
// tiles of 256 queries for sequences of 256 42 us against 33.
constexpr int kSmaxKeys = 64;

template <int DK, int RB>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(DK <= 192 ? 2 : 1)))
void smax_bf16_kernel(SmaxCall c, float* partials) {
    constexpr int SUB = (DK + 63) / 64;          // 64-wide sub-slabs of a key row
    constexpr int KS = DK / 16;                  // MFMA k-steps
    constexpr int STAGE = SUB * kSmaxKeys * 64;  // bf16 elements
    constexpr int BM = 128 * RB;
    __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE];
    __shared__ float red[4];
    const int per_head = c.qtiles * c.splits;
    // this XCD's heads, and the block's place among those that take them
    const bool by_xcd = c.heads_q % 8 == 0;
    const int nh = by_xcd ? c.heads_q / 8 : c.heads_q;
    const int h0 = by_xcd ? (blockIdx.x & 7) * nh : 0, L = by_xcd ? blockIdx.x >> 3 : blockIdx.x;
    const int h = h0 + (c.tile_major ? L % nh : L / per_head);
    const int rest = c.tile_major ? L / nh : L % per_head;
    const int t = rest / c.splits, split = rest - t * c.splits;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float top = -INFINITY;
    Query g;
    // long sequences come first, and of each its last query tile; behind the
    // last sequence are tiles that none fills
    if (find_query<BM>(c, t, g)) {
        const int Lq = g.q1 - g.q0, Lk = g.k1 - g.k0;
        const int i0 = ((Lq + BM - 1) / BM - 1 - g.tile) * BM;  // late tiles first
        const int shift = Lk - Lq;
        const int nq = min(BM, Lq - i0);
        const int end_all = c.causal ? min(Lk, i0 + nq + shift) : Lk;
        // in whole key tiles
        const int tiles = (max(end_all, 0) + kSmaxKeys - 1) / kSmaxKeys;
        const int begin = (int)((int64_t)tiles * split / c.splits) * kSmaxKeys;
        const int end = min(end_all, (int)((int64_t)tiles * (split + 1) / c.splits) * kSmaxKeys);
        if (begin < end) {
            const int D = c.head_dim;
            const uint16_t* qb = reinterpret_cast<const uint16_t*>(c.q) + (int64_t)h * c.q_head;
            const int hk = h / (c.heads_q / c.heads_k);
            const uint16_t* kb = reinterpret_cast<const uint16_t*>(c.k) + (int64_t)hk * c.k_head;
            // the wave's queries: row block r, k-step s
            bf::bf16x8 a[RB][KS];
            int row[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                row[r] = min(i0 + wave * 32 * RB + 32 * r + (lane & 31), Lq - 1);
                const uint16_t* src = qb + (int64_t)(g.q0 + row[r]) * c.q_token + 8 * (lane >> 5);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (16 * s + 8 * (lane >> 5) < D) v = gld(reinterpret_cast<const uint4*>(src + 16 * s));
                    a[r][s] = __builtin_bit_cast(bf::bf16x8, v);
                }
            }
            // key tile at j0 into a stage: wave w copies 16 keys of every sub-slab
            auto copy = [&](int j0, uint16_t* stage) {
                const uint16_t* base = kb + (int64_t)(g.k0 + j0) * c.k_token;
                const int last = Lk - 1 - j0;  // >= 0
                const __amdgpu_buffer_rsrc_t r = bf::resource(base, 0x7fffffff);
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int grp = wave * 2 + q;
                        const int key = grp * 8 + (lane >> 3);
                        const int ch = (lane & 7) ^ bf::swz<64>(key);
                        const uint32_t off = u * 64 + ch * 8 < D
                            ? (uint32_t)(min(key, last) * (int)c.k_token + u * 64 + ch * 8) * 2u : 0x80000000u;
                        __builtin_amdgcn_raw_ptr_buffer_load_lds(
                            r, (bf::lds_void*)(stage + (u * kSmaxKeys + grp * 8) * 64), 16, off, 0, 0, 0);
                    }
            };
            constexpr int CPS = 2 * SUB;  // copies of a wave and stage
            // first and last key that every / any of the wave's queries sees
            const int wi0 = i0 + wave * 32 * RB;
            const int every = c.causal ? min(wi0, Lq - 1) + shift : Lk - 1;
            const int any = c.causal ? min(wi0 + 32 * RB - 1, Lq - 1) + shift : Lk - 1;
            auto tile = [&](int j0, const uint16_t* stage) {
                if (j0 > any) return;
                bf::f32x16 acc[RB][2];
#pragma unroll
                for (int r = 0; r < RB; ++r)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[r][j][e] = 0.f;
                bf::bf16x8 b[3][2];
                auto read = [&](int s, bf::bf16x8 (&f)[2]) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        f[j] = bf::frag_rows<64>(stage + (s / 4) * kSmaxKeys * 64, 32 * j + (lane & 31),
                                             2 * (s % 4) + (lane >> 5));
                };
                // two k-steps ahead, in this order: left to itself the compiler
                // puts each read right before its use
                read(0, b[0]);
                read(1, b[1]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    if (s + 2 < KS) read(s + 2, b[(s + 2) % 3]);
#pragma unroll
                    for (int r = 0; r < RB; ++r)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            acc[r][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[s % 3][j], a[r][s], acc[r][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
                // operands exchanged: register e of lane l is key 8 (e / 4) +
                // 4 (l / 32) + e % 4 of the block, query l % 32
                if (j0 + kSmaxKeys - 1 > every) {
#pragma unroll
                    for (int r = 0; r < RB; ++r)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int key = j0 + 32 * j + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
                                const int lim = c.causal ? row[r] + shift : Lk - 1;
                                if (key > lim) acc[r][j][e] = -INFINITY;
                            }
                }
                float m[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int r = 0; r < RB; ++r)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        m[e & 3] = max_nan(max_nan(m[e & 3], acc[r][0][e]), acc[r][1][e]);
                top = max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
            };
            const int n = (end - begin + kSmaxKeys - 1) / kSmaxKeys;
            // a copy behind the last key repeats it: every stage may be filled
            auto start = [&](int i) { return min(begin + i * kSmaxKeys, Lk - 1); };
            copy(start(0), s0);
            copy(start(1), s1);
            for (int i = 0; i < n; i += 3) {
#pragma unroll
                for (int u = 0; u < 3; ++u) {
                    if (i + u >= n) break;
                    bf::wait_vmcnt<CPS>();  // this tile's copies, not the next one's
                    bf::lds_barrier();
                    copy(start(i + u + 2), u == 0 ? s2 : u == 1 ? s0 : s1);
                    tile(begin + (i + u) * kSmaxKeys, u == 0 ? s0 : u == 1 ? s1 : s2);
                }
            }
            bf::wait_vmcnt<0>();
        }
    }
    top = block_max(top, red);
    if (threadIdx.x == 0) gst(partials + (int64_t)h * per_head + rest, top * c.scale);
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

// bf16 rows that start on 16 bytes and hold whole 16-byte chunks, of a size
// that the registers hold
bool smax_chunked(const SmaxCall& c) {
    auto ok = [](const void* p, int64_t token, int64_t head) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && token % 8 == 0 && head % 8 == 0;
    };
    return c.bf16 && c.head_dim % 8 == 0 && c.head_dim <= 256 && ok(c.q, c.q_token, c.q_head) &&
           ok(c.k, c.k_token, c.k_head) && c.k_token <= (1 << 22);
}

namespace {

template <int DK>
void smax_launch(const SmaxCall& c, unsigned grid, float* partials, hipStream_t st) {
    if (c.tile == 256)
        smax_bf16_kernel<DK, 2><<<grid, 256, 0, st>>>(c, partials);
    else
        smax_bf16_kernel<DK, 1><<<grid, 256, 0, st>>>(c, partials);
}

}  // namespace

int64_t smax_plan(SmaxCall& c, int cus, bool chunked) {
    const int64_t seq = c.sequences < c.tq ? c.sequences : c.tq;
    // short sequences on tiles of 128 queries
    c.tile = !chunked ? kSmaxTile : c.tq < (int64_t)kSmaxLong * seq ? 128 : 256;
    c.qtiles = (int)(c.tq / c.tile + seq);
    // few query tiles: the keys are split too, for about four workgroups a
    // compute unit
    const int64_t have = (int64_t)c.qtiles * c.heads_q, want = 4 * (int64_t)cus;
    const int64_t ktiles = (c.tk + kSmaxTile - 1) / kSmaxTile;
    c.splits = (int)std::max<int64_t>(1, std::min(have > 0 ? (want + have / 2) / have : 1, ktiles));
    // the keys of the heads that one XCD serves, against its L2 of 4 MB
    const int64_t kv = c.heads_q % 8 == 0 ? std::max(1, c.heads_k / 8) : c.heads_k;
    c.tile_major = kv * c.tk * c.head_dim * 2 <= (4 << 20);
    return (int64_t)c.qtiles * c.splits * c.heads_q;
}

hipError_t launch_smax(const SmaxCall& c, float* partials, float* smax_q, float* smax_k, int accumulate,
                       hipStream_t st) {
    const int per_head = c.qtiles * c.splits;
    if (per_head > 0) {
        const unsigned grid = (unsigned)(per_head * (int64_t)c.heads_q);
        if (c.tile == kSmaxTile)
            smax_any_kernel<<<grid, 256, 0, st>>>(c, partials);
        else if (c.head_dim <= 64)
            smax_launch<64>(c, grid, partials, st);
        else if (c.head_dim <= 96)
            smax_launch<96>(c, grid, partials, st);
        else if (c.head_dim <= 128)
            smax_launch<128>(c, grid, partials, st);
        else if (c.head_dim <= 192)
            smax_launch<192>(c, grid, partials, st);
        else
            smax_launch<256>(c, grid, partials, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    smax_finalize_kernel<<<c.heads_k, 256, 0, st>>>(partials, per_head, c.heads_q / c.heads_k, accumulate,
                                                    smax_q, smax_k);
    return hipGetLastError();
}

}  // namespace muon
