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
#include "tile_bf16.h"

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

// ---- bf16 on the matrix cores ------------------------------------------------

// Row tile `mt` as find_group, and the group's number of row tiles before it;
// total: row tiles of all groups.
template <int BM>
__device__ __forceinline__ int count_tiles(const ExpertCall& c) {
    const int lane = threadIdx.x & 63;
    int total = 0;
    for (int e0 = 0; e0 < c.experts; e0 += 64) {
        int r0 = 0, r1 = 0;
        if (e0 + lane < c.experts) group_rows(c, e0 + lane, r0, r1);
        total += (r1 - r0 + BM - 1) / BM;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) total += __shfl_xor(total, off, 64);
    return __builtin_amdgcn_readfirstlane(total);
}

// Workgroup b runs on XCD b % 8, each with an L2 of its own.  Rounds of 256
// tiles deal runs of 32 consecutive tiles to the XCDs, so the tiles that run
// on one XCD at a time share operand panels, and neighbouring XCDs work on
// the same expert, whose panels then come from the memory-side cache; what is
// left after the last whole round is cut into 8 runs.
__device__ __forceinline__ int dealt_tile(int b, int total) {
    const int x = b & 7, t = b >> 3;
    const int full = total / 256;
    if (t < 32 * full) return ((t / 32) * 8 + x) * 32 + t % 32;
    const int rest = total - 256 * full, per = (rest + 7) / 8;
    const int u = t - 32 * full;
    const int tile = x * per + u;
    return u < per && tile < rest ? 256 * full + tile : -1;
}

// Tile lt of a group of R row tiles and NT column tiles: rows fastest within
// runs of 8 row tiles, so that concurrent tiles share column panels too.
__device__ __forceinline__ void tile_of(int lt, int R, int NT, int& mt, int& nt) {
    const int g = lt / (8 * NT);
    const int in = lt - g * 8 * NT;
    const int rows = min(8, R - 8 * g);
    nt = in / rows;
    mt = 8 * g + in - nt * rows;
}

constexpr int kBM = 256, kBN = 256;

template <class C>
__device__ __forceinline__ void rows_tile(const ExpertCall& c, const bf::Operand& p, const bf::Operand& q, int K,
                                          int rows, int cols, uint16_t* out, const bf::Stages& st) {
    bf::f32x16 acc[C::FM][C::FN];
    bf::product<C>(acc, p, q, K, st);
    const int64_t ld = c.ld_c;
    bf::for_each_chunk<C>(acc, reinterpret_cast<float*>(st.p0), rows, [&](int r, int c8, const float* v) {
        if (r < rows && c8 < cols) gst(reinterpret_cast<uint4*>(out + r * ld + c8), bf::pack8(v));
    });
}

// Forward and input gradient on 256 x 256 tiles of eight waves.  A group's
// last row tile takes the shorter kind that holds its rows.
template <ExpertOp OP, int CAP>
__global__ __launch_bounds__(512) void expert_rows_kernel(ExpertCall c, ExpertPtrs<CAP> w, int ntiles) {
    __shared__ __attribute__((aligned(1024))) uint16_t lp0[bf::kSlab], lq0[bf::kSlab], lp1[bf::kSlab], lq1[bf::kSlab];
    const bf::Stages st{lp0, lq0, lp1, lq1};
    const int tile = dealt_tile(blockIdx.x, count_tiles<kBM>(c) * ntiles);
    if (tile < 0) return;
    Group g;
    if (!find_group<kBM>(c, tile / ntiles, g)) return;
    const int R = (g.row1 - g.row0 + kBM - 1) / kBM;
    // g.tile counts whole rows of tiles: the tile's place within the group
    int mt, nt;
    tile_of(g.tile * ntiles + tile % ntiles, R, ntiles, mt, nt);
    constexpr bool QKM = OP == kExpertGradInput;
    const int N = QKM ? c.cols : c.rows, K = QKM ? c.rows : c.cols;
    const int i0 = g.row0 + mt * kBM, j0 = nt * kBN;
    const int rows = min(kBM, g.row1 - i0), cols = min(kBN, N - j0);
    const uint16_t* a = reinterpret_cast<const uint16_t*>(c.a) + (int64_t)i0 * c.ld_a;
    const bf::Operand p{a, c.ld_a, 2 * ((int64_t)(rows - 1) * c.ld_a + K)};
    const uint16_t* we = reinterpret_cast<const uint16_t*>(w.w[g.e]);
    const bf::Operand q = QKM ? bf::Operand{we + j0, c.ld_w, 2 * ((int64_t)(K - 1) * c.ld_w + N - j0)}
                              : bf::Operand{we + (int64_t)j0 * c.ld_w, c.ld_w, 2 * ((int64_t)(cols - 1) * c.ld_w + K)};
    uint16_t* out = reinterpret_cast<uint16_t*>(c.c) + (int64_t)i0 * c.ld_c + j0;
    if (rows > 128)
        rows_tile<bf::Cfg<256, kBN, 2, 4, false, QKM>>(c, p, q, K, rows, cols, out, st);
    else if (rows > 64)
        rows_tile<bf::Cfg<128, kBN, 2, 4, false, QKM>>(c, p, q, K, rows, cols, out, st);
    else
        rows_tile<bf::Cfg<64, kBN, 2, 4, false, QKM>>(c, p, q, K, rows, cols, out, st);
}

// Weight gradient on 128 x 128 tiles of four waves, two workgroups a compute
// unit: a group's rows are a short K, so the tile's result is much of the
// traffic, and one workgroup writes while the other multiplies.
template <int CAP>
__global__ __launch_bounds__(256) void expert_weight_kernel(ExpertCall c, ExpertPtrs<CAP> w, int mtiles, int ntiles) {
    using C = bf::Cfg<128, 128, 2, 2, true, true>;
    __shared__ __attribute__((aligned(1024))) uint16_t lp0[8192], lq0[8192], lp1[8192], lq1[8192];
    const bf::Stages st{lp0, lq0, lp1, lq1};
    const int per = mtiles * ntiles;
    const int tile = dealt_tile(blockIdx.x, per * c.experts);
    if (tile < 0) return;
    const int e = tile / per;
    int r0, r1, mt, nt;
    group_rows(c, e, r0, r1);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    r1 = __builtin_amdgcn_readfirstlane(r1);
    if (c.accumulate && r1 == r0) return;
    tile_of(tile - e * per, mtiles, ntiles, mt, nt);
    const int i0 = mt * 128, j0 = nt * 128, K = r1 - r0;
    const int rows = min(128, c.rows - i0), cols = min(128, c.cols - j0);
    const bf::Operand p{reinterpret_cast<const uint16_t*>(c.b) + (int64_t)r0 * c.ld_b + i0, c.ld_b,
                        2 * ((int64_t)(K - 1) * c.ld_b + c.rows - i0)};
    const bf::Operand q{reinterpret_cast<const uint16_t*>(c.a) + (int64_t)r0 * c.ld_a + j0, c.ld_a,
                        2 * ((int64_t)(K - 1) * c.ld_a + c.cols - j0)};
    bf::f32x16 acc[C::FM][C::FN];
    bf::product<C>(acc, p, q, K, st);
    const int64_t ld = c.ld_w;
    float* const of = reinterpret_cast<float*>(w.w[e]) + (int64_t)i0 * ld + j0;
    uint16_t* const ob = reinterpret_cast<uint16_t*>(w.w[e]) + (int64_t)i0 * ld + j0;
    const bool add = c.accumulate != 0;
    float* const band = reinterpret_cast<float*>(lp0);
    if (c.out_bf16) {
        bf::for_each_chunk<C>(acc, band, rows, [&](int r, int c8, const float* v) {
            if (r >= rows || c8 >= cols) return;
            uint4* o = reinterpret_cast<uint4*>(ob + r * ld + c8);
            float s[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) s[x] = v[x];
            if (add) {
                const uint4 old = gld(o);
                const uint32_t u[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    s[x] += __builtin_bit_cast(float, (x & 1) ? (u[x >> 1] & 0xffff0000u) : (u[x >> 1] << 16));
            }
            gst(o, bf::pack8(s));
        });
    } else {
        bf::for_each_chunk<C>(acc, band, rows, [&](int r, int c8, const float* v) {
            if (r >= rows || c8 >= cols) return;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float4* o = reinterpret_cast<float4*>(of + r * ld + c8 + 4 * half);
                float4 s = make_float4(v[4 * half], v[4 * half + 1], v[4 * half + 2], v[4 * half + 3]);
                if (add) {
                    const float4 old = gld(o);
                    s = make_float4(s.x + old.x, s.y + old.y, s.z + old.z, s.w + old.w);
                }
                gst(o, s);
            }
        });
    }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// bf16 operands whose rows all start on 16 bytes and hold whole 16-byte
// chunks; anything else takes the 64 x 64 tiles.
bool chunked(ExpertOp op, const ExpertCall& c, const void* const* w) {
    if (!c.bf16 || c.rows % 8 || c.cols % 8 || c.ld_a % 8 || c.ld_w % 8 || !aligned16(c.a)) return false;
    if (op == kExpertGradWeight ? (c.ld_b % 8 || !aligned16(c.b)) : (c.ld_c % 8 || !aligned16(c.c))) return false;
    for (int e = 0; e < c.experts; ++e)
        if (!aligned16(w[e])) return false;
    return true;
}

template <int CAP>
hipError_t launch_bf16(ExpertOp op, const ExpertCall& c, const ExpertPtrs<CAP>& w, hipStream_t st) {
    // dealt_tile covers every tile where the grid holds at least as many
    // blocks, in whole groups of 8
    auto grid = [](int64_t tiles) { return (unsigned)((tiles + 7) / 8 * 8); };
    if (op == kExpertGradWeight) {
        const int mt = (c.rows + 127) / 128, nt = (c.cols + 127) / 128;
        expert_weight_kernel<CAP><<<grid((int64_t)c.experts * mt * nt), 256, 0, st>>>(c, w, mt, nt);
    } else {
        const int64_t mt = c.tokens / kBM + (c.tokens < c.experts ? c.tokens : c.experts);
        const int nt = ((op == kExpertForward ? c.rows : c.cols) + kBN - 1) / kBN;
        if (op == kExpertForward)
            expert_rows_kernel<kExpertForward, CAP><<<grid(mt * nt), 512, 0, st>>>(c, w, nt);
        else
            expert_rows_kernel<kExpertGradInput, CAP><<<grid(mt * nt), 512, 0, st>>>(c, w, nt);
    }
    return hipGetLastError();
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
    return chunked(op, c, ptrs) ? launch_bf16<CAP>(op, c, w, st) : launch_any<CAP>(op, c, w, st);
}

}  // namespace

hipError_t launch_expert(ExpertOp op, const ExpertCall& c, const void* const* w, hipStream_t st) {
    return c.experts <= kExpertsSmall ? launch_cap<kExpertsSmall>(op, c, w, st)
                                      : launch_cap<kMaxExperts>(op, c, w, st);
}

}  // namespace muon
