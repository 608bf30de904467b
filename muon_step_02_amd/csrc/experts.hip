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

#include <type_traits>

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

// ---- fp32 of any alignment and size: 64 x 64 tiles -------------------------
//
// Bound by the fp32 matrix cores: 4 experts of 2049 x 4097 with 1024 rows 93
// TFLOP/s forward, 97 and 101 back (the library's fp32 product 154 at 8192^3); a
// call of few tiles by the 0.45 us of matrix work that a tile has in each 32-deep
// slab: 2 experts of 2613 x 3776 with 8 rows forward 126 us, 3776 x 2613 back 206.

// A tile of the result, one value at a time: rounded once, from the fp32 sum.
// Old values are loaded all before the first store: a load behind a store
// would wait for it.
__device__ __forceinline__ void put_tile(const any::f32x16& acc, float* out, int64_t ld, int rows, int cols,
                                         int accumulate) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = 32 * (wave & 1) + (lane & 31), row0 = 32 * (wave >> 1) + 4 * (lane >> 5);
    if (col >= cols) return;
    float v[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int row = row0 + 8 * (r >> 2) + (r & 3);
        v[r] = acc[r];
        if (accumulate && row < rows) v[r] += gld(out + (int64_t)row * ld + col);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int row = row0 + 8 * (r >> 2) + (r & 3);
        if (row < rows) gst(out + (int64_t)row * ld + col, v[r]);
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
    const any::Operand p{reinterpret_cast<const float*>(c.a) + (int64_t)i0 * c.ld_a, c.ld_a, nrows};
    const float* we = reinterpret_cast<const float*>(w.w[g.e]);
    const any::Operand q{we + (OP == kExpertForward ? (int64_t)j0 * c.ld_w : j0), c.ld_w, ncols};
    const any::f32x16 acc = any::product<false, OP == kExpertGradInput>(p, q, 0, K, lds);
    put_tile(acc, reinterpret_cast<float*>(c.c) + (int64_t)i0 * c.ld_c + j0, c.ld_c, nrows, ncols, 0);
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
    const any::Operand p{reinterpret_cast<const float*>(c.b) + (int64_t)r0 * c.ld_b + i0, c.ld_b, nrows};
    const any::Operand q{reinterpret_cast<const float*>(c.a) + (int64_t)r0 * c.ld_a + j0, c.ld_a, ncols};
    const any::f32x16 acc = any::product<true, true>(p, q, 0, r1 - r0, lds);
    put_tile(acc, reinterpret_cast<float*>(w.w[e]) + (int64_t)i0 * c.ld_w + j0, c.ld_w, nrows, ncols, c.accumulate);
}

// ---- bf16 on the matrix cores ------------------------------------------------

// Row tiles of all groups.
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

// Workgroup b runs on XCD b % 8, each with an L2 of its own.  Rounds of 8 S
// tiles deal runs of S consecutive tiles to the XCDs (S: the workgroups one
// XCD runs at a time), so those share operand panels, and neighbouring XCDs work on
// the same expert, whose panels then come from the memory-side cache; what is
// left after the last whole round is cut into 8 runs.
template <int S>
__device__ __forceinline__ int dealt_tile(int b, int total) {
    const int x = b & 7, t = b >> 3;
    const int full = total / (8 * S);
    if (t < S * full) return ((t / S) * 8 + x) * S + t % S;
    const int rest = total - 8 * S * full, per = (rest + 7) / 8;
    const int u = t - S * full;
    const int tile = x * per + u;
    return u < per && tile < rest ? 8 * S * full + tile : -1;
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

// Where tile (mt, nt) of BM x BN lies: its group, first row and operands.
struct RowsTile {
    bf::Operand p, q;
    uint16_t* out;
    int K, rows, cols;
};

// False: no tile for this workgroup.  S: workgroups an XCD runs at a time.
template <ExpertOp OP, int BM, int BN, int S, int CAP>
__device__ __forceinline__ bool rows_tile_of(const ExpertCall& c, const ExpertPtrs<CAP>& w, int ntiles, RowsTile& t) {
    const int tile = dealt_tile<S>(blockIdx.x, count_tiles<BM>(c) * ntiles);
    if (tile < 0) return false;
    Group g;
    if (!find_group<BM>(c, tile / ntiles, g)) return false;
    const int n = g.row1 - g.row0, R = (n + BM - 1) / BM;
    // g.tile counts whole rows of tiles: the tile's place within the group
    int mt, nt;
    tile_of(g.tile * ntiles + tile % ntiles, R, ntiles, mt, nt);
    // the group's rows in R equal tiles: tiles that share a weight panel run
    // at one speed and find it in the L2 (320 rows as 160 + 160 instead of
    // 256 + 64: 763 -> 739 us over 64 experts)
    const int H = ((n + R - 1) / R + 7) / 8 * 8;
    constexpr bool QKM = OP == kExpertGradInput;
    const int N = QKM ? c.cols : c.rows, K = QKM ? c.rows : c.cols;
    const int i0 = g.row0 + mt * H, j0 = nt * BN;
    t.K = K;
    t.rows = min(H, g.row1 - i0);
    t.cols = min(BN, N - j0);
    if (t.rows <= 0) return false;
    const uint16_t* a = reinterpret_cast<const uint16_t*>(c.a) + (int64_t)i0 * c.ld_a;
    t.p = bf::Operand{a, c.ld_a, 2 * ((int64_t)(t.rows - 1) * c.ld_a + K)};
    const uint16_t* we = reinterpret_cast<const uint16_t*>(w.w[g.e]);
    t.q = QKM ? bf::Operand{we + j0, c.ld_w, 2 * ((int64_t)(K - 1) * c.ld_w + N - j0)}
              : bf::Operand{we + (int64_t)j0 * c.ld_w, c.ld_w, 2 * ((int64_t)(t.cols - 1) * c.ld_w + K)};
    t.out = reinterpret_cast<uint16_t*>(c.c) + (int64_t)i0 * c.ld_c + j0;
    return true;
}

template <class C, class S>
__device__ __forceinline__ void rows_product(const ExpertCall& c, const RowsTile& t, const S& st) {
    bf::f32x16 acc[C::FM][C::FN];
    bf::zero<C>(acc);
    if constexpr (std::is_same<S, bf::TurnStages>::value)
        bf::product_in_turns<C>(acc, t.p, t.q, t.K, t.rows, st);
    else
        bf::product<C>(acc, t.p, t.q, t.K, st);
    const int64_t ld = c.ld_c;
    bf::for_each_chunk<C>(acc, reinterpret_cast<float*>(st.q[0]), t.rows, [&](int r, int c8, const float* v) {
        if (r < t.rows && c8 < t.cols) gst(reinterpret_cast<uint4*>(t.out + r * ld + c8), bf::pack8(v));
    });
}

// Forward and input gradient on 256 x 256 tiles of eight waves, or the shorter
// kind that holds the tile's rows.
//
// 32768 rows over 61 of 64 experts, 2048 x 7168: 880 us, 1.09 PFLOP/s of
// products that count (13% more are computed for rows that pad a tile); 64
// experts with 512 rows each 780 us, 1.24 PFLOP/s; one expert with all those rows
// 682 us, 1.41 PFLOP/s, where the library's dense product takes 618.  With both
// waves of a SIMD reading and multiplying at the same time (product()) the three
// took 1000, 880 and 786 us.  What bounds it now are the matrix cores' power (the
// dense product of zeros takes 535 us, the library's 530) and the weights, which
// two or three row tiles share.
template <ExpertOp OP, int CAP>
__global__ __launch_bounds__(512) void expert_rows_kernel(ExpertCall c, ExpertPtrs<CAP> w, int ntiles) {
    constexpr int S = kBN * 64;
    __shared__ __attribute__((aligned(1024))) uint16_t p0[S], p1[S], q0[S], q1[S], q2[S];
    const bf::TurnStages st{{p0, p1}, {q0, q1, q2}};
    RowsTile t;
    if (!rows_tile_of<OP, kBM, kBN, 32>(c, w, ntiles, t)) return;
    constexpr bool QKM = OP == kExpertGradInput;
    if (t.rows > 192)
        rows_product<bf::Cfg<256, kBN, 2, 4, false, QKM>>(c, t, st);
    else if (t.rows > 128)
        rows_product<bf::Cfg<192, kBN, 2, 4, false, QKM>>(c, t, st);
    else if (t.rows > 64)
        rows_product<bf::Cfg<128, kBN, 2, 4, false, QKM>>(c, t, st);
    else
        rows_product<bf::Cfg<64, kBN, 2, 4, false, QKM>>(c, t, st);
}

// Launches whose 256 x 256 tiles would leave compute units idle: 128 x 128
// tiles of four waves, two workgroups a compute unit (see mid_tiles).
constexpr int kMidM = 128, kMidN = 128;

template <ExpertOp OP, int CAP>
__global__ __launch_bounds__(256) void expert_mid_kernel(ExpertCall c, ExpertPtrs<CAP> w, int ntiles) {
    constexpr int S = kMidN * 64;
    __shared__ __attribute__((aligned(1024))) uint16_t l0[S], l1[S], l2[S], l3[S];
    const bf::Stages<2> st{{l0, l2}, {l1, l3}};
    RowsTile t;
    if (!rows_tile_of<OP, kMidM, kMidN, 64>(c, w, ntiles, t)) return;
    constexpr bool QKM = OP == kExpertGradInput;
    if (t.rows > 64)
        rows_product<bf::Cfg<128, kMidN, 2, 2, false, QKM>>(c, t, st);
    else
        rows_product<bf::Cfg<64, kMidN, 2, 2, false, QKM>>(c, t, st);
}

// Few rows a group: reading the weights is what it takes.  32 x 64 tiles of
// two waves, four stages, three workgroups a compute unit: three slabs of 8 KB
// of weights in flight each, and enough tiles to go round.  HBM bounds it: 64
// rows over 41 of 64 experts (1.2 GB of weights) 202-206 us, 5.9 TB/s, where the
// 256 x 256 tiles took 300 (328 of them for 256 compute units).
constexpr int kFewM = 32, kFewN = 64;
// Mean rows of a group up to which it is taken.  64 experts of 2048 x 7168,
// against the 256 x 256 tiles: forward at 32 rows 334 and 347 us (at 1 row 311
// and 336), input gradient at 4 rows 324 and 350, at 16 rows 357 and 354.
constexpr int kFewRows[2] = {32, 12};

template <ExpertOp OP, int CAP>
__global__ __launch_bounds__(128) void expert_few_kernel(ExpertCall c, ExpertPtrs<CAP> w, int ntiles) {
    constexpr int SP = kFewM * 64, SQ = kFewN * 64;
    __shared__ __attribute__((aligned(1024))) uint16_t p0[SP], p1[SP], p2[SP], p3[SP], q0[SQ], q1[SQ], q2[SQ], q3[SQ];
    const bf::Stages<4> st{{p0, p1, p2, p3}, {q0, q1, q2, q3}};
    RowsTile t;
    if (!rows_tile_of<OP, kFewM, kFewN, 96>(c, w, ntiles, t)) return;
    rows_product<bf::Cfg<kFewM, kFewN, 1, 2, false, OP == kExpertGradInput, 64, 4>>(c, t, st);
}

// Four values of a result, or as many as its row still holds, at the alignment
// of 16 (8) bytes or, LOOSE, of one value.
template <bool LOOSE>
__device__ __forceinline__ float4 load4(const float* p, int left) {
    typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
    if (!LOOSE) return gld(reinterpret_cast<const float4*>(p));
    if (left >= 4) {
        const f4 v = *(const MUON_GLOBAL f4*)p;
        return make_float4(v.x, v.y, v.z, v.w);
    }
    return make_float4(left > 0 ? gld(p) : 0.f, left > 1 ? gld(p + 1) : 0.f, left > 2 ? gld(p + 2) : 0.f, 0.f);
}
template <bool LOOSE>
__device__ __forceinline__ float4 load4(const uint16_t* p, int left) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
    uint2 w = make_uint2(0, 0);
    if (!LOOSE) {
        w = gld(reinterpret_cast<const uint2*>(p));
    } else if (left >= 4) {
        const u2 v = *(const MUON_GLOBAL u2*)p;
        w = make_uint2(v.x, v.y);
    } else {
        if (left > 0) w.x = gld(p);
        if (left > 1) w.x |= (uint32_t)gld(p + 1) << 16;
        if (left > 2) w.y = gld(p + 2);
    }
    return make_float4(bf16_bits_to_f32(w.x & 0xffff), bf16_bits_to_f32(w.x >> 16), bf16_bits_to_f32(w.y & 0xffff),
                       bf16_bits_to_f32(w.y >> 16));
}
template <bool LOOSE>
__device__ __forceinline__ void store4(float* p, int left, const float4& v) {
    typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
    if (!LOOSE) {
        if (left > 0) gst(reinterpret_cast<float4*>(p), v);
    } else if (left >= 4) {
        *(MUON_GLOBAL f4*)p = f4{v.x, v.y, v.z, v.w};
    } else {
        if (left > 0) gst(p, v.x);
        if (left > 1) gst(p + 1, v.y);
        if (left > 2) gst(p + 2, v.z);
    }
}
template <bool LOOSE>
__device__ __forceinline__ void store4(uint16_t* p, int left, const float4& v) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
    const uint16_t a = f32_to_bf16_bits(v.x), b = f32_to_bf16_bits(v.y), c = f32_to_bf16_bits(v.z),
                   d = f32_to_bf16_bits(v.w);
    const uint2 w = make_uint2(a | (uint32_t)b << 16, c | (uint32_t)d << 16);
    if (!LOOSE) {
        if (left > 0) gst(reinterpret_cast<uint2*>(p), w);
    } else if (left >= 4) {
        *(MUON_GLOBAL u2*)p = u2{w.x, w.y};
    } else {
        if (left > 0) gst(p, a);
        if (left > 1) gst(p + 1, b);
        if (left > 2) gst(p + 2, c);
    }
}

// The tile at `out`, rounded once, or added to what it holds: old values are
// loaded one band ahead.  mine: the wave's 16 x TN floats of LDS.
template <class C, class T, bool ADD, bool LOOSE>
__device__ __forceinline__ void store_result(const bf::f32x16 (&acc)[C::FM][C::FN], float* mine, T* out, int64_t ld,
                                             int rows, int cols) {
    constexpr int P = bf::wave_pieces<C>();
    float4 old[2][P];
    const int col = bf::wave_col<C>();
    auto load_old = [&](int b) {
        if constexpr (ADD) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                // behind the last row (and, not LOOSE, column): any value in range
                const int r = min(bf::wave_row<C>(b, i), rows - 1);
                old[b & 1][i] = load4<LOOSE>(out + r * ld + (LOOSE ? col : min(col, cols - 4)), cols - col);
            }
        }
    };
    load_old(0);
    bf::for_each_piece<C>(acc, mine, [&](int b) { if (b + 1 < C::TM / 16) load_old(b + 1); },
                          [&](int b, int i, int r, int, float4 v) {
        if constexpr (ADD) {
            const float4& o = old[b & 1][i];
            v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
        }
        if (r < rows) store4<LOOSE>(out + r * ld + col, cols - col, v);
    });
}

// Weight gradient on 128 x 256 tiles of four waves, two workgroups a compute
// unit: a group's rows are a short K, so reading and writing dW is most of
// the traffic, and one workgroup does it while the other multiplies.  With
// accumulate the old values of a band are loaded one band ahead.  64 experts of
// 2048 x 7168 with 512 rows each, added to fp32: 1.93 ms (1.47 with 64 rows,
// where reading and writing dW is all; 256 x 256 tiles of eight waves 2.04,
// 128 x 128 tiles 2.11, dW in 128-byte pieces from the accumulators 2.04);
// written, 1.52 ms in fp32 and 1.21 in bf16: the products (0.82 at the library's
// rate) and the stores of dW overlap in part only.  A workgroup walks all rows
// of its group: few tiles with many rows leave compute units idle (one expert of
// 128 x 256 with 32768 rows is one workgroup and 325 us).
constexpr int kWM = 128, kWN = 256;

template <int CAP, bool OBF, bool ADD>
__global__ __launch_bounds__(256, 2) void expert_weight_kernel(ExpertCall c, ExpertPtrs<CAP> w, int mtiles, int ntiles) {
    using C = bf::Cfg<kWM, kWN, 2, 2, true, true, 32, 3>;
    constexpr int SP = kWM * 32, SQ = kWN * 32;
    __shared__ __attribute__((aligned(1024))) uint16_t lp0[SP], lq0[SQ], lp1[SP], lq1[SQ], lp2[SP], lq2[SQ];
    const bf::Stages<3> st{{lp0, lp1, lp2}, {lq0, lq1, lq2}};
    const int per = mtiles * ntiles;
    const int tile = dealt_tile<64>(blockIdx.x, per * c.experts);
    if (tile < 0) return;
    const int e = tile / per;
    int r0, r1, mt, nt;
    group_rows(c, e, r0, r1);
    r0 = __builtin_amdgcn_readfirstlane(r0);
    r1 = __builtin_amdgcn_readfirstlane(r1);
    if (ADD && r1 == r0) return;
    tile_of(tile - e * per, mtiles, ntiles, mt, nt);
    const int i0 = mt * kWM, j0 = nt * kWN, K = r1 - r0;
    const int rows = min(kWM, c.rows - i0), cols = min(kWN, c.cols - j0);
    const bf::Operand p{reinterpret_cast<const uint16_t*>(c.b) + (int64_t)r0 * c.ld_b + i0, c.ld_b,
                        2 * ((int64_t)(K - 1) * c.ld_b + c.rows - i0)};
    const bf::Operand q{reinterpret_cast<const uint16_t*>(c.a) + (int64_t)r0 * c.ld_a + j0, c.ld_a,
                        2 * ((int64_t)(K - 1) * c.ld_a + c.cols - j0)};
    using T = typename std::conditional<OBF, uint16_t, float>::type;
    bf::f32x16 acc[C::FM][C::FN];
    bf::zero<C>(acc);
    bf::product<C>(acc, p, q, K, st);
    __syncthreads();  // every wave has read its last fragments
    const int wave = threadIdx.x >> 6;
    store_result<C, T, ADD, false>(acc, reinterpret_cast<float*>(wave < 2 ? lq0 : lq1) + wave % 2 * 16 * C::TN,
                                   reinterpret_cast<T*>(w.w[e]) + (int64_t)i0 * c.ld_w + j0, c.ld_w, rows, cols);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// bf16 operands whose rows all start on 16 bytes and hold whole 16-byte
// chunks: copied to LDS as they are.  Others go through registers.
bool chunked(ExpertOp op, const ExpertCall& c, const void* const* w) {
    if (!c.bf16 || c.rows % 8 || c.cols % 8 || c.ld_a % 8 || c.ld_w % 8 || !aligned16(c.a)) return false;
    if (op == kExpertGradWeight ? (c.ld_b % 8 || !aligned16(c.b)) : (c.ld_c % 8 || !aligned16(c.c))) return false;
    for (int e = 0; e < c.experts; ++e)
        if (!aligned16(w[e])) return false;
    return true;
}

// Whether 128 x 128 tiles take less time than 256 x 256 ones: in hundredths of
// a microsecond for each slab of K, a round of 256 big tiles takes 110, and the
// launch 8 more for their longer start (in proportion to K as the rest is, over
// the 16 to 112 slabs measured); a round of 512 small ones, two a compute unit,
// 115, of up to 256 76.  Measured, big and small: 8 experts of 1024 x 1024, 512 rows each
// (64 and 256 tiles) 26.0 and 16.0 us; 16 of 2048 x 2048, 256 rows (128 and
// 512) 41.9 and 41.4; 64 of 2048 x 7168, 128 rows (512 and 1024) 359 and 390; 8
// of 2056 outputs, 512 rows, K = 1000 (144 and 544) 29.0 and 40.9.
bool mid_tiles(int64_t big, int64_t mid) {
    const int64_t tb = (big + 255) / 256 * 110 + 8;
    const int64_t rest = mid % 512;
    const int64_t tm = mid / 512 * 115 + (rest == 0 ? 0 : rest <= 256 ? 76 : 115);
    return tm < tb;
}

// A launch holds fewer than 2^32 threads.
bool launch_fits(int64_t blocks, int threads) { return blocks * threads <= UINT32_MAX; }

template <int CAP>
hipError_t launch_bf16(ExpertOp op, const ExpertCall& c, const ExpertPtrs<CAP>& w, hipStream_t st) {
    // dealt_tile covers every tile where the grid holds at least as many
    // blocks, in whole groups of 8
    auto grid = [](int64_t tiles) { return (unsigned)((tiles + 7) / 8 * 8); };
    if (op == kExpertGradWeight) {
        const int mt = (c.rows + kWM - 1) / kWM, nt = (c.cols + kWN - 1) / kWN;
        const unsigned n = grid((int64_t)c.experts * mt * nt);
        if (!launch_fits(n, 256)) return hipErrorInvalidConfiguration;
        if (c.out_bf16) {
            if (c.accumulate)
                expert_weight_kernel<CAP, true, true><<<n, 256, 0, st>>>(c, w, mt, nt);
            else
                expert_weight_kernel<CAP, true, false><<<n, 256, 0, st>>>(c, w, mt, nt);
        } else {
            if (c.accumulate)
                expert_weight_kernel<CAP, false, true><<<n, 256, 0, st>>>(c, w, mt, nt);
            else
                expert_weight_kernel<CAP, false, false><<<n, 256, 0, st>>>(c, w, mt, nt);
        }
    } else {
        const int N = op == kExpertForward ? c.rows : c.cols;
        auto tiles = [&](int64_t groups, int64_t rows, int bm, int bn) {
            return groups * ((rows + bm - 1) / bm) * ((N + bn - 1) / bn);
        };
        const int64_t mean = (c.tokens + c.experts - 1) / c.experts;
        const bool few = mean <= kFewRows[op];
        // as if every group had the mean rows
        const bool mid = !few && mid_tiles(tiles(c.experts, mean, kBM, kBN), tiles(c.experts, mean, kMidM, kMidN));
        const int bm = few ? kFewM : mid ? kMidM : kBM, bn = few ? kFewN : mid ? kMidN : kBN;
        const int64_t mt = c.tokens / bm + (c.tokens < c.experts ? c.tokens : c.experts);
        const int nt = (N + bn - 1) / bn;
        const unsigned n = grid(mt * nt);
        if (!launch_fits(n, few ? 128 : mid ? 256 : 512)) return hipErrorInvalidConfiguration;
        if (op == kExpertForward) {
            if (few)
                expert_few_kernel<kExpertForward, CAP><<<n, 128, 0, st>>>(c, w, nt);
            else if (mid)
                expert_mid_kernel<kExpertForward, CAP><<<n, 256, 0, st>>>(c, w, nt);
            else
                expert_rows_kernel<kExpertForward, CAP><<<n, 512, 0, st>>>(c, w, nt);
        } else {
            if (few)
                expert_few_kernel<kExpertGradInput, CAP><<<n, 128, 0, st>>>(c, w, nt);
            else if (mid)
                expert_mid_kernel<kExpertGradInput, CAP><<<n, 256, 0, st>>>(c, w, nt);
            else
                expert_rows_kernel<kExpertGradInput, CAP><<<n, 512, 0, st>>>(c, w, nt);
        }
    }
    return hipGetLastError();
}

// ---- bf16 of any alignment and size -------------------------------------------

// T x T tiles of four waves through registers; blocks as in the fp32 kernels.
// Bound by the registers' way into LDS and by value-aligned accesses: 8 experts
// of 1001 x 2057, 512 rows each, forward 53 us (317 TFLOP/s; 34 us at 1000 x
// 2056 on the kernels above), input gradient 75, weight gradient 92; 4 of 2049 x
// 4097, 1024 rows each, 228, 248 and 245 us; 2 experts of 2613 x 3776 with 8 rows
// forward 56 us, input gradient of 3777 x 2613 153.
template <ExpertOp OP, int T, int CAP>
__global__ __launch_bounds__(256) void expert_rows_loose_kernel(ExpertCall c, ExpertPtrs<CAP> w, int ntiles) {
    constexpr bool QKM = OP == kExpertGradInput;
    using C = bf::Cfg<T, T, 2, 2, false, QKM>;
    __shared__ __attribute__((aligned(1024))) uint16_t l0[T * 64], l1[T * 64], l2[T * 64], l3[T * 64];
    const bf::Stages<2> st{{l0, l2}, {l1, l3}};
    const int mt = blockIdx.x / ntiles, nt = blockIdx.x - mt * ntiles;
    Group g;
    if (!find_group<T>(c, mt, g)) return;
    const int i0 = g.row0 + g.tile * T, j0 = nt * T;
    const int N = QKM ? c.cols : c.rows, K = QKM ? c.rows : c.cols;
    const int rows = min(T, g.row1 - i0), cols = min(T, N - j0);
    const uint16_t* we = reinterpret_cast<const uint16_t*>(w.w[g.e]);
    const bf::AnyOperand p{reinterpret_cast<const uint16_t*>(c.a) + (int64_t)i0 * c.ld_a, c.ld_a, rows};
    const bf::AnyOperand q{we + (QKM ? j0 : (int64_t)j0 * c.ld_w), c.ld_w, cols};
    bf::f32x16 acc[C::FM][C::FN];
    bf::zero<C>(acc);
    bf::product_any<C>(acc, p, q, K, st);
    store_result<C, uint16_t, false, true>(acc, reinterpret_cast<float*>(l0) + (threadIdx.x >> 6) * 16 * C::TN,
                                           reinterpret_cast<uint16_t*>(c.c) + (int64_t)i0 * c.ld_c + j0, c.ld_c, rows,
                                           cols);
}

template <int T, int CAP, bool OBF, bool ADD>
__global__ __launch_bounds__(256) void expert_weight_loose_kernel(ExpertCall c, ExpertPtrs<CAP> w, int mtiles, int ntiles) {
    using C = bf::Cfg<T, T, 2, 2, true, true>;
    __shared__ __attribute__((aligned(1024))) uint16_t l0[T * 64], l1[T * 64], l2[T * 64], l3[T * 64];
    const bf::Stages<2> st{{l0, l2}, {l1, l3}};
    const int per = mtiles * ntiles;
    const int e = blockIdx.x / per, rest = blockIdx.x - e * per;
    const int mt = rest / ntiles, nt = rest - mt * ntiles;
    int r0, r1;
    group_rows(c, e, r0, r1);
    if (ADD && r1 == r0) return;
    const int i0 = mt * T, j0 = nt * T;
    const int rows = min(T, c.rows - i0), cols = min(T, c.cols - j0);
    const bf::AnyOperand p{reinterpret_cast<const uint16_t*>(c.b) + (int64_t)r0 * c.ld_b + i0, c.ld_b, rows};
    const bf::AnyOperand q{reinterpret_cast<const uint16_t*>(c.a) + (int64_t)r0 * c.ld_a + j0, c.ld_a, cols};
    bf::f32x16 acc[C::FM][C::FN];
    bf::zero<C>(acc);
    bf::product_any<C>(acc, p, q, r1 - r0, st);
    using O = typename std::conditional<OBF, uint16_t, float>::type;
    store_result<C, O, ADD, true>(acc, reinterpret_cast<float*>(l0) + (threadIdx.x >> 6) * 16 * C::TN,
                                  reinterpret_cast<O*>(w.w[e]) + (int64_t)i0 * c.ld_w + j0, c.ld_w, rows, cols);
}

template <int T, int CAP>
hipError_t launch_loose(ExpertOp op, const ExpertCall& c, const ExpertPtrs<CAP>& w, hipStream_t st) {
    const int64_t nr = (c.rows + T - 1) / T, nc = (c.cols + T - 1) / T;
    const int64_t mt = c.tokens / T + (c.tokens < c.experts ? c.tokens : c.experts);
    if (!launch_fits(op == kExpertGradWeight ? c.experts * nr * nc : mt * (op == kExpertForward ? nr : nc), 256))
        return hipErrorInvalidConfiguration;
    if (op == kExpertGradWeight) {
        const unsigned n = (unsigned)(c.experts * nr * nc);
        if (c.out_bf16) {
            if (c.accumulate)
                expert_weight_loose_kernel<T, CAP, true, true><<<n, 256, 0, st>>>(c, w, (int)nr, (int)nc);
            else
                expert_weight_loose_kernel<T, CAP, true, false><<<n, 256, 0, st>>>(c, w, (int)nr, (int)nc);
        } else {
            if (c.accumulate)
                expert_weight_loose_kernel<T, CAP, false, true><<<n, 256, 0, st>>>(c, w, (int)nr, (int)nc);
            else
                expert_weight_loose_kernel<T, CAP, false, false><<<n, 256, 0, st>>>(c, w, (int)nr, (int)nc);
        }
    } else if (op == kExpertForward)
        expert_rows_loose_kernel<kExpertForward, T, CAP><<<(unsigned)(mt * nr), 256, 0, st>>>(c, w, (int)nr);
    else
        expert_rows_loose_kernel<kExpertGradInput, T, CAP><<<(unsigned)(mt * nc), 256, 0, st>>>(c, w, (int)nc);
    return hipGetLastError();
}

template <int CAP>
hipError_t launch_any(ExpertOp op, const ExpertCall& c, const ExpertPtrs<CAP>& w, hipStream_t st) {
    const int T = any::kTile;
    const int64_t nr = (c.rows + T - 1) / T, nc = (c.cols + T - 1) / T;
    // at most this many row tiles: every group may end in a ragged one
    const int64_t mt = c.tokens / T + (c.tokens < c.experts ? c.tokens : c.experts);
    const int64_t tiles = op == kExpertGradWeight ? c.experts * nr * nc : mt * (op == kExpertForward ? nr : nc);
    if (c.bf16) {
        // 128 x 128 tiles where they fill the chip twice (4 experts of 2049 x
        // 4097, 1024 rows: 227 us), else 64 x 64
        return tiles >= 4 * 1024 ? launch_loose<128, CAP>(op, c, w, st) : launch_loose<64, CAP>(op, c, w, st);
    }
    if (!launch_fits(tiles, 256)) return hipErrorInvalidConfiguration;
    if (op == kExpertGradWeight)
        expert_weight_any_kernel<CAP><<<(unsigned)(c.experts * nr * nc), 256, 0, st>>>(c, w, (int)nr, (int)nc);
    else if (op == kExpertForward)
        expert_rows_any_kernel<kExpertForward, CAP><<<(unsigned)(mt * nr), 256, 0, st>>>(c, w, (int)nr);
    else
        expert_rows_any_kernel<kExpertGradInput, CAP><<<(unsigned)(mt * nc), 256, 0, st>>>(c, w, (int)nc);
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
