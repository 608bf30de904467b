// bf16 product tiles on the matrix cores (gfx950) for operands that are not
// padded: C[i][j] = sum_k P[i][k] Q[j][k] over rows that end anywhere, a K of
// any multiple of 8, and any leading dimension that is a multiple of 8.
//
// A workgroup of WM x WN waves computes BM x BN, each wave a block of 32 x 32
// MFMA tiles (v_mfma_f32_32x32x16_bf16, fp32 accumulation).  K advances in
// slabs of BK (32 or 64), copied global -> LDS with buffer_load_dwordx4 ... lds (16 bytes
// per lane, no registers in between).  The copies go through buffer resources
// that end where the operand does: a row or k behind the end reads as zero,
// so ragged ends need no branch and no memory traffic, and a value that lies
// behind an end, a NaN included, never reaches a sum.
//
// An operand is stored with k along its rows (K-contiguous: rows are the
// tile's rows) or k-major (rows are k).  k-major slabs are copied as they are
// and gathered with the transposing LDS read (ds_read_b64_tr_b16).
#pragma once

#include <utility>

#include "muon_internal.h"

namespace muon {
namespace bf {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

// PKM, QKM: the operand is stored k-major.  BK: k per slab; NS: LDS stages.
template <int BM_, int BN_, int WM_, int WN_, bool PKM_, bool QKM_, int BK_ = 64, int NS_ = 2>
struct Cfg {
    static constexpr int BK = BK_, NS = NS_;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr bool PKM = PKM_, QKM = QKM_;
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int TM = BM / WM, TN = BN / WN;
    static constexpr int FM = TM / 32, FN = TN / 32;
    static constexpr int CH = BK / 8;                          // 16-byte chunks of a K-contiguous row
    static constexpr int LPS = (BM + BN) * BK / 512 / NW;      // copies of a wave and stage
    static_assert(FM >= 1 && FN >= 1 && BM % 32 == 0 && BN % 64 == 0, "32 x 32 blocks per wave");
    static_assert(BM * BK / 512 % NW == 0 && BN * BK / 512 % NW == 0, "slab copies split evenly over the waves");
    static_assert((BK == 32 || BK == 64) && NS >= 2 && NS <= 5, "");
    static_assert(32 * BN % (8 * NT) == 0, "epilogue chunks split evenly over the threads");
};

// One operand of a tile.  K-contiguous: row i at base + i * ld, `bytes` from
// base to the end of the last valid row.  k-major: k at base + k * ld, `bytes`
// from base to the end of the last valid k.
struct Operand {
    const uint16_t* base;
    int64_t ld;
    int64_t bytes;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const uint16_t* base, int64_t bytes) {
    const int32_t n = bytes <= 0 ? 0 : bytes > 0x7fffffff ? 0x7fffffff : (int32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, n, 0x00020000);
}

// LDS slab of a K-contiguous operand: BK bf16 (8 or 4 chunks of 16 bytes) per
// row, chunk c at position c ^ swz(row): the 16 lanes of one LDS cycle read one
// chunk of 16 consecutive rows, on 16 different positions of the 64 banks.
template <int BK = 64>
__device__ __forceinline__ int swz(int row) { return BK == 64 ? (row >> 1) & 7 : (row >> 2) & 3; }
// k-major slab of W columns: chunk c of row k at c ^ swzk(k): the 4 rows x 64
// bytes of a transposing read lie on disjoint quarters of the banks (a row of
// 64 columns is half of them).
template <int W>
__device__ __forceinline__ int swzk(int k) { return W == 64 ? (k & 2) << 1 : (k & 3) << 2; }

// Copies of k [k0, k0 + BK) of R rows into an LDS slab; NW waves share them.
// Lane l of a copy fills chunk position l % CH of row l / CH.
template <int R, int NW, int BK>
__device__ __forceinline__ void copy_rows(const Operand& o, int64_t k0, int64_t K, uint16_t* slab, int wave,
                                          int lane) {
    constexpr int CH = BK / 8, RPC = 64 / CH;  // chunks of a row, rows of a copy
    const __amdgpu_buffer_rsrc_t r = resource(o.base + k0, o.bytes - 2 * k0);
    const int left = K - k0 < BK ? (int)(K - k0) : BK;  // a multiple of 8
#pragma unroll
    for (int q = 0; q < R / RPC / NW; ++q) {
        const int grp = wave * (R / RPC / NW) + q;
        const int row = grp * RPC + lane / CH;
        const int c = (lane % CH) ^ swz<BK>(row);
        // a chunk behind K would be the next row's: pushed out of range
        const uint32_t off = c * 8 < left ? (uint32_t)(row * (int)o.ld + c * 8) * 2u : 0x80000000u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(slab + grp * RPC * BK), 16, off, 0, 0, 0);
    }
}

// ... of a k-major operand: BK rows k of W columns.
template <int W, int NW, int BK>
__device__ __forceinline__ void copy_kmajor(const Operand& o, int64_t k0, uint16_t* slab, int wave, int lane) {
    constexpr int CQ = W / 8, RPK = 64 / CQ;  // chunks of a row, rows of a copy
    static_assert(CQ <= 64 && (BK / RPK) % NW == 0, "k-major copies split evenly over the waves");
    const __amdgpu_buffer_rsrc_t r = resource(o.base + k0 * o.ld, o.bytes - 2 * k0 * o.ld);
#pragma unroll
    for (int q = 0; q < BK / RPK / NW; ++q) {
        const int grp = wave * (BK / RPK / NW) + q;
        const int k = grp * RPK + lane / CQ;
        const uint32_t off = (uint32_t)(k * (int)o.ld + (((lane % CQ) ^ swzk<W>(k)) * 8)) * 2u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(slab + grp * RPK * W), 16, off, 0, 0, 0);
    }
}

// MFMA operand fragment: lane l holds row l % 32, k = 8 (l / 32) + 0..7.
template <int BK = 64>
__device__ __forceinline__ bf16x8 frag_rows(const uint16_t* slab, int row, int chunk) {
    return *reinterpret_cast<const bf16x8*>(slab + row * BK + ((chunk ^ swz<BK>(row)) << 3));
}
// ... from a k-major slab of W columns, as two transposing 8-byte reads: in
// each group of 16 lanes, lane a + 4 b addresses row b, columns 4a ... 4a + 3
// of a 4 x 16 block and receives column (lane % 16) of rows 0 ... 3.
template <int W>
__device__ __forceinline__ bf16x8 frag_kmajor(const uint16_t* slab, int k0, int n0, int lane) {
    const int g = lane >> 4, s16 = lane & 15;
    const int n = n0 + 16 * (g & 1) + 4 * (s16 & 3);
    i16x4 h[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int k = k0 + 8 * (g >> 1) + 4 * t + (s16 >> 2);
        const uint16_t* p = slab + k * W + (((n >> 3) ^ swzk<W>(k)) << 3) + (n & 7);
        h[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(p));
    }
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// LDS stages, one array per operand and stage, each its own __shared__
// variable: the compiler then knows that a copy into one leaves the others
// alone.
template <int NS>
struct Stages {
    uint16_t *p[NS], *q[NS];
};

template <class C>
struct Frags {
    bf16x8 a[C::FM], b[C::FN];
};

template <class C>
__device__ __forceinline__ void read_frags(const uint16_t* sp, const uint16_t* sq, int kk, int wm, int wn,
                                           int lane, Frags<C>& f) {
    const int row = lane & 31, chunk = 2 * kk + (lane >> 5);
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
        f.a[i] = C::PKM ? frag_kmajor<C::BM>(sp, 16 * kk, wm * C::TM + i * 32, lane)
                        : frag_rows<C::BK>(sp, wm * C::TM + i * 32 + row, chunk);
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
        f.b[j] = C::QKM ? frag_kmajor<C::BN>(sq, 16 * kk, wn * C::TN + j * 32, lane)
                        : frag_rows<C::BK>(sq, wn * C::TN + j * 32 + row, chunk);
}

// Blocks of rows [I0, I1).
template <class C, int I0, int I1>
__device__ __forceinline__ void mfma_rows(f32x16 (&acc)[C::FM][C::FN], const Frags<C>& f) {
#pragma unroll
    for (int i = I0; i < I1; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}
template <class C>
__device__ __forceinline__ void mfma_frags(f32x16 (&acc)[C::FM][C::FN], const Frags<C>& f) {
    mfma_rows<C, 0, C::FM>(acc, f);
}

template <class C>
__device__ __forceinline__ void copy_p(const Operand& p, int64_t k0, int64_t K, uint16_t* sp, int wave, int lane) {
    if constexpr (C::PKM)
        copy_kmajor<C::BM, C::NW, C::BK>(p, k0, sp, wave, lane);
    else
        copy_rows<C::BM, C::NW, C::BK>(p, k0, K, sp, wave, lane);
}
template <class C>
__device__ __forceinline__ void copy_q(const Operand& q, int64_t k0, int64_t K, uint16_t* sq, int wave, int lane) {
    if constexpr (C::QKM)
        copy_kmajor<C::BN, C::NW, C::BK>(q, k0, sq, wave, lane);
    else
        copy_rows<C::BN, C::NW, C::BK>(q, k0, K, sq, wave, lane);
}

template <class C>
__device__ __forceinline__ void copy_stage(const Operand& p, const Operand& q, int64_t k0, int64_t K,
                                           uint16_t* sp, uint16_t* sq, int wave, int lane) {
    copy_p<C>(p, k0, K, sp, wave, lane);
    copy_q<C>(q, k0, K, sq, wave, lane);
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// Workgroup barrier without a memory fence: the wave's own LDS reads are
// waited for, copies in flight stay in flight (__syncthreads() would wait for
// them).
__device__ __forceinline__ void lds_barrier() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0) only
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// The LDS reads of the next k-step go out two at a time between the first
// MFMAs of this one.
template <int NR, int NM, int T = 0>
__device__ __forceinline__ void interleave() {
    constexpr int G = (NR + 1) / 2;
    if constexpr (T < G && T < NM) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, (T + 1) * 2 <= NR ? 2 : 1, 0);  // DS read
        interleave<NR, NM, T + 1>();
    } else if constexpr (NM > T) {
        __builtin_amdgcn_sched_group_barrier(0x008, NM - T, 0);
    }
}

// f(integral_constant 0), ..., f(integral_constant N - 1): indices that are
// constants before any loop is unrolled, so that every LDS access names its
// array (an access that could be to any array waits for every copy in flight).
template <class F, int... I>
__device__ __forceinline__ void unrolled_(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
    unrolled_(f, std::make_integer_sequence<int, N>{});
}

template <class C>
__device__ __forceinline__ void zero(f32x16 (&acc)[C::FM][C::FN]) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
}

// acc += the tile over k [0, K).  All stages are filled up front; while the
// MFMAs of a k-step (16 deep) run, the fragments of the next are read into
// the other registers.  The last k-step's MFMAs are issued after the barrier
// that frees the slab's stage, so the matrix cores have work while the waves
// meet; the copy of slab kt + NS goes into that stage.  Copies in flight stay
// in flight at the barriers.
template <class C>
__device__ __forceinline__ void product(f32x16 (&acc)[C::FM][C::FN], const Operand& p, const Operand& q,
                                        int64_t K, const Stages<C::NS>& st) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int KT = (int)((K + C::BK - 1) / C::BK);
    if (KT == 0) return;
    constexpr int KS = C::BK / 16, NS = C::NS;
    constexpr int NR = (C::PKM ? 2 : 1) * C::FM + (C::QKM ? 2 : 1) * C::FN;
    // behind K every copy reads zeros, without memory traffic: copies and waits
    // need no condition (the compiler would wait for the path of a condition
    // that leaves the most copies in flight)
    unrolled<NS>([&](auto u) { copy_stage<C>(p, q, u * C::BK, K, st.p[u], st.q[u], wave, lane); });
    wait_vmcnt<(NS - 1) * C::LPS>();
    lds_barrier();
    Frags<C> f[2];
    read_frags<C>(st.p[0], st.q[0], 0, wm, wn, lane, f[0]);
    auto slab = [&](auto u, int kt) {
        constexpr int next = (u + 1) % NS;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            if (kk < KS - 1) {
                read_frags<C>(st.p[u], st.q[u], kk + 1, wm, wn, lane, f[(kk + 1) & 1]);
            } else {
                // slab kt + 1 has landed once only the copies of the
                // slabs after it are outstanding
                wait_vmcnt<(NS - 2) * C::LPS>();
                lds_barrier();
                copy_stage<C>(p, q, (int64_t)(kt + NS) * C::BK, K, st.p[u], st.q[u], wave, lane);
                read_frags<C>(st.p[next], st.q[next], 0, wm, wn, lane, f[0]);
            }
            mfma_frags<C>(acc, f[kk & 1]);
            interleave<NR, C::FM * C::FN>();
        }
    };
    // Whole turns over the stages with no way out between: where one joins the
    // loop's end the compiler takes the copies of both paths to be in flight, and
    // the next turn's first LDS reads wait for them (128 x 128 tiles: 48.5 -> 46.2
    // us for 16 experts of 1024 x 4096 with 256 rows; the bf16 weight gradients of
    // 64 of 2048 x 7168 with 512: 1238 -> 1197).  The kernel for few rows, which
    // has four stages and HBM to wait for, is faster with that wait (205 and 211 us
    // for 64 rows).
    if constexpr (NS < 4) {
        int kt = 0;
        for (; kt + NS <= KT; kt += NS)
            unrolled<NS>([&](auto u) { slab(u, kt + u); });
        unrolled<NS - 1>([&](auto u) {
            if (kt + u < KT) slab(u, kt + u);
        });
    } else {
        for (int kt0 = 0; kt0 < KT; kt0 += NS)
            unrolled<NS>([&](auto u) {
                if (kt0 + u < KT) slab(u, kt0 + u);
            });
    }
    wait_vmcnt<0>();
}

struct TurnStages {
    uint16_t *p[2], *q[3];
};

// As product(), for eight waves, two on each SIMD, of which the waves of the
// tile's lower half run one phase behind those of its upper half: on every
// SIMD one wave has the matrix cores to itself while the other reads its
// operands.  A slab is four phases, each ended by a barrier: the fragments of
// two k-steps are read and copies issued, then multiplied, twice.
//
// The two halves read a stage in phases 4 kt ... 4 kt + 3 (slab kt, the lower half
// from 4 kt + 1), so a stage is free from phase 4 kt + 4 on.  P (rows) has two
// stages: slab kt + 1 is copied from the first phase of slab kt on.  Q (the
// weights, which come from farther away) has three: slab kt + 2 is copied from
// the third phase of slab kt on, and stays in flight at the wait there, which
// is for slab kt + 1: the upper half waits in phase 4 kt + 2, the lower one in 4 kt
// + 3, and the first read is in 4 kt + 4.
//
// rows: the tile's valid rows.  Where they end 32 rows or more before the tile
// does, the lower half leaves its last row of blocks out.
template <class C>
__device__ __forceinline__ void product_in_turns(f32x16 (&acc)[C::FM][C::FN], const Operand& p, const Operand& q,
                                                 int64_t K, int rows, const TurnStages& st) {
    static_assert(C::NW == 8 && C::WM == 2 && C::BK == 64, "two waves a SIMD, slabs of two times two k-steps");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int KT = (int)((K + C::BK - 1) / C::BK);
    if (KT == 0) return;
    constexpr int LQ = C::BN * C::BK / 512 / C::NW;  // copies of a wave and slab of Q
    copy_q<C>(q, 0, K, st.q[0], wave, lane);
    copy_p<C>(p, 0, K, st.p[0], wave, lane);
    copy_q<C>(q, C::BK, K, st.q[1], wave, lane);
    wait_vmcnt<LQ>();
    lds_barrier();
    // a barrier that no LDS read or copy is moved over
    auto meet = []() {
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_s_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (wm == 1) meet();
    const bool whole = wm == 0 || rows > C::BM - 32;
    Frags<C> f[2];
    auto multiply = [&]() {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) mfma_rows<C, 0, C::FM - 1>(acc, f[h]);
        if (whole)
#pragma unroll
            for (int h = 0; h < 2; ++h) mfma_rows<C, C::FM - 1, C::FM>(acc, f[h]);
        __builtin_amdgcn_sched_barrier(0);
        meet();
    };
    auto slab = [&](auto u, int kt) {
        constexpr int up = u % 2, uq = u % 3;
        read_frags<C>(st.p[up], st.q[uq], 0, wm, wn, lane, f[0]);
        read_frags<C>(st.p[up], st.q[uq], 1, wm, wn, lane, f[1]);
        copy_p<C>(p, (int64_t)(kt + 1) * C::BK, K, st.p[1 - up], wave, lane);
        lds_barrier();
        multiply();
        read_frags<C>(st.p[up], st.q[uq], 2, wm, wn, lane, f[0]);
        read_frags<C>(st.p[up], st.q[uq], 3, wm, wn, lane, f[1]);
        copy_q<C>(q, (int64_t)(kt + 2) * C::BK, K, st.q[(u + 2) % 3], wave, lane);
        wait_vmcnt<LQ>();
        lds_barrier();
        multiply();
    };
    // whole turns over the stages with no way out between: where one joins the
    // loop's end the compiler takes the copies of both paths to be in flight
    int kt = 0;
    for (; kt + 6 <= KT; kt += 6)
        unrolled<6>([&](auto u) { slab(u, kt + u); });
    unrolled<5>([&](auto u) {
        if (kt + u < KT) slab(u, kt + u);
    });
    if (wm == 0) meet();
    wait_vmcnt<0>();
}

// ---- operands of any alignment ----------------------------------------------
// The same slabs through registers: a chunk of 8 bf16 at any address (one
// 16-byte load where the row holds it whole, single values at its end), then
// a 16-byte write to its place in the slab.

// 16 bytes at the alignment of a bf16: gfx950 allows unaligned global accesses.
typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ uint4 chunk_any(const uint16_t* p, int64_t left) {
    if (left >= 8) {
        const u32x4h u = *(const MUON_GLOBAL u32x4h*)p;
        return make_uint4(u.x, u.y, u.z, u.w);
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < left) w[e >> 1] |= (uint32_t)gld(p + e) << 16 * (e & 1);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// rows x K of an operand stored K-contiguous, K x cols of one stored k-major.
struct AnyOperand {
    const uint16_t* base;
    int64_t ld;
    int n;  // rows, or columns
};

// Chunk f of this thread for the slab at k0, and its place in it.  R: the
// tile's rows (columns); NT threads.
template <int R, int NT, bool KM>
__device__ __forceinline__ uint4 fetch_any(const AnyOperand& o, int64_t k0, int64_t K, int f) {
    const int ch = f * NT + threadIdx.x;
    if constexpr (KM) {
        const int64_t k = k0 + ch / (R / 8);
        const int c = ch % (R / 8) * 8;
        return chunk_any(o.base + k * o.ld + c, k < K ? o.n - c : 0);
    } else {
        const int row = ch / 8;
        const int64_t k = k0 + ch % 8 * 8;
        return chunk_any(o.base + row * o.ld + k, row < o.n ? K - k : 0);
    }
}
template <int R, int NT, bool KM>
__device__ __forceinline__ void put_any(uint16_t* slab, const uint4& v, int f) {
    const int ch = f * NT + threadIdx.x;
    const int row = ch / (KM ? R / 8 : 8), c = ch % (KM ? R / 8 : 8);
    *reinterpret_cast<uint4*>(slab + row * (KM ? R : 64) + ((c ^ (KM ? swzk<R>(row) : swz<64>(row))) << 3)) = v;
}

// acc += the tile over k [0, K): the registers of slab kt + 2 are loaded and
// those of slab kt + 1 written while slab kt is multiplied.
template <class C>
__device__ __forceinline__ void product_any(f32x16 (&acc)[C::FM][C::FN], const AnyOperand& p, const AnyOperand& q,
                                            int64_t K, const Stages<2>& st) {
    static_assert(C::BK == 64, "64-deep slabs");
    constexpr int NP = C::BM * 8 / C::NT, NQ = C::BN * 8 / C::NT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int KT = (int)((K + 63) / 64);
    if (KT == 0) return;
    uint4 rp[NP], rq[NQ];
    auto fetch = [&](int kt) {
#pragma unroll
        for (int f = 0; f < NP; ++f) rp[f] = fetch_any<C::BM, C::NT, C::PKM>(p, (int64_t)kt * 64, K, f);
#pragma unroll
        for (int f = 0; f < NQ; ++f) rq[f] = fetch_any<C::BN, C::NT, C::QKM>(q, (int64_t)kt * 64, K, f);
    };
    auto put = [&](uint16_t* sp, uint16_t* sq) {
#pragma unroll
        for (int f = 0; f < NP; ++f) put_any<C::BM, C::NT, C::PKM>(sp, rp[f], f);
#pragma unroll
        for (int f = 0; f < NQ; ++f) put_any<C::BN, C::NT, C::QKM>(sq, rq[f], f);
    };
    fetch(0);
    put(st.p[0], st.q[0]);
    if (KT > 1) fetch(1);
    __syncthreads();
    for (int kt0 = 0; kt0 < KT; kt0 += 2) {
        unrolled<2>([&](auto u) {
            const int kt = kt0 + u;
            if (kt >= KT) return;
            Frags<C> f[2];
            read_frags<C>(st.p[u], st.q[u], 0, wm, wn, lane, f[0]);
            if (kt + 1 < KT) put(st.p[1 - u], st.q[1 - u]);
            if (kt + 2 < KT) fetch(kt + 2);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                if (kk < 3) read_frags<C>(st.p[u], st.q[u], kk + 1, wm, wn, lane, f[(kk + 1) & 1]);
                mfma_frags<C>(acc, f[kk & 1]);
            }
            __syncthreads();
        });
    }
}

// Epilogue band (32 rows in fp32, in LDS): column c of row r at
// c ^ ((r & 4) << 3) ^ ((r >> 3) << 4), so that the two half-waves of an
// accumulator store (rows r and r + 4) lie 32 banks apart.
template <class C>
__device__ __forceinline__ int band_at(int r, int c) {
    return r * C::BN + (c ^ ((r & 4) << 3) ^ ((r >> 3) << 4));
}

// Passes the tile through LDS (`band`, 32 x BN floats) in bands of 32 rows:
// put(row, column, values) for every chunk of 8 columns.
template <class C, class F>
__device__ __forceinline__ void for_each_chunk(const f32x16 (&acc)[C::FM][C::FN], float* band, int rows, F&& put) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / C::WN, wn = wave % C::WN;
#pragma unroll
    for (int b = 0; b < C::BM / 32; ++b) {
        if (b * 32 >= rows) break;  // uniform
        __syncthreads();
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            if (wm * C::TM + i * 32 == b * 32) {
#pragma unroll
                for (int j = 0; j < C::FN; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        band[band_at<C>(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3),
                                        wn * C::TN + j * 32 + (lane & 31))] = acc[i][j][r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 32 * C::BN / 8 / C::NT; ++q) {
            const unsigned ch = q * C::NT + threadIdx.x;
            const int rr = ch / (C::BN / 8), c8 = ch % (C::BN / 8) * 8;
            const float4 a0 = *reinterpret_cast<const float4*>(band + band_at<C>(rr, c8));
            const float4 a1 = *reinterpret_cast<const float4*>(band + band_at<C>(rr, c8) + 4);
            const float v[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
            put(b * 32 + rr, c8, v);
        }
    }
    __syncthreads();
}

// The tile by waves, without a barrier: each wave passes its own rows through
// `mine` (16 x TN floats of LDS), 16 rows at a time, and gets them back four
// columns a lane, a row's TN columns side by side.  put(b, q, row, column,
// values) for piece q of band b.  ahead(b) is called before band b is put:
// loads for band b + 1 belong there.
template <class C>
constexpr int wave_pieces() { return 16 * C::TN / 256; }
template <class C>
__device__ __forceinline__ int wave_row(int b, int q) {
    return (threadIdx.x >> 6) / C::WN * C::TM + b * 16 + (q * 64 + (threadIdx.x & 63)) / (C::TN / 4);
}
template <class C>
__device__ __forceinline__ int wave_col() {
    return (threadIdx.x >> 6) % C::WN * C::TN + (threadIdx.x & 63) % (C::TN / 4) * 4;
}
template <class C, class A, class F>
__device__ __forceinline__ void for_each_piece(const f32x16 (&acc)[C::FM][C::FN], float* mine, A&& ahead, F&& put) {
    static_assert(64 % (C::TN / 4) == 0, "a piece is whole rows");
    const int lane = threadIdx.x & 63;
    // rows r and r + 4 of a store lie 32 banks apart (a row of 32 columns is
    // no longer than that)
    auto at = [](int r, int c) { return r * C::TN + (C::TN >= 64 ? c ^ ((r & 4) << 3) : c); };
#pragma unroll
    for (int b = 0; b < C::TM / 16; ++b) {
        ahead(b);
        // the wave's own earlier reads of `mine` are done: LDS is in order
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int r = 0; r < 8; ++r)
                mine[at(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3), j * 32 + (lane & 31))] = acc[b / 2][j][b % 2 * 8 + r];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < wave_pieces<C>(); ++q)
            put(b, q, wave_row<C>(b, q), wave_col<C>(),
                *reinterpret_cast<const float4*>(mine + at((q * 64 + lane) / (C::TN / 4), lane % (C::TN / 4) * 4)));
        __builtin_amdgcn_wave_barrier();
    }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
    uint4 o;
    o.x = (uint32_t)f32_to_bf16_bits(v[0]) | ((uint32_t)f32_to_bf16_bits(v[1]) << 16);
    o.y = (uint32_t)f32_to_bf16_bits(v[2]) | ((uint32_t)f32_to_bf16_bits(v[3]) << 16);
    o.z = (uint32_t)f32_to_bf16_bits(v[4]) | ((uint32_t)f32_to_bf16_bits(v[5]) << 16);
    o.w = (uint32_t)f32_to_bf16_bits(v[6]) | ((uint32_t)f32_to_bf16_bits(v[7]) << 16);
    return o;
}

}  // namespace bf
}  // namespace muon
