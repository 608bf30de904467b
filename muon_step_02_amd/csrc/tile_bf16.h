// bf16 product tiles on the matrix cores (gfx950) for operands that are not
// padded: C[i][j] = sum_k P[i][k] Q[j][k] over rows that end anywhere, a K of
// any multiple of 8, and any leading dimension that is a multiple of 8.
//
// A workgroup of WM x WN waves computes BM x BN, each wave a block of 32 x 32
// MFMA tiles (v_mfma_f32_32x32x16_bf16, fp32 accumulation).  K advances in
// slabs of 64, copied global -> LDS with buffer_load_dwordx4 ... lds (16 bytes
// per lane, no registers in between).  The copies go through buffer resources
// that end where the operand does: a row or k behind the end reads as zero,
// so ragged ends need no branch and no memory traffic, and a value that lies
// behind an end, a NaN included, never reaches a sum.
//
// An operand is stored with k along its rows (K-contiguous: rows are the
// tile's rows) or k-major (rows are k).  k-major slabs are copied as they are
// and gathered with the transposing LDS read (ds_read_b64_tr_b16).
#pragma once

#include "muon_internal.h"

namespace muon {
namespace bf {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kBK = 64;      // k per slab
constexpr int kSlab = 16384;  // bf16 elements of an LDS array (256 rows)

// PKM, QKM: the operand is stored k-major.
template <int BM_, int BN_, int WM_, int WN_, bool PKM_, bool QKM_>
struct Cfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr bool PKM = PKM_, QKM = QKM_;
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int TM = BM / WM, TN = BN / WN;
    static constexpr int FM = TM / 32, FN = TN / 32;
    static constexpr int RB = 32;  // rows of an epilogue band
    static_assert(FM >= 1 && FN >= 1 && BM % 64 == 0 && BN % 64 == 0, "32 x 32 blocks per wave");
    static_assert((BM / 8) % NW == 0 && (BN / 8) % NW == 0, "slab copies split evenly over the waves");
    static_assert(RB * BN % (8 * NT) == 0, "epilogue chunks split evenly over the threads");
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

// LDS slab of a K-contiguous operand: 64 bf16 (8 chunks of 16 bytes) per row,
// chunk c at position c ^ swz(row): the 16 lanes of one LDS cycle read one
// chunk of 16 consecutive rows, on 16 different positions of the 64 banks.
__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }
// k-major slab of W columns: chunk c of row k at c ^ swzk(k): the 4 rows x 64
// bytes of a transposing read lie on disjoint quarters of the banks.
__device__ __forceinline__ int swzk(int k) { return (k & 3) << 2; }

// Copies of k [k0, k0 + 64) of R rows into an LDS slab; NW waves share them.
// Lane l of a copy fills chunk position l % 8 of row l / 8.
template <int R, int NW>
__device__ __forceinline__ void copy_rows(const Operand& o, int64_t k0, int64_t K, uint16_t* slab, int wave,
                                          int lane) {
    const __amdgpu_buffer_rsrc_t r = resource(o.base + k0, o.bytes - 2 * k0);
    const int left = K - k0 < kBK ? (int)(K - k0) : kBK;  // a multiple of 8
#pragma unroll
    for (int q = 0; q < R / 8 / NW; ++q) {
        const int grp = wave * (R / 8 / NW) + q;
        const int row = grp * 8 + (lane >> 3);
        const int c = (lane & 7) ^ swz(row);
        // a chunk behind K would be the next row's: pushed out of range
        const uint32_t off = c * 8 < left ? (uint32_t)(row * (int)o.ld + c * 8) * 2u : 0x80000000u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(slab + grp * 8 * kBK), 16, off, 0, 0, 0);
    }
}

// ... of a k-major operand: 64 rows k of W columns.
template <int W, int NW>
__device__ __forceinline__ void copy_kmajor(const Operand& o, int64_t k0, uint16_t* slab, int wave, int lane) {
    constexpr int CQ = W / 8, RPK = 64 / CQ;  // chunks of a row, rows of a copy
    static_assert(CQ <= 64 && (kBK / RPK) % NW == 0, "k-major copies split evenly over the waves");
    const __amdgpu_buffer_rsrc_t r = resource(o.base + k0 * o.ld, o.bytes - 2 * k0 * o.ld);
#pragma unroll
    for (int q = 0; q < kBK / RPK / NW; ++q) {
        const int grp = wave * (kBK / RPK / NW) + q;
        const int k = grp * RPK + lane / CQ;
        const uint32_t off = (uint32_t)(k * (int)o.ld + (((lane % CQ) ^ swzk(k)) * 8)) * 2u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(slab + grp * RPK * W), 16, off, 0, 0, 0);
    }
}

// MFMA operand fragment: lane l holds row l % 32, k = 8 (l / 32) + 0..7.
__device__ __forceinline__ bf16x8 frag_rows(const uint16_t* slab, int row, int chunk) {
    return *reinterpret_cast<const bf16x8*>(slab + row * kBK + ((chunk ^ swz(row)) << 3));
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
        const uint16_t* p = slab + k * W + (((n >> 3) ^ swzk(k)) << 3) + (n & 7);
        h[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(p));
    }
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// Two stages of one array per operand, each its own __shared__ variable: the
// compiler then knows that a copy into one leaves the others alone.
struct Stages {
    uint16_t *p0, *q0, *p1, *q1;
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
                        : frag_rows(sp, wm * C::TM + i * 32 + row, chunk);
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
        f.b[j] = C::QKM ? frag_kmajor<C::BN>(sq, 16 * kk, wn * C::TN + j * 32, lane)
                        : frag_rows(sq, wn * C::TN + j * 32 + row, chunk);
}

template <class C>
__device__ __forceinline__ void mfma_frags(f32x16 (&acc)[C::FM][C::FN], const Frags<C>& f) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}

template <class C>
__device__ __forceinline__ void copy_stage(const Operand& p, const Operand& q, int64_t k0, int64_t K,
                                           uint16_t* sp, uint16_t* sq, int wave, int lane) {
    if constexpr (C::PKM)
        copy_kmajor<C::BM, C::NW>(p, k0, sp, wave, lane);
    else
        copy_rows<C::BM, C::NW>(p, k0, K, sp, wave, lane);
    if constexpr (C::QKM)
        copy_kmajor<C::BN, C::NW>(q, k0, sq, wave, lane);
    else
        copy_rows<C::BN, C::NW>(q, k0, K, sq, wave, lane);
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

// acc = the tile over k [0, K).  Both stages are filled up front; while the
// MFMAs of a k-step (16 deep) run, the fragments of the next are read into
// the other registers.  The last k-step's MFMAs are issued after the barrier
// that frees the slab's stage, so the matrix cores have work while the waves
// meet; the copy of slab kt + 2 goes into that stage.
template <class C>
__device__ __forceinline__ void product(f32x16 (&acc)[C::FM][C::FN], const Operand& p, const Operand& q,
                                        int64_t K, const Stages& st) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / C::WN, wn = wave % C::WN;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    const int KT = (int)((K + kBK - 1) / kBK);
    if (KT == 0) return;
    constexpr int KS = kBK / 16;
    constexpr int NR = (C::PKM ? 2 : 1) * C::FM + (C::QKM ? 2 : 1) * C::FN;
    copy_stage<C>(p, q, 0, K, st.p0, st.q0, wave, lane);
    // behind K every copy reads zeros: the second stage is filled either way
    copy_stage<C>(p, q, kBK, K, st.p1, st.q1, wave, lane);
    constexpr int LPS = (C::BM / 8 + C::BN / 8) / C::NW;
    wait_vmcnt<LPS>();
    __syncthreads();
    Frags<C> f[2];
    read_frags<C>(st.p0, st.q0, 0, wm, wn, lane, f[0]);
    for (int kt0 = 0; kt0 < KT; kt0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int kt = kt0 + u;
            if (kt < KT) {
                uint16_t* const sp = u ? st.p1 : st.p0;
                uint16_t* const sq = u ? st.q1 : st.q0;
                const uint16_t* const np = u ? st.p0 : st.p1;
                const uint16_t* const nq = u ? st.q0 : st.q1;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    if (kk + 1 < KS) {
                        read_frags<C>(sp, sq, kk + 1, wm, wn, lane, f[(kk + 1) & 1]);
                    } else {
                        wait_vmcnt<0>();
                        __syncthreads();
                        if (kt + 2 < KT) copy_stage<C>(p, q, (int64_t)(kt + 2) * kBK, K, sp, sq, wave, lane);
                        read_frags<C>(np, nq, 0, wm, wn, lane, f[0]);
                    }
                    mfma_frags<C>(acc, f[kk & 1]);
                    interleave<NR, C::FM * C::FN>();
                }
            }
        }
    }
    wait_vmcnt<0>();
}

// Epilogue band (32 rows in fp32, in LDS): column c of row r at
// c ^ ((r & 4) << 3) ^ ((r >> 3) << 4), so that the two half-waves of an
// accumulator store (rows r and r + 4) lie 32 banks apart.
template <class C>
__device__ __forceinline__ int band_at(int r, int c) {
    return r * C::BN + (c ^ ((r & 4) << 3) ^ ((r >> 3) << 4));
}

// Passes the tile row band by row band through LDS (`band`, 32 x BN floats):
// put(row, column, values) for 8 consecutive columns, column a multiple of 8.
template <class C, class F>
__device__ __forceinline__ void for_each_chunk(const f32x16 (&acc)[C::FM][C::FN], float* band, int rows, F&& put) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / C::WN, wn = wave % C::WN;
#pragma unroll
    for (int b = 0; b < C::BM / C::RB; ++b) {
        if (b * C::RB >= rows) break;  // uniform
        __syncthreads();
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            if (wm * C::TM + i * 32 == b * C::RB) {
#pragma unroll
                for (int j = 0; j < C::FN; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        band[band_at<C>(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3), wn * C::TN + j * 32 + (lane & 31))] =
                            acc[i][j][r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < C::RB * C::BN / 8 / C::NT; ++q) {
            const int ch = q * C::NT + threadIdx.x;
            const int rr = ch / (C::BN / 8), c8 = (ch % (C::BN / 8)) * 8;
            const float4 a0 = *reinterpret_cast<const float4*>(band + band_at<C>(rr, c8));
            const float4 a1 = *reinterpret_cast<const float4*>(band + band_at<C>(rr, c8) + 4);
            const float v[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
            put(b * C::RB + rr, c8, v);
        }
    }
    __syncthreads();
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
