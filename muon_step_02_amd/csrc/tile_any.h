// A 64 x 64 product tile in fp32 for operands of any type, alignment, leading
// dimension and size (gfx950): C[i][j] = sum_k P[i][k] Q[j][k].
//
// Slabs of 32 k are read into registers (16 bytes a thread where the row
// allows it, whatever its alignment), widened to fp32 and laid out k-major in
// LDS; four waves hold a 32 x 32 block each and run v_mfma_f32_32x32x2f32.
// One such instruction keeps a SIMD busy for 64 cycles and needs two 4-byte
// LDS reads a lane, so the matrix cores are what bounds it (157 TFLOP/s);
// the registers of slab k + 1 are loaded while slab k is multiplied.
#pragma once

#include "muon_internal.h"

namespace muon {
namespace any {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4u __attribute__((ext_vector_type(4), aligned(2)));

constexpr int kTile = 64;
constexpr int kBK = 32;  // 64: LDS for two workgroups a compute unit only, 90 -> 62 TFLOP/s
constexpr int kF = kTile * kBK / 1024;  // 4-value loads of a thread, operand and slab
constexpr int kLd = 68;  // LDS row of 64 values, padded

struct Lds {
    float p[2][kBK * kLd];
    float q[2][kBK * kLd];
};

// An operand's 64 rows: element (i, k) at base[i * ld + k] (KM false) or
// base[k * ld + i] (KM true); rows i >= n and k >= K read as zero.
struct Operand {
    const void* base;
    int64_t ld;
    int n;
};

__device__ __forceinline__ float4 load4_any(const void* base, int bf16, int64_t off, int valid) {
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    if (valid >= 4) {
        if (bf16) {
            const u16x4u u = *(const MUON_GLOBAL u16x4u*)(reinterpret_cast<const uint16_t*>(base) + off);
            r = make_float4(bf16_bits_to_f32(u.x), bf16_bits_to_f32(u.y), bf16_bits_to_f32(u.z),
                            bf16_bits_to_f32(u.w));
        } else {
            const f32x4u u = *(const MUON_GLOBAL f32x4u*)(reinterpret_cast<const float*>(base) + off);
            r = make_float4(u.x, u.y, u.z, u.w);
        }
    } else if (valid > 0) {
        float v[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < valid)
                v[e] = bf16 ? bf16_bits_to_f32(gld(reinterpret_cast<const uint16_t*>(base) + off + e))
                            : gld(reinterpret_cast<const float*>(base) + off + e);
        r = make_float4(v[0], v[1], v[2], 0.f);
    }
    return r;
}

// Load f of thread t for the slab at k0: row t / 8 + 32 f, k 4 (t % 8) ... + 3,
// or with KM rows 4 (t % 16) ... + 3 of k t / 16 + 16 f.
template <bool KM>
__device__ __forceinline__ float4 fetch(const Operand& o, int bf16, int64_t k0, int64_t K, int f) {
    const int t = threadIdx.x;
    if (KM) {
        const int64_t k = k0 + (t >> 4) + 16 * f;
        const int i = (t & 15) * 4;
        return load4_any(o.base, bf16, k * o.ld + i, k < K ? o.n - i : 0);
    }
    const int i = (t >> 3) + 32 * f;
    const int64_t k = k0 + (t & 7) * 4;
    const int64_t left = K - k;
    return load4_any(o.base, bf16, (int64_t)i * o.ld + k, i < o.n ? (left > 4 ? 4 : (int)left) : 0);
}

template <bool KM>
__device__ __forceinline__ void put(float* s, const float4& v, int f) {
    const int t = threadIdx.x;
    if (KM) {
        *reinterpret_cast<float4*>(s + ((t >> 4) + 16 * f) * kLd + (t & 15) * 4) = v;
    } else {
        float* d = s + (t & 7) * 4 * kLd + (t >> 3) + 32 * f;
        d[0] = v.x;
        d[kLd] = v.y;
        d[2 * kLd] = v.z;
        d[3 * kLd] = v.w;
    }
}

// The tile over k [0, K); 256 threads.  Wave w holds rows 32 (w / 2) and
// columns 32 (w % 2): register r of lane l is row 8 (r / 4) + 4 (l / 32) +
// r % 4, column l % 32 of that block.
template <bool PKM, bool QKM>
__device__ __forceinline__ f32x16 product(const Operand& p, const Operand& q, int bf16, int64_t K,
                                          Lds& s) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int pi = 32 * (wave >> 1) + (lane & 31), qi = 32 * (wave & 1) + (lane & 31);
    f32x16 acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.f;
    if (K <= 0) return acc;
    __syncthreads();  // a previous tile's reads are done
    float4 np[kF], nq[kF];
#pragma unroll
    for (int f = 0; f < kF; ++f) {
        np[f] = fetch<PKM>(p, bf16, 0, K, f);
        nq[f] = fetch<QKM>(q, bf16, 0, K, f);
    }
#pragma unroll
    for (int f = 0; f < kF; ++f) {
        put<PKM>(s.p[0], np[f], f);
        put<QKM>(s.q[0], nq[f], f);
    }
    __syncthreads();
    int cur = 0;
    for (int64_t k0 = 0; k0 < K; k0 += kBK) {
        const bool more = k0 + kBK < K;
        if (more) {
#pragma unroll
            for (int f = 0; f < kF; ++f) {
                np[f] = fetch<PKM>(p, bf16, k0 + kBK, K, f);
                nq[f] = fetch<QKM>(q, bf16, k0 + kBK, K, f);
            }
        }
        const float* sp = s.p[cur] + (lane >> 5) * kLd + pi;
        const float* sq = s.q[cur] + (lane >> 5) * kLd + qi;
#pragma unroll
        for (int k = 0; k < kBK; k += 2)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(sp[k * kLd], sq[k * kLd], acc, 0, 0, 0);
        if (more) {
#pragma unroll
            for (int f = 0; f < kF; ++f) {
                put<PKM>(s.p[cur ^ 1], np[f], f);
                put<QKM>(s.q[cur ^ 1], nq[f], f);
            }
        }
        __syncthreads();
        cur ^= 1;
    }
    return acc;
}

}  // namespace any
}  // namespace muon
