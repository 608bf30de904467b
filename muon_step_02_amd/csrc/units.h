// Rows in units of 16 bytes a lane, at any alignment of an element and with
// ragged ends (grads.hip, layernorm.hip, rotary.hip, router.hip).
#pragma once

#include "muon_internal.h"

namespace muon {

// 16 or 8 bytes at the alignment of an element: rows of any leading dimension
// are read with full-width loads (gfx950 allows unaligned global accesses).
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32h __attribute__((aligned(2)));
typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));

// V elements of a row as they are in memory.
template <bool BF, int V>
struct Raw {
    static constexpr int W = BF ? V / 2 : V;  // 32-bit words
    uint32_t w[W];
    __device__ __forceinline__ float at(int e) const {
        if (!BF) return __builtin_bit_cast(float, w[e]);
        return __builtin_bit_cast(float, (e & 1) ? (w[e / 2] & 0xffff0000u) : (w[e / 2] << 16));
    }
};

// The V elements at offset `off`; `left`: elements the row still holds.  FULL:
// at least V of them, known without looking.  NT: whole units are not kept in the
// caches.
//
// A unit that the row ends within loads what the row holds, two bf16 at a time,
// and waits for none of it before the last.  (10^6 bf16 rows of 5, sum of squares
// and clip: 10.4 and 22.7 us; one element at a time, each waited for, 12.6 and 26.6;
// V loads always, of the last element in place of those behind it, 14.4 and 29.8.
// 200000 rows of 65: 12.2 and 24.8, 12.5 and 25.7, 14.1 and 28.2; 2000 vectors of
// 1001: 42 and 90, 47 and 100, 43 and 93.)
template <bool BF, int V, bool FULL, bool NT = false>
__device__ __forceinline__ Raw<BF, V> load_raw(const void* base, int64_t off, int64_t left) {
    Raw<BF, V> r;
    if (FULL || left >= V) {
        if constexpr (!BF) {
            const MUON_GLOBAL u32x4u* p = (const MUON_GLOBAL u32x4u*)(reinterpret_cast<const float*>(base) + off);
            const u32x4u u = NT ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w[i] = u[i];
        } else if constexpr (V == 8) {
            const MUON_GLOBAL u32x4h* p = (const MUON_GLOBAL u32x4h*)(reinterpret_cast<const uint16_t*>(base) + off);
            const u32x4h u = NT ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w[i] = u[i];
        } else {
            const MUON_GLOBAL u32x2h* p = (const MUON_GLOBAL u32x2h*)(reinterpret_cast<const uint16_t*>(base) + off);
            const u32x2h u = NT ? __builtin_nontemporal_load(p) : *p;
            r.w[0] = u[0];
            r.w[1] = u[1];
        }
    } else {
#pragma unroll
        for (int i = 0; i < Raw<BF, V>::W; ++i) r.w[i] = 0;
#pragma unroll
        for (int i = 0; i < Raw<BF, V>::W; ++i) {
            if constexpr (BF) {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + off + 2 * i;
                if (2 * i >= left) break;
                if (2 * i + 1 < left)
                    r.w[i] = *(const MUON_GLOBAL u32h*)p;
                else
                    r.w[i] = gld(p);
            } else if (i < left) {
                r.w[i] = gld(reinterpret_cast<const uint32_t*>(base) + off + i);
            }
        }
    }
    return r;
}

template <int V, bool OBF, bool FULL>
__device__ __forceinline__ void store_unit(void* base, int64_t off, int64_t left, const float* v) {
    if (FULL || left >= V) {
        if constexpr (!OBF) {
            u32x4u o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = __builtin_bit_cast(uint32_t, v[e]);
            *(MUON_GLOBAL u32x4u*)(reinterpret_cast<float*>(base) + off) = o;
        } else {
            uint32_t w[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                w[i] = (uint32_t)f32_to_bf16_bits(v[2 * i]) | (uint32_t)f32_to_bf16_bits(v[2 * i + 1]) << 16;
            uint16_t* p = reinterpret_cast<uint16_t*>(base) + off;
            if constexpr (V == 8)
                *(MUON_GLOBAL u32x4h*)p = u32x4h{w[0], w[1], w[2], w[3]};
            else
                *(MUON_GLOBAL u32x2h*)p = u32x2h{w[0], w[1]};
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (e < left) {
                if (OBF)
                    gst(reinterpret_cast<uint16_t*>(base) + off + e, f32_to_bf16_bits(v[e]));
                else
                    gst(reinterpret_cast<float*>(base) + off + e, v[e]);
            }
        }
    }
}

}  // namespace muon
