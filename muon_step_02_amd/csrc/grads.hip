// Global gradient norm over many tensors, and the clip to it (gfx950).
//
//   norm  = sqrt(sum over tensors and elements of g^2)
//   scale = max_norm / norm where norm > max_norm, else 1
//   out   = g * scale
//
// ("Por qué AdamW para entrenar modelos de lenguaje, y qué está cambiando",
// gustavoai.dev, section "Por qué AdamW, y por qué con esos números": before
// g enters the moments, a norm above 1 is rescaled to 1.)
//
// Both passes are bound by HBM: the norm reads every gradient once, the clip
// reads it again and writes the output.  Squares are formed and added up in
// 64 bits: the fp64 rate leaves room (one conversion and one fused
// multiply-add per element, a fifth of what the vector units do in the time
// the loads take), and no gradient that fp32 can hold overflows or vanishes
// in its square.  Every sum has a fixed order, so results are bitwise
// repeatable: block b takes chunks b, b + blocks, ... of the group.
//
// Measured: the norm of 192 fp32 gradients of 2048 x 7168 (11.3 GB) 1.81-1.86
// ms, 6.1-6.2 TB/s, where a large in-place multiplication moves 5.9 TB/s; the
// norm of 470 MB of bf16, at any row padding, 82-87 us, 5.4-5.7 TB/s.  Behind
// 940 MB of writes, which the memory-side cache has yet to write back, the same
// norm takes 140 us.  That is the clip's first pass where clips follow each
// other: 235 M bf16 values to fp32 take 112-148 + 252 us (5.6 TB/s in the second
// pass), 235 M fp32 values in place 531 in all.  The clip of 17 M fp32 values (67
// MB, the second read from the memory-side cache) takes 13 + 25 us.  Four vectors
// of 1024 values: 5 us in one workgroup, launch latency and two dependent loads.
#include <type_traits>

#include "inputs.h"

namespace muon {

namespace {

// 16 or 8 bytes at the alignment of an element: rows of any leading dimension
// are read with full-width loads (gfx950 allows unaligned global accesses).
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));
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
// at least V of them, known without looking.
template <bool BF, int V, bool FULL>
__device__ __forceinline__ Raw<BF, V> load_raw(const void* base, int64_t off, int64_t left) {
    Raw<BF, V> r;
    if (FULL || left >= V) {
        if constexpr (!BF) {
            const u32x4u u = *(const MUON_GLOBAL u32x4u*)(reinterpret_cast<const float*>(base) + off);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w[i] = u[i];
        } else if constexpr (V == 8) {
            const u32x4h u = *(const MUON_GLOBAL u32x4h*)(reinterpret_cast<const uint16_t*>(base) + off);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w[i] = u[i];
        } else {
            const u32x2h u = *(const MUON_GLOBAL u32x2h*)(reinterpret_cast<const uint16_t*>(base) + off);
            r.w[0] = u[0];
            r.w[1] = u[1];
        }
    } else {
#pragma unroll
        for (int i = 0; i < Raw<BF, V>::W; ++i) r.w[i] = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (e < left) {
                if (BF)
                    r.w[e / 2] |= (uint32_t)gld(reinterpret_cast<const uint16_t*>(base) + off + e) << 16 * (e & 1);
                else
                    r.w[e] = gld(reinterpret_cast<const uint32_t*>(base) + off + e);
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

template <int CAP>
__device__ __forceinline__ int grad_tensor_of(const GradGroup<CAP>& grp, int chunk) {
    int lo = 0, hi = grp.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (grp.chunk_prefix[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Where a thread's units of a chunk lie: unit u of the tensor is row u / upr,
// elements (u % upr) * V ... of that row (upr units a row).  One division for
// the first unit; the others are 256 units further on each.
struct Walk {
    int64_t r, c;       // row, unit within the row
    int64_t dr, dc;     // 256 units further
    int64_t upr, rows;
    __device__ __forceinline__ Walk(int64_t u, int64_t upr_, int64_t rows_) : upr(upr_), rows(rows_) {
        if (rows == 1) {
            r = 0;
            c = u;
            dr = 0;
            dc = 256;
        } else if (upr <= 0xffffffffll && u <= 0xffffffffll) {
            r = (uint32_t)u / (uint32_t)upr;
            c = u - r * upr;
            dr = 256u / (uint32_t)upr;
            dc = 256 - dr * upr;
        } else {
            r = u / upr;
            c = u - r * upr;
            dr = 256 / upr;
            dc = 256 - dr * upr;
        }
    }
    __device__ __forceinline__ bool inside() const { return r < rows && c < upr; }
    __device__ __forceinline__ void next() {
        r += dr;
        c += dc;
        if (rows > 1 && c >= upr) {
            c -= upr;
            ++r;
        }
    }
};

// Whether every unit of a chunk is whole: then no lane looks at its end.
__device__ __forceinline__ bool whole(int64_t rows, int64_t cols, int V, int64_t first) {
    return cols % V == 0 && first + kGradUnits <= rows * (cols / V);
}

template <bool BF, bool FULL>
__device__ __forceinline__ void chunk_sumsq(const void* g, int64_t rows, int64_t cols, int64_t ld,
                                            int64_t first, int tid, double (&acc)[4]) {
    constexpr int V = BF ? 8 : 4, Q = kGradUnits / 256;
    Walk w(first + tid, (cols + V - 1) / V, rows);
    Raw<BF, V> x[Q];
    // every load first, so that all are in flight together
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        x[q] = load_raw<BF, V, FULL>(g, w.r * ld + w.c * V, w.inside() ? cols - w.c * V : 0);
        w.next();
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const double d = (double)x[q].at(e);
            acc[e & 3] = fma(d, d, acc[e & 3]);
        }
}

// A chunk in units of 16 bytes of the wider type: bf16 gradients go to an fp32
// output in half units, so that its stores are whole 16 bytes a lane too.
template <bool BF, bool OBF, bool FULL>
__device__ __forceinline__ void chunk_scale(const void* g, void* out, int64_t rows, int64_t cols,
                                            int64_t ld, int64_t ld_out, int64_t first, int tid, float scale) {
    constexpr int H = BF && !OBF ? 2 : 1;  // parts of a unit
    constexpr int V = (BF ? 8 : 4) / H, Q = kGradUnits / 256 * H;
    const Walk w0(first * H + tid, (cols + V * H - 1) / (V * H) * H, rows);
    Raw<BF, V> x[Q];
    Walk w = w0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        x[q] = load_raw<BF, V, FULL>(g, w.r * ld + w.c * V, w.inside() ? cols - w.c * V : 0);
        w.next();
    }
    w = w0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = x[q].at(e) * scale;
        store_unit<V, OBF, FULL>(out, w.r * ld_out + w.c * V, w.inside() ? cols - w.c * V : 0, v);
        w.next();
    }
}

// Chunks b, b + blocks, ... of a group; tid: the thread's place among the 256
// that share a chunk.
template <int CAP>
__device__ __forceinline__ void group_sumsq(const GradGroup<CAP>& grp, int b, int blocks, int tid,
                                            double (&acc)[4]) {
    const int chunks = grp.chunk_prefix[grp.count];
    for (int ch = b; ch < chunks; ch += blocks) {
        const int t = grad_tensor_of(grp, ch);
        const int64_t first = (int64_t)(ch - grp.chunk_prefix[t]) * kGradUnits;
        const int64_t rows = grp.rows[t], cols = grp.cols[t], ld = grp.ld_g[t];
        const bool bf = grp.bf16[t];
        if (whole(rows, cols, bf ? 8 : 4, first)) {
            if (bf)
                chunk_sumsq<true, true>(grp.g[t], rows, cols, ld, first, tid, acc);
            else
                chunk_sumsq<false, true>(grp.g[t], rows, cols, ld, first, tid, acc);
        } else {
            if (bf)
                chunk_sumsq<true, false>(grp.g[t], rows, cols, ld, first, tid, acc);
            else
                chunk_sumsq<false, false>(grp.g[t], rows, cols, ld, first, tid, acc);
        }
    }
}

// The chunks in the order opposite to the sum's: what it read last is the
// likeliest to be left in the memory-side cache.
template <int CAP>
__device__ __forceinline__ void group_scale(const GradGroup<CAP>& grp, int b, int blocks, int tid, float scale) {
    const int chunks = grp.chunk_prefix[grp.count];
    for (int k = b; k < chunks; k += blocks) {
        const int ch = chunks - 1 - k;
        const int t = grad_tensor_of(grp, ch);
        // nothing to do in place where nothing is clipped
        if (scale == 1.f && grp.out[t] == grp.g[t]) continue;
        const int64_t first = (int64_t)(ch - grp.chunk_prefix[t]) * kGradUnits;
        const int64_t rows = grp.rows[t], cols = grp.cols[t], lg = grp.ld_g[t], lo = grp.ld_out[t];
        const bool full = whole(rows, cols, grp.bf16[t] ? 8 : 4, first);
        auto go = [&](auto bf, auto obf) {
            if (full)
                chunk_scale<bf, obf, true>(grp.g[t], grp.out[t], rows, cols, lg, lo, first, tid, scale);
            else
                chunk_scale<bf, obf, false>(grp.g[t], grp.out[t], rows, cols, lg, lo, first, tid, scale);
        };
        if (grp.bf16[t]) {
            if (grp.out_bf16[t]) go(std::true_type{}, std::true_type{}); else go(std::true_type{}, std::false_type{});
        } else {
            if (grp.out_bf16[t]) go(std::false_type{}, std::true_type{}); else go(std::false_type{}, std::false_type{});
        }
    }
}

// Sum over the workgroup, the same value in every thread, in a fixed order.
template <int NT>
__device__ __forceinline__ double block_sum(double s, double* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    double t = red[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) t += red[w];
    return t;
}

__device__ __forceinline__ float clip_scale(double sumsq, float max_norm, float* norm_out,
                                            float* scale_out, bool write) {
    const double norm = sqrt(sumsq);
    const float scale = norm > (double)max_norm ? (float)((double)max_norm / norm) : 1.f;
    if (write) {
        if (norm_out) gst(norm_out, (float)norm);
        if (scale_out) gst(scale_out, scale);
    }
    return scale;
}

template <int NT>
__device__ __forceinline__ double partials_sum(const double* partials, int n, double* red) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += NT) s += gld(partials + i);
    return block_sum<NT>(s, red);
}

template <int CAP>
__global__ __launch_bounds__(256) void grad_sumsq_kernel(GradGroup<CAP> grp, int blocks,
                                                         double* partials) {
    __shared__ double red[4];
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    group_sumsq(grp, blockIdx.x, blocks, threadIdx.x, acc);
    const double tot = block_sum<256>((acc[0] + acc[1]) + (acc[2] + acc[3]), red);
    if (threadIdx.x == 0) gst(partials + blockIdx.x, tot);
}

__global__ __launch_bounds__(256) void grad_finalize_kernel(const double* partials, int n,
                                                            float max_norm, float* norm_out,
                                                            float* scale_out) {
    __shared__ double red[4];
    const double s = partials_sum<256>(partials, n, red);
    clip_scale(s, max_norm, norm_out, scale_out, threadIdx.x == 0);
}

template <int CAP>
__global__ __launch_bounds__(256) void grad_scale_kernel(GradGroup<CAP> grp, int blocks,
                                                         const double* partials, int n,
                                                         float max_norm, float* norm_out,
                                                         float* scale_out) {
    __shared__ double red[4];
    const double s = partials_sum<256>(partials, n, red);
    const float scale = clip_scale(s, max_norm, norm_out, scale_out, blockIdx.x == 0 && threadIdx.x == 0);
    group_scale(grp, blockIdx.x, blocks, threadIdx.x, scale);
}

// Everything by one workgroup; each 256 of its threads take a chunk.
constexpr int kSingleThreads = 1024;

template <int CAP>
__global__ __launch_bounds__(kSingleThreads) void grad_single_kernel(GradGroup<CAP> grp, int clip, float max_norm,
                                                                     float* norm_out, float* scale_out) {
    __shared__ double red[kSingleThreads / 64];
    const int team = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8), tid = threadIdx.x & 255;
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    group_sumsq(grp, team, kSingleThreads / 256, tid, acc);
    // the barrier within also keeps the outputs behind every read of the sum
    const double s = block_sum<kSingleThreads>((acc[0] + acc[1]) + (acc[2] + acc[3]), red);
    const float scale = clip_scale(s, max_norm, norm_out, scale_out, threadIdx.x == 0);
    if (clip) group_scale(grp, team, kSingleThreads / 256, tid, scale);
}

}  // namespace

template <int CAP>
hipError_t launch_grad_sumsq(const GradGroup<CAP>& g, int blocks, double* partials, hipStream_t st) {
    grad_sumsq_kernel<CAP><<<blocks, 256, 0, st>>>(g, blocks, partials);
    return hipGetLastError();
}

hipError_t launch_grad_finalize(const double* partials, int nparts, float max_norm, float* norm_out,
                                float* scale_out, hipStream_t st) {
    grad_finalize_kernel<<<1, 256, 0, st>>>(partials, nparts, max_norm, norm_out, scale_out);
    return hipGetLastError();
}

template <int CAP>
hipError_t launch_grad_scale(const GradGroup<CAP>& g, int blocks, const double* partials, int nparts,
                             float max_norm, float* norm_out, float* scale_out, hipStream_t st) {
    grad_scale_kernel<CAP><<<blocks, 256, 0, st>>>(g, blocks, partials, nparts, max_norm, norm_out, scale_out);
    return hipGetLastError();
}

template <int CAP>
hipError_t launch_grad_single(const GradGroup<CAP>& g, int clip, float max_norm, float* norm_out,
                              float* scale_out, hipStream_t st) {
    grad_single_kernel<CAP><<<1, kSingleThreads, 0, st>>>(g, clip, max_norm, norm_out, scale_out);
    return hipGetLastError();
}

#define MUON_GRAD_GROUPS(CAP)                                                                        \
    template hipError_t launch_grad_sumsq<CAP>(const GradGroup<CAP>&, int, double*, hipStream_t);    \
    template hipError_t launch_grad_scale<CAP>(const GradGroup<CAP>&, int, const double*, int, float, \
                                               float*, float*, hipStream_t);                         \
    template hipError_t launch_grad_single<CAP>(const GradGroup<CAP>&, int, float, float*, float*,   \
                                                hipStream_t);
MUON_GRAD_GROUPS(kGradGroupSmall)
MUON_GRAD_GROUPS(kGradGroup)

}  // namespace muon
