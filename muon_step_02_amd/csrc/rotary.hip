// Rotary positions on the heads of queries and keys (gfx950).
//
// Pair i of a head of token t turns by a = position_t f_i:
//
//   (u, v) -> s (u cos a - v sin a, v cos a + u sin a)
//
// and back, for the gradient, by -a.  The pairs are neighbours (interleaved)
// or half the turning part apart; other elements are copied.
//
// Bound by HBM: every element is read and written once.  A workgroup takes a
// run of tokens of one tensor and forms their sines and cosines once, for all
// heads, in LDS.  Angles are formed in 64 bits and reduced to a part of a turn
// there: an fp32 product of a position and a frequency is off by up to 2^-24 of
// the angle, 0.06 radians at position 10^6.
#include <type_traits>

#include "block.h"
#include "units.h"

namespace muon {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;       // of a thread, all loaded before the first is used
constexpr int kTable = kRotaryPairs;  // (cosine, sine) pairs of a workgroup's tokens

// Where one tensor's units lie.  A unit is 2 V elements of a head: V pairs, or
// 2 V elements that are copied.
struct Place {
    int turning, before, after;  // units of the turning part, of what is left and right of it
    int tokens;                  // of a workgroup
    int parts;                   // workgroups of a token, where it has more units than one takes
    int blocks;
};

__host__ __device__ __forceinline__ int per_head(const Place& p) { return p.turning + p.before + p.after; }

template <bool BF>
Place place_of(const RotaryCall& c, const RotaryTensor& t, int64_t* blocks) {
    constexpr int V = BF ? 8 : 4, most = kThreads * kUnits;
    const bool copy = t.x != t.y;
    Place p;
    p.turning = (c.pairs + V - 1) / V;
    p.before = copy ? (c.first + 2 * V - 1) / (2 * V) : 0;
    p.after = copy ? (c.head_dim - c.first - 2 * c.pairs + 2 * V - 1) / (2 * V) : 0;
    const int64_t units = (int64_t)t.heads * per_head(p);
    p.parts = (int)((units + most - 1) / most);
    int64_t n = units > most ? 1 : most / units;
    if (n > kTable / c.pairs) n = kTable / c.pairs;
    if (n > c.tokens) n = c.tokens;
    p.tokens = (int)(n < 1 ? 1 : n);
    *blocks = (c.tokens + (int64_t)p.tokens - 1) / p.tokens * p.parts;
    p.blocks = (int)*blocks;
    return p;
}

struct RotaryPlaces {
    Place p[kRotaryTensors];
};

template <bool BF>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryCall c, RotaryPlaces places) {
    constexpr int V = BF ? 8 : 4;
    __shared__ float2 table[kTable];
    int block = blockIdx.x, which = 0;
    while (block >= places.p[which].blocks) block -= places.p[which++].blocks;
    const RotaryTensor t = c.t[which];
    const Place p = places.p[which];
    const int part = block % p.parts;
    const int token0 = block / p.parts * p.tokens;
    const int tokens = min(p.tokens, c.tokens - token0);
    const int units = per_head(p), per_token = t.heads * units;
    const int begin = part * kThreads * kUnits, end = min(begin + kThreads * kUnits, tokens * per_token);

    // this thread's units: read before the sines are formed
    Raw<BF, V> a[kUnits], b[kUnits];
    int token[kUnits], pair[kUnits], na[kUnits], nb[kUnits];
    int64_t to[kUnits];
    int apart[kUnits];
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        const int u = begin + q * kThreads + (int)threadIdx.x;
        const bool has = u < end;
        token[q] = has ? (uint32_t)u / (uint32_t)per_token : 0;
        const int r = has ? u - token[q] * per_token : 0;
        const int head = (uint32_t)r / (uint32_t)units;
        const int i = r - head * units;
        int first, n;  // the unit's first element, and those that its part has from there on
        pair[q] = -1;
        apart[q] = V;
        if (i < p.turning) {
            pair[q] = i * V;
            first = c.first + (c.interleaved ? 2 * V : V) * i;
            n = c.pairs - i * V;
            if (c.interleaved) {
                na[q] = 2 * n;
                nb[q] = 2 * n - V;
            } else {
                apart[q] = c.pairs;
                na[q] = nb[q] = n;
            }
        } else {
            const bool left = i < p.turning + p.before;
            const int k = 2 * V * (i - p.turning - (left ? 0 : p.before));
            first = left ? k : c.first + 2 * c.pairs + k;
            n = (left ? c.first : c.head_dim) - first;
            na[q] = n;
            nb[q] = n - V;
        }
        if (!has) na[q] = nb[q] = 0;
        const int64_t at = (token0 + token[q]) * t.x_token + head * t.x_head + first;
        to[q] = (token0 + token[q]) * t.y_token + head * t.y_head + first;
        a[q] = load_raw<BF, V, false>(t.x, at, na[q]);
        b[q] = load_raw<BF, V, false>(t.x, at + apart[q], nb[q]);
    }

    for (int i = threadIdx.x; i < tokens * c.pairs; i += kThreads) {
        const int k = (uint32_t)i / (uint32_t)c.pairs;
        constexpr double kPerTurn = 0.15915494309189533577;  // 1 / (2 pi)
        const double turns = gld(c.positions + token0 + k) * (gld(c.frequencies + i - k * c.pairs) * kPerTurn);
        float s, co;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &co);
        table[i] = make_float2(co * c.scale, (c.transpose ? -s : s) * c.scale);
    }
    __syncthreads();

#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        float x[V], y[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            x[e] = a[q].at(e);
            y[e] = b[q].at(e);
        }
        if (pair[q] >= 0) {
            const float2* cs = table + token[q] * c.pairs + pair[q];
            const int n = c.pairs - pair[q];  // pairs of the unit that exist
            if (c.interleaved) {
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const float2 f = cs[min(e, n - 1)], g = cs[min(e + V / 2, n - 1)];
                    const float u = x[2 * e], v = x[2 * e + 1], w = y[2 * e], z = y[2 * e + 1];
                    x[2 * e] = u * f.x - v * f.y;
                    x[2 * e + 1] = v * f.x + u * f.y;
                    y[2 * e] = w * g.x - z * g.y;
                    y[2 * e + 1] = z * g.x + w * g.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 f = cs[min(e, n - 1)];
                    const float u = x[e], v = y[e];
                    x[e] = u * f.x - v * f.y;
                    y[e] = v * f.x + u * f.y;
                }
            }
        }
        store_unit<V, BF, false>(t.y, to[q], na[q], x);
        store_unit<V, BF, false>(t.y, to[q] + apart[q], nb[q], y);
    }
}

template <bool BF>
int64_t places_of(const RotaryCall& c, RotaryPlaces* places) {
    int64_t blocks = 0;
    for (int i = 0; i < c.count; ++i) {
        int64_t n = 0;
        places->p[i] = place_of<BF>(c, c.t[i], &n);
        blocks += n;
    }
    return blocks;
}

template <bool BF>
hipError_t launch(const RotaryCall& c, hipStream_t st) {
    RotaryPlaces places{};
    const int64_t blocks = places_of<BF>(c, &places);
    rotary_kernel<BF><<<(int)blocks, kThreads, 0, st>>>(c, places);
    return hipGetLastError();
}

}  // namespace

bool rotary_fits(const RotaryCall& c) {
    RotaryPlaces places{};
    const int64_t blocks = c.bf16 ? places_of<true>(c, &places) : places_of<false>(c, &places);
    return blocks <= UINT32_MAX / kThreads;
}

hipError_t launch_rotary(const RotaryCall& c, hipStream_t st) {
    return c.bf16 ? launch<true>(c, st) : launch<false>(c, st);
}

}  // namespace muon
