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
constexpr int64_t kRotaryNontemporalBytes = (int64_t)96 << 20;
constexpr int kTable = kRotaryPairs;  // (cosine, sine) of a workgroup's tokens, whole units of them

// Where one tensor's units lie.  A unit is 2 V elements of a head: V pairs, or
// 2 V elements that are copied.
struct Place {
    int turning, before, after;  // units of the turning part, of what is left and right of it
    int tokens;                  // of a workgroup
    int parts;                   // workgroups of a token, where it has more units than one takes
    int blocks;
    float per_head, per_token;   // 1 / units of a head; of a token, 0 with several parts
};

struct RotaryPlaces {
    Place p[kRotaryTensors];
};

__host__ __device__ __forceinline__ int units_of(const Place& p) { return p.turning + p.before + p.after; }

// v / d for v below 2^14, with inv = 1 / d in fp32: (v + 1/2) / d is at least
// 1 / (2 d) from a whole number, and off by less than v 2^-22 / d.
__device__ __forceinline__ int divided(int v, float inv) { return (int)(((float)v + 0.5f) * inv); }

// INTER: neighbours are pairs.  WHOLE: no unit is cut short; a unit's two runs of V
// elements then lie half its part apart, so that the lanes of a load or store
// follow each other (runs side by side: 190 us for 806 MB of fp32 heads with 128
// elements copied and 32 pairs of neighbours).  NT: loads around the caches.
template <bool BF, bool INTER, bool WHOLE, bool NT>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryCall c, RotaryPlaces places) {
    constexpr int V = BF ? 8 : 4;
    // (cosine, sine) of a token's unit i, its pair 2 k + b, at [(token V / 2 + k)
    // units + i][b]: 16 bytes of a lane beside those of the lane with the next unit
    __shared__ __align__(16) float2 table[kTable];
    int block = blockIdx.x, which = 0;
    while (block >= places.p[which].blocks) block -= places.p[which++].blocks;
    const RotaryTensor t = c.t[which];
    const Place p = places.p[which];
    const int part = block % p.parts;
    const int token0 = block / p.parts * p.tokens;
    const int tokens = min(p.tokens, c.tokens - token0);
    const int units = units_of(p), per_token = t.heads * units;
    // the workgroup's units: `count` from unit `skipped` of head `head0` on
    const int begin = part * kThreads * kUnits, head0 = begin / units, skipped = begin - head0 * units;
    const int count = min(tokens * per_token - begin, kThreads * kUnits);

    // this thread's units: read before the sines are formed
    Raw<BF, V> a[kUnits], b[kUnits];
    int table_at[kUnits];  // -1: copied
    int64_t to[kUnits];
    int na[kUnits], nb[kUnits], apart[kUnits];
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        const int local = q * kThreads + (int)threadIdx.x;
        const bool has = local < count;
        const int v = skipped + (has ? local : 0);
        const int token = divided(v, p.per_token), r = v - token * per_token;
        const int h = divided(r, p.per_head), i = r - h * units, head = head0 + h;
        int first, n;  // the unit's first element, and those that its part has from there on
        table_at[q] = -1;
        if (i < p.turning) {
            table_at[q] = token * (V / 2) * p.turning + i;
            first = c.first + (INTER && !WHOLE ? 2 * V : V) * i;
            n = (INTER && !WHOLE ? 2 : 1) * (c.pairs - i * V);
            apart[q] = INTER && !WHOLE ? V : c.pairs;
        } else {
            const bool left = i < p.turning + p.before;
            const int k = (WHOLE ? V : 2 * V) * (i - p.turning - (left ? 0 : p.before));
            first = left ? k : c.first + 2 * c.pairs + k;
            n = (left ? c.first : c.head_dim) - first;
            apart[q] = !WHOLE ? V : V * (left ? p.before : p.after);
        }
        na[q] = has ? n : 0;
        nb[q] = has ? n - (INTER || table_at[q] < 0 ? V : 0) : 0;  // (!WHOLE)
        const int64_t at = (token0 + token) * t.x_token + head * t.x_head + first;
        to[q] = (token0 + token) * t.y_token + head * t.y_head + first;
        // (WHOLE: a thread without a unit reads the workgroup's first)
        a[q] = load_raw<BF, V, WHOLE, NT>(t.x, at, na[q]);
        b[q] = load_raw<BF, V, WHOLE, NT>(t.x, at + apart[q], nb[q]);
    }

    for (int i = threadIdx.x; i < tokens * c.pairs; i += kThreads) {
        const int k = (uint32_t)i / (uint32_t)c.pairs, pair = i - k * c.pairs;
        constexpr double kPerTurn = 0.15915494309189533577;  // 1 / (2 pi)
        const double turns = gld(c.positions + token0 + k) * (gld(c.frequencies + pair) * kPerTurn);
        float s, co;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &co);
        int unit = pair / V, e = pair % V;
        if (INTER && WHOLE) {
            const int half = pair >= c.pairs / 2, of = pair - half * (c.pairs / 2);
            unit = of / (V / 2);
            e = of % (V / 2) + half * (V / 2);
        }
        table[((k * (V / 2) + e / 2) * p.turning + unit) * 2 + (e & 1)] =
            make_float2(co * c.scale, (c.transpose ? -s : s) * c.scale);
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
        if (table_at[q] >= 0) {
            // (pairs behind the last, in a unit that is cut short, turn by anything)
            const float4* cs = reinterpret_cast<const float4*>(table) + table_at[q];
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                const float4 f = cs[k * p.turning];  // cosine, sine of pairs 2 k and 2 k + 1
                auto turn = [](float& u, float& v, float co, float s) {
                    const float w = u;
                    u = w * co - v * s;
                    v = v * co + w * s;
                };
                if (INTER) {
                    float* z = k < V / 4 ? x + 4 * k : y + 4 * k - V;
                    turn(z[0], z[1], f.x, f.y);
                    turn(z[2], z[3], f.z, f.w);
                } else {
                    turn(x[2 * k], y[2 * k], f.x, f.y);
                    turn(x[2 * k + 1], y[2 * k + 1], f.z, f.w);
                }
            }
        }
        if (WHOLE && na[q] <= 0) continue;
        store_unit<V, BF, WHOLE>(t.y, to[q], na[q], x);
        store_unit<V, BF, WHOLE>(t.y, to[q] + apart[q], nb[q], y);
    }
}

// The plan of a call: false where its workgroups cannot be numbered.
template <bool BF>
bool plan(const RotaryCall& c, RotaryPlaces* places, int64_t* blocks, bool* whole, bool* nontemporal) {
    constexpr int V = BF ? 8 : 4, most = kThreads * kUnits;
    int64_t bytes = 0;
    *blocks = 0;
    *whole = c.pairs % V == 0;
    for (int i = 0; i < c.count; ++i) {
        const RotaryTensor& t = c.t[i];
        Place& p = places->p[i];
        const bool copy = t.x != t.y;
        const int right = c.head_dim - c.first - 2 * c.pairs;
        p.turning = (c.pairs + V - 1) / V;
        p.before = copy ? (c.first + 2 * V - 1) / (2 * V) : 0;
        p.after = copy ? (right + 2 * V - 1) / (2 * V) : 0;
        if (copy && (c.first % (2 * V) || right % (2 * V))) *whole = false;
        const int64_t units = (int64_t)t.heads * units_of(p);
        p.parts = (int)((units + most - 1) / most);
        int64_t n = units > most ? 1 : most / units;
        n = n < kTable / (V * p.turning) ? n : kTable / (V * p.turning);
        n = n < c.tokens ? n : c.tokens;
        p.tokens = (int)n;
        p.per_head = 1.f / units_of(p);
        p.per_token = p.parts > 1 ? 0.f : 1.f / units;
        const int64_t b = (c.tokens + n - 1) / n * p.parts;
        p.blocks = (int)b;
        *blocks += b;
        bytes += (int64_t)c.tokens * t.heads * (copy ? c.head_dim : 2 * c.pairs) * (BF ? 2 : 4);
    }
    *nontemporal = bytes >= kRotaryNontemporalBytes;
    return *blocks <= UINT32_MAX / kThreads;
}

template <bool BF>
hipError_t launch(const RotaryCall& c, hipStream_t st) {
    RotaryPlaces places{};
    int64_t blocks = 0;
    bool whole = false, nontemporal = false;
    if (!plan<BF>(c, &places, &blocks, &whole, &nontemporal)) return hipErrorInvalidConfiguration;
    auto go = [&](auto inter, auto all, auto nt) {
        rotary_kernel<BF, inter.value, all.value, nt.value><<<(int)blocks, kThreads, 0, st>>>(c, places);
        return hipGetLastError();
    };
    using std::false_type;
    using std::true_type;
    auto with = [&](auto inter, auto all) { return nontemporal ? go(inter, all, true_type{}) : go(inter, all, false_type{}); };
    if (c.interleaved) return whole ? with(true_type{}, true_type{}) : with(true_type{}, false_type{});
    return whole ? with(false_type{}, true_type{}) : with(false_type{}, false_type{});
}

}  // namespace

bool rotary_fits(const RotaryCall& c) {
    RotaryPlaces places{};
    int64_t blocks;
    bool whole, nontemporal;
    return c.bf16 ? plan<true>(c, &places, &blocks, &whole, &nontemporal)
                  : plan<false>(c, &places, &blocks, &whole, &nontemporal);
}

hipError_t launch_rotary(const RotaryCall& c, hipStream_t st) {
    return c.bf16 ? launch<true>(c, st) : launch<false>(c, st);
}

}  // namespace muon
