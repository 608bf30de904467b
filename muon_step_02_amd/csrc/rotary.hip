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
// heads, in LDS.  A thread has one unit of two 16-byte runs (two units a thread:
// 124 us instead of 120 for 32768 tokens of 32 + 8 heads of 128 in bf16, four: 127;
// without sines 123 with two).  Angles are formed in 64 bits and reduced to a part
// of a turn there: an fp32 product of a position and a frequency is off by up to
// 2^-24 of the angle, 0.06 radians at position 10^6.
//
// Measured: that batch 113-121 us (5.6-5.9 TB/s), 4099 tokens of 128 fp32 heads of
// 192 with 32 pairs 133-140 (5.8-6.1), 16 tokens of 64 + 8 heads 3.7.
#include <type_traits>

#include "block.h"
#include "units.h"

namespace muon {

namespace {

constexpr int kThreads = 512;  // 256: 142 us for the fp32 heads below instead of 137, the same for bf16
// Bytes that a call reads from which they are not kept in the caches, which are
// left to what it writes.  With other inputs in every call: 16 to 96 MB 2-3% slower
// so, 128 MB the same and with a reader of y behind it 74 -> 70 us, 192 MB 71 -> 58
// (123 -> 104), 256 MB 94 -> 75 (162 -> 153), 336 MB 123 -> 113 (212 -> 204).
constexpr int64_t kRotaryNontemporalBytes = (int64_t)112 << 20;
constexpr int kTable = kRotaryPairs;  // (cosine, sine) of a workgroup's tokens, whole units of them

// Where one tensor's units lie.  A unit is 2 V elements of a head: V pairs, or
// 2 V elements that are copied.
struct Place {
    int turning, before, after;  // units of the turning part, of what is left and right of it
    int tokens;                  // of a workgroup
    int parts;                   // workgroups of a token, where it has more units than one takes
    int each;                    // units of such a workgroup
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

// How a head's parts (what turns, what is left and right of it) divide into units.
// kWhole: evenly; a unit's two runs of V elements then lie half its part apart, so
// that the lanes of a load or store follow each other (806 MB of fp32 heads with
// 128 elements copied and 32 pairs of neighbours 156 us, 190 with the runs side by
// side, two units a thread each).  kShifted: a part's last unit starts earlier and
// shares elements with the one before it.  Both form the same bits, and in place
// each has read its own before the workgroup's barrier, behind which they write.
// kShort: some part is shorter than the V pairs or elements that this needs, and is
// read and written one by one.  (60 MB of bf16 heads of 128: 20 us.  kShifted, heads
// of 80 with 10 pairs, 20, where ends one by one took 36; kShort, heads of 100 with
// 17 pairs from their fourth element on, 29.)
enum Cut { kWhole, kShifted, kShort };

// The first pair of the turning part's unit i, one that is not kWhole.
template <int V>
__device__ __forceinline__ int first_pair(int pairs, int i) { return max(0, min(i * V, pairs - V)); }

// INTER: neighbours are pairs.  NT: loads around the caches.
template <bool BF, bool INTER, Cut CUT, bool NT>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryCall c, RotaryPlaces places) {
    constexpr int V = BF ? 8 : 4;
    constexpr bool WHOLE = CUT == kWhole, FULL = CUT != kShort;
    // (cosine, sine) of a token's unit i, its pair 2 k + b, at [(token V / 2 + k)
    // units + i][b]: 16 bytes of a lane beside those of the lane with the next unit
    __shared__ __align__(16) float2 table[kTable];
    int block = blockIdx.x, which = 0;
#pragma unroll
    for (int i = 0; i + 1 < kRotaryTensors; ++i) {  // (a tensor that is not there has no workgroups)
        const bool next = which == i && block >= places.p[i].blocks;
        block -= next ? places.p[i].blocks : 0;
        which += next;
    }
    const RotaryTensor t = c.t[which];
    const Place p = places.p[which];
    const int part = block % p.parts;
    const int token0 = block / p.parts * p.tokens;
    const int tokens = min(p.tokens, c.tokens - token0);
    const int units = units_of(p), per_token = t.heads * units;
    // the workgroup's units: `count` from unit `skipped` of head `head0` on
    const int begin = part * p.each, head0 = begin / units, skipped = begin - head0 * units;
    const int count = min(tokens * per_token - begin, p.each);

    // this thread's unit, read before the sines are formed; one without any reads
    // the workgroup's first
    const bool has = (int)threadIdx.x < count;
    const int v = skipped + (has ? (int)threadIdx.x : 0);
    const int token = divided(v, p.per_token), r = v - token * per_token;
    const int h = divided(r, p.per_head), i = r - h * units, head = head0 + h;
    const bool turns = i < p.turning;
    // the unit's first element, where its other run is, and what the two have
    int first, apart, na, nb;
    if (turns) {
        const int k = WHOLE ? V * i : first_pair<V>(c.pairs, i) * (INTER ? 2 : 1);
        first = c.first + k;
        apart = INTER && !WHOLE ? V : c.pairs;
        na = (INTER ? 2 : 1) * c.pairs - k;
        nb = na - (INTER ? V : 0);
    } else {
        const bool left = i < p.turning + p.before;
        const int all = left ? c.first : c.head_dim - c.first - 2 * c.pairs;
        const int u = i - p.turning - (left ? 0 : p.before);
        const int k = WHOLE ? V * u : max(0, min(2 * V * u, all - 2 * V));
        first = k + (left ? 0 : c.first + 2 * c.pairs);
        apart = WHOLE ? V * (left ? p.before : p.after) : min(V, all - V);
        na = all;
        nb = all >= V ? V : 0;
    }
    if (!has) na = nb = 0;
    const int64_t from = (token0 + token) * t.x_token + head * t.x_head + first;
    const int64_t to = (token0 + token) * t.y_token + head * t.y_head + first;
    const Raw<BF, V> a = load_raw<BF, V, FULL, NT>(t.x, from, na);
    const Raw<BF, V> b = load_raw<BF, V, FULL, NT>(t.x, from + apart, nb);

    const int slots = p.turning * V;
    for (int j = threadIdx.x; j < tokens * slots; j += kThreads) {
        const int k = (uint32_t)j / (uint32_t)slots, unit = (j - k * slots) / V, e = j % V;
        int pair = first_pair<V>(c.pairs, unit) + e;
        if (INTER && WHOLE) pair = unit * (V / 2) + e % (V / 2) + (e < V / 2 ? 0 : c.pairs / 2);
        if (CUT == kShort && pair >= c.pairs) continue;
        constexpr double kPerTurn = 0.15915494309189533577;  // 1 / (2 pi)
        const double angle = gld(c.positions + token0 + k) * (gld(c.frequencies + pair) * kPerTurn);
        float s, co;
        sincospif(2.f * (float)(angle - rint(angle)), &s, &co);
        table[((k * (V / 2) + e / 2) * p.turning + unit) * 2 + (e & 1)] =
            make_float2(co * c.scale, (c.transpose ? -s : s) * c.scale);
    }
    // (a unit that shares elements must not find them turned)
    if (!WHOLE) __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): every load has returned
    __syncthreads();
    if (!has) return;

    float x[V], y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        x[e] = a.at(e);
        y[e] = b.at(e);
    }
    if (turns) {
        // (pairs behind the last, where there are fewer than V, turn by anything)
        const float4* cs = reinterpret_cast<const float4*>(table) + token * (V / 2) * p.turning + i;
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            const float4 f = cs[k * p.turning];  // cosine, sine of pairs 2 k and 2 k + 1
            auto turn = [](float& u, float& w, float co, float s) {
                const float old = u;
                u = fmaf(old, co, -(w * s));
                w = fmaf(w, co, old * s);
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
    store_unit<V, BF, FULL>(t.y, to, na, x);
    store_unit<V, BF, FULL>(t.y, to + apart, nb, y);
}

// The plan of a call: false where its workgroups cannot be numbered.
template <bool BF>
bool plan(const RotaryCall& c, RotaryPlaces* places, int64_t* blocks, Cut* cut, bool* nontemporal) {
    constexpr int V = BF ? 8 : 4, most = kThreads;
    int64_t bytes = 0;
    *blocks = 0;
    const int right = c.head_dim - c.first - 2 * c.pairs;
    bool whole = c.pairs % V == 0, cuts = c.pairs < V;
    for (int i = 0; i < c.count; ++i) {
        if (c.t[i].x == c.t[i].y) continue;
        whole = whole && c.first % (2 * V) == 0 && right % (2 * V) == 0;
        cuts = cuts || (c.first > 0 && c.first < V) || (right > 0 && right < V);
    }
    *cut = cuts ? kShort : whole ? kWhole : kShifted;
    for (int i = 0; i < c.count; ++i) {
        const RotaryTensor& t = c.t[i];
        Place& p = places->p[i];
        const bool copy = t.x != t.y;
        p.turning = (c.pairs + V - 1) / V;
        p.before = copy ? (c.first + 2 * V - 1) / (2 * V) : 0;
        p.after = copy ? (right + 2 * V - 1) / (2 * V) : 0;
        const int64_t units = (int64_t)t.heads * units_of(p);
        // in place, units that share elements stay in one workgroup
        static_assert(kRotaryPairs / V <= most, "a head's units");
        p.each = copy || *cut == kWhole ? most : most / p.turning * p.turning;
        p.parts = (int)((units + p.each - 1) / p.each);
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
    Cut cut = kWhole;
    bool nontemporal = false;
    if (!plan<BF>(c, &places, &blocks, &cut, &nontemporal)) return hipErrorInvalidConfiguration;
    using std::bool_constant;
    using std::integral_constant;
    auto go = [&](auto inter, auto how, auto nt) {
        rotary_kernel<BF, inter.value, how.value, nt.value><<<(int)blocks, kThreads, 0, st>>>(c, places);
        return hipGetLastError();
    };
    auto with = [&](auto inter, auto how) {
        return nontemporal ? go(inter, how, bool_constant<true>{}) : go(inter, how, bool_constant<false>{});
    };
    auto as = [&](auto how) {
        return c.interleaved ? with(bool_constant<true>{}, how) : with(bool_constant<false>{}, how);
    };
    switch (cut) {
        case kWhole: return as(integral_constant<Cut, kWhole>{});
        case kShifted: return as(integral_constant<Cut, kShifted>{});
        default: return as(integral_constant<Cut, kShort>{});
    }
}

}  // namespace

bool rotary_fits(const RotaryCall& c) {
    RotaryPlaces places{};
    int64_t blocks;
    Cut cut;
    bool nontemporal;
    return c.bf16 ? plan<true>(c, &places, &blocks, &cut, &nontemporal)
                  : plan<false>(c, &places, &blocks, &cut, &nontemporal);
}

hipError_t launch_rotary(const RotaryCall& c, hipStream_t st) {
    return c.bf16 ? launch<true>(c, st) : launch<false>(c, st);
}

}  // namespace muon
