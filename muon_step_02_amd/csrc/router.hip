// The router of a mixture-of-experts layer, and its gradient (gfx950).
//
//   p = softmax(z) over the experts of a token, lse = log sum exp z
//   chosen = the k largest logits, the lowest index first among equals
//   gates = p[chosen], or p[chosen] over their sum
//   counts, offsets = choices per expert and their prefix sums
//   rows = a choice's place in the order by (expert, token); order: the inverse
//   balance = E sum_e (counts_e / sum counts) (sum_t p_te / n)
//   z loss = sum_t lse_t^2 / n,   n = tokens with a logit above -inf
//
// Three launches.  A workgroup takes 64 tokens, a team of 1 to 64 lanes one of
// them at a time, with 8 (16 beyond 64 experts) logits a lane in registers.
// Which of the 64 tokens chose an expert is one 64-bit mask in LDS: its bits
// count the choices, and those below a token's own are the token's place among
// them, whatever order the bits were set in.  The second launch adds up the
// workgroups' counts and probabilities per expert, the third gives every choice
// its row.  At most 64 tokens go through one workgroup in one launch.
//
// 32768 tokens of 256 fp32 logits, 8 choices: 19 + 6.2 + 5.3 us (38 MB, 6.5 us at
// the rate of HBM), bound by vector instructions (5.5 million, 9 us of the first
// launch) and by the latencies before and behind them, which 4 waves a SIMD (64
// tokens a workgroup, two workgroups a compute unit; beyond 512 experts the kernel
// takes 132 registers and more, and there is one) leave open.  64 tokens of 64 bf16
// logits: 7.6 us, of which an empty kernel of this kind takes 4.  Tried
// without gain: the next token's logits read ahead (registers for 3 waves a SIMD:
// 24 us), every workgroup of the last launch adding up all counts itself in place
// of the launch between (38 us in all instead of 31, 15 instead of 13.5 for 65
// tokens).  The gradient, 32768 tokens of 64 bf16 logits: 8.5 us; 4099 of 61 fp32
// logits, renormalised: 5.6 us.
//
// Gradient, with g_e = B E counts_e / (sum counts n) + [e chosen] dgate:
//
//   dz = p (g - sum p g + 2 Z lse / n)
//
// where gates were divided by their sum, their part of dz is
// gate_j (dgate_j - sum gate dgate) instead.
#include <math.h>

#include <type_traits>
#include <utility>

#include "block.h"
#include "team.h"
#include "units.h"

namespace muon {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;

// e^x for x <= 0 (or NaN) by the base-2 instruction.  The product is rounded once
// more than e^x needs: the result is off by up to |x| 2^-24 of itself beside the
// instruction's own step, 2 u rms at x = -5 and 8 u at -20 (u = 2^-24).  For fp32
// logits the rounding of x = z - top costs as much; for bf16 ones that difference is
// as a rule exact, and this is the larger part.  Taken for the time: with the
// product's rest carried along (three instructions more) the gates of 256 experts,
// logits of deviation 2, are off by 1.05 u rms instead of 1.2, and forward calls take
// 1 to 3% longer (64 tokens 7.2 -> 7.4 us, 32768 of 256 experts 30.5 -> 31.0, of 64
// 19.6 -> 19.9).  Below 2^-126 it is zero.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269502f); }

// A token's logits over the L lanes of a team: lane l holds C from l * C on,
// -inf behind the last.
template <bool BF, int C>
__device__ __forceinline__ void load_logits(const void* base, int64_t off, int left, float* z) {
    constexpr int V = BF ? 8 : 4;
#pragma unroll
    for (int p = 0; p < C; p += V) {
        const Raw<BF, V> r = load_raw<BF, V, false>(base, off + p, left - p);
#pragma unroll
        for (int e = 0; e < V; ++e) z[p + e] = p + e < left ? r.at(e) : -INFINITY;
    }
}

struct Softmax {
    float top, total;  // largest logit, sum of exp(z - top)
    bool live;
};

// e = exp(z - top).  A token without any logit above -inf gets zeros.
template <int L, int C>
__device__ __forceinline__ Softmax softmax(const float* z, float* e) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < C; ++i) m = fmaxf(m, z[i]);  // (of a NaN and a number the number)
    m = team_reduce<L>(m, [](float a, float b) { return fmaxf(a, b); });
    Softmax s;
    s.live = m != -INFINITY;
    s.top = s.live ? m : 0.f;
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        e[i] = exp_of(z[i] - s.top);
        t += e[i];
    }
    s.total = team_sum<L>(t);
    s.live = s.live || s.total != s.total;  // a NaN counts
    return s;
}

// Logits as whole numbers in their order, both zeros alike: the maximum is one
// instruction without a look at NaNs, which come last, with what is taken.
constexpr int32_t kTaken = INT32_MIN;
constexpr int32_t kLowest = (int32_t)0x807fffff;  // -inf
__device__ __forceinline__ int32_t key_of(float z) {
    const int32_t b = __builtin_bit_cast(int32_t, z + 0.f);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float logit_of(int32_t key) {
    return __builtin_bit_cast(float, key ^ ((key >> 31) & 0x7fffffff));
}

// One choice of a team: its largest key, `top` (kLowest or less: none is left),
// taken out of the lane that holds it, the lowest index first among equals (lane
// l has the indices from l * C on).  Returns that lane's place of it, or -1.
template <int L, int C>
__device__ __forceinline__ int take(int32_t* key, int32_t& top) {
    int32_t m = key[0];
#pragma unroll
    for (int c = 1; c < C; ++c) m = max(m, key[c]);
    top = team_reduce<L>(m, [](int32_t a, int32_t b) { return max(a, b); });
    bool left = m == top && top > kLowest;
    if constexpr (L > 1) {
        const int lane = threadIdx.x & 63, l = lane % L;
        const uint64_t equal = __ballot(left);
        // (a team without one has no bits here, and no lane that is left)
        if constexpr (L == 64)
            left = left && l == __builtin_ctzll(equal | 1ull << 63);
        else
            left = left && l == __builtin_ctz((uint32_t)(equal >> (lane - l)) | 1u << 31);
    }
    int at = -1;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const bool hit = left && key[c] == top;
        key[c] = hit ? kTaken : key[c];
        at = hit ? c : at;
        left = left && !hit;
    }
    return at;
}

// Calls fn(integral_constant<int, 1>) ... fn(integral_constant<int, 15>).
template <class F, int... I>
__device__ __forceinline__ void turns_of(F&& fn, std::integer_sequence<int, I...>) {
    (fn(std::integral_constant<int, I + 1>{}), ...);
}
template <class F>
__device__ __forceinline__ void row_turns(F&& fn) {
    turns_of(fn, std::make_integer_sequence<int, 15>{});
}

// Up to kFew choices of a team of 16 lanes or more at once.  Of 16 groups of
// logits (the lanes' of equal place in their rows of 16) the k largest maxima
// bound the k-th largest logit from below; what reaches the bound, 8 to 16 logits
// as a rule, goes side by side to 16 lanes, where each counts those before it.
// Returns false, for the whole wave, where a team has more than 16 of them.
// About 220 vector instructions for the wave's teams, where one choice after the
// other takes 75 each.  Calls for 32768 tokens of 256 experts, one after the other
// and at once: 1 choice 24.7 and 25.7 us, 2 25.7 and 26.1, 3 26.6 and 26.4, 4 27.8
// and 26.8, 8 33.5 and 30.5.  More than 8 choices: of logits in no order, a wave has
// a team with more than 16 that reach the bound in 2% of cases with 8 choices, 18%
// with 9, 60% with 10 and nearly always with 12.
constexpr int kFew = 8;
template <int L, int C>
__device__ __forceinline__ bool take_few(const int32_t* key, int k, int2* slots, int32_t* chosen, float* logits) {
    const int lane = threadIdx.x & 63, l = lane % L, place = lane & 15;
    int32_t m = key[0];
#pragma unroll
    for (int c = 1; c < C; ++c) m = max(m, key[c]);
    auto larger = [](int32_t a, int32_t b) { return max(a, b); };
    if constexpr (L > 16) m = team_step<16>(m, larger);
    if constexpr (L > 32) m = team_step<32>(m, larger);
    int before = 0;
    row_turns([&](auto r) { before += (int32_t)lane_move<0x120 + r.value>((uint32_t)m) > m; });
    const int32_t bound = max(kLowest + 1, team_reduce<16>(before < k ? m : INT32_MAX,
                                                           [](int32_t a, int32_t b) { return min(a, b); }));
    int n = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) n += key[c] >= bound;
    // their places, in the order of the experts
    int upto = row_prefix(n), all = __builtin_amdgcn_ds_bpermute((lane | 15) << 2, upto);
    if constexpr (L > 16) {
        const int whole = wave_prefix(n);
        const int first = L == 64 ? 0 : __builtin_amdgcn_ds_bpermute(((lane & -L) - 1) << 2, whole);
        upto = whole - (lane < L ? 0 : first);
        all = __builtin_amdgcn_ds_bpermute((lane | (L - 1)) << 2, upto);
    }
    if (__ballot(all > 16)) return false;
    int at = upto - n;
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (key[c] >= bound) slots[at++] = make_int2(key[c], l * C + c);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int2 mine = place < all ? slots[place] : make_int2(kTaken, 0);
    before = 0;
    row_turns([&](auto r) {
        // lane p sees lane p - r: with p >= r an expert before its own
        const int32_t other = (int32_t)lane_move<0x120 + r.value>((uint32_t)mine.x);
        // (a lane without one has the lowest key, and what wraps round there is not used)
        before += other > (place >= r.value ? (int32_t)((uint32_t)mine.x - 1u) : mine.x);
    });
    if (l < 16 && place < all && before < k) {
        chosen[before] = mine.y;
        logits[before] = logit_of(mine.x);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return true;
}

// The exclusive prefix sums of n <= 1024 counts, and their sum at [n].
__device__ __forceinline__ void prefix_counts(int32_t* s, int n, int32_t* wave_sum) {
    constexpr int Q = kRouterMaxExperts / kThreads;  // counts of a thread
    int v[Q], sum = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int i = threadIdx.x * Q + q;
        v[q] = i < n ? s[i] : 0;
        sum += v[q];
    }
    const int upto = wave_prefix(sum);
    if ((threadIdx.x & 63) == 63) wave_sum[threadIdx.x >> 6] = upto;
    __syncthreads();  // every count is read, every wave's sum is there
    int at = upto - sum;
    for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) at += wave_sum[w];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int i = threadIdx.x * Q + q;
        if (i < n) s[i] = at;
        at += v[q];
    }
    if (threadIdx.x == kThreads - 1) s[n] = at;
    __syncthreads();
}

// The workgroup's sum in every thread.
__device__ __forceinline__ double add_up(double v, double* red) {
    v = wave_sum64(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = red[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += red[w];
    return s;
}

// The rows of one workgroup's choices: `first` + the place among the masks'
// tokens.  order behind the last row is -1.
__device__ __forceinline__ void put_rows(const RouterCall& c, const unsigned long long* mask, const int32_t* first,
                                         int32_t all, int token0, int tokens, const int32_t* chosen) {
    for (int i = threadIdx.x; i < tokens * c.top_k; i += kThreads) {
        const int e = chosen[i], t = (uint32_t)i / (uint32_t)c.top_k;
        const int64_t at = (int64_t)token0 * c.top_k + i;
        int row = -1;
        if (e >= 0) row = first[e] + __popcll(mask[e] & ((1ull << t) - 1));
        if (c.rows) gst(c.rows + at, row);
        if (c.order) {
            if (row >= 0) gst(c.order + row, (int32_t)at);
            if (at >= all) gst(c.order + at, -1);
        }
    }
}

// Dynamic LDS of the two kernels over tokens, in this order; every part is a
// multiple of 8 bytes.
struct RouterLds {
    unsigned long long* mask;  // [experts]
    int32_t* first;            // [experts + 1]
    float* probs;              // [waves][experts]
    int32_t* chosen;           // [64 * top_k]
    float* gates;              // [64 * top_k]
    float* lse;                // [64]
    int32_t* live;             // [64]
    __device__ __forceinline__ RouterLds(char* p, int experts, int top_k) {
        const int even = (experts + 1) & ~1;
        mask = reinterpret_cast<unsigned long long*>(p);
        first = reinterpret_cast<int32_t*>(mask + experts);
        probs = reinterpret_cast<float*>(first + even + 2);
        chosen = reinterpret_cast<int32_t*>(probs + kWaves * even);
        gates = reinterpret_cast<float*>(chosen + kRouterTokens * top_k);
        lse = gates + kRouterTokens * top_k;
        live = reinterpret_cast<int32_t*>(lse + kRouterTokens);
    }
};
size_t router_lds(int experts, int top_k) {
    const size_t even = ((size_t)experts + 1) & ~(size_t)1;
    return (size_t)experts * 8 + (even + 2) * 4 + kWaves * even * 4 + (size_t)kRouterTokens * (top_k + 1) * 8;
}

__device__ __forceinline__ void put_losses(const RouterCall& c, double balance, int64_t choices, double lse2,
                                           int32_t live) {
    if (c.live) gst(c.live, live);
    if (!c.losses) return;
    const double n = live > 0 ? live : 1;
    gst(c.losses, (float)(choices > 0 ? c.experts * (balance / (double)choices) / n : 0.0 * balance));
    gst(c.losses + 1, (float)(lse2 / n));
}

// Softmax, choices, gates, and the workgroup's sums.  ONE: the workgroup has
// every token, and does the rest too.
template <bool BF, int L, int C, bool ONE>
__global__ __launch_bounds__(kThreads) void router_choose_kernel(RouterCall c, RouterSpace s) {
    extern __shared__ __align__(16) char lds[];
    __shared__ double red[kWaves];
    __shared__ int32_t wave_sum[kWaves];
    constexpr int TEAMS = 64 / L;  // of a wave
    __shared__ int2 slots[L >= 16 ? kWaves * TEAMS : 1][16];
    const RouterLds m(lds, c.experts, c.top_k);
    const int lane = threadIdx.x & 63, l = lane % L, team = lane / L, wave = threadIdx.x >> 6;
    const int token0 = blockIdx.x * kRouterTokens, tokens = min(kRouterTokens, c.tokens - token0);
    for (int e = threadIdx.x; e < c.experts; e += kThreads) m.mask[e] = 0;
    for (int i = threadIdx.x; i < tokens * c.top_k; i += kThreads) m.chosen[i] = -1;
    if (threadIdx.x < kRouterTokens) {
        m.lse[threadIdx.x] = 0.f;
        m.live[threadIdx.x] = 0;
    }
    __syncthreads();

    float probs[C];
#pragma unroll
    for (int i = 0; i < C; ++i) probs[i] = 0.f;
    for (int first = wave * TEAMS; first < tokens; first += kWaves * TEAMS) {
        const int t = first + team;
        const bool has = t < tokens;
        float z[C], e[C];
        load_logits<BF, C>(c.logits, (int64_t)(token0 + (has ? t : 0)) * c.ld + l * C, has ? c.experts - l * C : 0, z);
        const Softmax x = softmax<L, C>(z, e);
        const float inv = x.live ? 1.f / x.total : 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) probs[i] = fmaf(e[i], inv, probs[i]);
        if (l == 0 && x.live) {
            m.lse[t] = x.top + logf(x.total);
            m.live[t] = 1;
        }
        // one choice after the other, by the lane that holds it
        int32_t key[C];
#pragma unroll
        for (int i = 0; i < C; ++i) key[i] = key_of(z[i]);
        if (__ballot(x.total != x.total))  // a NaN somewhere: its key could be any
#pragma unroll
            for (int i = 0; i < C; ++i) key[i] = z[i] == z[i] ? key[i] : kTaken;
        bool done = false;
        if constexpr (L >= 16)
            if (c.top_k <= kFew)
                done = take_few<L, C>(key, c.top_k, slots[wave * TEAMS + team], m.chosen + t * c.top_k,
                                      m.gates + t * c.top_k);
        for (int j = 0; j < (done ? 0 : c.top_k); ++j) {
            int32_t top;
            const int i = take<L, C>(key, top);
            if (i >= 0) {
                m.chosen[t * c.top_k + j] = l * C + i;
                m.gates[t * c.top_k + j] = logit_of(top);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // then its gates, by as many lanes as there are
        float sum = 0.f;
        for (int j = l; j < c.top_k; j += L) {
            if (!has) continue;
            float& g = m.gates[t * c.top_k + j];
            g = m.chosen[t * c.top_k + j] >= 0 ? exp_of(g - x.top) : 0.f;
            sum += g;
        }
        if (c.renormalize) sum = team_sum<L>(sum);
        // a NaN logit, which x.total has seen, makes its token's gates NaN
        float by = c.renormalize ? fmaf(0.f, x.total, sum) : x.total;
        if (by == 0.f) by = 1.f;
        if (has)
            for (int j = l; j < c.top_k; j += L) m.gates[t * c.top_k + j] /= by;
    }
    // the teams of a wave have the same experts in the same lanes
#pragma unroll
    for (int i = 0; i < C; ++i) probs[i] = across_teams<L>(probs[i]);
    const int even = (c.experts + 1) & ~1;
    if (team == 0)
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (l * C + i < c.experts) m.probs[wave * even + l * C + i] = probs[i];
    __syncthreads();

    const int64_t at = (int64_t)token0 * c.top_k;
    for (int i = threadIdx.x; i < tokens * c.top_k; i += kThreads) {
        const int e = m.chosen[i];
        if (e >= 0) atomicOr(m.mask + e, 1ull << ((uint32_t)i / (uint32_t)c.top_k));
        gst(c.chosen + at + i, e);
        gst(c.gates + at + i, m.gates[i]);
    }
    // the last wave: every token's logarithm (kRouterTokens are a wave's lanes)
    double lse2 = 0.0;
    int32_t alive = 0;
    if (wave == kWaves - 1) {
        const double lse = m.lse[lane];
        lse2 = wave_sum64(lse * lse);
        alive = __popcll(__ballot(m.live[lane] != 0));
        if (!ONE && lane == 0) {
            gst(s.lse + blockIdx.x, lse2);
            gst(s.live + blockIdx.x, alive);
        }
    }
    __syncthreads();
    double balance = 0.0;
    for (int e = threadIdx.x; e < c.experts; e += kThreads) {
        const int n = __popcll(m.mask[e]);
        float p = m.probs[e];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) p += m.probs[w * even + e];
        if (ONE) {
            m.first[e] = n;
            gst(c.counts + e, n);
            balance = fma((double)n, (double)p, balance);
        } else {
            gst(s.hist + (int64_t)blockIdx.x * c.experts + e, (uint8_t)n);
            gst(s.probs + (int64_t)blockIdx.x * c.experts + e, p);
        }
    }
    if (!ONE) return;
    balance = add_up(balance, red);  // (and every count is in LDS)
    prefix_counts(m.first, c.experts, wave_sum);
    const int32_t all = m.first[c.experts];
    for (int e = threadIdx.x; e <= c.experts; e += kThreads) gst(c.offsets + e, m.first[e]);
    if (c.rows || c.order) put_rows(c, m.mask, m.first, all, token0, tokens, m.chosen);
    if (threadIdx.x == kThreads - 1) put_losses(c, balance, all, lse2, alive);
}

// Per expert: the workgroups' choices before each workgroup, and the sums over
// all of them.  16 experts a workgroup; 64 threads an expert, each a run of
// workgroups.
constexpr int kJoinExperts = 16;

__global__ __launch_bounds__(1024) void router_join_kernel(RouterCall c, RouterSpace s) {
    __shared__ int32_t count[kJoinExperts][64];
    __shared__ double prob[kJoinExperts][64];
    const int x = threadIdx.x % kJoinExperts, run = threadIdx.x / kJoinExperts;
    const int e = blockIdx.x * kJoinExperts + x, each = (s.blocks + 63) / 64;
    const int b0 = min(run * each, s.blocks), b1 = min(b0 + each, s.blocks);
    int n = 0;
    double p = 0.0;
    if (e < c.experts)
        for (int b = b0; b < b1; ++b) {
            n += gld(s.hist + (int64_t)b * c.experts + e);
            p += gld(s.probs + (int64_t)b * c.experts + e);
        }
    count[x][run] = n;
    prob[x][run] = p;
    __syncthreads();
    {  // a wave an expert
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, mine = blockIdx.x * kJoinExperts + w;
        const int own = count[w][lane];
        const int upto = wave_prefix(own);
        count[w][lane] = upto - own;
        const double q = wave_sum64(prob[w][lane]);
        if (lane == 63 && mine < c.experts) {
            gst(c.counts + mine, upto);
            gst(s.total + mine, q);
        }
    }
    __syncthreads();
    if (e >= c.experts) return;
    n = count[x][run];
    for (int b = b0; b < b1; ++b) {
        gst(s.base + (int64_t)b * c.experts + e, n);
        n += gld(s.hist + (int64_t)b * c.experts + e);
    }
}

// A row for every choice; the first workgroup also writes offsets and losses.
__global__ __launch_bounds__(kThreads) void router_rows_kernel(RouterCall c, RouterSpace s) {
    extern __shared__ __align__(16) char lds[];
    __shared__ double red[kWaves];
    __shared__ int32_t wave_sum[kWaves];
    const RouterLds m(lds, c.experts, c.top_k);
    const int token0 = blockIdx.x * kRouterTokens, tokens = min(kRouterTokens, c.tokens - token0);
    for (int e = threadIdx.x; e < c.experts; e += kThreads) {
        m.mask[e] = 0;
        m.first[e] = gld(c.counts + e);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * c.top_k; i += kThreads) {
        const int e = gld(c.chosen + (int64_t)token0 * c.top_k + i);
        m.chosen[i] = e;
        if (e >= 0) atomicOr(m.mask + e, 1ull << ((uint32_t)i / (uint32_t)c.top_k));
    }
    prefix_counts(m.first, c.experts, wave_sum);  // (its barriers also order the masks)
    const int32_t all = m.first[c.experts];
    if (blockIdx.x == 0) {
        double balance = 0.0, lse2 = 0.0, live = 0.0;
        for (int e = threadIdx.x; e < c.experts; e += kThreads)
            balance = fma((double)gld(c.counts + e), gld(s.total + e), balance);
        for (int b = threadIdx.x; b < s.blocks; b += kThreads) {
            lse2 += gld(s.lse + b);
            live += gld(s.live + b);
        }
        balance = add_up(balance, red);
        lse2 = add_up(lse2, red);
        live = add_up(live, red);
        if (threadIdx.x == 0) put_losses(c, balance, all, lse2, (int32_t)live);
        for (int e = threadIdx.x; e <= c.experts; e += kThreads) gst(c.offsets + e, m.first[e]);
        __syncthreads();
    }
    if (!c.rows && !c.order) return;
    for (int e = threadIdx.x; e < c.experts; e += kThreads)
        m.first[e] += gld(s.base + (int64_t)blockIdx.x * c.experts + e);
    __syncthreads();
    put_rows(c, m.mask, m.first, all, token0, tokens, m.chosen);
}

template <bool BF, int L, int C>
__global__ __launch_bounds__(kThreads) void router_grad_kernel(RouterGradCall c) {
    __shared__ double red[kWaves];
    constexpr int TEAMS = 64 / L, V = BF ? 8 : 4;
    constexpr int K = C * L < kRouterMaxChoices ? C * L : kRouterMaxChoices, Q = (K + L - 1) / L;  // choices; of a lane
    const int lane = threadIdx.x & 63, l = lane % L, team = lane / L, wave = threadIdx.x >> 6;
    const float n = (float)max(gld(c.live), 1);
    // every token's gradient of the balance loss by its probabilities
    double choices = 0.0;
    for (int e = threadIdx.x; e < c.experts; e += kThreads) choices += gld(c.counts + e);
    choices = add_up(choices, red);
    float share[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = l * C + i;
        share[i] = e < c.experts && choices > 0.0
                       ? (float)((double)c.balance * c.experts / n * (gld(c.counts + e) / choices)) : 0.f;
    }
    const float zn = 2.f * c.z / n;
    for (int64_t first = ((int64_t)blockIdx.x * kWaves + wave) * TEAMS; first < c.tokens;
         first += (int64_t)gridDim.x * kWaves * TEAMS) {
        const int64_t t = first + team;
        const bool has = t < c.tokens;
        const int64_t at = (has ? t : 0) * c.ld;
        float z[C], p[C], own[C];  // own: the gates' part of what the expert gets
        load_logits<BF, C>(c.logits, at + l * C, has ? c.experts - l * C : 0, z);
        const Softmax x = softmax<L, C>(z, p);
        const float inv = x.live ? 1.f / x.total : 0.f;
        const float lse = x.live ? x.top + logf(x.total) : 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            p[i] *= inv;
            own[i] = 0.f;
        }
        if (c.dgates) {
            // a lane has every L-th choice: its expert and its gate's gradient
            int e[Q];
            float d[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int j = q * L + l;
                const bool there = has && j < c.top_k;
                e[q] = there ? gld(c.chosen + t * c.top_k + j) : -1;
                d[q] = there ? gld(c.dgates + t * c.top_k + j) : 0.f;
                if (e[q] >= c.experts) e[q] = -1;
                // (where there is no choice, dgates may be anything)
                d[q] = e[q] >= 0 ? d[q] : 0.f;
            }
            if (c.renormalize) {
                // the gates are a softmax over the chosen logits
                float w[Q], most = -INFINITY, sum = 0.f, along = 0.f;
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    w[q] = -INFINITY;
                    if (e[q] >= 0)
                        w[q] = BF ? bf16_bits_to_f32(gld(reinterpret_cast<const uint16_t*>(c.logits) + at + e[q]))
                                  : gld(reinterpret_cast<const float*>(c.logits) + at + e[q]);
                    most = fmaxf(most, w[q]);
                }
                most = team_reduce<L>(most, [](float a, float b) { return fmaxf(a, b); });
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    w[q] = e[q] >= 0 ? exp_of(w[q] - most) : 0.f;
                    sum += w[q];
                    along = fmaf(w[q], d[q], along);
                }
                sum = team_sum<L>(sum);
                along = team_sum<L>(along);
#pragma unroll
                for (int q = 0; q < Q; ++q) d[q] = e[q] >= 0 ? w[q] / sum * (d[q] - along / sum) : 0.f;
            }
            // to the lanes that have the experts, one choice after the other
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int n_of = min(L, c.top_k - q * L);
                for (int k = 0; k < n_of; ++k) {
                    const int from = (lane - l + k) << 2;
                    const int to = L > 1 ? __builtin_amdgcn_ds_bpermute(from, e[q]) : e[q];
                    const int bits = __builtin_bit_cast(int, d[q]);
                    const float v = __builtin_bit_cast(float, L > 1 ? __builtin_amdgcn_ds_bpermute(from, bits) : bits);
#pragma unroll
                    for (int i = 0; i < C; ++i) own[i] += l * C + i == to ? v : 0.f;
                }
            }
        }
        // by the probabilities; renormalised gates have none of it
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) dot = fmaf(p[i], share[i] + (c.renormalize ? 0.f : own[i]), dot);
        dot = team_sum<L>(dot) - zn * lse;
        float o[C];
#pragma unroll
        for (int i = 0; i < C; ++i)
            o[i] = c.renormalize ? fmaf(p[i], share[i] - dot, own[i]) : p[i] * (share[i] + own[i] - dot);
        if (has)
#pragma unroll
            for (int q = 0; q < C; q += V)
                store_unit<V, BF, false>(c.dlogits, t * c.ld_out + l * C + q, c.experts - l * C - q, o + q);
    }
}

// Calls fn(lanes of a team, logits a lane).
template <class F>
hipError_t with_team(int experts, F&& fn) {
    using std::integral_constant;
#define MUON_TEAM(L, C) fn(integral_constant<int, L>{}, integral_constant<int, C>{})
    if (experts <= 8) return MUON_TEAM(1, 8);
    if (experts <= 16) return MUON_TEAM(2, 8);
    if (experts <= 32) return MUON_TEAM(4, 8);
    if (experts <= 64) return MUON_TEAM(8, 8);
    if (experts <= 128) return MUON_TEAM(8, 16);
    if (experts <= 256) return MUON_TEAM(16, 16);
    if (experts <= 512) return MUON_TEAM(32, 16);
    return MUON_TEAM(64, 16);
#undef MUON_TEAM
}

template <bool BF>
hipError_t choose(const RouterCall& c, const RouterSpace& s, hipStream_t st) {
    const size_t lds = router_lds(c.experts, c.top_k);
    return with_team(c.experts, [&](auto l, auto n) {
        if (c.tokens <= kRouterTokens)
            router_choose_kernel<BF, l.value, n.value, true><<<1, kThreads, lds, st>>>(c, s);
        else
            router_choose_kernel<BF, l.value, n.value, false><<<s.blocks, kThreads, lds, st>>>(c, s);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_router(const RouterCall& c, const RouterSpace& s, hipStream_t st) {
    hipError_t e = c.bf16 ? choose<true>(c, s, st) : choose<false>(c, s, st);
    if (e != hipSuccess || c.tokens <= kRouterTokens) return e;
    router_join_kernel<<<(c.experts + kJoinExperts - 1) / kJoinExperts, 1024, 0, st>>>(c, s);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    router_rows_kernel<<<s.blocks, kThreads, router_lds(c.experts, c.top_k), st>>>(c, s);
    return hipGetLastError();
}

hipError_t launch_router_grad(const RouterGradCall& c, int cus, hipStream_t st) {
    auto go = [&](auto bf) {
        return with_team(c.experts, [&](auto l, auto n) {
            const int each = kWaves * (64 / l.value);
            const int64_t need = ((int64_t)c.tokens + each - 1) / each, most = (int64_t)cus * 8;
            const int blocks = (int)(need < most ? need : most);
            router_grad_kernel<bf.value, l.value, n.value><<<blocks, kThreads, 0, st>>>(c);
            return hipGetLastError();
        });
    };
    return c.bf16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace muon
