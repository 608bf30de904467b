// Layer norm over rows, and its gradient (gfx950).
//
//   mean = sum x / C  (or 0)     rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   xhat = (x - mean) rstd       y = xhat w + b
//
//   g  = dy w
//   dx = rstd (g - [center] sum g / C - xhat sum (g xhat) / C)
//   dw = sum over rows of dy xhat     db = sum over rows of dy
//
// Both directions are bound by HBM: the forward pass reads x and writes y, the
// gradient reads x and dy and writes dx, each once.  A row stays in the
// registers of its team of 8 to 1024 lanes from its load to its store, so the
// variance is the mean of the squared differences themselves, in a second sum
// over registers.  Workgroups walk over rows; weight and bias are read once each.
//
// A team of a wave or more reads its next row while it works on one.  That needs
// loads and stores without a branch around them: where one may be left out, the
// compiler waits for every access in flight instead of the loads it needs.  So
// rows are read and written through buffer resources of their own length: what
// lies behind a row reads as zero and is not written, a row that is not there
// has no length, and the last unit of a row whose length is no multiple of a
// unit starts earlier (its first elements are its neighbour's, computed twice).
#include <algorithm>
#include <type_traits>

#include "block.h"
#include "team.h"
#include "units.h"

namespace muon {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Rows of large tensors, read once, are not kept in the caches, which are left to
// what the call writes and the next one reads.  With other inputs in every call:
// gradients of 128 MB tensors 81 -> 70 us, of 192 MB 116 -> 98, of 256 MB 151 ->
// 126, with a reader of dx behind them 128 -> 107, 184 -> 161 and 239 -> 227 us;
// tensors of 16 to 64 MB took the same time either way, and a call on the same 34
// MB again and again 13 us instead of 16.  (Stores around the caches: forward
// passes over the same 470 MB in every call 90 -> 72 us, but a reader of y behind
// one loses more.)
constexpr int kNontemporal = 2;
constexpr int64_t kNontemporalBytes = (int64_t)96 << 20;  // of x

// `bytes` bytes from p on, the same in every lane of the wave.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_resource(const void* p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}

// V elements of weight or bias from column `at` on; `absent` without one.  Columns
// behind the last read as anything.
template <int V, bool WHOLE>
__device__ __forceinline__ void load_weight(const void* w, bool bf, int at, int cols, float absent, float* out) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = absent;
    } else if (!WHOLE) {
        // a last unit that is cut short
        for (int e = 0; e < V; ++e) {
            const int k = min(at + e, cols - 1);
            out[e] = bf ? bf16_bits_to_f32(gld(reinterpret_cast<const uint16_t*>(w) + k))
                        : gld(reinterpret_cast<const float*>(w) + k);
        }
    } else if (bf) {
        const auto r = row_resource(w, cols * 2);
        if constexpr (V == 8) {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, at * 2, 0, 0);
#pragma unroll
            for (int e = 0; e < 8; ++e) out[e] = bf16_bits_to_f32((uint16_t)(v[e / 2] >> 16 * (e & 1)));
        } else {
            const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, at * 2, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) out[e] = bf16_bits_to_f32((uint16_t)(v[e / 2] >> 16 * (e & 1)));
        }
    } else {
        const auto r = row_resource(w, cols * 4);
#pragma unroll
        for (int p = 0; p < V; p += 4) {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, (at + p) * 4, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) out[p + e] = __builtin_bit_cast(float, (uint32_t)v[e]);
        }
    }
}

// How rows end: with a whole unit; with one that starts earlier, so that it ends
// with the row; or within their only one.
enum RowEnd { kWhole, kShifted, kShort };

// Which elements of a row a lane of a team of L has: R units of V.  Unit i starts
// at column at[i]; kShifted: its first skip[i] elements are another unit's too (V:
// there is no such unit).
template <bool BF, RowEnd END, int L, int R>
struct Share {
    static constexpr int V = BF ? 8 : 4;
    static constexpr int kNowhere = 1 << 24;  // behind every row
    int at[R], skip[R];
    __device__ __forceinline__ Share(int l, int cols) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * L + l) * V;
            at[i] = c;
            skip[i] = 0;
            if (END == kShifted && c + V > cols) {
                at[i] = c < cols ? cols - V : L >= 64 ? kNowhere : 0;
                skip[i] = c < cols ? c - (cols - V) : V;
            }
        }
    }
    // whether element e of unit i is in the row, and this lane's to count
    __device__ __forceinline__ bool mine(int i, int e, int cols) const {
        return END == kShifted ? e >= skip[i] : END == kWhole ? at[i] < cols : at[i] + e < cols;
    }
    // a unit that a row of a team of this size may not have: smaller teams take the
    // rows that end before these
    static constexpr bool maybe(int i) { return R == 1 || 2 * i + 1 >= R; }
};

// A row, as it is in memory.
template <bool BF, RowEnd END, int L, int R>
struct Row {
    static constexpr int V = BF ? 8 : 4, ES = BF ? 2 : 4;
    Raw<BF, V> u[R];
    template <bool NT>
    __device__ __forceinline__ void read(const void* base, int64_t off, int cols, const Share<BF, END, L, R>& s, bool has) {
        if constexpr (L >= 64) {
            const auto r = row_resource(reinterpret_cast<const char*>(base) + off * ES, has ? cols * ES : 0);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, s.at[i] * ES, 0, NT ? kNontemporal : 0);
#pragma unroll
                for (int k = 0; k < 4; ++k) u[i].w[k] = v[k];
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int left = has ? cols - s.at[i] : 0;
                if (END == kShort) {
                    u[i] = load_raw<BF, V, false, NT>(base, off + s.at[i], left);
                } else {
                    // from the row's start where there is no such unit
                    const bool there = END == kShifted ? has && s.skip[i] < V : left > 0;
                    u[i] = load_raw<BF, V, true, NT>(base, off + (there ? s.at[i] : 0), V);
#pragma unroll
                    for (int k = 0; k < Raw<BF, V>::W; ++k) u[i].w[k] = there ? u[i].w[k] : 0;
                }
            }
        }
    }
    // NT: around the caches; for teams of a wave or more `nontemporal` says so (a
    // branch there, not a kernel: the aux bits of the two loads keep the compiler
    // from making one of them).
    template <bool NT>
    __device__ __forceinline__ void load(const void* base, int64_t off, int cols, const Share<BF, END, L, R>& s, bool has,
                                         bool nontemporal) {
        if (NT || (L >= 64 && nontemporal))
            read<true>(base, off, cols, s, has);
        else
            read<false>(base, off, cols, s, has);
    }
};

// Writes v, unit i of a row at a time.
template <bool BF, RowEnd END, int L, int R>
struct Out {
    static constexpr int V = BF ? 8 : 4, ES = BF ? 2 : 4;
    char* p;
    int cols;
    bool has;
    __device__ __forceinline__ Out(void* base, int64_t off, int cols_, bool has_)
        : p(reinterpret_cast<char*>(base) + off * ES), cols(cols_), has(has_) {}
    __device__ __forceinline__ void put(int i, const Share<BF, END, L, R>& s, const float* v) const {
        if constexpr (L >= 64) {
            u32x4 w;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = BF ? (uint32_t)f32_to_bf16_bits(v[2 * k]) | (uint32_t)f32_to_bf16_bits(v[2 * k + 1]) << 16
                          : __builtin_bit_cast(uint32_t, v[k]);
            __builtin_amdgcn_raw_buffer_store_b128(w, row_resource(p, has ? cols * ES : 0), s.at[i] * ES, 0, 0);
        } else if (has) {
            const int left = cols - s.at[i];
            if (END == kShort)
                store_unit<V, BF, false>(p, s.at[i], left, v);
            else if (END == kShifted ? s.skip[i] < V : left > 0)
                store_unit<V, BF, true>(p, s.at[i], V, v);
        }
    }
};

// Sums over a team.  The waves of a team of more lanes than a wave has meet in
// LDS, in one of two slots in turn, so that one barrier a sum is enough (a wave
// that writes a slot again has passed the other slot's barrier, which every wave
// reaches after it has read).  NT: threads of the workgroup.
template <int L, int NT>
struct TeamSum {
    float* red;  // [2][2 * waves]
    int slot = 0;
    __device__ __forceinline__ explicit TeamSum(float* r) : red(r) {}
    __device__ __forceinline__ void operator()(float& a, float& b, bool two) {
        constexpr int W = L > 64 ? L / 64 : 1, ALL = NT / 64;
        a = team_sum<(L > 64 ? 64 : L)>(a);
        if (two) b = team_sum<(L > 64 ? 64 : L)>(b);
        if constexpr (W > 1) {
            float* s = red + slot * 2 * ALL;
            const int w = threadIdx.x >> 6, w0 = w / W * W;
            if ((threadIdx.x & 63) == 0) {
                s[w] = a;
                s[ALL + w] = b;
            }
            __syncthreads();
            a = s[w0];
            b = s[ALL + w0];
#pragma unroll
            for (int i = 1; i < W; ++i) {
                a += s[w0 + i];
                b += s[ALL + w0 + i];
            }
            slot ^= 1;
        }
    }
};

__device__ __forceinline__ int64_t row_at(int row, int heads, int64_t token, int64_t head) {
    if (heads == 1) return row * token;
    const uint32_t t = (uint32_t)row / (uint32_t)heads;
    return t * token + (row - (int)t * heads) * head;
}

// The team of a thread; one of a wave or more is the same in all its lanes.
template <int L>
__device__ __forceinline__ int team_of() {
    const int t = threadIdx.x / L;
    return L >= 64 ? __builtin_amdgcn_readfirstlane(t) : t;
}

// Calls work(row buffer, first row of the workgroup's teams) for the rows first,
// first + stride, ...; with AHEAD, load(buffer, first) has read the next ones by
// then.
template <class B, bool AHEAD, class Load, class Work>
__device__ __forceinline__ void walk_rows(int64_t first, int64_t stride, int rows, Load&& load, Work&& work) {
    B a, b;
    if constexpr (!AHEAD) {
        for (; first < rows; first += stride) {
            load(a, first);
            work(a, first);
        }
        return;
    }
    load(a, first);
    while (true) {
        load(b, first + stride);
        work(a, first);
        first += stride;
        if (first >= rows) return;
        load(a, first + stride);
        work(b, first);
        first += stride;
        if (first >= rows) return;
    }
}

template <int L>
constexpr int threads_of() { return L > 128 ? L : 256; }

template <bool BF, RowEnd END, int L, int R, bool NT>
__global__ __launch_bounds__(threads_of<L>()) void norm_forward_kernel(NormCall c) {
    constexpr int V = BF ? 8 : 4, THREADS = threads_of<L>(), TEAMS = THREADS / L;
    __shared__ float red[L > 64 ? 4 * (THREADS / 64) : 1];
    const int l = threadIdx.x % L, team = team_of<L>();
    const Share<BF, END, L, R> s(l, c.cols);
    float w[R][V], b[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        load_weight<V, END != kShort>(c.weight, c.weight_bf16, s.at[i], c.cols, 1.f, w[i]);
        load_weight<V, END != kShort>(c.bias, c.weight_bf16, s.at[i], c.cols, 0.f, b[i]);
    }
    TeamSum<L, THREADS> sum(red);
    const float n = (float)c.cols;
    using Buffer = Row<BF, END, L, R>;
    auto load = [&](Buffer& x, int64_t first) {
        const int64_t row = first + team;
        const bool has = row < c.rows;
        x.template load<NT>(c.x, row_at(has ? (int)row : 0, c.heads, c.x_token, c.x_head), c.cols, s, has, c.nontemporal);
    };
    auto work = [&](const Buffer& x, int64_t first) {
        const int row = (int)first + team;
        const bool has = row < c.rows;
        float v[R][V], mean = 0.f, none = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = x.u[i].at(e);
        if (c.center) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    // (what is behind the row reads as zero)
                    mean += END == kShifted && s.maybe(i) && !s.mine(i, e, c.cols) ? 0.f : v[i][e];
            sum(mean, none, false);
            mean /= n;
        }
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[i][e] -= mean;
                const float d = !s.maybe(i) || s.mine(i, e, c.cols) ? v[i][e] : 0.f;
                sq = fmaf(d, d, sq);
            }
        sum(sq, none, false);
        const float rstd = 1.f / sqrtf(sq / n + c.eps);
        const Out<BF, END, L, R> out(c.out, has ? row_at(row, c.heads, c.out_token, c.out_head) : 0, c.cols, has);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = fmaf(v[i][e] * rstd, w[i][e], b[i][e]);
            out.put(i, s, o);
        }
        if (l == 0 && has) {
            if (c.mean) gst(c.mean + row, mean);
            if (c.rstd) gst(c.rstd + row, rstd);
        }
    };
    walk_rows<Buffer, L >= 64>((int64_t)blockIdx.x * TEAMS, (int64_t)gridDim.x * TEAMS, c.rows, load, work);
}

__device__ __forceinline__ void put_grad(void* p, bool bf, int accumulate, int col, double v) {
    if (bf) {
        uint16_t* q = reinterpret_cast<uint16_t*>(p) + col;
        if (accumulate) v += bf16_bits_to_f32(gld(q));
        gst(q, f32_to_bf16_bits((float)v));
    } else {
        float* q = reinterpret_cast<float*>(p) + col;
        if (accumulate) v += gld(q);
        gst(q, (float)v);
    }
}

// Threads of the gradient's workgroups: 256, or two teams that are wider than a
// wave, or one.  Each team adds its rows to sums of its own, and the workgroup hands
// on one sum a column: fewer, wider workgroups leave less to join.  Two fp32 teams of
// 384 or 512 lanes were slower than one (120 MB of rows of 2049 columns 78 us instead
// of 69, of 4096 68 instead of 65, of 3500 the same), and 1024 threads hold no two
// wider ones.
template <bool BF, int L>
constexpr int grad_threads() { return L <= 64 ? 256 : L <= (BF ? 512 : 256) ? 2 * L : L; }

// dx, and each workgroup's sums for dw and db over its rows.  The weight of a row
// of more than a wave is kept in LDS, which leaves those registers to the next row.
template <bool BF, RowEnd END, int L, int R, bool NT>
__global__ __launch_bounds__((grad_threads<BF, L>())) void norm_grad_kernel(NormCall c) {
    constexpr int V = BF ? 8 : 4, THREADS = grad_threads<BF, L>(), TEAMS = THREADS / L;
    constexpr bool WIDE = L > 64;
    __shared__ float red[WIDE ? 4 * (THREADS / 64) : 1];
    // the weight, then the teams' sums
    __shared__ __align__(16) float held[WIDE ? L * R * V : THREADS * R * V];
    const int l = threadIdx.x % L, team = team_of<L>();
    const Share<BF, END, L, R> s(l, c.cols);
    // (a wide row's values: 16 bytes of a lane beside those of the next)
    auto held_at = [&](int i, int e) { return ((i * (V / 4) + e / 4) * L + l) * 4 + e % 4; };
    float w[WIDE ? 1 : R][V], dw[R][V], db[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float v[V];
        load_weight<V, END != kShort>(c.weight, c.weight_bf16, s.at[i], c.cols, 1.f, v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (!WIDE)
                w[i][e] = v[e];
            else if (team == 0)
                held[held_at(i, e)] = v[e];
            dw[i][e] = db[i][e] = 0.f;
        }
    }
    if (WIDE) __syncthreads();
    TeamSum<L, THREADS> sum(red);
    const float n = (float)c.cols;
    struct Buffer {
        Row<BF, END, L, R> x, dy;
        float mean, rstd;
    };
    auto load = [&](Buffer& r, int64_t first) {
        const int64_t row = first + team;
        const bool has = row < c.rows;
        const int there = has ? (int)row : 0;
        r.x.template load<NT>(c.x, row_at(there, c.heads, c.x_token, c.x_head), c.cols, s, has, c.nontemporal);
        r.dy.template load<NT>(c.dy, row_at(there, c.heads, c.dy_token, c.dy_head), c.cols, s, has, c.nontemporal);
        r.mean = c.center ? gld(c.mean + there) : 0.f;
        r.rstd = gld(c.rstd + there);
    };
    auto work = [&](const Buffer& r, int64_t first) {
        const int row = (int)first + team;
        const bool has = row < c.rows;
        const float mu = has ? r.mean : 0.f, rs = has ? r.rstd : 0.f;
        auto weight = [&](int i, int e) { return WIDE ? held[held_at(i, e)] : w[WIDE ? 0 : i][e]; };
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float d = r.dy.u[i].at(e);
                if (END == kShifted && s.maybe(i)) d = s.mine(i, e, c.cols) ? d : 0.f;
                const float t = r.x.u[i].at(e) - mu, g = d * weight(i, e);
                dw[i][e] = fmaf(d * rs, t, dw[i][e]);
                db[i][e] += d;
                s1 = fmaf(g, t, s1);
                s2 += g;
            }
        if (!c.out) return;
        sum(s1, s2, c.center);
        // dx = rstd (g - sum(g) / C - (x - mean) rstd sum(g xhat) / C); rstd^3 as a
        // factor would leave fp32 for rows of tiny values
        const float a = -(s1 * rs / n) * rs, b = c.center ? -(s2 / n) : 0.f;
        const Out<BF, END, L, R> out(c.out, has ? row_at(row, c.heads, c.out_token, c.out_head) : 0, c.cols, has);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                o[e] = fmaf(r.x.u[i].at(e) - mu, a, fmaf(r.dy.u[i].at(e), weight(i, e), b)) * rs;
            out.put(i, s, o);
        }
    };
    // (Workgroups of one team of 768 or 1024 lanes do not read ahead: with 128
    // registers a lane a second row of four fp32 units has no room, one of two bf16
    // units spills on 1024 lanes and gains nothing on 768, 83 us either way for 120 MB
    // of rows of 12000 columns.  One of two fp32 units has room: 72 us instead of 74
    // for rows of 7168 columns, 73.4 instead of 74.1 for 5120.)
    walk_rows<Buffer, L <= 512>((int64_t)blockIdx.x * TEAMS, (int64_t)gridDim.x * TEAMS, c.rows, load, work);
    // the teams' sums, added in their order
    auto put = [&](int side, float (&acc)[R][V], void* out) {
        if (!out) return;
        float* p = c.partials + ((int64_t)side * gridDim.x + blockIdx.x) * c.cols;
        if constexpr (TEAMS > 1) {
            auto place = [&](int t, int i, int e) { return WIDE ? held_at(i, e) : ((t * R + i) * V + e) * L + l; };
            __syncthreads();
            if (!WIDE || team == 1)
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) held[place(team, i, e)] = acc[i][e];
            __syncthreads();
            if (team == 0)
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        for (int t = 1; t < TEAMS; ++t) acc[i][e] += held[place(t, i, e)];
        }
        if (team > 0) return;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (gridDim.x > 1 && s.mine(i, 0, c.cols) && s.mine(i, V - 1, c.cols)) {
#pragma unroll
                for (int e = 0; e < V; e += 4) store_unit<4, false, true>(p, s.at[i] + e, 4, &acc[i][e]);
                continue;
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (!s.mine(i, e, c.cols)) continue;
                if (gridDim.x == 1)
                    put_grad(out, c.grad_bf16, c.accumulate, s.at[i] + e, acc[i][e]);
                else
                    gst(p + s.at[i] + e, acc[i][e]);
            }
        }
    };
    put(0, dw, c.dweight);
    put(1, db, c.dbias);
}

// dw and db from the workgroups' sums: 64 columns a workgroup, each of its 16
// waves every 16th sum, eight of them in flight, added in 64 bits.
__global__ __launch_bounds__(1024) void norm_grad_join_kernel(NormCall c, int blocks) {
    __shared__ double part[16][64];
    void* out = blockIdx.y ? c.dbias : c.dweight;
    if (!out) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
    double s = 0.0;
    if (col < c.cols) {
        const float* p = c.partials + (int64_t)blockIdx.y * blocks * c.cols + col;
        int b = wave;
        for (; b + 7 * 16 < blocks; b += 8 * 16) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = gld(p + (int64_t)(b + 16 * i) * c.cols);
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        for (; b < blocks; b += 16) s += gld(p + (int64_t)b * c.cols);
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave || col >= c.cols) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][lane];
    put_grad(out, c.grad_bf16, c.accumulate, col, s);
}

// Calls fn(lanes of a team, units a lane) for a row of `units` 16-byte units: the
// smallest L * R that holds them, and lanes with at most 32 values each.  More
// units a lane rather than more waves a team, which meet at a barrier (120 MB of
// bf16 rows of 1536 columns on 192 lanes 52 us, on 64 lanes 41), and three units
// rather than four where they do, which leaves fewer lanes idle (rows of 2049
// columns on 256 lanes of two 65 us, on 128 of three 48).
template <bool BF, RowEnd END, class F>
hipError_t with_team(int units, F&& fn) {
    using std::integral_constant;
#define MUON_TEAM(L, R) \
    if (units <= L * R) return fn(integral_constant<int, L>{}, integral_constant<int, R>{})
    MUON_TEAM(8, 1);
    if constexpr (END != kShort) {
        MUON_TEAM(16, 1);
        MUON_TEAM(32, 1);
        MUON_TEAM(16, 3);
        MUON_TEAM(64, 1);
        MUON_TEAM(32, 3);
        MUON_TEAM(64, 2);
        MUON_TEAM(64, 3);
        MUON_TEAM(64, 4);
        MUON_TEAM(128, 3);
        MUON_TEAM(128, 4);
        MUON_TEAM(192, 4);
        MUON_TEAM(256, 4);
        MUON_TEAM(384, 4);
        MUON_TEAM(512, 4);
        if constexpr (!BF) {
            MUON_TEAM(384, 8);
            MUON_TEAM(512, 8);
        }
    }
    return hipErrorInvalidValue;  // (no row is longer)
}

// The same for the gradient, whose sums for dw and db take two registers a value:
// at most 24 values a lane, and 16 in teams of several waves.  (120 MB of fp32 rows
// of 1000 columns: 256 lanes of one unit 63 us, 64 of four 66; of 2047: 256 of two
// 68, 128 of four 73; of 2560: 384 of two 65, 192 of four 78; of 8192: 1024 of two
// 71, 512 of four 78.)
template <bool BF, RowEnd END, class F>
hipError_t with_grad_team(int units, F&& fn) {
    using std::integral_constant;
    MUON_TEAM(8, 1);
    if constexpr (END != kShort) {
        MUON_TEAM(16, 1);
        MUON_TEAM(32, 1);
        MUON_TEAM(16, 3);
        MUON_TEAM(64, 1);
        MUON_TEAM(32, 3);
        MUON_TEAM(64, 2);
        if constexpr (BF) {
            MUON_TEAM(128, 2);
            MUON_TEAM(192, 2);
            MUON_TEAM(256, 2);
            MUON_TEAM(384, 2);
            MUON_TEAM(512, 2);
            MUON_TEAM(768, 2);
            MUON_TEAM(1024, 2);
        } else {
            MUON_TEAM(64, 3);
            MUON_TEAM(256, 1);
            MUON_TEAM(192, 2);
            MUON_TEAM(256, 2);
            MUON_TEAM(384, 2);
            MUON_TEAM(512, 2);
            MUON_TEAM(768, 2);
            MUON_TEAM(1024, 2);
            MUON_TEAM(768, 4);
            MUON_TEAM(1024, 4);
        }
    }
#undef MUON_TEAM
    return hipErrorInvalidValue;
}

int units_of(int cols, bool bf) { return (cols + (bf ? 7 : 3)) / (bf ? 8 : 4); }

// Workgroups for `rows` rows, `teams` to a workgroup, `each` workgroups a
// compute unit at most.
int blocks_for(int rows, int teams, int cus, int each) {
    const int64_t need = ((int64_t)rows + teams - 1) / teams;
    return (int)(need < (int64_t)cus * each ? need : (int64_t)cus * each);
}

NormCall with_loads(NormCall c) {
    c.nontemporal = (int64_t)c.rows * c.cols * (c.bf16 ? 2 : 4) >= kNontemporalBytes;
    return c;
}

// Calls fn(whether rows are bf16, how they end).
template <class F>
hipError_t with_types(const NormCall& c, F&& fn) {
    using std::integral_constant;
    auto with = [&](auto bf) {
        constexpr int V = bf.value ? 8 : 4;
        if (c.cols % V == 0) return fn(bf, integral_constant<RowEnd, kWhole>{});
        return c.cols > V ? fn(bf, integral_constant<RowEnd, kShifted>{}) : fn(bf, integral_constant<RowEnd, kShort>{});
    };
    return c.bf16 ? with(std::true_type{}) : with(std::false_type{});
}

}  // namespace

hipError_t launch_norm_forward(const NormCall& call, int cus, hipStream_t st) {
    const NormCall c = with_loads(call);
    return with_types(c, [&](auto bf, auto end) {
        return with_team<bf.value, end.value>(units_of(c.cols, c.bf16), [&](auto l, auto r) {
            constexpr int NT = threads_of<l.value>();
            const int blocks = blocks_for(c.rows, NT / l.value, cus, NT > 256 ? 2 : 2048 / NT);
            if (l.value < 64 && c.nontemporal)
                norm_forward_kernel<bf.value, end.value, l.value, r.value, l.value < 64><<<blocks, NT, 0, st>>>(c);
            else
                norm_forward_kernel<bf.value, end.value, l.value, r.value, false><<<blocks, NT, 0, st>>>(c);
            return hipGetLastError();
        });
    });
}

int norm_grad_blocks(int32_t rows, int32_t cols, bool bf16, int cus) {
    int blocks = 0;
    auto count = [&](auto bf, auto l, auto r) {
        constexpr int NT = grad_threads<bf.value, l.value>();
        // as many as registers leave room for
        blocks = blocks_for(rows, NT / l.value, cus, l.value > 64 ? std::max(1, 1024 / NT) : r.value > 1 ? 2 : 4);
        return hipSuccess;
    };
    const int units = units_of(cols, bf16);
    (void)(bf16 ? with_grad_team<true, kWhole>(units, [&](auto l, auto r) { return count(std::true_type{}, l, r); })
                : with_grad_team<false, kWhole>(units, [&](auto l, auto r) { return count(std::false_type{}, l, r); }));
    return blocks;
}

hipError_t launch_norm_grad(const NormCall& call, int cus, hipStream_t st) {
    const NormCall c = with_loads(call);
    const int blocks = norm_grad_blocks(c.rows, c.cols, c.bf16, cus);
    hipError_t e = hipSuccess;
    if (blocks > 0) e = with_types(c, [&](auto bf, auto end) {
        return with_grad_team<bf.value, end.value>(units_of(c.cols, c.bf16), [&](auto l, auto r) {
            constexpr int NT = grad_threads<bf.value, l.value>();
            if (l.value < 64 && c.nontemporal)
                norm_grad_kernel<bf.value, end.value, l.value, r.value, l.value < 64><<<blocks, NT, 0, st>>>(c);
            else
                norm_grad_kernel<bf.value, end.value, l.value, r.value, false><<<blocks, NT, 0, st>>>(c);
            return hipGetLastError();
        });
    });
    if (e != hipSuccess || blocks == 1 || (!c.dweight && !c.dbias)) return e;
    norm_grad_join_kernel<<<dim3((c.cols + 63) / 64, 2), 1024, 0, st>>>(c, blocks);
    return hipGetLastError();
}

}  // namespace muon
