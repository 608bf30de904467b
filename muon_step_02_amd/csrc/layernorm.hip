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
// registers of its team of 8 to 512 lanes from its load to its store, so the
// variance is the mean of the squared differences themselves, in a second sum
// over registers.  Weight and bias are read once per workgroup, which then
// walks over rows.
#include <type_traits>

#include "block.h"
#include "team.h"
#include "units.h"

namespace muon {

namespace {

template <int L>
constexpr int threads_of() { return L > 256 ? L : 256; }

// V elements of weight or bias, `left` of them there; `absent` without one.
template <int V>
__device__ __forceinline__ void load_weight(const void* w, bool bf, int off, int left, float absent, float* out) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = absent;
    } else if (bf) {
        const Raw<true, V> r = load_raw<true, V, false>(w, off, left);
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = r.at(e);
    } else {
#pragma unroll
        for (int p = 0; p < V; p += 4) {
            const Raw<false, 4> r = load_raw<false, 4, false>(w, off + p, left - p);
#pragma unroll
            for (int e = 0; e < 4; ++e) out[p + e] = r.at(e);
        }
    }
}

// A team's row: lane l holds units l, l + L, ... of V elements.
template <bool BF, bool EVEN, int L, int R>
struct Row {
    static constexpr int V = BF ? 8 : 4;
    Raw<BF, V> u[R];
    __device__ __forceinline__ void load(const void* base, int64_t off, int cols, int l, bool has) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = (i * L + l) * V, left = has ? cols - c : 0;
            if (!EVEN) {
                u[i] = load_raw<BF, V, false>(base, off + c, left);
            } else if (left > 0) {
                u[i] = load_raw<BF, V, true>(base, off + c, V);
            } else {
#pragma unroll
                for (int k = 0; k < Raw<BF, V>::W; ++k) u[i].w[k] = 0;
            }
        }
    }
};

template <bool BF, bool EVEN>
__device__ __forceinline__ void store_row(void* base, int64_t off, int left, const float* v) {
    constexpr int V = BF ? 8 : 4;
    if (!EVEN)
        store_unit<V, BF, false>(base, off, left, v);
    else if (left > 0)
        store_unit<V, BF, true>(base, off, V, v);
}

// Sums over a team.  A team of more lanes than a wave has is a whole
// workgroup: its waves meet in LDS, in one of two slots in turn, so that one
// barrier a sum is enough (a wave that writes a slot again has passed the
// other slot's barrier, which every wave reaches after it has read).
template <int L>
struct TeamSum {
    float* red;  // [2][2 * waves]
    int slot = 0;
    __device__ __forceinline__ explicit TeamSum(float* r) : red(r) {}
    __device__ __forceinline__ void operator()(float& a, float& b, bool two) {
        constexpr int W = L > 64 ? L / 64 : 1;
        a = team_sum<(L > 64 ? 64 : L)>(a);
        if (two) b = team_sum<(L > 64 ? 64 : L)>(b);
        if constexpr (W > 1) {
            float* s = red + slot * 2 * W;
            const int w = threadIdx.x >> 6;
            if ((threadIdx.x & 63) == 0) {
                s[w] = a;
                s[W + w] = b;
            }
            __syncthreads();
            a = s[0];
            b = s[W];
#pragma unroll
            for (int i = 1; i < W; ++i) {
                a += s[i];
                b += s[W + i];
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

template <bool BF, bool EVEN, int L, int R>
__global__ __launch_bounds__(threads_of<L>()) void norm_forward_kernel(NormCall c) {
    constexpr int V = BF ? 8 : 4, TEAMS = threads_of<L>() / L;
    __shared__ float red[L > 64 ? 4 * (L / 64) : 1];
    const int l = threadIdx.x % L, team = threadIdx.x / L;
    float w[R][V], b[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int col = (i * L + l) * V;
        load_weight<V>(c.weight, c.weight_bf16, col, c.cols - col, 1.f, w[i]);
        load_weight<V>(c.bias, c.weight_bf16, col, c.cols - col, 0.f, b[i]);
    }
    TeamSum<L> sum(red);
    const float n = (float)c.cols;
    for (int64_t first = (int64_t)blockIdx.x * TEAMS; first < c.rows; first += (int64_t)gridDim.x * TEAMS) {
        const int row = (int)first + team;
        const bool has = row < c.rows;
        Row<BF, EVEN, L, R> x;
        x.load(c.x, has ? row_at(row, c.heads, c.x_token, c.x_head) : 0, c.cols, l, has);
        float v[R][V], mean = 0.f, none = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = x.u[i].at(e);
        if (c.center) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) mean += v[i][e];
            sum(mean, none, false);
            mean /= n;
        }
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int left = c.cols - (i * L + l) * V;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[i][e] -= mean;
                // places behind the row are not part of its variance
                const float d = (EVEN ? left > 0 : e < left) ? v[i][e] : 0.f;
                sq = fmaf(d, d, sq);
            }
        }
        sum(sq, none, false);
        const float rstd = 1.f / sqrtf(sq / n + c.eps);
        if (!has) continue;
        if (l == 0) {
            if (c.mean) gst(c.mean + row, mean);
            if (c.rstd) gst(c.rstd + row, rstd);
        }
        const int64_t at = row_at(row, c.heads, c.out_token, c.out_head);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int col = (i * L + l) * V;
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = fmaf(v[i][e] * rstd, w[i][e], b[i][e]);
            store_row<BF, EVEN>(c.out, at + col, c.cols - col, v[i]);
        }
    }
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

// dx, and each workgroup's sums for dw and db over its rows.
template <bool BF, bool EVEN, int L, int R>
__global__ __launch_bounds__(threads_of<L>()) void norm_grad_kernel(NormCall c) {
    constexpr int V = BF ? 8 : 4, NT = threads_of<L>(), TEAMS = NT / L;
    __shared__ float red[L > 64 ? 4 * (L / 64) : NT * R * V];
    const int l = threadIdx.x % L, team = threadIdx.x / L;
    float w[R][V], dw[R][V], db[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int col = (i * L + l) * V;
        load_weight<V>(c.weight, c.weight_bf16, col, c.cols - col, 1.f, w[i]);
#pragma unroll
        for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = 0.f;
    }
    TeamSum<L> sum(red);
    const float n = (float)c.cols;
    for (int64_t first = (int64_t)blockIdx.x * TEAMS; first < c.rows; first += (int64_t)gridDim.x * TEAMS) {
        const int row = (int)first + team;
        const bool has = row < c.rows;
        Row<BF, EVEN, L, R> x, dy;
        x.load(c.x, has ? row_at(row, c.heads, c.x_token, c.x_head) : 0, c.cols, l, has);
        dy.load(c.dy, has ? row_at(row, c.heads, c.dy_token, c.dy_head) : 0, c.cols, l, has);
        const float mean = has && c.center ? gld(c.mean + row) : 0.f, rstd = has ? gld(c.rstd + row) : 0.f;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float hat = (x.u[i].at(e) - mean) * rstd, d = dy.u[i].at(e), g = d * w[i][e];
                dw[i][e] = fmaf(d, hat, dw[i][e]);
                db[i][e] += d;
                s1 = fmaf(g, hat, s1);
                s2 += g;
            }
        if (!c.out) continue;
        sum(s1, s2, c.center);
        s1 /= n;
        s2 = c.center ? s2 / n : 0.f;
        if (!has) continue;
        const int64_t at = row_at(row, c.heads, c.out_token, c.out_head);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int col = (i * L + l) * V;
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float hat = (x.u[i].at(e) - mean) * rstd, g = dy.u[i].at(e) * w[i][e];
                o[e] = rstd * (g - s2 - hat * s1);
            }
            store_row<BF, EVEN>(c.out, at + col, c.cols - col, o);
        }
    }
    // the teams' sums, added in their order
    auto put = [&](int side, float (&acc)[R][V], void* out) {
        if (!out) return;
        if constexpr (TEAMS > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) red[(team * R + i) * L * V + l * V + e] = acc[i][e];
            __syncthreads();
            for (int col = threadIdx.x; col < c.cols; col += NT) {
                float s = red[col];
                for (int t = 1; t < TEAMS; ++t) s += red[t * R * L * V + col];
                if (gridDim.x == 1)
                    put_grad(out, c.grad_bf16, c.accumulate, col, s);
                else
                    gst(c.partials + ((int64_t)side * gridDim.x + blockIdx.x) * c.cols + col, s);
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int col = (i * L + l) * V;
                if (gridDim.x == 1) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (col + e < c.cols) put_grad(out, c.grad_bf16, c.accumulate, col + e, acc[i][e]);
                } else {
                    float* p = c.partials + ((int64_t)side * gridDim.x + blockIdx.x) * c.cols;
#pragma unroll
                    for (int h = 0; h < V; h += 4)
                        store_unit<4, false, false>(p, col + h, c.cols - col - h, &acc[i][h]);
                }
            }
        }
    };
    put(0, dw, c.dweight);
    put(1, db, c.dbias);
}

// dw and db from the workgroups' sums: 64 columns a workgroup, each of its 16
// waves every 16th sum, in 64 bits.
__global__ __launch_bounds__(1024) void norm_grad_join_kernel(NormCall c, int blocks) {
    __shared__ double part[16][64];
    void* out = blockIdx.y ? c.dbias : c.dweight;
    if (!out) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
    double s = 0.0;
    if (col < c.cols) {
        const float* p = c.partials + (int64_t)blockIdx.y * blocks * c.cols + col;
        for (int b = wave; b < blocks; b += 16) s += gld(p + (int64_t)b * c.cols);
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave || col >= c.cols) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) s += part[i][lane];
    put_grad(out, c.grad_bf16, c.accumulate, col, s);
}

// Calls fn(lanes of a team, units a lane) for a row of `units` 16-byte units.
template <bool BF, class F>
hipError_t with_team(int units, F&& fn) {
    using std::integral_constant;
#define MUON_TEAM(L, R) fn(integral_constant<int, L>{}, integral_constant<int, R>{})
    if (units <= 8) return MUON_TEAM(8, 1);
    if (units <= 16) return MUON_TEAM(16, 1);
    if (units <= 32) return MUON_TEAM(32, 1);
    if (units <= 64) return MUON_TEAM(64, 1);
    if (units <= 128) return MUON_TEAM(64, 2);
    if (units <= 256) return MUON_TEAM(256, 1);
    if (units <= 512) return MUON_TEAM(256, 2);
    if (units <= 1024) return MUON_TEAM(256, 4);
    if (BF || units <= 2048) return MUON_TEAM(512, 4);
    return MUON_TEAM(512, 8);
#undef MUON_TEAM
}

int units_of(int cols, bool bf) { return (cols + (bf ? 7 : 3)) / (bf ? 8 : 4); }

// Workgroups for `rows` rows, `teams` to a workgroup, `each` workgroups a
// compute unit at most.
int blocks_for(int rows, int teams, int cus, int each) {
    const int64_t need = ((int64_t)rows + teams - 1) / teams;
    return (int)(need < (int64_t)cus * each ? need : (int64_t)cus * each);
}

template <class F>
hipError_t with_types(const NormCall& c, F&& fn) {
    const bool even = c.cols % (c.bf16 ? 8 : 4) == 0;
    if (c.bf16) return even ? fn(std::true_type{}, std::true_type{}) : fn(std::true_type{}, std::false_type{});
    return even ? fn(std::false_type{}, std::true_type{}) : fn(std::false_type{}, std::false_type{});
}

}  // namespace

hipError_t launch_norm_forward(const NormCall& c, int cus, hipStream_t st) {
    return with_types(c, [&](auto bf, auto even) {
        return with_team<bf.value>(units_of(c.cols, c.bf16), [&](auto l, auto r) {
            constexpr int NT = threads_of<l.value>();
            const int blocks = blocks_for(c.rows, NT / l.value, cus, NT > 256 ? 2 : 8);
            norm_forward_kernel<bf.value, even.value, l.value, r.value><<<blocks, NT, 0, st>>>(c);
            return hipGetLastError();
        });
    });
}

int norm_grad_blocks(int32_t rows, int32_t cols, bool bf16, int cus) {
    int blocks = 0;
    // (a unit's lanes do not depend on its type)
    (void)with_team<false>(units_of(cols, bf16), [&](auto l, auto) {
        constexpr int NT = threads_of<l.value>();
        blocks = blocks_for(rows, NT / l.value, cus, NT > 256 ? 1 : 2);
        return hipSuccess;
    });
    return blocks;
}

hipError_t launch_norm_grad(const NormCall& c, int cus, hipStream_t st) {
    const int blocks = norm_grad_blocks(c.rows, c.cols, c.bf16, cus);
    hipError_t e = hipSuccess;
    if (blocks > 0) e = with_types(c, [&](auto bf, auto even) {
        return with_team<bf.value>(units_of(c.cols, c.bf16), [&](auto l, auto r) {
            norm_grad_kernel<bf.value, even.value, l.value, r.value><<<blocks, threads_of<l.value>(), 0, st>>>(c);
            return hipGetLastError();
        });
    });
    if (e != hipSuccess || blocks == 1 || (!c.dweight && !c.dbias)) return e;
    norm_grad_join_kernel<<<dim3((c.cols + 63) / 64, 2), 1024, 0, st>>>(c, blocks);
    return hipGetLastError();
}

}  // namespace muon
