// C ABI of the operators around the products and the logits (block.h):
// validation, workspace layout and launches.
#include <math.h>

#include <algorithm>

#include "block.h"
#include "context.h"

using namespace muon;

namespace {

constexpr int64_t kMaxSpan = (int64_t)1 << 40;  // elements from a tensor's first to its last
constexpr int64_t kMaxRows = INT32_MAX / 2;

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// ---- tensors of heads --------------------------------------------------------

bool strides_ok(const muon_heads& t, int64_t tokens, int64_t width) {
    if (t.heads < 1 || t.token < 0 || t.head < 0 || t.token > kMaxSpan || t.head > kMaxSpan) return false;
    if (tokens == 0) return true;
    const __int128 span = (__int128)(tokens - 1) * t.token + (__int128)(t.heads - 1) * t.head + width;
    return span <= kMaxSpan;
}

// Whether no two elements of the tensor are one.
bool distinct(const muon_heads& t, int64_t tokens, int64_t width) {
    if (tokens <= 1) return t.heads == 1 || t.head >= width;
    if (t.heads == 1) return t.token >= width;
    if (t.head >= width && t.token >= (t.heads - 1) * t.head + width) return true;
    return t.token >= width && t.head >= (tokens - 1) * t.token + width;
}

muon_status check_heads(const muon_heads* t, int64_t tokens, int64_t width, int32_t dtype, bool write) {
    if (!t || !strides_ok(*t, tokens, width)) return MUON_ERR_INVALID_ARG;
    if (write && !distinct(*t, tokens, width)) return MUON_ERR_INVALID_ARG;
    if (tokens == 0) return MUON_OK;
    if (!t->data) return MUON_ERR_INVALID_ARG;
    return misaligned(t->data, elem_bytes(dtype)) ? MUON_ERR_UNALIGNED : MUON_OK;
}

// The bytes from row to row of the tensor: exactly where its rows are evenly
// spaced, else with the gaps between a token's heads (or a head's tokens).
Rect heads_rect(const muon_heads& t, int64_t tokens, int64_t width, int32_t dtype, bool write, int owner) {
    const size_t es = elem_bytes(dtype);
    // (what is no stride apart is one)
    int64_t outer = t.token > 0 ? tokens : 1, so = t.token, inner = t.head > 0 ? t.heads : 1, si = t.head;
    if (inner == 1) return rect_of(t.data, outer, width, so, es, write, owner);
    if (outer == 1) return rect_of(t.data, inner, width, si, es, write, owner);
    if (si > so) {
        std::swap(outer, inner);
        std::swap(so, si);
    }
    const int64_t run = (inner - 1) * si + width;
    if (si >= width && so == inner * si) return rect_of(t.data, outer * inner, width, si, es, write, owner);
    if (so >= run) return rect_of(t.data, outer, run, so, es, write, owner);
    return run_of(t.data, (size_t)((outer - 1) * so + run) * es, write, owner);
}

bool same_place(const muon_heads& a, const muon_heads& b) {
    return a.data == b.data && a.token == b.token && a.head == b.head && a.heads == b.heads;
}

// The ranges of one call: what it writes shares no bytes with anything else.
struct Ranges {
    static constexpr int kMost = 16;
    Rect r[kMost];
    int n = 0;
    int add(const Rect& x) {
        if (x.hi <= x.lo) return -1;
        r[n] = x;
        r[n].owner = n;
        return n++;
    }
    int run(const void* p, size_t bytes, bool write) { return p && bytes ? add(run_of(p, bytes, write, 0)) : -1; }
    // two ranges that are one tensor, read and written in place
    void together(int a, int b) {
        if (a >= 0 && b >= 0) r[b].owner = r[a].owner;
    }
    bool clash() const {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((r[i].write || r[j].write) && r[i].owner != r[j].owner && collide(r[i], r[j])) return true;
        return false;
    }
};

int cus_of(muon_handle h) { return 8 * h->cus_per_xcd; }

// ---- layer norm ----------------------------------------------------------------

muon_status check_norm(const muon_layernorm* n, int32_t heads) {
    if (!n || heads < 1) return MUON_ERR_INVALID_ARG;
    if (n->tokens < 0 || n->tokens > kMaxRows / heads || n->cols < 1 || n->cols > kNormMaxCols)
        return MUON_ERR_INVALID_ARG;
    if (!valid_dtype(n->dtype) || !valid_dtype(n->weight_dtype) || (n->center != 0 && n->center != 1))
        return MUON_ERR_INVALID_ARG;
    if (!finite(n->eps) || n->eps < 0.f) return MUON_ERR_INVALID_ARG;
    return MUON_OK;
}

NormCall norm_call(const muon_layernorm* n, const muon_heads* x, const muon_heads* out) {
    NormCall c{};
    c.x = x->data;
    c.x_token = x->token;
    c.x_head = x->head;
    if (out) {
        c.out = out->data;
        c.out_token = out->token;
        c.out_head = out->head;
    }
    c.weight = n->weight;
    c.rows = (int32_t)(n->tokens * x->heads);
    c.heads = x->heads;
    c.cols = (int32_t)n->cols;
    c.bf16 = n->dtype == MUON_BF16;
    c.weight_bf16 = n->weight_dtype == MUON_BF16;
    c.center = n->center;
    c.eps = n->eps;
    return c;
}

size_t norm_workspace_bytes(const muon_layernorm* n, int32_t heads, int cus) {
    const int blocks = norm_grad_blocks((int32_t)(n->tokens * heads), (int32_t)n->cols, n->dtype == MUON_BF16, cus);
    return align_up((size_t)blocks * 2 * n->cols * sizeof(float) + 256, 256);
}

// ---- router --------------------------------------------------------------------

muon_status check_router(const muon_router* r) {
    if (!r) return MUON_ERR_INVALID_ARG;
    if (r->experts < 1 || r->experts > kRouterMaxExperts || r->top_k < 1 || r->top_k > kRouterMaxChoices ||
        r->top_k > r->experts || !valid_dtype(r->dtype) || (r->renormalize != 0 && r->renormalize != 1))
        return MUON_ERR_INVALID_ARG;
    if (r->tokens < 0 || r->tokens > kRouterMaxTokens || r->tokens > kMaxRows / r->top_k || r->ld < r->experts ||
        r->ld > kMaxSpan)
        return MUON_ERR_INVALID_ARG;
    if (r->tokens > 0 && r->ld > kMaxSpan / r->tokens) return MUON_ERR_INVALID_ARG;
    return MUON_OK;
}

size_t router_space(const muon_router* r, char* base, RouterSpace* s) {
    const int64_t blocks = (r->tokens + kRouterTokens - 1) / kRouterTokens;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = base + at;
        at = align_up(at + bytes, 256);
        return p;
    };
    const size_t cells = (size_t)blocks * r->experts;
    RouterSpace t{};
    t.total = reinterpret_cast<double*>(take((size_t)r->experts * 8));
    t.lse = reinterpret_cast<double*>(take((size_t)blocks * 8));
    t.live = reinterpret_cast<int32_t*>(take((size_t)blocks * 4));
    t.base = reinterpret_cast<int32_t*>(take(cells * 4));
    t.probs = reinterpret_cast<float*>(take(cells * 4));
    t.hist = reinterpret_cast<uint8_t*>(take(cells));
    t.blocks = (int32_t)blocks;
    if (s) *s = t;
    return at;
}

}  // namespace

extern "C" {

muon_status muon_layernorm_forward(muon_handle h, const muon_layernorm* n, const muon_heads* x,
                                   const muon_heads* y, float* mean, float* rstd, void* stream) {
    if (!h || !x || !y) return MUON_ERR_INVALID_ARG;
    muon_status st = check_norm(n, x->heads);
    if (st == MUON_OK) st = check_heads(x, n->tokens, n->cols, n->dtype, false);
    if (st == MUON_OK) st = check_heads(y, n->tokens, n->cols, n->dtype, true);
    if (st != MUON_OK) return st;
    if (y->heads != x->heads) return MUON_ERR_INVALID_ARG;
    const size_t wb = elem_bytes(n->weight_dtype);
    if (misaligned(n->weight, wb) || misaligned(n->bias, wb) || misaligned(mean, 4) || misaligned(rstd, 4))
        return MUON_ERR_UNALIGNED;
    if (n->tokens == 0) return MUON_OK;
    const size_t rows = (size_t)n->tokens * x->heads;
    Ranges r;
    const int ix = r.add(heads_rect(*x, n->tokens, n->cols, n->dtype, false, 0));
    const int iy = r.add(heads_rect(*y, n->tokens, n->cols, n->dtype, true, 0));
    if (same_place(*x, *y)) r.together(ix, iy);
    r.run(n->weight, n->cols * wb, false);
    r.run(n->bias, n->cols * wb, false);
    r.run(mean, rows * 4, true);
    r.run(rstd, rows * 4, true);
    if (r.clash()) return MUON_ERR_OVERLAP;
    NormCall c = norm_call(n, x, y);
    c.bias = n->bias;
    c.mean = mean;
    c.rstd = rstd;
    DeviceGuard g(h->device);
    return hip_status(launch_norm_forward(c, cus_of(h), reinterpret_cast<hipStream_t>(stream)));
}

muon_status muon_layernorm_workspace_size(muon_handle h, const muon_layernorm* n, int32_t heads, size_t* bytes) {
    if (!h || !bytes) return MUON_ERR_INVALID_ARG;
    const muon_status st = check_norm(n, heads);
    if (st != MUON_OK) return st;
    *bytes = norm_workspace_bytes(n, heads, cus_of(h));
    return MUON_OK;
}

muon_status muon_layernorm_grad(muon_handle h, const muon_layernorm* n, const muon_heads* x,
                                const muon_heads* dy, const float* mean, const float* rstd,
                                const muon_heads* dx, void* dweight, void* dbias, int32_t grad_dtype,
                                int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
    if (!h || !x || !dy) return MUON_ERR_INVALID_ARG;
    muon_status st = check_norm(n, x->heads);
    if (st == MUON_OK) st = check_heads(x, n->tokens, n->cols, n->dtype, false);
    if (st == MUON_OK) st = check_heads(dy, n->tokens, n->cols, n->dtype, false);
    if (st == MUON_OK && dx) st = check_heads(dx, n->tokens, n->cols, n->dtype, true);
    if (st != MUON_OK) return st;
    if (dy->heads != x->heads || (dx && dx->heads != x->heads)) return MUON_ERR_INVALID_ARG;
    if (!dx && !dweight && !dbias) return MUON_ERR_INVALID_ARG;
    if (!valid_dtype(grad_dtype) || (accumulate != 0 && accumulate != 1)) return MUON_ERR_INVALID_ARG;
    if (n->tokens > 0 && (!rstd || (n->center && !mean))) return MUON_ERR_INVALID_ARG;
    const size_t wb = elem_bytes(n->weight_dtype), gb = elem_bytes(grad_dtype);
    if (misaligned(n->weight, wb) || misaligned(mean, 4) || misaligned(rstd, 4) || misaligned(dweight, gb) ||
        misaligned(dbias, gb))
        return MUON_ERR_UNALIGNED;
    const size_t need = norm_workspace_bytes(n, x->heads, cus_of(h));
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < need) return MUON_ERR_WORKSPACE;
    const size_t rows = (size_t)n->tokens * x->heads;
    Ranges r;
    if (n->tokens > 0) {
        const int ix = r.add(heads_rect(*x, n->tokens, n->cols, n->dtype, false, 0));
        const int id = r.add(heads_rect(*dy, n->tokens, n->cols, n->dtype, false, 0));
        if (dx) {
            const int io = r.add(heads_rect(*dx, n->tokens, n->cols, n->dtype, true, 0));
            if (same_place(*x, *dx)) r.together(ix, io);
            if (same_place(*dy, *dx)) {
                // (where x, dy and dx are one, they all are)
                if (r.r[io].owner == ix) r.together(ix, id);
                r.together(id, io);
            }
        }
    }
    r.run(n->weight, n->cols * wb, false);
    r.run(n->center ? mean : nullptr, rows * 4, false);
    r.run(rstd, rows * 4, false);
    r.run(dweight, n->cols * gb, true);
    r.run(dbias, n->cols * gb, true);
    r.run(workspace, need, true);
    if (r.clash()) return MUON_ERR_OVERLAP;
    NormCall c = norm_call(n, x, dx);
    c.dy = dy->data;
    c.dy_token = dy->token;
    c.dy_head = dy->head;
    c.mean = const_cast<float*>(mean);
    c.rstd = const_cast<float*>(rstd);
    c.dweight = dweight;
    c.dbias = dbias;
    c.partials = reinterpret_cast<float*>(workspace);
    c.grad_bf16 = grad_dtype == MUON_BF16;
    c.accumulate = accumulate;
    DeviceGuard g(h->device);
    return hip_status(launch_norm_grad(c, cus_of(h), reinterpret_cast<hipStream_t>(stream)));
}

muon_status muon_rotary_frequencies(const muon_rotary_plan* p, double* out) {
    if (!p || !out || p->pairs < 1 || p->pairs > kRotaryPairs) return MUON_ERR_INVALID_ARG;
    if (!isfinite(p->base) || p->base <= 0.0) return MUON_ERR_INVALID_ARG;
    if (p->scaling < MUON_ROTARY_NONE || p->scaling > MUON_ROTARY_PARTS) return MUON_ERR_INVALID_ARG;
    if (p->scaling != MUON_ROTARY_NONE && (!isfinite(p->factor) || p->factor <= 0.0)) return MUON_ERR_INVALID_ARG;
    if (p->scaling == MUON_ROTARY_BASE && p->pairs < 2) return MUON_ERR_INVALID_ARG;
    if (p->scaling == MUON_ROTARY_PARTS &&
        (!isfinite(p->context) || p->context <= 0.0 || !isfinite(p->low) || !isfinite(p->high) || p->low >= p->high))
        return MUON_ERR_INVALID_ARG;
    double base = p->base;
    if (p->scaling == MUON_ROTARY_BASE) base *= pow(p->factor, p->pairs / (p->pairs - 1.0));
    for (int i = 0; i < p->pairs; ++i) {
        double f = pow(base, -(double)i / p->pairs);
        if (p->scaling == MUON_ROTARY_LINEAR) f /= p->factor;
        if (p->scaling == MUON_ROTARY_PARTS) {
            constexpr double kTurn = 6.28318530717958647693;
            const double k = std::min(1.0, std::max(0.0, (p->context * f / kTurn - p->low) / (p->high - p->low)));
            f *= k + (1.0 - k) / p->factor;
        }
        out[i] = f;
    }
    return MUON_OK;
}

muon_status muon_rotary(muon_handle h, const muon_positions* r, const muon_heads* x, const muon_heads* y, int n,
                        int transpose, void* stream) {
    if (!h || !r || !x || !y || n < 1 || n > kRotaryTensors) return MUON_ERR_INVALID_ARG;
    if (r->tokens < 0 || r->tokens > kMaxRows || r->head_dim < 1 || r->head_dim > 65536 || r->pairs < 1 ||
        r->pairs > kRotaryPairs || r->first < 0 || r->first > r->head_dim - 2 * r->pairs ||
        !valid_dtype(r->dtype) || (r->interleaved != 0 && r->interleaved != 1) ||
        (transpose != 0 && transpose != 1) || !finite(r->scale))
        return MUON_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        if (x[i].heads != y[i].heads || x[i].heads > 65536) return MUON_ERR_INVALID_ARG;
        muon_status st = check_heads(&x[i], r->tokens, r->head_dim, r->dtype, false);
        if (st == MUON_OK) st = check_heads(&y[i], r->tokens, r->head_dim, r->dtype, true);
        if (st != MUON_OK) return st;
    }
    if (r->tokens == 0) return MUON_OK;
    if (!r->positions || !r->frequencies) return MUON_ERR_INVALID_ARG;
    if (misaligned(r->positions, 4) || misaligned(r->frequencies, 8)) return MUON_ERR_UNALIGNED;
    RotaryCall c{};
    Ranges ranges;
    for (int i = 0; i < n; ++i) {
        c.t[i] = RotaryTensor{x[i].data, y[i].data, x[i].token, x[i].head, y[i].token, y[i].head, x[i].heads};
        const int ix = ranges.add(heads_rect(x[i], r->tokens, r->head_dim, r->dtype, false, 0));
        const int iy = ranges.add(heads_rect(y[i], r->tokens, r->head_dim, r->dtype, true, 0));
        if (same_place(x[i], y[i])) ranges.together(ix, iy);
    }
    ranges.run(r->positions, (size_t)r->tokens * 4, false);
    ranges.run(r->frequencies, (size_t)r->pairs * 8, false);
    if (ranges.clash()) return MUON_ERR_OVERLAP;
    c.count = n;
    c.positions = r->positions;
    c.frequencies = r->frequencies;
    c.tokens = (int32_t)r->tokens;
    c.head_dim = r->head_dim;
    c.first = r->first;
    c.pairs = r->pairs;
    c.interleaved = r->interleaved;
    c.transpose = transpose;
    c.bf16 = r->dtype == MUON_BF16;
    c.scale = r->scale;
    if (!rotary_fits(c)) return MUON_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    return hip_status(launch_rotary(c, reinterpret_cast<hipStream_t>(stream)));
}

muon_status muon_router_workspace_size(muon_handle h, const muon_router* r, size_t* bytes) {
    if (!h || !bytes) return MUON_ERR_INVALID_ARG;
    const muon_status st = check_router(r);
    if (st != MUON_OK) return st;
    *bytes = router_space(r, nullptr, nullptr);
    return MUON_OK;
}

muon_status muon_router_forward(muon_handle h, const muon_router* r, const muon_routing* out, void* workspace,
                                size_t workspace_bytes, void* stream) {
    if (!h || !out) return MUON_ERR_INVALID_ARG;
    const muon_status st = check_router(r);
    if (st != MUON_OK) return st;
    if (!out->counts || !out->offsets || (r->tokens > 0 && (!r->logits || !out->chosen || !out->gates)))
        return MUON_ERR_INVALID_ARG;
    const void* words[] = {out->chosen, out->gates, out->counts, out->offsets,
                           out->rows,   out->order, out->live,   out->losses};
    for (const void* p : words)
        if (misaligned(p, 4)) return MUON_ERR_UNALIGNED;
    if (misaligned(r->logits, elem_bytes(r->dtype))) return MUON_ERR_UNALIGNED;
    const size_t need = router_space(r, nullptr, nullptr);
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < need) return MUON_ERR_WORKSPACE;
    const size_t choices = (size_t)r->tokens * r->top_k * 4;
    Ranges ranges;
    if (r->tokens > 0)
        ranges.add(rect_of(r->logits, r->tokens, r->experts, r->ld, elem_bytes(r->dtype), false, 0));
    ranges.run(out->chosen, choices, true);
    ranges.run(out->gates, choices, true);
    ranges.run(out->counts, (size_t)r->experts * 4, true);
    ranges.run(out->offsets, (size_t)(r->experts + 1) * 4, true);
    ranges.run(out->rows, choices, true);
    ranges.run(out->order, choices, true);
    ranges.run(out->live, 4, true);
    ranges.run(out->losses, 8, true);
    ranges.run(workspace, need, true);
    if (ranges.clash()) return MUON_ERR_OVERLAP;
    RouterCall c{};
    c.logits = r->logits;
    c.ld = r->ld;
    c.tokens = (int32_t)r->tokens;
    c.experts = r->experts;
    c.top_k = r->top_k;
    c.bf16 = r->dtype == MUON_BF16;
    c.renormalize = r->renormalize;
    c.chosen = out->chosen;
    c.gates = out->gates;
    c.rows = out->rows;
    c.order = out->order;
    c.counts = out->counts;
    c.offsets = out->offsets;
    c.live = out->live;
    c.losses = out->losses;
    RouterSpace s;
    router_space(r, reinterpret_cast<char*>(workspace), &s);
    DeviceGuard g(h->device);
    return hip_status(launch_router(c, s, reinterpret_cast<hipStream_t>(stream)));
}

muon_status muon_router_grad(muon_handle h, const muon_router* r, const int32_t* chosen, const int32_t* counts,
                             const int32_t* live, const float* dgates, float balance, float z, void* dlogits,
                             int64_t ld_dlogits, void* stream) {
    if (!h) return MUON_ERR_INVALID_ARG;
    const muon_status st = check_router(r);
    if (st != MUON_OK) return st;
    if (!finite(balance) || !finite(z)) return MUON_ERR_INVALID_ARG;
    if (ld_dlogits < r->experts || ld_dlogits > kMaxSpan || (r->tokens > 0 && ld_dlogits > kMaxSpan / r->tokens))
        return MUON_ERR_INVALID_ARG;
    if (r->tokens == 0) return MUON_OK;
    if (!r->logits || !chosen || !counts || !live || !dlogits) return MUON_ERR_INVALID_ARG;
    const size_t es = elem_bytes(r->dtype);
    if (misaligned(r->logits, es) || misaligned(dlogits, es) || misaligned(chosen, 4) || misaligned(counts, 4) ||
        misaligned(live, 4) || misaligned(dgates, 4))
        return MUON_ERR_UNALIGNED;
    const size_t choices = (size_t)r->tokens * r->top_k * 4;
    Ranges ranges;
    ranges.add(rect_of(r->logits, r->tokens, r->experts, r->ld, es, false, 0));
    ranges.add(rect_of(dlogits, r->tokens, r->experts, ld_dlogits, es, true, 0));
    ranges.run(chosen, choices, false);
    ranges.run(counts, (size_t)r->experts * 4, false);
    ranges.run(live, 4, false);
    ranges.run(dgates, choices, false);
    if (ranges.clash()) return MUON_ERR_OVERLAP;
    RouterGradCall c{};
    c.logits = r->logits;
    c.ld = r->ld;
    c.tokens = (int32_t)r->tokens;
    c.experts = r->experts;
    c.top_k = r->top_k;
    c.bf16 = r->dtype == MUON_BF16;
    c.renormalize = r->renormalize;
    c.chosen = chosen;
    c.counts = counts;
    c.live = live;
    c.dgates = dgates;
    c.dlogits = dlogits;
    c.ld_out = ld_dlogits;
    c.balance = balance;
    c.z = z;
    DeviceGuard g(h->device);
    return hip_status(launch_router_grad(c, cus_of(h), reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
