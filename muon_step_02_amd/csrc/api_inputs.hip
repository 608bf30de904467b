// C ABI of the operators on what the optimizer step consumes (inputs.h):
// validation, workspace layout and launches.
#include <string.h>

#include <algorithm>
#include <new>

#include "context.h"
#include "inputs.h"

using namespace muon;

namespace {

// Whether a written range shares bytes with any other range, one owner's
// ranges among themselves excepted.  Sorts `r`.
bool any_collision(Rect* r, int n) {
    std::sort(r, r + n, [](const Rect& a, const Rect& b) { return a.lo < b.lo; });
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n && r[j].lo < r[i].hi; ++j)
            if ((r[i].write || r[j].write) && r[i].owner != r[j].owner && collide(r[i], r[j])) return true;
    return false;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// ---- gradient norm and clip ------------------------------------------------

constexpr int64_t kMaxChunks = INT32_MAX / 4;

bool dense(const muon_grad& g, bool clip) {
    return g.rows == 1 || (g.ld_grad == g.cols && (!clip || g.ld_out == g.cols));
}

// Chunks of one tensor: of its rows, or of all of it where they follow each
// other without gaps.
int64_t grad_chunks(const muon_grad& g, bool clip) {
    if (g.rows == 0 || g.cols == 0) return 0;
    const int64_t v = g.grad_dtype == MUON_BF16 ? 8 : 4;
    const bool d = dense(g, clip);
    const int64_t rows = d ? 1 : g.rows, cols = d ? g.rows * g.cols : g.cols;
    const int64_t units = rows * ((cols + v - 1) / v);
    return (units + kGradUnits - 1) / kGradUnits;
}

muon_status check_grad(const muon_grad& g) {
    constexpr int64_t lim = (int64_t)1 << 40;
    if (g.rows < 0 || g.cols < 0 || g.rows > lim || g.cols > lim || !valid_dtype(g.grad_dtype))
        return MUON_ERR_INVALID_ARG;
    if (g.rows > 0 && g.cols > 0 && g.cols > lim / g.rows) return MUON_ERR_INVALID_ARG;
    if (g.ld_grad < g.cols || (g.rows > 1 && g.ld_grad > lim / g.rows)) return MUON_ERR_INVALID_ARG;
    if (g.out && (!valid_dtype(g.out_dtype) || g.ld_out < g.cols || (g.rows > 1 && g.ld_out > lim / g.rows)))
        return MUON_ERR_INVALID_ARG;
    return MUON_OK;
}

muon_status check_grads(const muon_grad* gs, int n, bool clip, int64_t* chunks) {
    if (!gs || n < 1) return MUON_ERR_INVALID_ARG;
    int64_t total = 0;
    for (int i = 0; i < n; ++i) {
        const muon_grad& g = gs[i];
        const muon_status st = check_grad(g);
        if (st != MUON_OK) return st;
        if (g.rows == 0 || g.cols == 0) continue;
        if (!g.grad || (clip && !g.out)) return MUON_ERR_INVALID_ARG;
        if (misaligned(g.grad, elem_bytes(g.grad_dtype)) || (clip && misaligned(g.out, elem_bytes(g.out_dtype))))
            return MUON_ERR_UNALIGNED;
        total += grad_chunks(g, clip);
        if (total > kMaxChunks) return MUON_ERR_INVALID_ARG;
    }
    *chunks = total;
    return MUON_OK;
}

// Outputs share no memory with each other or with any gradient, but for the
// gradient a tensor is clipped in place of.
muon_status check_grad_overlap(const muon_grad* gs, int n) {
    Rect* r = new (std::nothrow) Rect[2 * (size_t)n];
    if (!r) return MUON_ERR_HIP;
    int k = 0;
    muon_status st = MUON_OK;
    for (int i = 0; i < n; ++i) {
        const muon_grad& g = gs[i];
        if (g.rows == 0 || g.cols == 0) continue;
        const size_t es = elem_bytes(g.grad_dtype), eo = elem_bytes(g.out_dtype);
        const Rect a = rect_of(g.grad, g.rows, g.cols, g.ld_grad, es, false, i);
        const Rect b = rect_of(g.out, g.rows, g.cols, g.ld_out, eo, true, i);
        const bool same = g.out == g.grad && es == eo && (g.rows == 1 || g.ld_out == g.ld_grad);
        if (!same && collide(a, b)) st = MUON_ERR_OVERLAP;
        r[k++] = a;
        r[k++] = b;
    }
    if (st == MUON_OK && any_collision(r, k)) st = MUON_ERR_OVERLAP;
    delete[] r;
    return st;
}

size_t grad_workspace_bytes(int n) {
    // one partial sum per block, one block more per launch at most
    const size_t parts = kGradBlocks + ((size_t)n + kGradGroup - 1) / kGradGroup;
    return align_up(parts * sizeof(double), 256);
}

// The workspace and the scalars, all of them written, share no memory with each
// other or with a tensor: blocks read one while others write the other.
muon_status check_grad_scalars(const muon_grad* gs, int n, bool clip, const float* norm_out,
                               const float* scale_out, const void* workspace) {
    Rect w[3];
    int k = 0;
    w[k++] = run_of(workspace, grad_workspace_bytes(n), true, 0);
    if (norm_out) w[k++] = run_of(norm_out, 4, true, 1);
    if (scale_out) w[k++] = run_of(scale_out, 4, true, 2);
    for (int i = 1; i < k; ++i)
        for (int j = 0; j < i; ++j)
            if (collide(w[i], w[j])) return MUON_ERR_OVERLAP;
    for (int t = 0; t < n; ++t) {
        const muon_grad& g = gs[t];
        if (g.rows == 0 || g.cols == 0) continue;
        const Rect a = rect_of(g.grad, g.rows, g.cols, g.ld_grad, elem_bytes(g.grad_dtype), false, 0);
        const Rect b = clip ? rect_of(g.out, g.rows, g.cols, g.ld_out, elem_bytes(g.out_dtype), true, 0) : a;
        for (int i = 0; i < k; ++i)
            if (collide(w[i], a) || collide(w[i], b)) return MUON_ERR_OVERLAP;
    }
    return MUON_OK;
}

// Calls fn(group, chunks of the group) for the tensors of each launch.
template <int CAP, class F>
hipError_t for_each_grad_group(const muon_grad* gs, int n, bool clip, F&& fn) {
    GradGroup<CAP> grp;
    memset(&grp, 0, sizeof(grp));
    int64_t chunks = 0;
    auto flush = [&]() -> hipError_t {
        if (grp.count == 0) return hipSuccess;
        grp.chunk_prefix[grp.count] = (int32_t)chunks;
        const hipError_t e = fn(grp, chunks);
        grp.count = 0;
        chunks = 0;
        return e;
    };
    for (int i = 0; i < n; ++i) {
        const muon_grad& g = gs[i];
        const int64_t c = grad_chunks(g, clip);
        if (c == 0) continue;
        if (grp.count == CAP) {
            const hipError_t e = flush();
            if (e != hipSuccess) return e;
        }
        const int k = grp.count++;
        const bool d = dense(g, clip);
        grp.g[k] = g.grad;
        grp.out[k] = clip ? g.out : nullptr;
        grp.rows[k] = d ? 1 : g.rows;
        grp.cols[k] = d ? g.rows * g.cols : g.cols;
        grp.ld_g[k] = d ? 0 : g.ld_grad;
        grp.ld_out[k] = d ? 0 : g.ld_out;
        grp.chunk_prefix[k] = (int32_t)chunks;
        grp.bf16[k] = g.grad_dtype == MUON_BF16;
        grp.out_bf16[k] = g.out_dtype == MUON_BF16;
        chunks += c;
    }
    return flush();
}

template <int CAP>
hipError_t grad_launches(const muon_grad* gs, int n, bool clip, int64_t total, float max_norm,
                         float* norm_out, float* scale_out, double* partials, hipStream_t s) {
    // One workgroup does it all where there is little to do: one launch.
    if (n <= CAP && total <= kGradSingle && total > 0)
        return for_each_grad_group<CAP>(gs, n, clip, [&](const GradGroup<CAP>& g, int64_t) {
            return launch_grad_single<CAP>(g, clip, max_norm, norm_out, scale_out, s);
        });
    // blocks in proportion to the chunks, kGradBlocks of them at most together
    auto blocks_of = [&](int64_t chunks) {
        if (total <= kGradBlocks) return (int)chunks;
        return (int)std::max<int64_t>(1, chunks * kGradBlocks / total);
    };
    int parts = 0;
    hipError_t e = for_each_grad_group<CAP>(gs, n, clip, [&](const GradGroup<CAP>& g, int64_t chunks) {
        const int b = blocks_of(chunks);
        const hipError_t r = launch_grad_sumsq<CAP>(g, b, partials + parts, s);
        parts += b;
        return r;
    });
    if (e != hipSuccess) return e;
    if (!clip || total == 0) return launch_grad_finalize(partials, parts, max_norm, norm_out, scale_out, s);
    bool first = true;
    return for_each_grad_group<CAP>(gs, n, clip, [&](const GradGroup<CAP>& g, int64_t chunks) {
        const hipError_t r = launch_grad_scale<CAP>(g, blocks_of(chunks), partials, parts, max_norm,
                                                    first ? norm_out : nullptr, first ? scale_out : nullptr, s);
        first = false;
        return r;
    });
}

muon_status grad_call(muon_handle h, const muon_grad* gs, int n, bool clip, float max_norm,
                      float* norm_out, float* scale_out, void* workspace, size_t workspace_bytes,
                      void* stream) {
    if (!h) return MUON_ERR_INVALID_ARG;
    int64_t chunks = 0;
    muon_status st = check_grads(gs, n, clip, &chunks);
    if (st != MUON_OK) return st;
    if (!finite(max_norm) || max_norm <= 0.f) return MUON_ERR_INVALID_ARG;
    if (!clip && !norm_out && !scale_out) return MUON_ERR_INVALID_ARG;
    if (misaligned(norm_out, 4) || misaligned(scale_out, 4)) return MUON_ERR_UNALIGNED;
    if (clip) {
        st = check_grad_overlap(gs, n);
        if (st != MUON_OK) return st;
    }
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < grad_workspace_bytes(n))
        return MUON_ERR_WORKSPACE;
    st = check_grad_scalars(gs, n, clip, norm_out, scale_out, workspace);
    if (st != MUON_OK) return st;
    DeviceGuard g(h->device);
    double* partials = reinterpret_cast<double*>(workspace);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return hip_status(n <= kGradGroupSmall
                          ? grad_launches<kGradGroupSmall>(gs, n, clip, chunks, max_norm, norm_out, scale_out, partials, s)
                          : grad_launches<kGradGroup>(gs, n, clip, chunks, max_norm, norm_out, scale_out, partials, s));
}

// ---- products grouped by expert --------------------------------------------

constexpr int64_t kMaxWidth = 1 << 20;

muon_status check_experts(const muon_experts* ex, const int32_t* offsets, int64_t tokens) {
    if (!ex || !ex->weights || !offsets) return MUON_ERR_INVALID_ARG;
    if (ex->experts < 1 || ex->experts > kMaxExperts || !valid_dtype(ex->dtype)) return MUON_ERR_INVALID_ARG;
    if (ex->rows < 1 || ex->cols < 1 || ex->rows > kMaxWidth || ex->cols > kMaxWidth || ex->ld < ex->cols ||
        ex->ld > kMaxWidth)
        return MUON_ERR_INVALID_ARG;
    if (tokens < 0 || tokens > INT32_MAX / 2) return MUON_ERR_INVALID_ARG;
    if (misaligned(offsets, 4)) return MUON_ERR_UNALIGNED;
    for (int e = 0; e < ex->experts; ++e) {
        if (!ex->weights[e]) return MUON_ERR_INVALID_ARG;
        if (misaligned(ex->weights[e], elem_bytes(ex->dtype))) return MUON_ERR_UNALIGNED;
    }
    return MUON_OK;
}

muon_status check_tokens(const void* p, int64_t ld, int64_t width, int64_t tokens, int32_t dtype) {
    if (ld < width || ld > kMaxWidth) return MUON_ERR_INVALID_ARG;
    if (tokens == 0) return MUON_OK;
    if (!p) return MUON_ERR_INVALID_ARG;
    return misaligned(p, elem_bytes(dtype)) ? MUON_ERR_UNALIGNED : MUON_OK;
}

// The experts' matrices and `n` more ranges: a written one shares no bytes
// with any other (owner -1: the experts', which may repeat where only read).
muon_status check_expert_overlap(const muon_experts* ex, bool write, const Rect* more, int n) {
    Rect* r = new (std::nothrow) Rect[(size_t)ex->experts + n];
    if (!r) return MUON_ERR_HIP;
    int k = 0;
    for (int e = 0; e < ex->experts; ++e)
        r[k++] = rect_of(ex->weights[e], ex->rows, ex->cols, ex->ld, elem_bytes(ex->dtype), write, e);
    for (int i = 0; i < n; ++i) {
        if (more[i].hi <= more[i].lo) continue;
        r[k] = more[i];
        r[k++].owner = ex->experts + i;
    }
    const bool bad = any_collision(r, k);
    delete[] r;
    return bad ? MUON_ERR_OVERLAP : MUON_OK;
}

Rect tokens_rect(const void* p, int64_t tokens, int64_t width, int64_t ld, int32_t dtype, bool write) {
    if (tokens == 0) return Rect{0, 0, 0, 1, false, 0};
    return rect_of(p, tokens, width, ld, elem_bytes(dtype), write, 0);
}

// launch_expert finds out which tiles a call takes, and refuses the sizes whose
// tiles no launch holds.
muon_status expert_status(hipError_t e) { return e == hipErrorInvalidConfiguration ? MUON_ERR_INVALID_ARG : hip_status(e); }

bool grid_fits(int64_t a, int64_t b, int64_t c) { return a * b <= INT32_MAX / (c > 0 ? c : 1); }

muon_status expert_rows(ExpertOp op, muon_handle h, const muon_experts* ex, const int32_t* offsets,
                        const void* x, int64_t ld_x, void* y, int64_t ld_y, int64_t tokens, void* stream) {
    if (!h) return MUON_ERR_INVALID_ARG;
    muon_status st = check_experts(ex, offsets, tokens);
    if (st != MUON_OK) return st;
    const int64_t wx = op == kExpertForward ? ex->cols : ex->rows;
    const int64_t wy = op == kExpertForward ? ex->rows : ex->cols;
    st = check_tokens(x, ld_x, wx, tokens, ex->dtype);
    if (st == MUON_OK) st = check_tokens(y, ld_y, wy, tokens, ex->dtype);
    if (st != MUON_OK) return st;
    // the smallest tiles: 32 x 64
    if (!grid_fits(tokens / 32 + ex->experts, (wy + 63) / 64, 1)) return MUON_ERR_INVALID_ARG;
    const Rect more[3] = {tokens_rect(x, tokens, wx, ld_x, ex->dtype, false),
                          tokens_rect(y, tokens, wy, ld_y, ex->dtype, true),
                          rect_of(offsets, 1, ex->experts + 1, ex->experts + 1, 4, false, 0)};
    st = check_expert_overlap(ex, false, more, 3);
    if (st != MUON_OK) return st;
    if (tokens == 0) return MUON_OK;
    ExpertCall c{};
    c.offsets = offsets;
    c.a = x;
    c.c = y;
    c.ld_a = ld_x;
    c.ld_c = ld_y;
    c.ld_w = ex->ld;
    c.tokens = tokens;
    c.experts = ex->experts;
    c.rows = (int32_t)ex->rows;
    c.cols = (int32_t)ex->cols;
    c.bf16 = ex->dtype == MUON_BF16;
    DeviceGuard g(h->device);
    return expert_status(launch_expert(op, c, ex->weights, reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

muon_status muon_grad_workspace_size(muon_handle h, const muon_grad* gs, int n, size_t* bytes) {
    if (!h || !bytes || !gs || n < 1) return MUON_ERR_INVALID_ARG;
    *bytes = grad_workspace_bytes(n);
    return MUON_OK;
}

muon_status muon_grad_norm(muon_handle h, const muon_grad* gs, int n, float max_norm, float* norm_out,
                           float* scale_out, void* workspace, size_t workspace_bytes, void* stream) {
    return grad_call(h, gs, n, false, max_norm, norm_out, scale_out, workspace, workspace_bytes, stream);
}

muon_status muon_grad_clip(muon_handle h, const muon_grad* gs, int n, float max_norm, float* norm_out,
                           float* scale_out, void* workspace, size_t workspace_bytes, void* stream) {
    return grad_call(h, gs, n, true, max_norm, norm_out, scale_out, workspace, workspace_bytes, stream);
}

muon_status muon_expert_forward(muon_handle h, const muon_experts* ex, const int32_t* offsets,
                                const void* x, int64_t ld_x, void* y, int64_t ld_y, int64_t tokens,
                                void* stream) {
    return expert_rows(kExpertForward, h, ex, offsets, x, ld_x, y, ld_y, tokens, stream);
}

muon_status muon_expert_grad_input(muon_handle h, const muon_experts* ex, const int32_t* offsets,
                                   const void* dy, int64_t ld_dy, void* dx, int64_t ld_dx,
                                   int64_t tokens, void* stream) {
    return expert_rows(kExpertGradInput, h, ex, offsets, dy, ld_dy, dx, ld_dx, tokens, stream);
}

muon_status muon_expert_grad_weight(muon_handle h, const muon_experts* grads, const int32_t* offsets,
                                    const void* x, int64_t ld_x, const void* dy, int64_t ld_dy,
                                    int64_t tokens, int32_t dtype, int accumulate, void* stream) {
    if (!h) return MUON_ERR_INVALID_ARG;
    muon_status st = check_experts(grads, offsets, tokens);
    if (st != MUON_OK) return st;
    if (!valid_dtype(dtype) || (accumulate != 0 && accumulate != 1)) return MUON_ERR_INVALID_ARG;
    // fp32 products rounded to bf16 gradients have no use here
    if (dtype == MUON_F32 && grads->dtype == MUON_BF16) return MUON_ERR_INVALID_ARG;
    st = check_tokens(x, ld_x, grads->cols, tokens, dtype);
    if (st == MUON_OK) st = check_tokens(dy, ld_dy, grads->rows, tokens, dtype);
    if (st != MUON_OK) return st;
    if (!grid_fits((grads->rows + 63) / 64, (grads->cols + 63) / 64, grads->experts)) return MUON_ERR_INVALID_ARG;
    const Rect more[3] = {tokens_rect(x, tokens, grads->cols, ld_x, dtype, false),
                          tokens_rect(dy, tokens, grads->rows, ld_dy, dtype, false),
                          rect_of(offsets, 1, grads->experts + 1, grads->experts + 1, 4, false, 0)};
    st = check_expert_overlap(grads, true, more, 3);
    if (st != MUON_OK) return st;
    ExpertCall c{};
    c.offsets = offsets;
    c.a = x;
    c.b = dy;
    c.ld_a = ld_x;
    c.ld_b = ld_dy;
    c.ld_w = grads->ld;
    c.tokens = tokens;
    c.experts = grads->experts;
    c.rows = (int32_t)grads->rows;
    c.cols = (int32_t)grads->cols;
    c.bf16 = dtype == MUON_BF16;
    c.out_bf16 = grads->dtype == MUON_BF16;
    c.accumulate = accumulate;
    DeviceGuard g(h->device);
    return expert_status(launch_expert(kExpertGradWeight, c, grads->weights, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Elements from the first to the last of (tokens, heads, head_dim) values.
__int128 span(int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim) {
    return tokens > 0 ? (__int128)(tokens - 1) * token + (__int128)(heads - 1) * head + dim : 0;
}

// parts: the most partial maxima either kernel's plan has for these sizes.
muon_status check_qk(const muon_qk* s, SmaxCall* c, int64_t* parts, muon_handle h) {
    if (!s) return MUON_ERR_INVALID_ARG;
    if (s->heads_q < 1 || s->heads_k < 1 || s->heads_q % s->heads_k || s->heads_q > 65536 ||
        s->head_dim < 1 || s->head_dim > 65536 || s->sequences < 1 || s->sequences > (1 << 20) ||
        !valid_dtype(s->dtype) || (s->causal != 0 && s->causal != 1))
        return MUON_ERR_INVALID_ARG;
    if (s->tokens_q < 0 || s->tokens_k < 0 || s->tokens_q > INT32_MAX / 2 || s->tokens_k > INT32_MAX / 2)
        return MUON_ERR_INVALID_ARG;
    if (!finite(s->scale) || s->scale <= 0.f) return MUON_ERR_INVALID_ARG;
    constexpr int64_t lim = (int64_t)1 << 40;
    if (s->q_token < 0 || s->q_head < 0 || s->k_token < 0 || s->k_head < 0 || s->q_token > lim ||
        s->q_head > lim || s->k_token > lim || s->k_head > lim)
        return MUON_ERR_INVALID_ARG;
    if (span(s->tokens_q, s->q_token, s->heads_q, s->q_head, s->head_dim) > lim ||
        span(s->tokens_k, s->k_token, s->heads_k, s->k_head, s->head_dim) > lim)
        return MUON_ERR_INVALID_ARG;
    c->q = s->q;
    c->k = s->k;
    c->tq = s->tokens_q;
    c->tk = s->tokens_k;
    c->q_token = s->q_token;
    c->q_head = s->q_head;
    c->k_token = s->k_token;
    c->k_head = s->k_head;
    c->cu_q = s->cu_q;
    c->cu_k = s->cu_k;
    c->sequences = s->sequences;
    c->heads_q = s->heads_q;
    c->heads_k = s->heads_k;
    c->head_dim = s->head_dim;
    c->bf16 = s->dtype == MUON_BF16;
    c->causal = s->causal;
    c->scale = s->scale;
    const bool fast = smax_chunked(*c);
    const int64_t other = smax_plan(*c, 8 * h->cus_per_xcd, !fast);
    const int64_t taken = smax_plan(*c, 8 * h->cus_per_xcd, fast);
    *parts = std::max(other, taken);
    // a launch of 256 threads a part holds fewer than 2^32
    return *parts > INT32_MAX || taken > UINT32_MAX / 256 ? MUON_ERR_INVALID_ARG : MUON_OK;
}

// Outputs and workspace share no memory with anything else of the call: blocks
// write them while others read the rest.
muon_status check_qk_overlap(const muon_qk* s, const float* smax_q, const float* smax_k, const void* workspace,
                             size_t workspace_bytes) {
    const size_t es = elem_bytes(s->dtype), cu = (size_t)(s->sequences + 1) * 4;
    const size_t q = (size_t)span(s->tokens_q, s->q_token, s->heads_q, s->q_head, s->head_dim) * es;
    const size_t k = (size_t)span(s->tokens_k, s->k_token, s->heads_k, s->k_head, s->head_dim) * es;
    Rect r[7];
    int n = 0;
    auto add = [&](const void* p, size_t bytes, bool write) {
        if (bytes) r[n] = run_of(p, bytes, write, n), ++n;
    };
    add(s->q, q, false);
    add(s->k, k, false);
    add(s->cu_q, cu, false);
    add(s->cu_k, cu, false);
    add(workspace, workspace_bytes, true);
    add(smax_q, smax_q ? (size_t)s->heads_q * 4 : 0, true);
    add(smax_k, smax_k ? (size_t)s->heads_k * 4 : 0, true);
    return any_collision(r, n) ? MUON_ERR_OVERLAP : MUON_OK;
}

size_t smax_workspace_bytes(int64_t parts) { return align_up((size_t)parts * sizeof(float) + 256, 256); }

}  // namespace

extern "C" {

muon_status muon_qk_smax_workspace_size(muon_handle h, const muon_qk* qk, size_t* bytes) {
    if (!h || !bytes) return MUON_ERR_INVALID_ARG;
    SmaxCall c{};
    int64_t parts = 0;
    const muon_status st = check_qk(qk, &c, &parts, h);
    if (st != MUON_OK) return st;
    *bytes = smax_workspace_bytes(parts);
    return MUON_OK;
}

muon_status muon_qk_smax(muon_handle h, const muon_qk* qk, float* smax_q, float* smax_k, int accumulate,
                         void* workspace, size_t workspace_bytes, void* stream) {
    if (!h) return MUON_ERR_INVALID_ARG;
    SmaxCall c{};
    int64_t parts = 0;
    muon_status st = check_qk(qk, &c, &parts, h);
    if (st != MUON_OK) return st;
    if (!smax_q && !smax_k) return MUON_ERR_INVALID_ARG;
    if (accumulate != 0 && accumulate != 1) return MUON_ERR_INVALID_ARG;
    if (!c.cu_q || !c.cu_k || (c.tq > 0 && !c.q) || (c.tk > 0 && !c.k)) return MUON_ERR_INVALID_ARG;
    const size_t es = elem_bytes(qk->dtype);
    if (misaligned(c.q, es) || misaligned(c.k, es) || misaligned(c.cu_q, 4) || misaligned(c.cu_k, 4) ||
        misaligned(smax_q, 4) || misaligned(smax_k, 4))
        return MUON_ERR_UNALIGNED;
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < smax_workspace_bytes(parts))
        return MUON_ERR_WORKSPACE;
    st = check_qk_overlap(qk, smax_q, smax_k, workspace, smax_workspace_bytes(parts));
    if (st != MUON_OK) return st;
    DeviceGuard g(h->device);
    return hip_status(launch_smax(c, reinterpret_cast<float*>(workspace), smax_q, smax_k, accumulate,
                                  reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
