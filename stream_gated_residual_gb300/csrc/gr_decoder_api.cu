// C entries of the decoder parts around the Gated Residual (embedding, layer norm, linear attention
// and their gradients): host-side validation, dispatch, status codes. Contracts in include/gr.h.
#include <math.h>

#include "gr_internal.h"
#include "gr_mixer.h"

namespace gr {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t width(int dtype) { return dtype == GR_BF16 ? 2 : 4; }
bool real_dtype(int dtype) { return dtype == GR_F32 || dtype == GR_BF16; }
int as_status(cudaError_t e) { return e == cudaSuccess ? GR_OK : GR_E_CUDA; }

// A buffer of a call: where it starts and how many bytes the call may touch.
struct Span {
    const void* p;
    size_t n;
};
bool meet(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}

int check_embedding(const gr_embedding* e) {
    if (!e) return GR_E_NULL;
    if (e->n_tokens < 0 || e->n_tokens > (int64_t(1) << 40) || e->n_vocab < 1 ||
        e->n_vocab > 0x7fffffffLL || e->d_model < 8 || e->d_model % 8 != 0 || e->d_model > GR_MAX_D ||
        (e->n_branch != 1 && e->n_branch != kBranches))
        return GR_E_SHAPE;
    if (!real_dtype(e->table_dtype) || !real_dtype(e->state_dtype) ||
        (e->id_bits != 32 && e->id_bits != 64))
        return GR_E_DTYPE;
    return GR_OK;
}

int check_norm(const gr_norm* n) {
    if (!n) return GR_E_NULL;
    if (n->n_tokens < 0 || n->n_tokens > (int64_t(1) << 40) || n->d_model < 8 || n->d_model % 8 != 0 ||
        n->d_model > GR_MAX_D || (n->n_group != 1 && n->n_group != kBranches))
        return GR_E_SHAPE;
    if (!real_dtype(n->dtype)) return GR_E_DTYPE;
    if (!(n->eps >= 0.0f) || !isfinite(n->eps)) return GR_E_EPS;
    return GR_OK;
}

int check_mixer(const gr_mixer* m) {
    if (!m) return GR_E_NULL;
    if (m->n_tokens < 0 || m->n_tokens > 0x7fffffffLL || m->n_seqs < 0 || m->n_heads < 1 ||
        int64_t(m->n_seqs) * m->n_heads > 0x7fffffffLL || m->d_key < 8 || m->d_key % 8 != 0 ||
        m->d_key > GR_MAX_HEAD || m->d_value < 8 || m->d_value % 8 != 0 || m->d_value > GR_MAX_HEAD)
        return GR_E_SHAPE;
    if (!real_dtype(m->dtype)) return GR_E_DTYPE;
    return GR_OK;
}

// One rows argument with its extent: what the strides reach from the first element to the last.
struct Rows {
    const gr_rows* r;
    int64_t n, h, d;
    size_t w;
    bool token_major() const { return n <= 1 || r->token_stride >= (h - 1) * r->head_stride + d; }
    int64_t extent() const { return (n - 1) * r->token_stride + (h - 1) * r->head_stride + d; }
    Span span() const { return {r->data, n > 0 ? size_t(extent()) * w : 0}; }
    int check(bool output) const {
        if (n == 0) return GR_OK;
        if (!r->data) return GR_E_NULL;
        const int64_t ts = r->token_stride, hs = r->head_stride, most = int64_t(1) << 46;
        if ((n > 1 && (ts < d || ts > most / n)) || (h > 1 && (hs < d || hs > most / h)) ||
            ts < 0 || hs < 0)
            return GR_E_SHAPE;
        if (!aligned(r->data, 16) || (n > 1 && size_t(ts) * w % 16 != 0) ||
            (h > 1 && size_t(hs) * w % 16 != 0))
            return GR_E_ALIGN;
        if (output && !token_major() && h > 1 && hs < (n - 1) * ts + d) return GR_E_SHAPE;
        return GR_OK;
    }
    // Whether two rows arguments may touch a common byte. Views of one fused buffer do not: their
    // tokens' rows lie between each other's (the same token stride), their heads' (the same head
    // stride), or, at the same two strides, the heads of every token or the tokens of every head.
    bool meets(const Rows& o) const {
        if (!meet(span(), o.span())) return false;
        if (w != o.w) return true;
        const int64_t gap = (int64_t(reinterpret_cast<uintptr_t>(o.r->data)) -
                             int64_t(reinterpret_cast<uintptr_t>(r->data))) / int64_t(w);
        const int64_t ts = r->token_stride, hs = r->head_stride;
        const bool same_t = n > 1 && ts == o.r->token_stride, same_h = h > 1 && hs == o.r->head_stride;
        auto mod = [](int64_t x, int64_t y) { return ((x % y) + y) % y; };
        // blocks of `mine` and `its` elements that repeat with one period, beside each other in it
        auto beside = [&](int64_t g, int64_t period, int64_t mine, int64_t its) {
            const int64_t at = mod(g, period);
            return at >= mine && at + its <= period;
        };
        if (same_t && beside(gap, ts, (h - 1) * hs + d, (o.h - 1) * o.r->head_stride + o.d)) return false;
        if (same_h && beside(gap, hs, (n - 1) * ts + d, (o.n - 1) * o.r->token_stride + o.d)) return false;
        // `count` rows at the inner stride within each outer period, the later block not past its end
        auto between = [&](int64_t outer, int64_t inner, int64_t count) {
            const int64_t mine = (count - 1) * inner + d, its = (count - 1) * inner + o.d;
            if (mine > outer || its > outer) return false;
            const int64_t after = mod(gap, outer), ahead = mod(-gap, outer);
            return (after + its <= outer && beside(after, inner, d, o.d)) ||
                   (ahead + mine <= outer && beside(ahead, inner, o.d, d));
        };
        return !(same_t && same_h && (between(ts, hs, h) || between(hs, ts, n)));
    }
    MixRows mix() const {
        // strides of a dimension of one are never used to step, but reach the tensor maps
        return {r->data, n > 1 ? r->token_stride : h * (h > 1 ? r->head_stride : d),
                h > 1 ? r->head_stride : d};
    }
};

bool tc_shape(const gr_mixer* m) {
    return m->dtype == GR_BF16 && (m->d_key == 64 || m->d_key == 128) &&
           (m->d_value == 64 || m->d_value == 128);
}

// Workspace of a prompt, or of its gradient: on the tensor cores all three passes at once where they
// have the same shape (d_key == d_value), else one after another. Both forms' needs are covered: a row's
// strides may be beyond what the tensor cores' copies take.
size_t mixer_workspace(const gr_mixer* m, bool gradient) {
    const int64_t N = m->n_tokens;
    const int B = m->n_seqs, H = m->n_heads, dk = m->d_key, dv = m->d_value;
    size_t need = mix_simt_workspace(N, B, H, dk, dv);
    auto cover = [&](size_t n) { need = need > n ? need : n; };
    if (gradient) cover(mix_simt_workspace(N, B, H, dv, dk));
    if (tc_shape(m)) {
        cover(mix_tc_workspace(N, B, H, dk, dv, 1));
        if (gradient && dk == dv) cover(mix_tc_workspace(N, B, H, dk, dv, 3));
    }
    return need;
}

// Passes over the same rows: three in one launch on the tensor cores, else one after another.
int run_mix(const MixArgs* p, int passes, void* ws, cudaStream_t st) {
    bool tc = true;
    for (int i = 0; i < passes; ++i) tc = tc && mix_tc_supported(p[i]);
    if (tc && passes == 3) return as_status(launch_mix_tc(p, passes, ws, st));
    for (int i = 0; i < passes; ++i) {
        const cudaError_t e =
            mix_tc_supported(p[i]) ? launch_mix_tc(p + i, 1, ws, st) : launch_mix_simt(p[i], ws, st);
        if (e != cudaSuccess) return GR_E_CUDA;
    }
    return GR_OK;
}

size_t state_bytes(const gr_mixer* m, int64_t n) {
    return size_t(n) * m->n_heads * m->d_key * m->d_value * 4;
}

// seq_starts and the workspace, as every packed call takes them.
int check_packed(const gr_mixer* m, bool gradient, const int32_t* starts, void* ws,
                 size_t ws_bytes) {
    if (!starts && m->n_seqs != 1) return GR_E_NULL;
    if (!aligned(starts, 4)) return GR_E_ALIGN;
    const size_t need = mixer_workspace(m, gradient);
    if (need && (!ws || ws_bytes < need)) return GR_E_SIZE;
    if (need && !aligned(ws, 256)) return GR_E_ALIGN;
    return GR_OK;
}

MixArgs mix_args(const gr_mixer* m, const Rows& a, const Rows& b, const Rows& c, const Rows& out,
                 const float* log_decay, const int32_t* starts) {
    MixArgs p{};
    p.n_tokens = m->n_tokens;
    p.n_seqs = m->n_seqs;
    p.n_heads = m->n_heads;
    p.da = int(a.d);
    p.dc = int(c.d);
    p.dtype = m->dtype;
    p.a = a.mix(), p.b = b.mix(), p.c = c.mix(), p.out = out.mix();
    p.log_decay = log_decay;
    p.starts = starts;
    p.mr = p.dc, p.mc = 1;
    return p;
}

}  // namespace
}  // namespace gr

using namespace gr;

extern "C" {

int gr_embed(const gr_embedding* e, const void* table, const void* ids, void* R, void* stream) {
    int st = check_embedding(e);
    if (st) return st;
    if (e->n_tokens == 0) return GR_OK;
    if (!table || !ids || !R) return GR_E_NULL;
    if (!aligned(table, 16) || !aligned(R, 16) || !aligned(ids, e->id_bits / 8)) return GR_E_ALIGN;
    const size_t N = size_t(e->n_tokens), D = size_t(e->d_model);
    const Span out{R, N * e->n_branch * D * width(e->state_dtype)};
    if (meet(out, {table, size_t(e->n_vocab) * D * width(e->table_dtype)}) ||
        meet(out, {ids, N * size_t(e->id_bits / 8)}))
        return GR_E_ALIAS;
    if ((st = usable_device())) return st;
    return as_status(launch_embed(e->n_tokens, e->n_vocab, e->d_model, e->n_branch, e->table_dtype,
                                  e->state_dtype, e->id_bits, e->scale, ids, table, R,
                                  static_cast<cudaStream_t>(stream)));
}

int gr_embed_backward_workspace_size(const gr_embedding* e, size_t* bytes) {
    const int st = check_embedding(e);
    if (st) return st;
    if (!bytes) return GR_E_NULL;
    *bytes = embed_backward_workspace(e->n_tokens, e->d_model);
    return GR_OK;
}

int gr_embed_backward(const gr_embedding* e, const float* dR, const void* ids, float* dtable,
                      int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_embedding(e);
    if (st) return st;
    if (!dtable) return GR_E_NULL;
    if (e->n_tokens == 0 && accumulate) return GR_OK;
    const size_t N = size_t(e->n_tokens), D = size_t(e->d_model);
    const size_t need = embed_backward_workspace(e->n_tokens, e->d_model);
    if (N > 0 && (!dR || !ids || !workspace)) return GR_E_NULL;
    if (!aligned(dR, 16) || !aligned(dtable, 16) || !aligned(ids, e->id_bits / 8) ||
        !aligned(workspace, 256))
        return GR_E_ALIGN;
    if (workspace_bytes < need) return GR_E_SIZE;
    const Span out{dtable, size_t(e->n_vocab) * D * 4}, ws{workspace, need};
    const Span in[2] = {{dR, N * e->n_branch * D * 4}, {ids, N * size_t(e->id_bits / 8)}};
    if (meet(out, ws) || meet(out, in[0]) || meet(out, in[1]) || meet(ws, in[0]) || meet(ws, in[1]))
        return GR_E_ALIAS;
    if ((st = usable_device())) return st;
    return as_status(launch_embed_backward(e->n_tokens, e->n_vocab, e->d_model, e->n_branch,
                                           e->id_bits, e->scale, dR, ids, dtable, accumulate != 0,
                                           workspace, static_cast<cudaStream_t>(stream)));
}

int gr_layer_norm(const gr_norm* n, const void* x, const float* weight, const float* bias, void* y,
                  float* mean, float* rstd, void* stream) {
    int st = check_norm(n);
    if (st) return st;
    if (n->n_tokens == 0) return GR_OK;
    if (!x || !weight || !y) return GR_E_NULL;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(y, 16) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return GR_E_ALIGN;
    const size_t rows = size_t(n->n_tokens) * n->n_group, D = size_t(n->d_model);
    const Span in[3] = {{x, rows * D * width(n->dtype)}, {weight, n->n_group * D * 4},
                        {bias, n->n_group * D * 4}};
    const Span out[3] = {{y, in[0].n}, {mean, rows * 4}, {rstd, rows * 4}};
    for (int a = 0; a < 3; ++a) {
        for (int b = 0; b < 3; ++b)
            if (meet(out[a], in[b]) && !(a == 0 && b == 0 && x == y)) return GR_E_ALIAS;
        for (int b = a + 1; b < 3; ++b)
            if (meet(out[a], out[b])) return GR_E_ALIAS;
    }
    if ((st = usable_device())) return st;
    return as_status(launch_layer_norm(n->n_tokens, n->d_model, n->n_group, n->dtype, n->eps, x,
                                       weight, bias, y, mean, rstd,
                                       static_cast<cudaStream_t>(stream)));
}

int gr_layer_norm_backward_workspace_size(const gr_norm* n, size_t* bytes) {
    const int st = check_norm(n);
    if (st) return st;
    if (!bytes) return GR_E_NULL;
    *bytes = layer_norm_backward_workspace(n->n_tokens, n->d_model, n->n_group);
    return GR_OK;
}

int gr_layer_norm_backward(const gr_norm* n, const float* dy, const void* x, const float* weight,
                           const float* mean, const float* rstd, float* dx, float* dweight,
                           float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_norm(n);
    if (st) return st;
    if (!dweight) return GR_E_NULL;
    const size_t rows = size_t(n->n_tokens) * n->n_group, D = size_t(n->d_model);
    if (rows > 0 && (!dy || !x || !weight || !mean || !rstd || !dx || !workspace)) return GR_E_NULL;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(weight, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dx, 16) || !aligned(dweight, 16) || !aligned(dbias, 16) ||
        !aligned(workspace, 256))
        return GR_E_ALIGN;
    const size_t need = layer_norm_backward_workspace(n->n_tokens, n->d_model, n->n_group);
    if (workspace_bytes < need) return GR_E_SIZE;
    const size_t per = n->n_group * D * 4;
    const Span in[5] = {{dy, rows * D * 4}, {x, rows * D * width(n->dtype)}, {weight, per},
                        {mean, rows * 4}, {rstd, rows * 4}};
    const Span out[4] = {{dx, rows * D * 4}, {dweight, per}, {dbias, per}, {workspace, need}};
    for (int a = 0; a < 4; ++a) {
        for (int b = 0; b < 5; ++b)
            if (meet(out[a], in[b]) && !(a == 0 && b == 0 && dx == dy)) return GR_E_ALIAS;
        for (int b = a + 1; b < 4; ++b)
            if (meet(out[a], out[b])) return GR_E_ALIAS;
    }
    if ((st = usable_device())) return st;
    return as_status(launch_layer_norm_backward(n->n_tokens, n->d_model, n->n_group, n->dtype, dy, x,
                                                weight, mean, rstd, dx, dweight, dbias, workspace,
                                                static_cast<cudaStream_t>(stream)));
}

const char* gr_mixer_path(const gr_mixer* m) {
    if (check_mixer(m) != GR_OK) return "invalid";
    return tc_shape(m) ? "mixer_tc" : "mixer_simt";
}

int gr_linear_attention_workspace_size(const gr_mixer* m, int gradient, size_t* bytes) {
    const int st = check_mixer(m);
    if (st) return st;
    if (!bytes) return GR_E_NULL;
    *bytes = mixer_workspace(m, gradient != 0);
    return GR_OK;
}

int gr_linear_attention(const gr_mixer* m, const gr_rows* q, const gr_rows* k, const gr_rows* v,
                        const float* log_decay, const int32_t* seq_starts, const float* state_in,
                        const gr_rows* o, float* state_out, void* workspace, size_t workspace_bytes,
                        void* stream) {
    int st = check_mixer(m);
    if (st) return st;
    if (m->n_seqs == 0 || (m->n_tokens == 0 && !state_out)) return GR_OK;
    if (!q || !k || !v || !o || !log_decay) return GR_E_NULL;
    const int64_t N = m->n_tokens, H = m->n_heads;
    const size_t w = width(m->dtype);
    const Rows in[3] = {{q, N, H, m->d_key, w}, {k, N, H, m->d_key, w}, {v, N, H, m->d_value, w}};
    const Rows out{o, N, H, m->d_value, w};
    for (const Rows& r : in)
        if ((st = r.check(false))) return st;
    if ((st = out.check(true))) return st;
    if ((st = check_packed(m, false, seq_starts, workspace, workspace_bytes))) return st;
    if (!aligned(log_decay, 4) || !aligned(state_in, 16) || !aligned(state_out, 16)) return GR_E_ALIGN;
    const size_t ns = state_bytes(m, m->n_seqs);
    const Span so{state_out, ns}, si{state_in, ns}, ws{workspace, mixer_workspace(m, false)};
    const Span flat[2] = {{log_decay, size_t(H) * 4},
                          {seq_starts, (size_t(m->n_seqs) + 1) * sizeof(int32_t)}};
    for (const Rows& r : in)
        if (out.meets(r) || meet(so, r.span()) || meet(ws, r.span())) return GR_E_ALIAS;
    for (const Span& f : flat)
        if (meet(out.span(), f) || meet(so, f) || meet(ws, f)) return GR_E_ALIAS;
    if (meet(out.span(), si) || meet(out.span(), so) || meet(out.span(), ws) || meet(ws, si) ||
        meet(ws, so) || (state_in != state_out && meet(si, so)))
        return GR_E_ALIAS;
    if ((st = usable_device())) return st;
    MixArgs p = mix_args(m, in[0], in[1], in[2], out, log_decay, seq_starts);
    p.m_in = state_in;
    p.m_out = state_out;
    p.weight = 1.0f;
    p.outer = m->scale;
    return run_mix(&p, 1, workspace, static_cast<cudaStream_t>(stream));
}

int gr_linear_attention_step(const gr_mixer* m, const gr_rows* q, const gr_rows* k,
                             const gr_rows* v, const float* log_decay, float* state,
                             int64_t n_slots, const int32_t* slots, const gr_rows* o, void* stream) {
    int st = check_mixer(m);
    if (st) return st;
    const int64_t N = m->n_tokens, H = m->n_heads;
    if (n_slots < 0 || n_slots > (int64_t(1) << 31) || N * H > 0x7fffffffLL) return GR_E_SHAPE;
    if (N == 0) return GR_OK;
    if (!q || !k || !v || !o || !log_decay || (!state && n_slots > 0)) return GR_E_NULL;
    const size_t w = width(m->dtype);
    const Rows in[3] = {{q, N, H, m->d_key, w}, {k, N, H, m->d_key, w}, {v, N, H, m->d_value, w}};
    const Rows out{o, N, H, m->d_value, w};
    for (const Rows& r : in)
        if ((st = r.check(false))) return st;
    if ((st = out.check(true))) return st;
    if (!aligned(log_decay, 4) || !aligned(state, 16) || !aligned(slots, 4)) return GR_E_ALIGN;
    const Span ss{state, state_bytes(m, n_slots)};
    const Span flat[2] = {{log_decay, size_t(H) * 4}, {slots, size_t(N) * 4}};
    for (const Rows& r : in)
        if (out.meets(r) || meet(ss, r.span())) return GR_E_ALIAS;
    for (const Span& f : flat)
        if (meet(out.span(), f) || meet(ss, f)) return GR_E_ALIAS;
    if (meet(out.span(), ss)) return GR_E_ALIAS;
    if ((st = usable_device())) return st;
    return as_status(launch_mix_step(N, int(H), m->d_key, m->d_value, m->dtype, m->scale, in[0].mix(),
                                     in[1].mix(), in[2].mix(), log_decay, state, n_slots, slots,
                                     out.mix(), static_cast<cudaStream_t>(stream)));
}

int gr_linear_attention_backward(const gr_mixer* m, const gr_rows* dO, const gr_rows* q,
                                 const gr_rows* k, const gr_rows* v, const float* log_decay,
                                 const int32_t* seq_starts, const float* state_in,
                                 const float* dstate_out, const gr_rows* dq, const gr_rows* dk,
                                 const gr_rows* dv, float* dstate_in, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    int st = check_mixer(m);
    if (st) return st;
    if (m->n_seqs == 0 || (m->n_tokens == 0 && !dstate_in)) return GR_OK;
    if (!dO || !q || !k || !v || !dq || !dk || !dv || !log_decay) return GR_E_NULL;
    const int64_t N = m->n_tokens, H = m->n_heads;
    const size_t w = width(m->dtype);
    const Rows in[4] = {{dO, N, H, m->d_value, w}, {q, N, H, m->d_key, w}, {k, N, H, m->d_key, w},
                        {v, N, H, m->d_value, w}};
    const Rows out[3] = {{dq, N, H, m->d_key, w}, {dk, N, H, m->d_key, w}, {dv, N, H, m->d_value, w}};
    for (const Rows& r : in)
        if ((st = r.check(false))) return st;
    for (const Rows& r : out)
        if ((st = r.check(true))) return st;
    if ((st = check_packed(m, true, seq_starts, workspace, workspace_bytes))) return st;
    if (!aligned(log_decay, 4) || !aligned(state_in, 16) || !aligned(dstate_out, 16) ||
        !aligned(dstate_in, 16))
        return GR_E_ALIGN;
    const size_t ns = state_bytes(m, m->n_seqs);
    const Span so{dstate_in, ns}, ws{workspace, mixer_workspace(m, true)};
    const Span flat[4] = {{log_decay, size_t(H) * 4},
                          {seq_starts, (size_t(m->n_seqs) + 1) * sizeof(int32_t)},
                          {state_in, ns},
                          {dstate_out, ns}};
    for (int a = 0; a < 3; ++a) {
        for (const Rows& r : in)
            if (out[a].meets(r)) return GR_E_ALIAS;
        for (int b = a + 1; b < 3; ++b)
            if (out[a].meets(out[b])) return GR_E_ALIAS;
        for (const Span& f : flat)
            if (meet(out[a].span(), f)) return GR_E_ALIAS;
        if (meet(out[a].span(), so) || meet(out[a].span(), ws)) return GR_E_ALIAS;
    }
    for (const Rows& r : in)
        if (meet(so, r.span()) || meet(ws, r.span())) return GR_E_ALIAS;
    for (const Span& f : flat) {
        // dstate_in may be dstate_out itself (and that none of the others)
        const bool onto = &f == &flat[3] && dstate_out == dstate_in;
        if (meet(ws, f) || (!onto && meet(so, f))) return GR_E_ALIAS;
    }
    if (meet(so, ws)) return GR_E_ALIAS;
    if ((st = usable_device())) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    MixArgs p[3];
    // dq_t = scale S_t dO_t: forwards over (dO, v, k) with the state transposed
    p[0] = mix_args(m, in[0], in[3], in[2], out[0], log_decay, seq_starts);
    p[0].m_in = state_in;
    p[0].mr = 1, p[0].mc = m->d_value;
    p[0].weight = 1.0f;
    p[0].outer = m->scale;
    // dk_t = G_t v_t: backwards over (v, dO, q), G transposed
    p[1] = mix_args(m, in[3], in[0], in[1], out[1], log_decay, seq_starts);
    p[1].m_in = dstate_out;
    p[1].mr = 1, p[1].mc = m->d_value;
    p[1].reverse = true;
    p[1].weight = m->scale;
    p[1].outer = 1.0f;
    // dv_t = G_tᵀ k_t: backwards over (k, q, dO); its G goes on to the incoming state
    p[2] = mix_args(m, in[2], in[1], in[0], out[2], log_decay, seq_starts);
    p[2].m_in = dstate_out;
    p[2].m_out = dstate_in;
    p[2].reverse = true;
    p[2].weight = m->scale;
    p[2].outer = 1.0f;
    // dv apart where its shape is another one, or where it writes what dk still reads
    const int together = m->d_key != m->d_value || (dstate_in && dstate_in == dstate_out) ? 2 : 3;
    if ((st = run_mix(p, together, workspace, s))) return st;
    return together == 3 ? GR_OK : run_mix(p + 2, 1, workspace, s);
}

}  // extern "C"
