// C entries of the gated feed-forward sublayer and of FP8 blocks: host-side validation, the steps of a call,
// status codes. Contracts in include/gr.h.
#include <initializer_list>

#include "gr_check.h"
#include "gr_feed.h"

namespace gr {
namespace {

int check_feed(const gr_feed* f, bool fp8) {
    if (!f) return GR_E_NULL;
    if (fp8 ? f->dtype != GR_FP8 : !real_dtype(f->dtype)) return GR_E_DTYPE;
    const int step = fp8 ? 16 : 8;
    if (f->n_tokens < 0 || f->n_tokens > 0x7fffffffLL || f->d_model < step || f->d_model % step != 0 ||
        f->d_model > GR_MAX_D || f->d_ff < step || f->d_ff % step != 0 || f->d_ff > GR_MAX_FF ||
        (f->activation != GR_SILU && f->activation != GR_GELU))
        return GR_E_SHAPE;
    return GR_OK;
}

int check_blocks(const gr_blocks* b) {
    if (!b) return GR_E_NULL;
    if (!real_dtype(b->dtype)) return GR_E_DTYPE;
    if (b->n_rows < 0 || b->n_matrix < 1 || b->n_rows > (int64_t(1) << 40) / b->n_matrix || b->n_cols < 16 ||
        b->n_cols % 16 != 0 || b->n_cols > GR_MAX_FF || (b->block_rows != 1 && b->block_rows != kBlock) ||
        b->n_rows * b->n_matrix > 0x7fffffffLL / ceil_div(b->n_cols, kBlock))
        return GR_E_SHAPE;
    return GR_OK;
}

int check_product(const gr_product* p) {
    if (!p) return GR_E_NULL;
    if (p->n_tokens < 0 || p->n_tokens > 0x7fffffffLL || p->d_in < 16 || p->d_in % 16 != 0 ||
        p->d_in > GR_MAX_FF || p->d_out < 8 || p->d_out % 8 != 0 || p->d_out > 2 * GR_MAX_FF)
        return GR_E_SHAPE;
    return GR_OK;
}

int check_buffers(std::initializer_list<Span> aligned_in, std::initializer_list<Span> bytes_in,
                  std::initializer_list<Span> out, const Span& ws, size_t ws_bytes) {
    for (const auto& s : aligned_in)
        if (!s.p && s.n) return GR_E_NULL;
    for (const auto& s : bytes_in)
        if (!s.p && s.n) return GR_E_NULL;
    for (const auto& s : out)
        if (!s.p && s.n) return GR_E_NULL;
    for (const auto& s : aligned_in)
        if (!aligned(s.p, 16)) return GR_E_ALIGN;
    for (const auto& s : out)
        if (!aligned(s.p, 16)) return GR_E_ALIGN;
    if (ws.n && (!ws.p || ws_bytes < ws.n)) return GR_E_SIZE;
    if (ws.n && !aligned(ws.p, 256)) return GR_E_ALIGN;
    for (const auto* o = out.begin(); o != out.end(); ++o) {
        for (const auto& s : aligned_in)
            if (meet(*o, s)) return GR_E_ALIAS;
        for (const auto& s : bytes_in)
            if (meet(*o, s)) return GR_E_ALIAS;
        for (const auto* q = out.begin(); q != o; ++q)
            if (meet(*o, *q)) return GR_E_ALIAS;
        if (meet(*o, ws)) return GR_E_ALIAS;
    }
    for (const auto& s : aligned_in)
        if (meet(ws, s)) return GR_E_ALIAS;
    for (const auto& s : bytes_in)
        if (meet(ws, s)) return GR_E_ALIAS;
    return GR_OK;
}

// The workspace in parts, each from a 256-byte boundary on.
struct Parts {
    char* base;
    size_t used = 0;
    bool ok = true;
    template <typename T = void> T* take(size_t bytes) {
        if (bytes == SIZE_MAX) {   // a call that cannot be planned
            ok = false;
            return nullptr;
        }
        char* p = base ? base + used : nullptr;
        used += align256(bytes);
        return reinterpret_cast<T*>(p);
    }
};

struct FeedParts {
    void *h = nullptr, *dpre = nullptr;              // gr_feed_forward and its gradient
    float* parts = nullptr;                          // bf16 and FP8: sums over ranges of k
    void* terms = nullptr;                           // fp32: operands as bf16 terms, and such sums
    uint8_t *xc = nullptr, *xs = nullptr;            // FP8: x in blocks
    uint8_t *hc = nullptr, *hs = nullptr;            // and h
    uint8_t *w_in = nullptr, *w_out = nullptr;       // and the weights' scales
    size_t bytes = 0;
    bool ok;
    FeedParts(const gr_feed* f, bool gradient, void* base) {
        Parts w{static_cast<char*>(base)};
        const size_t N = size_t(f->n_tokens), D = size_t(f->d_model), F = size_t(f->d_ff);
        if (f->dtype == GR_FP8) {
            xc = w.take<uint8_t>(N * D);
            xs = w.take<uint8_t>(token_scale_bytes(N, D));
            hc = w.take<uint8_t>(N * F);
            hs = w.take<uint8_t>(token_scale_bytes(N, F));
            w_in = w.take<uint8_t>(2 * ceil_div(F, kBlock) * scale_pitch(D));
            w_out = w.take<uint8_t>(ceil_div(D, kBlock) * scale_pitch(F));
            if (N > 0) parts = w.take<float>(tc_feed_fp8_workspace(f->n_tokens, f->d_model, f->d_ff));
        } else if (f->dtype == GR_F32) {
            if (N > 0) terms = w.take(f32_feed_workspace(f->n_tokens, f->d_model, f->d_ff, gradient));
        } else {
            h = w.take(N * F * 2);
            if (gradient) dpre = w.take(2 * N * F * 2);
            if (N > 0)
                parts = w.take<float>(tc_feed_workspace(f->n_tokens, f->d_model, f->d_ff, gradient));
        }
        bytes = w.used;
        ok = w.ok;
    }
};

// gr_fp8_matmul: both operands' scales as the product takes them, and its parts.
struct ProductParts {
    uint8_t *a, *b;
    float* parts;
    size_t bytes;
    bool ok;
    ProductParts(const gr_product* p, void* base) {
        Parts w{static_cast<char*>(base)};
        a = w.take<uint8_t>(token_scale_bytes(p->n_tokens, p->d_in));
        b = w.take<uint8_t>(ceil_div(p->d_out, kBlock) * scale_pitch(p->d_in));
        parts = w.take<float>(tc_product_fp8_workspace(p->n_tokens, p->d_out, p->d_in));
        bytes = w.used;
        ok = w.ok;
    }
};

}  // namespace
}  // namespace gr

using namespace gr;

extern "C" {

int gr_feed_workspace_size(const gr_feed* f, int gradient, size_t* bytes) {
    const int st = check_feed(f, f && f->dtype == GR_FP8 && !gradient);
    if (st) return st;
    if (!bytes) return GR_E_NULL;
    const FeedParts p(f, gradient != 0, nullptr);
    if (!p.ok) return GR_E_SHAPE;
    *bytes = p.bytes;
    return GR_OK;
}

int gr_feed_forward(const gr_feed* f, const void* x, const void* w_in, const void* w_out, void* y, void* pre,
                    void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_feed(f, false);
    if (st) return st;
    if (f->n_tokens == 0) return GR_OK;
    const int64_t N = f->n_tokens;
    const int D = f->d_model, F = f->d_ff;
    const size_t w = width(f->dtype), nd = size_t(N) * D * w, fd = size_t(F) * D * w;
    const FeedParts p(f, false, workspace);
    if (!p.ok) return GR_E_SHAPE;
    if ((st = check_buffers({{x, nd}, {w_in, 2 * fd}, {w_out, fd}}, {},
                            {{y, nd}, {pre, pre ? 2 * size_t(N) * F * w : 0}}, {workspace, p.bytes},
                            workspace_bytes)))
        return st;
    if ((st = usable_device())) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (f->dtype == GR_F32)
        return as_status(f32_feed_forward(N, D, F, f->activation, static_cast<const float*>(x),
                                          static_cast<const float*>(w_in), static_cast<const float*>(w_out),
                                          static_cast<float*>(y), static_cast<float*>(pre), p.terms, s));
    cudaError_t e = tc_gated(N, D, F, f->activation, x, w_in, p.h, pre, p.parts, s);
    if (e == cudaSuccess) e = tc_product(N, D, F, N, p.h, true, w_out, true, y, p.parts, s);
    return as_status(e);
}

int gr_feed_forward_backward(const gr_feed* f, const void* dy, const void* x, const void* w_in,
                             const void* w_out, const void* pre, void* dx, void* dw_in, void* dw_out,
                             void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_feed(f, false);
    if (st) return st;
    const int64_t N = f->n_tokens;
    const int D = f->d_model, F = f->d_ff;
    const size_t w = width(f->dtype), nd = size_t(N) * D * w, fd = size_t(F) * D * w;
    const FeedParts p(f, true, workspace);
    if (!p.ok) return GR_E_SHAPE;
    const size_t weights = N > 0 ? fd : 0;   // without tokens only the weights' gradients are touched
    if ((st = check_buffers({{dy, nd}, {x, nd}, {w_in, 2 * weights}, {w_out, weights},
                             {pre, 2 * size_t(N) * F * w}}, {},
                            {{dx, nd}, {dw_in, 2 * fd}, {dw_out, fd}}, {workspace, p.bytes}, workspace_bytes)))
        return st;
    if ((st = usable_device())) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) {
        cudaError_t e = cudaMemsetAsync(dw_in, 0, 2 * fd, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dw_out, 0, fd, s);
        return as_status(e);
    }
    if (f->dtype == GR_F32)
        return as_status(f32_feed_backward(N, D, F, f->activation, static_cast<const float*>(dy),
                                           static_cast<const float*>(x), static_cast<const float*>(w_in),
                                           static_cast<const float*>(w_out), static_cast<const float*>(pre),
                                           static_cast<float*>(dx), static_cast<float*>(dw_in),
                                           static_cast<float*>(dw_out), p.terms, s));
    cudaError_t e = tc_gated_grad(N, D, F, f->activation, dy, w_out, pre, p.dpre, p.h, p.parts, s);
    if (e == cudaSuccess) e = tc_product(N, D, 2 * F, N, p.dpre, true, w_in, false, dx, p.parts, s);
    if (e == cudaSuccess) e = tc_product(2 * F, D, N, INT64_MAX, p.dpre, false, x, false, dw_in, p.parts, s);
    if (e == cudaSuccess) e = tc_product(D, F, N, INT64_MAX, dy, false, p.h, false, dw_out, p.parts, s);
    return as_status(e);
}

int gr_fp8_encode_blocks(const gr_blocks* b, const void* m, uint8_t* codes, uint8_t* scales, void* stream) {
    int st = check_blocks(b);
    if (st) return st;
    if (b->n_rows == 0) return GR_OK;
    if (!m || !codes || !scales) return GR_E_NULL;
    if (!aligned(m, 16) || !aligned(codes, 16)) return GR_E_ALIGN;
    const size_t n = size_t(b->n_matrix) * b->n_rows * b->n_cols;
    const Span in{m, n * width(b->dtype)}, c{codes, n},
        s{scales, size_t(b->n_matrix) * ceil_div(b->n_rows, b->block_rows) * ceil_div(b->n_cols, kBlock)};
    if (meet(in, c) || meet(in, s) || meet(c, s)) return GR_E_ALIAS;
    if ((st = usable_device())) return st;
    return as_status(launch_encode_blocks(b->n_matrix, b->n_rows, b->n_cols, b->block_rows, b->dtype, m, codes,
                                          scales, static_cast<cudaStream_t>(stream)));
}

int gr_fp8_matmul_workspace_size(const gr_product* p, size_t* bytes) {
    const int st = check_product(p);
    if (st) return st;
    if (!bytes) return GR_E_NULL;
    *bytes = 0;
    if (p->n_tokens == 0) return GR_OK;
    const ProductParts w(p, nullptr);
    if (!w.ok) return GR_E_SHAPE;
    *bytes = w.bytes;
    return GR_OK;
}

int gr_fp8_matmul(const gr_product* p, const uint8_t* a, const uint8_t* a_scales, const uint8_t* b,
                  const uint8_t* b_scales, void* out, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_product(p);
    if (st) return st;
    if (p->n_tokens == 0) return GR_OK;
    const size_t N = size_t(p->n_tokens), K = size_t(p->d_in), O = size_t(p->d_out), nb = ceil_div(K, kBlock);
    const ProductParts w(p, workspace);
    if (!w.ok) return GR_E_SHAPE;
    if ((st = check_buffers({{a, N * K}, {b, O * K}}, {{a_scales, N * nb}, {b_scales, ceil_div(O, kBlock) * nb}},
                            {{out, N * O * 2}}, {workspace, w.bytes}, workspace_bytes)))
        return st;
    if ((st = usable_device())) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tc_takes_rows(N, K, a_scales, b_scales))
        return as_status(tc_product_fp8(N, O, K, {a, a_scales, b, b_scales, true}, out, w.parts, s));
    cudaError_t e = launch_fp8_operands(nullptr, 0, 0, nullptr, nullptr, {a_scales, w.a, int64_t(N), int(nb), true},
                                        {b_scales, w.b, int64_t(ceil_div(O, kBlock)), int(nb), false}, s);
    if (e == cudaSuccess) e = tc_product_fp8(N, O, K, {a, w.a, b, w.b}, out, w.parts, s);
    return as_status(e);
}

int gr_feed_forward_fp8(const gr_feed* f, const void* x, const uint8_t* w_in, const uint8_t* w_in_scales,
                        const uint8_t* w_out, const uint8_t* w_out_scales, void* y, void* workspace,
                        size_t workspace_bytes, void* stream) {
    int st = check_feed(f, true);
    if (st) return st;
    if (f->n_tokens == 0) return GR_OK;
    const int64_t N = f->n_tokens;
    const int D = f->d_model, F = f->d_ff;
    const size_t nd = size_t(N) * D * 2, fd = size_t(F) * D, db = ceil_div(D, kBlock), fb = ceil_div(F, kBlock);
    const FeedParts p(f, false, workspace);
    if (!p.ok) return GR_E_SHAPE;
    if ((st = check_buffers({{x, nd}, {w_in, 2 * fd}, {w_out, fd}},
                            {{w_in_scales, 2 * fb * db}, {w_out_scales, fb * db}}, {{y, nd}},
                            {workspace, p.bytes}, workspace_bytes)))
        return st;
    if ((st = usable_device())) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_fp8_operands(x, N, D, p.xc, p.xs,
                                        {w_in_scales, p.w_in, int64_t(2 * fb), int(db), false},
                                        {w_out_scales, p.w_out, int64_t(db), int(fb), false}, s);
    if (e == cudaSuccess)
        e = tc_gated_fp8(N, D, F, f->activation, {p.xc, p.xs, w_in, p.w_in}, p.hc, p.hs, p.parts, s);
    if (e == cudaSuccess) e = tc_product_fp8(N, D, F, {p.hc, p.hs, w_out, p.w_out}, y, p.parts, s);
    return as_status(e);
}

}  // extern "C"
