// C ABI of the layer operators: argument validation, workspace layout and the kernel sequence of
// each entry point.  See include/lora_layer.h for the contract.
#include <cmath>
#include <initializer_list>

#include "lm_layer.h"
#include "lm_ptx.cuh"

using namespace lm;

namespace {

#define LL_TRY(expr)                    \
    do {                                \
        const lm_status _s = (expr);    \
        if (_s != LM_OK) return _s;     \
    } while (0)

lm_status launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? LM_OK : report_error(LM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

lm_status need(const void* p, size_t align, const char* name) {
    if (!p) return report_error(LM_ERR_NULL, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align != 0)
        return report_error(LM_ERR_ALIGN, "%s is not %zu-byte aligned", name, align);
    return LM_OK;
}

lm_status want(const void* p, size_t align, const char* name) { return p ? need(p, align, name) : LM_OK; }

lm_status must_be_null(const void* p, const char* name, const char* why) {
    return p ? report_error(LM_ERR_SHAPE, "%s is given %s", name, why) : LM_OK;
}

lm_status check_tokens(int64_t T, int64_t most) {
    if (T < 0 || T > most) return report_error(LM_ERR_SHAPE, "T = %lld is not in [0, %lld]", (long long)T, (long long)most);
    return LM_OK;
}

struct Span {
    const void* p;
    size_t bytes;
    const char* name;
};

bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

lm_status check_alias(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& in : ins)
            if (overlap(*o, in)) return report_error(LM_ERR_ALIAS, "%s overlaps %s", o->name, in.name);
        for (const Span* q = o + 1; q != outs.end(); ++q)
            if (overlap(*o, *q)) return report_error(LM_ERR_ALIAS, "%s overlaps %s", o->name, q->name);
    }
    return LM_OK;
}

// ------------------------------------------------------------------ attention
// test hook (attn_debug_inject)
thread_local int32_t g_starve = 0;
thread_local uint64_t g_wait_ns = 0;

constexpr int64_t kMaxTokens = int64_t(1) << 20;

lm_status check_attn_shape(int64_t T, int32_t hq, int32_t hk, int32_t d) {
    LL_TRY(check_tokens(T, kMaxTokens));
    if (hq < 1 || hk < 1 || hq > 1024 || hq % hk != 0)
        return report_error(LM_ERR_SHAPE, "hq = %d, hk = %d: the key/value heads must divide the query heads (at most 1024)", hq, hk);
    if (d < 8 || d > 128 || d % 8 != 0) return report_error(LM_ERR_SHAPE, "d = %d must be a multiple of 8 in [8, 128]", d);
    return LM_OK;
}

lm_status check_attn(const lm_attn* a) {
    if (!a) return report_error(LM_ERR_NULL, "a is NULL");
    if (!std::isfinite(a->scale)) return report_error(LM_ERR_SHAPE, "scale is not finite");
    // (a capped score's absolute error is up to 2^-21 cap, and scale / cap has to be a number)
    if (!(a->cap == 0.f || (a->cap >= 0x1p-14f && a->cap <= 0x1p12f)) || !std::isfinite(3.f * a->scale / (a->cap == 0.f ? 1.f : a->cap)))
        return report_error(LM_ERR_SHAPE, "cap = %g must be 0 or in [2^-14, 2^12], and 3 scale / cap finite", a->cap);
    if (a->window < 0) return report_error(LM_ERR_SHAPE, "window = %d must be 0 or positive", a->window);
    LL_TRY(want(a->slopes, 4, "slopes"));
    if (a->cu_docs) {
        LL_TRY(need(a->cu_docs, 4, "cu_docs"));
        if (a->n_docs < 1) return report_error(LM_ERR_SHAPE, "n_docs = %d must be positive", a->n_docs);
        LL_TRY(want(a->prefix, 4, "prefix"));
    } else {
        LL_TRY(must_be_null(a->prefix, "prefix", "without cu_docs"));
    }
    return LM_OK;
}

lm_status check_heads(const lm_heads* t, int64_t T, int heads, int d, const char* name) {
    if (!t) return report_error(LM_ERR_NULL, "%s is NULL", name);
    LL_TRY(need(t->p, 16, name));
    const int64_t most = int64_t(1) << 38;  // bytes of a stride fit the tensor map's 40 bits
    if (t->token_stride % 8 || t->head_stride % 8 || t->token_stride < d || t->head_stride < d || t->token_stride > most ||
        t->head_stride > most)
        return report_error(LM_ERR_SHAPE, "%s: strides %lld (tokens), %lld (heads) must be multiples of 8, at least d", name,
                            (long long)t->token_stride, (long long)t->head_stride);
    return LM_OK;
}

Span heads_span(const lm_heads* t, int64_t T, int heads, int d, const char* name) {
    return Span{t->p, T ? (size_t)((T - 1) * t->token_stride + (heads - 1) * t->head_stride + d) * 2 : 0, name};
}

int64_t whole_tiles(int64_t T) { return (T + 127) / 128 * 128; }

struct AttnPlan {
    size_t rng, delta, nlse, total;
};

AttnPlan plan_attn(int64_t T, int32_t hq) {
    AttnPlan P;
    P.rng = 256;  // after the error word
    P.delta = (P.rng + (size_t)T * sizeof(TokRange) + 255) & ~size_t(255);
    P.nlse = P.delta + (size_t)whole_tiles(T) * hq * 4;  // (a multiple of 512 bytes)
    P.total = P.nlse + (size_t)whole_tiles(T) * hq * 4;
    return P;
}

AttnParams attn_params(int64_t T, int32_t hq, int32_t hk, int32_t d, const lm_heads* q, const lm_heads* k,
                       const lm_heads* v, const lm_attn* a, void* ws) {
    AttnParams p{};
    p.T = (int32_t)T;
    p.Tp = (int32_t)whole_tiles(T);
    p.hq = hq;
    p.hk = hk;
    p.d = d;
    p.d16 = (d + 15) / 16 * 16;
    p.scale = a->scale;
    p.cap = a->cap;
    p.slopes = a->slopes;
    p.rng = a->cu_docs ? reinterpret_cast<const TokRange*>(static_cast<char*>(ws) + plan_attn(T, hq).rng) : nullptr;
    p.causal = a->causal;
    p.window = a->window;
    p.cu_docs = a->cu_docs;
    p.n_docs = a->n_docs;
    p.q = {q->p, q->token_stride, q->head_stride};
    p.k = {k->p, k->token_stride, k->head_stride};
    p.v = {v->p, v->token_stride, v->head_stride};
    p.err = static_cast<int32_t*>(ws);
    p.wait_ns = g_wait_ns ? g_wait_ns : kDefaultWaitNs;
    p.starve = g_starve;
    return p;
}

// the table of who sees whom; one document needs none
lm_status attn_ranges(const lm_attn* a, const AttnParams& p, cudaStream_t st) {
    if (!p.rng) return LM_OK;
    LaunchTag tag("attn.ranges", st);
    return launched(launch_attn_ranges(*a, p.T, const_cast<TokRange*>(p.rng), st), "attn ranges launch");
}

}  // namespace

extern "C" lm_status attn_workspace_size(int64_t T, int32_t hq, int32_t hk, int32_t d, size_t* bytes) {
    LL_TRY(check_attn_shape(T, hq, hk, d));
    if (!bytes) return report_error(LM_ERR_NULL, "bytes is NULL");
    *bytes = plan_attn(T, hq).total;
    return LM_OK;
}

extern "C" lm_status attn_debug_inject(int32_t kernel_mask, uint64_t wait_ns) {
    if (kernel_mask < 0 || kernel_mask > 7) return report_error(LM_ERR_SHAPE, "kernel_mask = %d is not in [0, 7]", kernel_mask);
    g_starve = kernel_mask;
    g_wait_ns = wait_ns;
    return LM_OK;
}

extern "C" lm_status attn_fwd(int64_t T, int32_t hq, int32_t hk, int32_t d, const lm_heads* q, const lm_heads* k,
                              const lm_heads* v, const lm_attn* a, uint16_t* O, int8_t* O_lo, float* lse, void* ws,
                              size_t ws_bytes, lm_stream stream) {
    LL_TRY(check_attn_shape(T, hq, hk, d));
    LL_TRY(check_attn(a));
    LL_TRY(check_heads(q, T, hq, d, "q"));
    LL_TRY(check_heads(k, T, hk, d, "k"));
    LL_TRY(check_heads(v, T, hk, d, "v"));
    LL_TRY(need(O, 32, "O"));
    LL_TRY(want(O_lo, 32, "O_lo"));
    LL_TRY(need(lse, 32, "lse"));
    LL_TRY(need(ws, 32, "ws"));
    const AttnPlan P = plan_attn(T, hq);
    if (ws_bytes < P.total) return report_error(LM_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, P.total);
    LL_TRY(check_alias({{O, (size_t)T * hq * d * 2, "O"}, {O_lo, (size_t)T * hq * ((d + 15) / 16 * 16), "O_lo"},
                        {lse, (size_t)T * hq * 4, "lse"}, {ws, P.total, "ws"}},
                       {heads_span(q, T, hq, d, "q"), heads_span(k, T, hk, d, "k"), heads_span(v, T, hk, d, "v")}));
    if (T == 0) return LM_OK;
    int sms = 0;
    LL_TRY(device_ready(&sms));
    cudaStream_t st = (cudaStream_t)stream;
    AttnParams p = attn_params(T, hq, hk, d, q, k, v, a, ws);
    p.out = O;
    p.out_lo = O_lo;
    p.lse = lse;
    LL_TRY(attn_ranges(a, p, st));
    LaunchTag tag("attn.fwd", st);
    return launch_attn_fwd(p, sms, st);
}

extern "C" lm_status attn_bwd(int64_t T, int32_t hq, int32_t hk, int32_t d, const lm_heads* q, const lm_heads* k,
                              const lm_heads* v, const lm_heads* dO, const uint16_t* O, const int8_t* O_lo,
                              const float* lse, const lm_attn* a, uint16_t* dQ, uint16_t* dK, uint16_t* dV, void* ws,
                              size_t ws_bytes, lm_stream stream) {
    LL_TRY(check_attn_shape(T, hq, hk, d));
    LL_TRY(check_attn(a));
    LL_TRY(check_heads(q, T, hq, d, "q"));
    LL_TRY(check_heads(k, T, hk, d, "k"));
    LL_TRY(check_heads(v, T, hk, d, "v"));
    LL_TRY(check_heads(dO, T, hq, d, "dO"));
    LL_TRY(need(O, 32, "O"));
    LL_TRY(want(O_lo, 32, "O_lo"));
    LL_TRY(need(lse, 32, "lse"));
    LL_TRY(need(dQ, 32, "dQ"));
    LL_TRY(need(dK, 32, "dK"));
    LL_TRY(need(dV, 32, "dV"));
    LL_TRY(need(ws, 32, "ws"));
    const AttnPlan P = plan_attn(T, hq);
    if (ws_bytes < P.total) return report_error(LM_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, P.total);
    const size_t bq = (size_t)T * hq * d * 2, bk = (size_t)T * hk * d * 2;
    LL_TRY(check_alias({{dQ, bq, "dQ"}, {dK, bk, "dK"}, {dV, bk, "dV"}, {ws, P.total, "ws"}},
                       {heads_span(q, T, hq, d, "q"), heads_span(k, T, hk, d, "k"), heads_span(v, T, hk, d, "v"),
                        heads_span(dO, T, hq, d, "dO"), {O, bq, "O"}, {O_lo, (size_t)T * hq * ((d + 15) / 16 * 16), "O_lo"},
                        {lse, (size_t)T * hq * 4, "lse"}}));
    if (T == 0) return LM_OK;
    int sms = 0;
    LL_TRY(device_ready(&sms));
    cudaStream_t st = (cudaStream_t)stream;
    AttnParams p = attn_params(T, hq, hk, d, q, k, v, a, ws);
    p.dO = {dO->p, dO->token_stride, dO->head_stride};
    p.O = O;
    p.O_lo = O_lo;
    p.lse_in = lse;
    p.out = dQ;
    p.dK = dK;
    p.dV = dV;
    float* delta = reinterpret_cast<float*>(static_cast<char*>(ws) + P.delta);
    float* nlse = reinterpret_cast<float*>(static_cast<char*>(ws) + P.nlse);
    p.ndelta = delta;
    p.nlse = nlse;
    {
        LaunchTag tag("attn.delta", st);
        LL_TRY(launched(launch_attn_delta(p, *a, delta, nlse, const_cast<TokRange*>(p.rng), st), "attn delta launch"));
    }
    return launch_attn_bwd(p, sms, st);
}

// ------------------------------------------------------------------ addnorm
namespace {
lm_status check_addnorm(int64_t T, int64_t d, const lm_addnorm* n, const uint16_t* y) {
    LL_TRY(check_tokens(T, int64_t(1) << 30));
    if (d < 32 || d > 16384 || d % 32 != 0)
        return report_error(LM_ERR_SHAPE, "d = %lld must be a multiple of 32 in [32, 16384]", (long long)d);
    if (!n) return report_error(LM_ERR_NULL, "n is NULL");
    if ((n->h_dtype != LM_BF16 && n->h_dtype != LM_F32) || (n->w_dtype != LM_BF16 && n->w_dtype != LM_F32))
        return report_error(LM_ERR_DTYPE, "h_dtype = %d or w_dtype = %d is not known", n->h_dtype, n->w_dtype);
    if (!std::isfinite(n->alpha) || !std::isfinite(n->w_offset)) return report_error(LM_ERR_SHAPE, "alpha or w_offset is not finite");
    if (!(n->eps > 0.f) || !std::isfinite(n->eps)) return report_error(LM_ERR_SHAPE, "eps = %g must be positive", n->eps);
    if (!y && !n->w_in) return report_error(LM_ERR_NULL, "y and w_in are both NULL: nothing to do");
    if (!y) {
        LL_TRY(must_be_null(n->w_post, "w_post", "without y"));
        LL_TRY(must_be_null(n->gate, "gate", "without y"));
    }
    LL_TRY(want(y, 32, "y"));
    LL_TRY(want(n->w_in, 32, "w_in"));
    LL_TRY(want(n->w_post, 32, "w_post"));
    return want(n->gate, 32, "gate");
}

AddNormParams addnorm_params(int64_t T, int64_t d, const void* h, const uint16_t* y, const lm_addnorm* n) {
    AddNormParams p{};
    p.T = T;
    p.d = (int32_t)d;
    p.h = h;
    p.y = y;
    p.w_in = n->w_in;
    p.w_post = n->w_post;
    p.gate = n->gate;
    p.alpha = n->alpha;
    p.eps = n->eps;
    p.w_offset = n->w_offset;
    p.h_f32 = n->h_dtype == LM_F32;
    p.w_f32 = n->w_dtype == LM_F32;
    return p;
}
}  // namespace

extern "C" lm_status addnorm_workspace_size(int64_t T, int64_t d, size_t* bytes) {
    LL_TRY(check_tokens(T, int64_t(1) << 30));
    if (d < 32 || d > 16384 || d % 32 != 0)
        return report_error(LM_ERR_SHAPE, "d = %lld must be a multiple of 32 in [32, 16384]", (long long)d);
    if (!bytes) return report_error(LM_ERR_NULL, "bytes is NULL");
    *bytes = 256 + addnorm_part_bytes(T, d);
    return LM_OK;
}

extern "C" lm_status addnorm_fwd(int64_t T, int64_t d, const void* h, const uint16_t* y, const lm_addnorm* n, void* h_out,
                                 uint16_t* x, float* rstd_y, float* rstd_h, lm_stream stream) {
    LL_TRY(check_addnorm(T, d, n, y));
    LL_TRY(need(h, 32, "h"));
    if (y) LL_TRY(need(h_out, 32, "h_out"));
    if (n->w_in) {
        LL_TRY(need(x, 32, "x"));
        LL_TRY(need(rstd_h, 32, "rstd_h"));
    }
    if (n->w_post) LL_TRY(need(rstd_y, 32, "rstd_y"));
    const size_t hb = (size_t)T * d * (n->h_dtype == LM_F32 ? 4 : 2), xb = (size_t)T * d * 2, rb = (size_t)T * 4;
    const size_t wb = (size_t)d * (n->w_dtype == LM_F32 ? 4 : 2);
    LL_TRY(check_alias({{y ? h_out : nullptr, hb, "h_out"}, {n->w_in ? x : nullptr, xb, "x"},
                        {n->w_post ? rstd_y : nullptr, rb, "rstd_y"}, {n->w_in ? rstd_h : nullptr, rb, "rstd_h"}},
                       {{h, hb, "h"}, {y, xb, "y"}, {n->w_in, wb, "w_in"}, {n->w_post, wb, "w_post"}, {n->gate, wb, "gate"}}));
    if (T == 0) return LM_OK;
    int sms = 0;
    LL_TRY(device_ready(&sms));
    AddNormParams p = addnorm_params(T, d, h, y, n);
    p.h_out = h_out;
    p.x = x;
    p.rstd_y = rstd_y;
    p.rstd_h = rstd_h;
    cudaStream_t st = (cudaStream_t)stream;
    LaunchTag tag("addnorm.fwd", st);
    return launched(launch_addnorm_fwd(p, st), "addnorm forward launch");
}

extern "C" lm_status addnorm_bwd(int64_t T, int64_t d, const void* h, const uint16_t* y, const void* dh_out,
                                 const uint16_t* dx, const float* rstd_y, const float* rstd_h, const lm_addnorm* n,
                                 void* dh, uint16_t* dy, float* dw_in, float* dw_post, float* dgate, void* ws,
                                 size_t ws_bytes, lm_stream stream) {
    LL_TRY(check_addnorm(T, d, n, y));
    LL_TRY(need(h, 32, "h"));
    LL_TRY(want(dh_out, 32, "dh_out"));
    LL_TRY(need(dh, 32, "dh"));
    if (y) LL_TRY(need(dy, 32, "dy"));
    if (n->w_in) {
        LL_TRY(need(dx, 32, "dx"));
        LL_TRY(need(rstd_h, 32, "rstd_h"));
    } else {
        LL_TRY(must_be_null(dx, "dx", "without w_in"));
        LL_TRY(must_be_null(dw_in, "dw_in", "without w_in"));
    }
    if (n->w_post) LL_TRY(need(rstd_y, 32, "rstd_y"));
    else LL_TRY(must_be_null(dw_post, "dw_post", "without w_post"));
    if (!n->gate) LL_TRY(must_be_null(dgate, "dgate", "without gate"));
    LL_TRY(want(dw_in, 32, "dw_in"));
    LL_TRY(want(dw_post, 32, "dw_post"));
    LL_TRY(want(dgate, 32, "dgate"));
    LL_TRY(need(ws, 32, "ws"));
    const size_t total = 256 + addnorm_part_bytes(T, d);
    if (ws_bytes < total) return report_error(LM_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, total);
    const size_t hb = (size_t)T * d * (n->h_dtype == LM_F32 ? 4 : 2), xb = (size_t)T * d * 2, rb = (size_t)T * 4;
    const size_t wb = (size_t)d * (n->w_dtype == LM_F32 ? 4 : 2), gb = (size_t)d * 4;
    LL_TRY(check_alias({{dh, hb, "dh"}, {y ? dy : nullptr, xb, "dy"}, {dw_in, gb, "dw_in"}, {dw_post, gb, "dw_post"},
                        {dgate, gb, "dgate"}, {ws, total, "ws"}},
                       {{h, hb, "h"}, {y, xb, "y"}, {dh_out, hb, "dh_out"}, {dx, xb, "dx"}, {rstd_y, rb, "rstd_y"},
                        {rstd_h, rb, "rstd_h"}, {n->w_in, wb, "w_in"}, {n->w_post, wb, "w_post"}, {n->gate, wb, "gate"}}));
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) {  // sums over no tokens
        for (float* g : {dw_in, dw_post, dgate})
            if (g) LL_TRY(launched(cudaMemsetAsync(g, 0, gb, st), "cudaMemsetAsync"));
        return LM_OK;
    }
    int sms = 0;
    LL_TRY(device_ready(&sms));
    AddNormParams p = addnorm_params(T, d, h, y, n);
    p.dh_out = dh_out;
    p.dx = dx;
    p.rstd_y_in = rstd_y;
    p.rstd_h_in = rstd_h;
    p.dh = dh;
    p.dy = dy;
    p.dw_in = dw_in;
    p.dw_post = dw_post;
    p.dgate = dgate;
    p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
    LaunchTag tag("addnorm.bwd", st);
    return launched(launch_addnorm_bwd(p, st), "addnorm backward launch");
}

// ------------------------------------------------------------------ logprob
namespace {
lm_status check_logprob(int64_t T, int64_t V, int64_t ld, const void* logits, int32_t dtype, const void* targets,
                        int32_t index, float scale) {
    LL_TRY(check_tokens(T, (int64_t(1) << 31) - 1));
    if (V < 1 || V > (int64_t(1) << 30)) return report_error(LM_ERR_SHAPE, "V = %lld is not in [1, 2^30]", (long long)V);
    if (ld < V || ld > (int64_t(1) << 40)) return report_error(LM_ERR_SHAPE, "ld = %lld is smaller than V = %lld", (long long)ld, (long long)V);
    if (dtype != LM_BF16 && dtype != LM_F32) return report_error(LM_ERR_DTYPE, "dtype = %d is not known", dtype);
    if (index != LM_I32 && index != LM_I64) return report_error(LM_ERR_DTYPE, "index = %d is not known", index);
    if (!(scale > 0.f) || !std::isfinite(scale)) return report_error(LM_ERR_SHAPE, "scale = %g must be positive", scale);
    LL_TRY(need(logits, dtype == LM_F32 ? 4 : 2, "logits"));
    return need(targets, index == LM_I64 ? 8 : 4, "targets");
}

size_t logit_bytes(int64_t T, int64_t V, int64_t ld, int32_t dtype) {
    return T ? (size_t)((T - 1) * ld + V) * (dtype == LM_F32 ? 4 : 2) : 0;
}

LogprobParams logprob_params(int64_t T, int64_t V, int64_t ld, const void* logits, int32_t dtype, const void* targets,
                             int32_t index, float scale) {
    LogprobParams p{};
    p.T = T;
    p.V = V;
    p.ld = ld;
    p.logits = logits;
    p.f32 = dtype == LM_F32;
    p.targets = targets;
    p.i64 = index == LM_I64;
    p.scale = scale;
    return p;
}
}  // namespace

extern "C" lm_status logprob_fwd(int64_t T, int64_t V, int64_t ld, const void* logits, int32_t dtype, const void* targets,
                                 int32_t index, float scale, int32_t k, float* logp, float* entropy, float* lse,
                                 int32_t* top_ids, float* top_logp, lm_stream stream) {
    LL_TRY(check_logprob(T, V, ld, logits, dtype, targets, index, scale));
    if (k < 0 || k > kMaxTop || k > V) return report_error(LM_ERR_SHAPE, "k = %d is not in [0, %d] or larger than V", k, kMaxTop);
    LL_TRY(need(logp, 4, "logp"));
    LL_TRY(want(entropy, 4, "entropy"));
    LL_TRY(need(lse, 4, "lse"));
    if (k) {
        LL_TRY(need(top_ids, 4, "top_ids"));
        LL_TRY(need(top_logp, 4, "top_logp"));
    } else {
        LL_TRY(must_be_null(top_ids, "top_ids", "with k = 0"));
        LL_TRY(must_be_null(top_logp, "top_logp", "with k = 0"));
    }
    const size_t rb = (size_t)T * 4;
    LL_TRY(check_alias({{logp, rb, "logp"}, {entropy, rb, "entropy"}, {lse, rb, "lse"}, {top_ids, rb * k, "top_ids"},
                        {top_logp, rb * k, "top_logp"}},
                       {{logits, logit_bytes(T, V, ld, dtype), "logits"},
                        {targets, (size_t)T * (index == LM_I64 ? 8 : 4), "targets"}}));
    if (T == 0) return LM_OK;
    int sms = 0;
    LL_TRY(device_ready(&sms));
    LogprobParams p = logprob_params(T, V, ld, logits, dtype, targets, index, scale);
    p.k = k;
    p.logp = logp;
    p.entropy = entropy;
    p.lse = lse;
    p.top_ids = top_ids;
    p.top_logp = top_logp;
    cudaStream_t st = (cudaStream_t)stream;
    LaunchTag tag("logprob.fwd", st);
    return launched(launch_logprob_fwd(p, st), "logprob forward launch");
}

extern "C" lm_status logprob_bwd(int64_t T, int64_t V, int64_t ld, const void* logits, int32_t dtype, const void* targets,
                                 int32_t index, float scale, const float* lse, const float* entropy, const float* dlogp,
                                 const float* dentropy, void* dlogits, int64_t ld_out, lm_stream stream) {
    LL_TRY(check_logprob(T, V, ld, logits, dtype, targets, index, scale));
    if (ld_out < V || ld_out > (int64_t(1) << 40))
        return report_error(LM_ERR_SHAPE, "ld_out = %lld is smaller than V = %lld", (long long)ld_out, (long long)V);
    LL_TRY(need(lse, 4, "lse"));
    LL_TRY(want(dlogp, 4, "dlogp"));
    LL_TRY(want(dentropy, 4, "dentropy"));
    if (dentropy) LL_TRY(need(entropy, 4, "entropy"));
    LL_TRY(need(dlogits, dtype == LM_F32 ? 4 : 2, "dlogits"));
    const size_t rb = (size_t)T * 4;
    const bool in_place = dlogits == logits && ld_out == ld;
    LL_TRY(check_alias({{dlogits, logit_bytes(T, V, ld_out, dtype), "dlogits"}},
                       {{in_place ? nullptr : logits, logit_bytes(T, V, ld, dtype), "logits"},
                        {targets, (size_t)T * (index == LM_I64 ? 8 : 4), "targets"}, {lse, rb, "lse"},
                        {entropy, rb, "entropy"}, {dlogp, rb, "dlogp"}, {dentropy, rb, "dentropy"}}));
    if (T == 0) return LM_OK;
    int sms = 0;
    LL_TRY(device_ready(&sms));
    LogprobParams p = logprob_params(T, V, ld, logits, dtype, targets, index, scale);
    p.lse_in = lse;
    p.entropy_in = entropy;
    p.dlogp = dlogp;
    p.dentropy = dentropy;
    p.dlogits = dlogits;
    p.ld_out = ld_out;
    cudaStream_t st = (cudaStream_t)stream;
    LaunchTag tag("logprob.bwd", st);
    return launched(launch_logprob_bwd(p, st), "logprob backward launch");
}
