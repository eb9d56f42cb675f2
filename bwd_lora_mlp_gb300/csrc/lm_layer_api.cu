// C ABI of the layer operators: argument validation, workspace layout and the kernel sequence of
// each entry point.  See include/lora_layer.h for the contract.
#include <cfloat>
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
    p.T = p.Tk = (int32_t)T;
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

// ------------------------------------------------------------------ cross attention
namespace {
lm_status check_cross_shape(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk, int32_t d) {
    LL_TRY(check_attn_shape(Tq, hq, hk, d));
    if (Tk < 0 || Tk > kMaxTokens) return report_error(LM_ERR_SHAPE, "Tk = %lld is not in [0, %lld]", (long long)Tk, (long long)kMaxTokens);
    return LM_OK;
}

lm_status check_cross(const lm_cross* a) {
    if (!a) return report_error(LM_ERR_NULL, "a is NULL");
    if (!(a->scale > 0.f)) return report_error(LM_ERR_SHAPE, "scale = %g must be positive", a->scale);
    lm_attn like{};
    like.scale = a->scale;
    like.cap = a->cap;
    LL_TRY(check_attn(&like));
    if (!a->cu_q) {
        LL_TRY(must_be_null(a->cu_k, "cu_k", "without cu_q"));
        return must_be_null(a->k_len, "k_len", "without cu_q");
    }
    LL_TRY(need(a->cu_q, 4, "cu_q"));
    LL_TRY(need(a->cu_k, 4, "cu_k"));
    LL_TRY(want(a->k_len, 4, "k_len"));
    if (a->n_docs < 1 || a->n_docs > 1 << 30) return report_error(LM_ERR_SHAPE, "n_docs = %d is not in [1, 2^30]", a->n_docs);
    return LM_OK;
}

Span docs_span(const int32_t* p, int64_t n, const char* name) { return Span{p, (size_t)n * 4, name}; }

struct CrossPlan {
    FewPlan few;
    size_t qrange, krange, qseen, kseen, delta, nlse, part_ml, part_o, part_dkv, part_dq, total;
};

CrossPlan plan_cross(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk, int32_t d) {
    CrossPlan P;
    P.few = plan_few(Tq, Tk, hq, hk);
    size_t at = 256;  // after the error word
    auto take = [&at](size_t bytes) {
        const size_t here = at;
        at = (at + bytes + 255) & ~size_t(255);
        return here;
    };
    const size_t rows = (size_t)Tq * hq * (P.few.parts > 1 ? P.few.parts : 0);
    P.qrange = take((size_t)Tq * sizeof(int2));
    P.krange = take((size_t)Tk * sizeof(int2));
    P.qseen = take((size_t)whole_tiles(Tq) / 8);
    P.kseen = take((size_t)whole_tiles(Tk) / 8);
    P.delta = take((size_t)whole_tiles(Tq) * hq * 4);
    P.nlse = take((size_t)whole_tiles(Tq) * hq * 4);
    P.part_ml = take(rows * sizeof(float2));
    P.part_o = take(rows * d * sizeof(float));
    const size_t forward = at;  // (the backward's parts lie where the forward's were)
    at = P.part_ml;
    const BwdParts most = most_parts(Tq, Tk, hq, hk);
    P.part_dkv = take(most.k > 1 ? (size_t)most.k * 2 * Tk * hk * d * sizeof(float) : 0);
    P.part_dq = take(most.q > 1 ? (size_t)most.q * Tq * hq * d * sizeof(float) : 0);
    P.total = at > forward ? at : forward;
    return P;
}

// the parameters of both directions, and who sees whom (a launch with documents)
lm_status cross_begin(AttnParams* p, const CrossPlan& P, int64_t Tq, int64_t Tk, int32_t hq, int32_t hk, int32_t d,
                      const lm_heads* q, const lm_heads* k, const lm_heads* v, const lm_cross* a, void* ws, cudaStream_t st) {
    lm_attn like{};
    like.scale = a->scale;
    like.cap = a->cap;
    *p = attn_params(Tq, hq, hk, d, q, k, v, &like, ws);
    p->Tk = (int32_t)Tk;
    if (!a->cu_q) return LM_OK;
    char* base = static_cast<char*>(ws);
    const CrossTables t{reinterpret_cast<int2*>(base + P.qrange), reinterpret_cast<int2*>(base + P.krange),
                        reinterpret_cast<uint4*>(base + P.qseen), reinterpret_cast<uint4*>(base + P.kseen)};
    p->qrange = t.qrange;
    p->krange = t.krange;
    p->qseen = t.qseen;
    p->kseen = t.kseen;
    LaunchTag tag("cross.ranges", st);
    return launched(launch_cross_ranges(*a, Tq, Tk, t, st), "cross ranges launch");
}
}  // namespace

extern "C" lm_status cross_workspace_size(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk, int32_t d, size_t* bytes) {
    LL_TRY(check_cross_shape(Tq, Tk, hq, hk, d));
    if (!bytes) return report_error(LM_ERR_NULL, "bytes is NULL");
    *bytes = plan_cross(Tq, Tk, hq, hk, d).total;
    return LM_OK;
}

extern "C" lm_status cross_fwd(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk, int32_t d, const lm_heads* q, const lm_heads* k,
                               const lm_heads* v, const lm_cross* a, uint16_t* O, int8_t* O_lo, float* lse, void* ws,
                               size_t ws_bytes, lm_stream stream) {
    LL_TRY(check_cross_shape(Tq, Tk, hq, hk, d));
    LL_TRY(check_cross(a));
    LL_TRY(check_heads(q, Tq, hq, d, "q"));
    LL_TRY(check_heads(k, Tk, hk, d, "k"));
    LL_TRY(check_heads(v, Tk, hk, d, "v"));
    LL_TRY(need(O, 32, "O"));
    LL_TRY(want(O_lo, 32, "O_lo"));
    LL_TRY(need(lse, 32, "lse"));
    LL_TRY(need(ws, 32, "ws"));
    const CrossPlan P = plan_cross(Tq, Tk, hq, hk, d);
    if (ws_bytes < P.total) return report_error(LM_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, P.total);
    const size_t ob = (size_t)Tq * hq * d * 2, lob = (size_t)Tq * hq * ((d + 15) / 16 * 16), lb = (size_t)Tq * hq * 4;
    LL_TRY(check_alias({{O, ob, "O"}, {O_lo, lob, "O_lo"}, {lse, lb, "lse"}, {ws, P.total, "ws"}},
                       {heads_span(q, Tq, hq, d, "q"), heads_span(k, Tk, hk, d, "k"), heads_span(v, Tk, hk, d, "v"),
                        docs_span(a->cu_q, int64_t{a->n_docs} + 1, "cu_q"), docs_span(a->cu_k, int64_t{a->n_docs} + 1, "cu_k"),
                        docs_span(a->k_len, a->n_docs, "k_len")}));
    if (Tq == 0) return LM_OK;
    int sms = 0;
    LL_TRY(device_ready(&sms));
    cudaStream_t st = (cudaStream_t)stream;
    if (Tk == 0) {  // nothing is seen
        LL_TRY(launched(cudaMemsetAsync(O, 0, ob, st), "cudaMemsetAsync"));
        if (O_lo) LL_TRY(launched(cudaMemsetAsync(O_lo, 0, lob, st), "cudaMemsetAsync"));
        return launched(launch_fill(lse, (int64_t)Tq * hq, -INFINITY, st), "fill launch");
    }
    AttnParams p;
    LL_TRY(cross_begin(&p, P, Tq, Tk, hq, hk, d, q, k, v, a, ws, st));
    p.out = O;
    p.out_lo = O_lo;
    p.lse = lse;
    p.splits = P.few.splits;
    p.parts = P.few.parts;
    p.rows = P.few.tokens;
    p.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + P.part_ml);
    p.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + P.part_o);
    LaunchTag tag("cross.fwd", st);
    return launch_cross_fwd(p, sms, st);
}

extern "C" lm_status cross_bwd(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk, int32_t d, const lm_heads* q, const lm_heads* k,
                               const lm_heads* v, const lm_heads* dO, const uint16_t* O, const int8_t* O_lo, const float* lse,
                               const lm_cross* a, uint16_t* dQ, uint16_t* dK, uint16_t* dV, void* ws, size_t ws_bytes,
                               lm_stream stream) {
    LL_TRY(check_cross_shape(Tq, Tk, hq, hk, d));
    LL_TRY(check_cross(a));
    LL_TRY(check_heads(q, Tq, hq, d, "q"));
    LL_TRY(check_heads(k, Tk, hk, d, "k"));
    LL_TRY(check_heads(v, Tk, hk, d, "v"));
    LL_TRY(check_heads(dO, Tq, hq, d, "dO"));
    LL_TRY(need(O, 32, "O"));
    LL_TRY(want(O_lo, 32, "O_lo"));
    LL_TRY(need(lse, 32, "lse"));
    LL_TRY(need(dQ, 32, "dQ"));
    LL_TRY(need(dK, 32, "dK"));
    LL_TRY(need(dV, 32, "dV"));
    LL_TRY(need(ws, 32, "ws"));
    const CrossPlan P = plan_cross(Tq, Tk, hq, hk, d);
    if (ws_bytes < P.total) return report_error(LM_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, P.total);
    const size_t bq = (size_t)Tq * hq * d * 2, bk = (size_t)Tk * hk * d * 2;
    LL_TRY(check_alias({{dQ, bq, "dQ"}, {dK, bk, "dK"}, {dV, bk, "dV"}, {ws, P.total, "ws"}},
                       {heads_span(q, Tq, hq, d, "q"), heads_span(k, Tk, hk, d, "k"), heads_span(v, Tk, hk, d, "v"),
                        heads_span(dO, Tq, hq, d, "dO"), {O, bq, "O"}, {O_lo, (size_t)Tq * hq * ((d + 15) / 16 * 16), "O_lo"},
                        {lse, (size_t)Tq * hq * 4, "lse"}, docs_span(a->cu_q, int64_t{a->n_docs} + 1, "cu_q"),
                        docs_span(a->cu_k, int64_t{a->n_docs} + 1, "cu_k"), docs_span(a->k_len, a->n_docs, "k_len")}));
    if (Tq == 0 && Tk == 0) return LM_OK;
    int sms = 0;
    LL_TRY(device_ready(&sms));
    cudaStream_t st = (cudaStream_t)stream;
    if (Tq == 0 || Tk == 0) {  // nothing is seen
        if (bq) LL_TRY(launched(cudaMemsetAsync(dQ, 0, bq, st), "cudaMemsetAsync"));
        if (bk) LL_TRY(launched(cudaMemsetAsync(dK, 0, bk, st), "cudaMemsetAsync"));
        if (bk) LL_TRY(launched(cudaMemsetAsync(dV, 0, bk, st), "cudaMemsetAsync"));
        return LM_OK;
    }
    AttnParams p;
    LL_TRY(cross_begin(&p, P, Tq, Tk, hq, hk, d, q, k, v, a, ws, st));
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
    const BwdParts parts = plan_parts(Tq, Tk, hq, hk, d, a->cu_q ? a->n_docs : 1);
    p.kparts = parts.k;
    p.qparts = parts.q;
    p.part_dkv = reinterpret_cast<float*>(static_cast<char*>(ws) + P.part_dkv);
    p.part_dq = reinterpret_cast<float*>(static_cast<char*>(ws) + P.part_dq);
    {
        LaunchTag tag("cross.delta", st);
        LL_TRY(launched(launch_attn_delta(p, lm_attn{}, delta, nlse, nullptr, st), "cross delta launch"));
    }
    return launch_cross_bwd(p, sms, st);
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

// ------------------------------------------------------------------ qkrope
namespace {
// Whether two strided tensors share no element.  Rows of the one may lie between rows of the other: with equal
// token strides, or equal head strides, it is enough that their places modulo that stride are apart.
struct Strided {
    const lm_heads* t;
    int64_t T;
    int heads, d;
    const char* name;
};
bool apart(const Strided& a, const Strided& b) {
    if (!overlap(heads_span(a.t, a.T, a.heads, a.d, a.name), heads_span(b.t, b.T, b.heads, b.d, b.name))) return true;
    auto between = [](const Strided& x, const Strided& y, int64_t period, int64_t ex, int64_t ey) {
        if (ex > period || ey > period) return false;
        const int64_t off = (reinterpret_cast<intptr_t>(y.t->p) - reinterpret_cast<intptr_t>(x.t->p)) / 2;
        const int64_t at = ((off % period) + period) % period;
        return at >= ex && at + ey <= period;
    };
    auto row = [](const Strided& x) { return (x.heads - 1) * x.t->head_stride + x.d; };
    auto column = [](const Strided& x) { return (x.T - 1) * x.t->token_stride + x.d; };
    return (a.t->token_stride == b.t->token_stride && between(a, b, a.t->token_stride, row(a), row(b))) ||
           (a.t->head_stride == b.t->head_stride && between(a, b, a.t->head_stride, column(a), column(b)));
}
// an output's own tokens and heads must not share elements
lm_status check_own(const Strided& a) {
    if ((a.heads - 1) * a.t->head_stride + a.d <= a.t->token_stride || (a.T - 1) * a.t->token_stride + a.d <= a.t->head_stride)
        return LM_OK;
    return report_error(LM_ERR_ALIAS, "%s: its tokens and heads overlap", a.name);
}
bool same_place(const lm_heads* a, const lm_heads* b) {
    return a->p == b->p && a->token_stride == b->token_stride && a->head_stride == b->head_stride;
}

lm_status check_qkrope_shape(int64_t T, int32_t hq, int32_t hk, int32_t d) {
    LL_TRY(check_tokens(T, (int64_t(1) << 31) - 1));
    if (hq < 1 || hk < 0 || hq > 1024 || hk > 1024)
        return report_error(LM_ERR_SHAPE, "hq = %d must be in [1, 1024], hk = %d in [0, 1024]", hq, hk);
    if (d < 8 || d > 256 || d % 8 != 0) return report_error(LM_ERR_SHAPE, "d = %d must be a multiple of 8 in [8, 256]", d);
    return LM_OK;
}

lm_status check_qkrope(const lm_qkrope* r, int32_t hk, int32_t d) {
    if (!r) return report_error(LM_ERR_NULL, "r is NULL");
    if (r->rot < 0 || r->rot > d || r->rot % 8 != 0)
        return report_error(LM_ERR_SHAPE, "rot = %d must be a multiple of 8 in [0, d]", r->rot);
    if (!r->rot && !r->norm) return report_error(LM_ERR_SHAPE, "neither a norm nor a rotation: nothing to do");
    if (r->pos_index != LM_I32 && r->pos_index != LM_I64) return report_error(LM_ERR_DTYPE, "pos_index = %d is not known", r->pos_index);
    if (r->w_dtype != LM_BF16 && r->w_dtype != LM_F32) return report_error(LM_ERR_DTYPE, "w_dtype = %d is not known", r->w_dtype);
    if (r->rot) {
        if (r->axes < 1) return report_error(LM_ERR_SHAPE, "axes = %d must be positive", r->axes);
        LL_TRY(need(r->inv_freq, 4, "inv_freq"));
        LL_TRY(want(r->pos, r->pos_index == LM_I64 ? 8 : 4, "pos"));
        LL_TRY(want(r->axis, 4, "axis"));
        if (r->axes > 1) {
            LL_TRY(need(r->pos, 4, "pos"));
            LL_TRY(need(r->axis, 4, "axis"));
        }
        if (!std::isfinite(r->factor)) return report_error(LM_ERR_SHAPE, "factor is not finite");
    } else {
        LL_TRY(must_be_null(r->inv_freq, "inv_freq", "with rot = 0"));
        LL_TRY(must_be_null(r->pos, "pos", "with rot = 0"));
        LL_TRY(must_be_null(r->axis, "axis", "with rot = 0"));
    }
    if (r->norm) {
        // (the kernels' reciprocal root takes subnormals for 0, and a head of zeros would be 0 x inf)
        if (!(r->eps >= FLT_MIN) || !std::isfinite(r->eps))
            return report_error(LM_ERR_SHAPE, "eps = %g must be at least 2^-126", r->eps);
        if (!std::isfinite(r->w_offset)) return report_error(LM_ERR_SHAPE, "w_offset is not finite");
        LL_TRY(want(r->w_q, r->w_dtype == LM_F32 ? 4 : 2, "w_q"));
        LL_TRY(want(r->w_k, r->w_dtype == LM_F32 ? 4 : 2, "w_k"));
        if (!hk) LL_TRY(must_be_null(r->w_k, "w_k", "without keys"));
    } else {
        LL_TRY(must_be_null(r->w_q, "w_q", "without a norm"));
        LL_TRY(must_be_null(r->w_k, "w_k", "without a norm"));
    }
    return LM_OK;
}

// outputs against each other and against what is read; an output may be the input at the same index of `over`
lm_status check_rope_places(std::initializer_list<Strided> outs, std::initializer_list<Strided> over,
                            std::initializer_list<Strided> ins, std::initializer_list<Span> flat_outs,
                            std::initializer_list<Span> flat) {
    for (const Strided* o = outs.begin(); o != outs.end(); ++o) {
        if (!o->t) continue;
        LL_TRY(check_own(*o));
        for (const Strided* q = o + 1; q != outs.end(); ++q)
            if (q->t && !apart(*o, *q)) return report_error(LM_ERR_ALIAS, "%s overlaps %s", o->name, q->name);
        for (const Strided* q = over.begin(); q != over.end(); ++q)
            if (q->t && !(q - over.begin() == o - outs.begin() && same_place(o->t, q->t)) && !apart(*o, *q))
                return report_error(LM_ERR_ALIAS, "%s overlaps %s", o->name, q->name);
        for (const Strided& q : ins)
            if (q.t && !apart(*o, q)) return report_error(LM_ERR_ALIAS, "%s overlaps %s", o->name, q.name);
        const Span s = heads_span(o->t, o->T, o->heads, o->d, o->name);
        for (const Span& f : flat)
            if (overlap(s, f)) return report_error(LM_ERR_ALIAS, "%s overlaps %s", o->name, f.name);
        for (const Span& f : flat_outs)
            if (overlap(s, f)) return report_error(LM_ERR_ALIAS, "%s overlaps %s", o->name, f.name);
    }
    for (const Span* o = flat_outs.begin(); o != flat_outs.end(); ++o) {
        for (const std::initializer_list<Strided>* l : {&over, &ins})
            for (const Strided& q : *l)
                if (q.t && overlap(*o, heads_span(q.t, q.T, q.heads, q.d, q.name)))
                    return report_error(LM_ERR_ALIAS, "%s overlaps %s", o->name, q.name);
        for (const Span& f : flat)
            if (overlap(*o, f)) return report_error(LM_ERR_ALIAS, "%s overlaps %s", o->name, f.name);
        for (const Span* q = o + 1; q != flat_outs.end(); ++q)
            if (overlap(*o, *q)) return report_error(LM_ERR_ALIAS, "%s overlaps %s", o->name, q->name);
    }
    return LM_OK;
}

struct RopeFlat {
    Span inv_freq, pos, axis, w_q, w_k;
};
RopeFlat rope_flat(int64_t T, int32_t d, const lm_qkrope* r) {
    const size_t half = (size_t)r->rot / 2 * 4, wb = (size_t)d * (r->w_dtype == LM_F32 ? 4 : 2);
    return RopeFlat{{r->inv_freq, half, "inv_freq"},
                    {r->pos, (size_t)T * (r->rot ? r->axes : 0) * (r->pos_index == LM_I64 ? 8 : 4), "pos"},
                    {r->axis, half, "axis"},
                    {r->w_q, wb, "w_q"},
                    {r->w_k, wb, "w_k"}};
}

QkRopeParams qkrope_params(int64_t T, int32_t hq, int32_t hk, int32_t d, const lm_qkrope* r) {
    QkRopeParams p{};
    p.T = T;
    p.d = d;
    p.rot = r->rot;
    p.axes = r->rot ? r->axes : 1;
    p.inv_freq = r->inv_freq;
    p.pos = r->pos;
    p.axis = p.axes > 1 ? r->axis : nullptr;  // (one axis: all pairs are its)
    p.pos_i64 = r->pos_index == LM_I64;
    p.w_f32 = r->w_dtype == LM_F32;
    p.norm = r->norm != 0;
    p.interleaved = r->interleaved != 0;
    p.factor = r->factor;
    p.eps = r->eps;
    p.w_offset = r->w_offset;
    p.q.heads = hq;
    p.k.heads = hk;
    p.q.w = r->w_q;
    p.k.w = r->w_k;
    return p;
}
void side_in(RopeSide& S, const lm_heads* t) { S.x = t->p, S.x_ts = t->token_stride, S.x_hs = t->head_stride; }
void side_grad(RopeSide& S, const lm_heads* t) { S.dy = t->p, S.dy_ts = t->token_stride, S.dy_hs = t->head_stride; }
void side_out(RopeSide& S, const lm_heads* t) {
    S.y = const_cast<uint16_t*>(t->p), S.y_ts = t->token_stride, S.y_hs = t->head_stride;
}
}  // namespace

extern "C" lm_status qkrope_workspace_size(int64_t T, int32_t hq, int32_t hk, int32_t d, size_t* bytes) {
    LL_TRY(check_qkrope_shape(T, hq, hk, d));
    if (!bytes) return report_error(LM_ERR_NULL, "bytes is NULL");
    *bytes = 256 + qkrope_part_bytes(d);
    return LM_OK;
}

extern "C" lm_status qkrope_fwd(int64_t T, int32_t hq, int32_t hk, int32_t d, const lm_heads* q, const lm_heads* k,
                                const lm_qkrope* r, const lm_heads* q_out, const lm_heads* k_out, lm_stream stream) {
    LL_TRY(check_qkrope_shape(T, hq, hk, d));
    LL_TRY(check_qkrope(r, hk, d));
    LL_TRY(check_heads(q, T, hq, d, "q"));
    LL_TRY(check_heads(q_out, T, hq, d, "q_out"));
    if (hk) {
        LL_TRY(check_heads(k, T, hk, d, "k"));
        LL_TRY(check_heads(k_out, T, hk, d, "k_out"));
    } else {
        LL_TRY(must_be_null(k, "k", "with hk = 0"));
        LL_TRY(must_be_null(k_out, "k_out", "with hk = 0"));
    }
    if (T == 0) return LM_OK;
    const RopeFlat f = rope_flat(T, d, r);
    LL_TRY(check_rope_places({{q_out, T, hq, d, "q_out"}, {k_out, T, hk, d, "k_out"}}, {{q, T, hq, d, "q"}, {k, T, hk, d, "k"}}, {}, {},
                             {f.inv_freq, f.pos, f.axis, f.w_q, f.w_k}));
    int sms = 0;
    LL_TRY(device_ready(&sms));
    QkRopeParams p = qkrope_params(T, hq, hk, d, r);
    side_in(p.q, q);
    side_out(p.q, q_out);
    if (hk) {
        side_in(p.k, k);
        side_out(p.k, k_out);
    }
    cudaStream_t st = (cudaStream_t)stream;
    LaunchTag tag("qkrope.fwd", st);
    return launched(launch_qkrope(p, false, st), "qkrope forward launch");
}

extern "C" lm_status qkrope_bwd(int64_t T, int32_t hq, int32_t hk, int32_t d, const lm_heads* q, const lm_heads* k,
                                const lm_heads* dq, const lm_heads* dk, const lm_qkrope* r, const lm_heads* dq_in,
                                const lm_heads* dk_in, float* dw_q, float* dw_k, void* ws, size_t ws_bytes, lm_stream stream) {
    LL_TRY(check_qkrope_shape(T, hq, hk, d));
    LL_TRY(check_qkrope(r, hk, d));
    const bool norm = r->norm != 0;
    if (norm) LL_TRY(check_heads(q, T, hq, d, "q"));
    LL_TRY(check_heads(dq, T, hq, d, "dq"));
    LL_TRY(check_heads(dq_in, T, hq, d, "dq_in"));
    if (hk) {
        if (norm) LL_TRY(check_heads(k, T, hk, d, "k"));
        LL_TRY(check_heads(dk, T, hk, d, "dk"));
        LL_TRY(check_heads(dk_in, T, hk, d, "dk_in"));
    } else {
        LL_TRY(must_be_null(k, "k", "with hk = 0"));
        LL_TRY(must_be_null(dk, "dk", "with hk = 0"));
        LL_TRY(must_be_null(dk_in, "dk_in", "with hk = 0"));
        LL_TRY(must_be_null(dw_k, "dw_k", "with hk = 0"));
    }
    LL_TRY(want(dw_q, 4, "dw_q"));
    LL_TRY(want(dw_k, 4, "dw_k"));
    const size_t total = 256 + qkrope_part_bytes(d), gb = (size_t)d * 4;
    if (norm) {
        LL_TRY(need(ws, 32, "ws"));
        if (ws_bytes < total) return report_error(LM_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, total);
    } else {
        LL_TRY(must_be_null(dw_q, "dw_q", "without a norm"));
        LL_TRY(must_be_null(dw_k, "dw_k", "without a norm"));
    }
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) {  // sums over no tokens
        for (float* g : {dw_q, dw_k})
            if (g) LL_TRY(launched(cudaMemsetAsync(g, 0, gb, st), "cudaMemsetAsync"));
        return LM_OK;
    }
    const RopeFlat f = rope_flat(T, d, r);
    LL_TRY(check_rope_places({{dq_in, T, hq, d, "dq_in"}, {dk_in, T, hk, d, "dk_in"}}, {{dq, T, hq, d, "dq"}, {dk, T, hk, d, "dk"}},
                             {{norm ? q : nullptr, T, hq, d, "q"}, {norm ? k : nullptr, T, hk, d, "k"}},
                             {{dw_q, gb, "dw_q"}, {dw_k, gb, "dw_k"}, {norm ? ws : nullptr, total, "ws"}},
                             {f.inv_freq, f.pos, f.axis, f.w_q, f.w_k}));
    int sms = 0;
    LL_TRY(device_ready(&sms));
    QkRopeParams p = qkrope_params(T, hq, hk, d, r);
    if (norm) side_in(p.q, q);
    side_grad(p.q, dq);
    side_out(p.q, dq_in);
    p.q.dw = dw_q;
    if (hk) {
        if (norm) side_in(p.k, k);
        side_grad(p.k, dk);
        side_out(p.k, dk_in);
        p.k.dw = dw_k;
    }
    p.part = norm ? reinterpret_cast<float*>(static_cast<char*>(ws) + 256) : nullptr;
    LaunchTag tag("qkrope.bwd", st);
    return launched(launch_qkrope(p, true, st), "qkrope backward launch");
}

// ------------------------------------------------------------------ distill
namespace {
lm_status check_distill(int64_t T, int64_t V, int64_t ld, const void* logits, int32_t dtype, const lm_teacher* t,
                        const void* targets, int32_t index, float scale) {
    LL_TRY(check_tokens(T, (int64_t(1) << 31) - 1));
    if (V < 1 || V > (int64_t(1) << 30)) return report_error(LM_ERR_SHAPE, "V = %lld is not in [1, 2^30]", (long long)V);
    if (ld < V || ld > (int64_t(1) << 40)) return report_error(LM_ERR_SHAPE, "ld = %lld is smaller than V = %lld", (long long)ld, (long long)V);
    if (dtype != LM_BF16 && dtype != LM_F32) return report_error(LM_ERR_DTYPE, "dtype = %d is not known", dtype);
    if (!(scale > 0.f) || !std::isfinite(scale)) return report_error(LM_ERR_SHAPE, "scale = %g must be positive", scale);
    LL_TRY(need(logits, dtype == LM_F32 ? 4 : 2, "logits"));
    if (!t) return report_error(LM_ERR_NULL, "t is NULL");
    if (t->K < 1 || t->K > kMaxEntries) return report_error(LM_ERR_SHAPE, "K = %d is not in [1, %d]", t->K, kMaxEntries);
    if (t->index != LM_I32 && t->index != LM_I64) return report_error(LM_ERR_DTYPE, "index = %d of ids is not known", t->index);
    if (t->dtype != LM_BF16 && t->dtype != LM_F32) return report_error(LM_ERR_DTYPE, "dtype = %d of values is not known", t->dtype);
    LL_TRY(need(t->ids, t->index == LM_I64 ? 8 : 4, "ids"));
    LL_TRY(need(t->values, t->dtype == LM_F32 ? 4 : 2, "values"));
    if (!targets) return LM_OK;
    if (index != LM_I32 && index != LM_I64) return report_error(LM_ERR_DTYPE, "index = %d is not known", index);
    return need(targets, index == LM_I64 ? 8 : 4, "targets");
}

struct DistillIn {
    Span ids, values, targets;
};
DistillIn distill_in(int64_t T, const lm_teacher* t, const void* targets, int32_t index) {
    const size_t n = (size_t)T * t->K;
    return DistillIn{{t->ids, n * (t->index == LM_I64 ? 8 : 4), "ids"},
                     {t->values, n * (t->dtype == LM_F32 ? 4 : 2), "values"},
                     {targets, (size_t)T * (index == LM_I64 ? 8 : 4), "targets"}};
}

DistillParams distill_params(int64_t T, int64_t V, int64_t ld, const void* logits, int32_t dtype, const lm_teacher* t,
                             const void* targets, int32_t index, float scale) {
    DistillParams p{};
    p.T = T;
    p.V = V;
    p.ld = ld;
    p.logits = logits;
    p.f32 = dtype == LM_F32;
    p.i64 = t->index == LM_I64;
    p.t64 = index == LM_I64;
    p.v_f32 = t->dtype == LM_F32;
    p.rest = t->rest != 0;
    p.K = t->K;
    p.ids = t->ids;
    p.values = t->values;
    p.targets = targets;
    p.scale = scale;
    return p;
}
}  // namespace

extern "C" lm_status distill_fwd(int64_t T, int64_t V, int64_t ld, const void* logits, int32_t dtype, const lm_teacher* t,
                                 const void* targets, int32_t index, float scale, float* kl, float* logp, float* lse,
                                 float* saved, lm_stream stream) {
    LL_TRY(check_distill(T, V, ld, logits, dtype, t, targets, index, scale));
    LL_TRY(need(kl, 4, "kl"));
    LL_TRY(need(lse, 4, "lse"));
    LL_TRY(need(saved, 32, "saved"));
    if (targets) LL_TRY(need(logp, 4, "logp"));
    else LL_TRY(must_be_null(logp, "logp", "without targets"));
    const size_t rb = (size_t)T * 4;
    const DistillIn in = distill_in(T, t, targets, index);
    LL_TRY(check_alias({{kl, rb, "kl"}, {logp, rb, "logp"}, {lse, rb, "lse"}, {saved, rb * 8, "saved"}},
                       {{logits, logit_bytes(T, V, ld, dtype), "logits"}, in.ids, in.values, in.targets}));
    if (T == 0) return LM_OK;
    int sms = 0;
    LL_TRY(device_ready(&sms));
    DistillParams p = distill_params(T, V, ld, logits, dtype, t, targets, index, scale);
    p.kl = kl;
    p.logp = logp;
    p.lse = lse;
    p.saved = saved;
    cudaStream_t st = (cudaStream_t)stream;
    LaunchTag tag("distill.fwd", st);
    return launched(launch_distill_fwd(p, st), "distill forward launch");
}

extern "C" lm_status distill_bwd(int64_t T, int64_t V, int64_t ld, const void* logits, int32_t dtype, const lm_teacher* t,
                                 const void* targets, int32_t index, float scale, const float* saved, const float* dkl,
                                 const float* dlogp, void* dlogits, int64_t ld_out, lm_stream stream) {
    LL_TRY(check_distill(T, V, ld, logits, dtype, t, targets, index, scale));
    if (ld_out < V || ld_out > (int64_t(1) << 40))
        return report_error(LM_ERR_SHAPE, "ld_out = %lld is smaller than V = %lld", (long long)ld_out, (long long)V);
    LL_TRY(need(saved, 32, "saved"));
    LL_TRY(want(dkl, 4, "dkl"));
    LL_TRY(want(dlogp, 4, "dlogp"));
    if (!targets) LL_TRY(must_be_null(dlogp, "dlogp", "without targets"));
    LL_TRY(need(dlogits, dtype == LM_F32 ? 4 : 2, "dlogits"));
    const size_t rb = (size_t)T * 4;
    const bool in_place = dlogits == logits && ld_out == ld;
    const DistillIn in = distill_in(T, t, targets, index);
    LL_TRY(check_alias({{dlogits, logit_bytes(T, V, ld_out, dtype), "dlogits"}},
                       {{in_place ? nullptr : logits, logit_bytes(T, V, ld, dtype), "logits"}, in.ids, in.values, in.targets,
                        {saved, rb * 8, "saved"}, {dkl, rb, "dkl"}, {dlogp, rb, "dlogp"}}));
    if (T == 0) return LM_OK;
    int sms = 0;
    LL_TRY(device_ready(&sms));
    DistillParams p = distill_params(T, V, ld, logits, dtype, t, targets, index, scale);
    p.saved = const_cast<float*>(saved);
    p.dkl = dkl;
    p.dlogp = dlogp;
    p.dlogits = dlogits;
    p.ld_out = ld_out;
    cudaStream_t st = (cudaStream_t)stream;
    LaunchTag tag("distill.bwd", st);
    return launched(launch_distill_bwd(p, st), "distill backward launch");
}
