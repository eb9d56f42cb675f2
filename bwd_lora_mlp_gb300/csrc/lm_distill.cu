// Distillation from a teacher's top logits, with the log probabilities of given tokens (include/lora_layer.h).
//   x = scale z,  lse = log sum e^x,  q = e^{x - lse};  p the teacher's K entries, S their tokens
//   without rest  kl = sum_k p_k (log p_k - log q_k)                        dx_j = q_j - p_j
//   with rest     the same + p_r (log p_r - log q_r),  p_r = 1 - sum p,     dx_j = W q_j - p_j in S,
//                 q_r = sum of q outside S,  W = sum p + p_r                dx_j = q_j (W - p_r / q_r) elsewhere
// Forward: one pass over the logits.  With rest, the running maximum and sum leave the tokens of S out, so that q_r
// comes from its own terms and not from what 1 - sum q leaves: each vector has a byte in shared memory that says
// which of its logits are in S.  What the K entries add is asked for before the pass and summed after it; one
// thread joins the scalars.  The sum at scale 1 for the tokens' own log probabilities takes a second exponential
// only where scale is not 1.  Bound by memory in long rows: 4096 x 131072 with rest and tokens 181 us, 5.9 TB/s (0.87 of the
// copy rate); 8192 x 32000 with two exponentials 97 us, 5.4 TB/s; 1000 x 50257 with rest 27 us: six or seven rows an SM, whose
// beginnings and ends show.  (The second exponential by arithmetic, a polynomial of degree 5, instead of the exponential
// unit: 8192 x 32000 167 us instead of 123, for a quarter of the elements 131; rows asked for further ahead in L2: 185 to
// 192 us at 4096 x 131072.)
// Backward: one pass; outside S, dx_j = (W q_r - p_r) e^{x_j} / sum of e^x outside S, a share of at most 1, which no size
// of logits overflows.  The entries in a CTA's stretch are read before it is written and written after it.
// 4096 x 131072 322 us, 6.7 TB/s (0.98 of the copy rate); 8192 x 32000 173 us, 6.1; 1000 x 50257 28 us, 7.2 (its logits
// are in part still in L2).
#include <algorithm>

#include "lm_rows.cuh"

namespace lm {

constexpr int kMarks = 16384;     // vectors of a row (a CTA's segment) with a byte of their own
constexpr int kEntryWarps = kMaxEntries / 32;
// One row of `saved`: what the backward takes from the forward.
// Logarithms are of sums relative to a logit that is written beside them: with masks of the type's lowest
// value a sum's logarithm is nothing beside the maximum.
struct Saved {
    float top, l2, l1;  // the row's largest logit; log2 of sum e^{(z - top) scale}, of sum e^{z - top}
    float m, ml2;       // with rest: the same over the logits that are not entries, at scale; else m is the teacher's largest
    float coef, W, tl;  // others: coef times their share of e^x; entries: W q - p,  p = e^{y - tl}, or e^{(y - m) scale - tl}
};

__device__ __forceinline__ float teacher_at(const DistillParams& p, int64_t t, int k) {
    const int64_t i = t * p.K + k;
    return p.v_f32 ? static_cast<const float*>(p.values)[i]
                   : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.values)[i] << 16);
}
// log p of a value, but for a sum's logarithm: log probabilities are what they are, logits are taken relative to the
// row's largest before they are scaled, so that nothing is lost of their differences however far from 0 they lie
template <bool REST>
__device__ __forceinline__ float teacher_log(float y, float top, float scale) {
    return REST ? y : (y - top) * scale;
}
__device__ __forceinline__ int id_at(const DistillParams& p, int64_t t, int k) {
    const int64_t i = t * p.K + k;
    const int64_t v = p.i64 ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
    return v >= 0 && v < p.V ? (int)v : -1;
}
__device__ __forceinline__ int64_t hard_target(const DistillParams& p, int64_t t) {
    if (!p.targets) return -1;
    const int64_t v = p.t64 ? static_cast<const int64_t*>(p.targets)[t] : static_cast<const int32_t*>(p.targets)[t];
    return v >= 0 && v < p.V ? v : -1;
}

// A running maximum and the sums of e^{(z - m) scale} and e^{z - m}.
struct Part {
    float m, S, S1;
};
// 2^{(a - m) c}, 0 for a = -inf also where m is
__device__ __forceinline__ float brought(float a, float m, float c) {
    return a == -INFINITY ? 0.f : lp_ex2(fmaxf(a - m, -1e30f) * c);
}
template <int N, bool TWO>
__device__ __forceinline__ Part join_parts(Part s, float c) {
    float m = s.m;
#pragma unroll
    for (int o = N / 2; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    s.S *= brought(s.m, m, c);
    if (TWO) s.S1 *= brought(s.m, m, kL2e);
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
        s.S += __shfl_xor_sync(0xffffffffu, s.S, o);
        if (TWO) s.S1 += __shfl_xor_sync(0xffffffffu, s.S1, o);
    }
    if (m != m) s.S = s.S1 = m;
    s.m = m;
    return s;
}

// Which of entries k to k + 3 are of token id, and the first of those that are (beyond all entries: none)
__device__ __forceinline__ uint32_t same_of(const int* ids, int k, int id) {
    const int4 v = *reinterpret_cast<const int4*>(ids + k);
    return (v.x == id ? 1u : 0u) | (v.y == id ? 2u : 0u) | (v.z == id ? 4u : 0u) | (v.w == id ? 8u : 0u);
}
__device__ __forceinline__ int before(uint32_t same) { return same ? __ffs((int)same) - 1 : kMaxEntries; }

struct DistillShared {
    alignas(16) int ids[kMaxEntries];
    float red[kEntryWarps][2], sums[kEntryWarps][4];
    Part warp[kThreads / 32], seg[kMaxCluster];
};

template <bool F32, bool REST, bool TWO, int N>
__global__ void __launch_bounds__(N, 1024 / N) distill_fwd_kernel(const __grid_constant__ DistillParams p, int cluster) {
    __shared__ DistillShared sm;
    __shared__ uint4 marks4[REST ? kMarks / 16 : 1];
    uint8_t* marks = reinterpret_cast<uint8_t*>(marks4);
    griddep_launch_dependents();
    if (cluster > 1) cluster_arrive();  // (waited for where the CTAs write to the first one's shared memory)
    griddep_wait();
    constexpr int W = Row<F32>::kVec;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x / cluster;
    const int part = cluster > 1 ? (int)cluster_rank() : 0;
    const Row<F32> row{static_cast<const char*>(p.logits) + t * p.ld * (F32 ? 4 : 2)};
    const int64_t len = ((p.V + cluster - 1) / cluster + 63) / 64 * 64;  // segments of whole 64-element stretches
    const int64_t j0 = min(p.V, part * len), j1 = min(p.V, j0 + len);
    const float c = p.scale * kL2e;
    constexpr int U = 4;
    Scan<U, F32, N> pass(row, j0, j1);  // (its first loads are under way)
    const int64_t a = pass.a;
    const int nv = pass.nv;

    // ---- the entries: asked for here, and (but for their marks) looked at after the pass
    int id = -1;
    float y = -INFINITY, x = -INFINITY;
    if (tid < p.K) {
        id = id_at(p, t, tid);
        if (id >= 0 && part == 0) {
            y = teacher_at(p, t, tid);
            x = row.at(id);
        }
    }
    const int64_t target = tid == 0 && part == 0 ? hard_target(p, t) : -1;
    const float zt = target >= 0 ? row.at(target) : 0.f;
    if (REST) {
        if (tid < kMaxEntries) sm.ids[tid] = id;
        for (int i = tid; i < min(kMarks, nv + 15) / 16; i += N) marks4[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        if (id >= a && id < a + (int64_t)nv * W) {
            const int64_t v = (id - a) / W;
            const int i = (int)(v & (kMarks - 1));
            atomicOr(reinterpret_cast<uint32_t*>(marks4) + i / 4, 1u << (i % 4 * 8 + (int)(id - a - v * W)));
        }
        __syncthreads();
    }

    // ---- the pass
    Part s{-INFINITY, 0.f, 0.f};
    auto rise = [&](float big) {  // the running maximum follows, and the sums with it (a NaN comes here every time and stays)
        s.S *= brought(s.m, big, c);
        if (TWO) s.S1 *= brought(s.m, big, kL2e);
        s.m = max_nan(s.m, big);
    };
    auto entry_bits = [&](int64_t j) {  // where vectors share a byte: which of the W logits from j on are entries
        uint32_t b = 0;
        for (int k = 0; k < p.K; ++k) {
            const int64_t at = sm.ids[k] - j;
            if (sm.ids[k] >= 0 && (uint64_t)at < (uint64_t)W) b |= 1u << at;
        }
        return b;
    };
    pass.run([&](uint32_t (&w)[U][4], int64_t j, int) {
        if (REST) {
            const int v = (int)((j - a) / W);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint32_t b = marks[(v + u * N) & (kMarks - 1)];
                if (b) {
                    if (nv > kMarks) b = entry_bits(j + (int64_t)u * N * W);
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (b >> e & 1u) {
                            if (F32) w[u][e % 4] = 0xFF800000u;
                            else w[u][e / 2 % 4] = e & 1 ? (w[u][e / 2 % 4] & 0xFFFFu) | 0xFF800000u : (w[u][e / 2 % 4] & 0xFFFF0000u) | 0xFF80u;
                        }
                }
            }
        }
        const float big = largest<U, F32>(w);
        if (!(big <= s.m)) rise(big);
        if (s.m == -INFINITY) return;
        float2 S2[2] = {make_float2(s.S, 0.f), make_float2(0.f, 0.f)}, T2[2] = {make_float2(s.S1, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < W; e += 2) {
                const float2 d = __fadd2_rn(make_float2(logit<F32>(w[u], e), logit<F32>(w[u], e + 1)), make_float2(-s.m, -s.m));
                const float2 q = __fmul2_rn(d, make_float2(c, c));
                S2[u & 1] = __fadd2_rn(S2[u & 1], make_float2(lp_ex2(q.x), lp_ex2(q.y)));
                if (TWO) {
                    const float2 r = __fmul2_rn(d, make_float2(kL2e, kL2e));
                    T2[u & 1] = __fadd2_rn(T2[u & 1], make_float2(lp_ex2(r.x), lp_ex2(r.y)));
                }
            }
        s.S = (S2[0].x + S2[0].y) + (S2[1].x + S2[1].y);
        s.S1 = (T2[0].x + T2[0].y) + (T2[1].x + T2[1].y);
    }, [&](float z, int64_t j) {
        if (REST && (entry_bits(j) & 1u)) return;
        if (!(z <= s.m)) rise(z);
        if (z == -INFINITY) return;
        s.S += lp_ex2((z - s.m) * c);
        if (TWO) s.S1 += lp_ex2((z - s.m) * kL2e);
    });
    if (s.m != s.m) s.S = s.S1 = s.m;
    s = join_parts<32, TWO>(s, c);
    if (lane == 0) sm.warp[warp] = s;
    if (warp < kEntryWarps) {
        float yt = y, xt = x;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            yt = max_nan(yt, __shfl_xor_sync(0xffffffffu, yt, o));
            xt = max_nan(xt, __shfl_xor_sync(0xffffffffu, xt, o));
        }
        if (lane == 0) sm.red[warp][0] = yt, sm.red[warp][1] = xt;
    }
    const bool any = __syncthreads_or(id >= 0);
    s = join_parts<N / 32, TWO>(sm.warp[tid & (N / 32 - 1)], c);
    if (cluster > 1) {
        __syncwarp();
        cluster_wait();  // CTA 0 has started
        if (tid == 0) {
            st_first(&sm.seg[part].m, s.m);
            st_first(&sm.seg[part].S, s.S);
            st_first(&sm.seg[part].S1, s.S1);
        }
        __syncwarp();
        cluster_sync();
        if (part) return;
        const int i = tid & (kMaxCluster - 1);
        s = join_parts<kMaxCluster, TWO>(i < cluster ? sm.seg[i] : Part{-INFINITY, 0.f, 0.f}, c);
    }
    float ytop = -INFINITY, xtop = -INFINITY;
#pragma unroll
    for (int w = 0; w < kEntryWarps; ++w) {
        ytop = max_nan(ytop, sm.red[w][0]);
        xtop = max_nan(xtop, sm.red[w][1]);
    }
    const float top = REST && any ? max_nan(s.m, xtop) : s.m;  // the row's largest logit
    const bool empty = top == -INFINITY;
    // the teacher's weights, and (each token once) the entries' e^x; a sum over the entries, the same in all threads
    auto over_entries = [&](float v, int which) {
        if (warp < kEntryWarps) {
#pragma unroll
            for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) sm.sums[warp][which] = v;
        }
    };
    auto total_of = [&](int which) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kEntryWarps; ++w) v += sm.sums[w][which];
        return v;
    };
    const float yref = ytop == -INFINITY ? 0.f : ytop, ly = teacher_log<REST>(y, yref, p.scale);
    const float e = id >= 0 ? expf(ly) : 0.f;
    over_entries(e, 0);
    if (REST) {
        bool first = id >= 0 && warp < kEntryWarps;
        for (int k = 0; k < tid && first; k += 4) first = k + before(same_of(sm.ids, k, id)) >= tid;
        over_entries(first ? brought(x, top, c) : 0.f, 1);
        if (TWO) over_entries(first ? brought(x, top, kL2e) : 0.f, 2);
    }
    __syncthreads();
    const float E = total_of(0), rest = s.S * brought(s.m, top, c), total = REST ? rest + total_of(1) : rest, log_total = logf(total);
    // sum p (log p - log q); each log p - log q is formed before it is weighed: their sum is far smaller than its parts.
    // (But for a logit that the scale takes out of fp32, the lowest numbers of a type, whose share may be small enough.)
    auto weighed = [&](float pk, float lp, float z, float l) {  // l: log q = scale (z - top) + l
        const float dz = z - top, dx = dz * p.scale;
        return dx == -INFINITY && dz != dx ? pk * p.scale * -dz : pk * (lp - (dx + l));
    };
    const float log_E = REST ? 0.f : logf(E), p_k = e == 0.f ? 0.f : REST ? e : e / E;
    over_entries(p_k == 0.f ? 0.f : weighed(p_k, ly - log_E, x, -log_total), 3);
    __syncthreads();
    if (tid) return;

    // ---- the row's scalars
    const float lse = empty ? -INFINITY : fmaf(top, p.scale, log_total);
    float log_total1 = p.scale == 1.f ? log_total : NAN;  // (not wanted, and not formed, at another scale)
    if (TWO) {
        const float r1 = s.S1 * brought(s.m, top, kL2e);
        log_total1 = logf(REST ? r1 + total_of(2) : r1);
    }
    Saved o{top, log_total * kL2e, log_total1 * kL2e, 0.f, 0.f, 1.f, 1.f, 0.f};
    float kl = any ? total_of(3) : 0.f;
    if (REST) {
        const bool others = s.m != -INFINITY;  // some logit outside the entries weighs something
        const float pr = E != E ? E : others ? fmaxf(1.f - E, 0.f) : 0.f, lr = logf(s.S);
        // log (p_r / q_r): of the quotient, whose logarithm is small, where q_r is a number of ordinary size
        const float qr = rest / total;
        if (any) kl += !(pr > 0.f) ? pr : qr >= 1e-30f || !(qr == qr) ? pr * logf(pr / qr) : weighed(pr, logf(pr), s.m, lr - log_total);
        o.W = E + pr;
        o.m = others ? s.m : 0.f;
        o.ml2 = others ? lr * kL2e : INFINITY;
        o.coef = any && others ? fmaf(o.W, qr, -pr) : 0.f;
    } else {
        o.m = yref;
        o.tl = any && E != 0.f ? log_E : INFINITY;
        if (!any || E == 0.f) o.coef = o.W = 0.f;
    }
    if (empty) kl = any && E > 0.f ? INFINITY : 0.f;  // no distribution: what the teacher expects is infinitely far
    p.kl[t] = kl;
    p.lse[t] = lse;
    if (p.logp) p.logp[t] = target < 0 ? 0.f : empty ? -INFINITY : zt - top - log_total1;
    float4* out = reinterpret_cast<float4*>(p.saved + t * 8);
    out[0] = make_float4(o.top, o.l2, o.l1, o.m);
    out[1] = make_float4(o.ml2, o.coef, o.W, o.tl);
}

template <bool F32, bool REST, bool TWO, int N>
static cudaError_t fwd_rows(const DistillParams& p, int c, cudaStream_t st) {
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim = {(unsigned)c, 1, 1};
    return launch_pdl(distill_fwd_kernel<F32, REST, TWO, N>, dim3((unsigned)(p.T * c)), dim3(N), 0, st, &a, c > 1 ? 1 : 0, p, c);
}
template <bool F32, bool REST, bool TWO>
static cudaError_t fwd_launch(const DistillParams& p, cudaStream_t st) {
    // As for the log probabilities: a row is shared by a cluster where there are fewer rows than places for CTAs.
    int c = 1;
    while (c < kMaxCluster && p.T * c * 2 <= 152 * 1024 / kThreads && p.V / (c * 2) >= kThreads * 8) c *= 2;
    // A row of its own has half the threads: eight rows an SM instead of four, so that the beginning and end of a row, in
    // which it reads little, are a smaller part of its time.  (8192 x 32000 97 us instead of 109, 1000 x 50257 27 instead of
    // 31, 4096 x 131072 the same; a row of eight CTAs 5.2 us instead of 4.7.)
    return c == 1 ? fwd_rows<F32, REST, TWO, kThreads / 2>(p, c, st) : fwd_rows<F32, REST, TWO, kThreads>(p, c, st);
}
template <bool F32>
static cudaError_t fwd_forms(const DistillParams& p, cudaStream_t st) {
    const bool two = p.scale != 1.f && p.targets;
    if (p.rest) return two ? fwd_launch<F32, true, true>(p, st) : fwd_launch<F32, true, false>(p, st);
    return two ? fwd_launch<F32, false, true>(p, st) : fwd_launch<F32, false, false>(p, st);
}
cudaError_t launch_distill_fwd(const DistillParams& p, cudaStream_t st) {
    return p.f32 ? fwd_forms<true>(p, st) : fwd_forms<false>(p, st);
}

// ------------------------------------------------------------------ backward
// 16-byte vectors of a thread: a CTA takes a stretch of 1024 of them.  Small CTAs, many of them: each waits for its entries
// and their logits between its loads and its stores, and once more before the entries' own gradients.  (4096 x 131072 and
// 8192 x 32000: 128 threads of 8 vectors 322 and 173 us, of 10 320 and 172 but 2048 x 32000 44 instead of 42, of 6 337 and 185.
// With a slower search for tokens given twice, one entry a step, 8 vectors took 345 and 182, 256 threads of them 378 and 191,
// of 4 392 and 230, 512 of 8 409 and 216.)
constexpr int kDbThreads = 128, kDbVecs = 8;
static_assert(kDbThreads >= kMaxEntries, "a thread an entry");

template <bool F32, bool REST, bool TWO>
__global__ void __launch_bounds__(kDbThreads) distill_bwd_kernel(const __grid_constant__ DistillParams p, unsigned per_row) {
    __shared__ __align__(16) int ids[kMaxEntries];
    __shared__ float ps[kMaxEntries];
    griddep_launch_dependents();
    griddep_wait();
    constexpr int W = Row<F32>::kVec;
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x / per_row;
    const Row<F32> row{static_cast<const char*>(p.logits) + t * p.ld * (F32 ? 4 : 2)};
    char* out = static_cast<char*>(p.dlogits) + t * p.ld_out * (F32 ? 4 : 2);
    // stretches begin at the row's first 16-byte boundary; the first CTA also takes what is before it
    const int64_t a = min(p.V, row.head(0)), n = (int64_t)kDbThreads * kDbVecs * W;
    const int64_t s0 = a + (blockIdx.x - t * per_row) * n, s1 = min(p.V, s0 + n), from = s0 == a ? 0 : s0;
    const bool alike = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.p)) & 15) == 0;
    const int64_t at = hard_target(p, t);
    const float gk = p.dkl ? p.dkl[t] * p.scale : 0.f, gh = p.dlogp && at >= 0 ? p.dlogp[t] : 0.f;
    auto put = [&](int64_t j, float d) {
        if (F32) reinterpret_cast<float*>(out)[j] = d;
        else reinterpret_cast<uint16_t*>(out)[j] = (uint16_t)(pack_bf16x2(d, 0.f) & 0xFFFFu);
    };
    const float4 s_a = reinterpret_cast<const float4*>(p.saved + t * 8)[0], s_b = reinterpret_cast<const float4*>(p.saved + t * 8)[1];
    const Saved s{s_a.x, s_a.y, s_a.z, s_a.w, s_b.x, s_b.y, s_b.z, s_b.w};
    const float m = REST ? s.m : s.top, ml2 = REST ? s.ml2 : s.l2;  // of the logits that coef is a factor of
    const float c = p.scale * kL2e;
    const bool none = (gk == 0.f && gh == 0.f) || s.top == -INFINITY;  // the row's gradient is 0, whatever it holds
    uint4 raw[kDbVecs];
    if (alike && !none)
#pragma unroll
        for (int u = 0; u < kDbVecs; ++u) {
            const int64_t j = s0 + (u * kDbThreads + tid) * W;
            if (j + W <= s1) raw[u] = *reinterpret_cast<const uint4*>(row.p + j * (F32 ? 4 : 2));
        }
    // the entries of this stretch: their logits are read before anything is written over them.  (With rest the others'
    // share of e^x says nothing of them, so a row whose own log probability alone has a gradient asks for them too; what
    // the teacher thinks of them has no part in it then.)
    int id = -1;
    float x = 0.f;
    if (!none) {
        float pk = 0.f;
        if (tid < p.K && (REST || gk != 0.f)) {
            id = id_at(p, t, tid);
            if (id < from || id >= s1) id = -1;
            if (id >= 0) {
                x = row.at(id);
                // (with rest tl is 0, but this load then waits for the row's scalars, behind the stretch's own loads: 4096 x
                // 131072 321 us instead of 336)
                const float e = expf(teacher_log<REST>(teacher_at(p, t, tid), s.m, p.scale) - s.tl);
                pk = gk == 0.f ? 0.f : e;
            }
        }
        if (tid < kMaxEntries) ids[tid] = id, ps[tid] = pk;
        __syncthreads();
    }
    // with one scale, a token's own softmax outside the entries is their share of it times e^{(z - m)} / sum
    const float qr = !REST ? 1.f : s.ml2 == INFINITY ? 0.f : lp_ex2(fmaf(s.m - s.top, c, s.ml2 - s.l2));
    const float coef = gk == 0.f ? 0.f : s.coef, k0 = TWO ? gk * coef : fmaf(gk, coef, -gh * qr), k1 = -gh;
    auto soft = [&](float z) {
        float d = k0 * lp_ex2(fmaf(z - m, c, -ml2));
        if (TWO) d = fmaf(k1, lp_ex2(fmaf(z - s.top, kL2e, -s.l1)), d);
        return d;
    };
    auto grad = [&](int64_t j) { return none ? 0.f : soft(row.at(j)) + (j == at ? gh : 0.f); };
    if (s0 == a && tid < a) put(tid, grad(tid));
    if (alike) {
#pragma unroll
        for (int u = 0; u < kDbVecs; ++u) {
            const int64_t j = s0 + (u * kDbThreads + tid) * W;
            if (j + W <= s1) {
                float d[W];
                if (none) {
#pragma unroll
                    for (int e = 0; e < W; ++e) d[e] = 0.f;
                } else {
                    const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                    for (int e = 0; e < W; e += 2) {
                        const float2 z = make_float2(logit<F32>(w, e), logit<F32>(w, e + 1));
                        const float2 q = __ffma2_rn(__fadd2_rn(z, make_float2(-m, -m)), make_float2(c, c), make_float2(-ml2, -ml2));
                        float2 r = __fmul2_rn(make_float2(lp_ex2(q.x), lp_ex2(q.y)), make_float2(k0, k0));
                        if (TWO) {
                            const float2 l1 = __ffma2_rn(__fadd2_rn(z, make_float2(-s.top, -s.top)), make_float2(kL2e, kL2e),
                                                         make_float2(-s.l1, -s.l1));
                            r = __ffma2_rn(make_float2(k1, k1), make_float2(lp_ex2(l1.x), lp_ex2(l1.y)), r);
                        }
                        d[e] = r.x;
                        d[e + 1] = r.y;
                    }
                    if ((uint64_t)(at - j) < (uint64_t)W) {  // the target is one of these
#pragma unroll
                        for (int e = 0; e < W; ++e) d[e] += at - j == e ? gh : 0.f;
                    }
                }
                uint4 v;
                if (F32) v = make_uint4(__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3]));
                else v = make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]), pack_bf16x2(d[W - 4], d[W - 3]),
                                    pack_bf16x2(d[W - 2], d[W - 1]));
                *reinterpret_cast<uint4*>(out + j * (F32 ? 4 : 2)) = v;
            } else {
                for (int64_t i = j; i < s1; ++i) put(i, grad(i));
            }
        }
    } else {  // the rows of the two tensors lie differently: element by element
        for (int64_t j = s0 + tid; j < s1; j += kDbThreads) put(j, grad(j));
    }
    if (none) return;
    __syncthreads();
    if (id < 0) return;
    float pk = 0.f;
    for (int k = 0; k < p.K; k += 4) {
        uint32_t same = same_of(ids, k, id);
        if (same && k + before(same) < tid) return;  // (a token given twice is its first entry's)
        for (; same; same &= same - 1) pk += ps[k + before(same)];
    }
    const float q = lp_ex2(fmaf(x - s.top, c, -s.l2));
    float d = (gk == 0.f ? 0.f : gk * fmaf(s.W, q, -pk)) + (id == at ? gh : 0.f);
    if (gh != 0.f) d = fmaf(-gh, TWO ? lp_ex2(fmaf(x - s.top, kL2e, -s.l1)) : q, d);
    put(id, d);
}

template <bool F32, bool REST, bool TWO>
static cudaError_t bwd_launch(const DistillParams& p, cudaStream_t st) {
    const int64_t n = (int64_t)kDbThreads * kDbVecs * Row<F32>::kVec;
    const int64_t per_row = (p.V + n - 1) / n;
    if (p.T * per_row > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(distill_bwd_kernel<F32, REST, TWO>, dim3((unsigned)(p.T * per_row)), dim3(kDbThreads), 0, st, nullptr, 0, p,
                      (unsigned)per_row);
}
template <bool F32>
static cudaError_t bwd_forms(const DistillParams& p, cudaStream_t st) {
    const bool two = p.scale != 1.f && p.dlogp;
    if (p.rest) return two ? bwd_launch<F32, true, true>(p, st) : bwd_launch<F32, true, false>(p, st);
    return two ? bwd_launch<F32, false, true>(p, st) : bwd_launch<F32, false, false>(p, st);
}
cudaError_t launch_distill_bwd(const DistillParams& p, cudaStream_t st) {
    return p.f32 ? bwd_forms<true>(p, st) : bwd_forms<false>(p, st);
}

}  // namespace lm
