// Cross attention forward (include/lora_layer.h): queries of T tokens, keys and values of another tensor of Tk.  The
// backward is in lm_cross_bwd.cu.
// The kernels are attention's own (lm_attn_fwd.cuh, lm_attn_bwd.cuh); what a query sees is an interval of keys whose
// ends do not decrease here too, read from tables of its own.  Few queries have another form of the forward: the rows
// of a tile are the heads of a group, token by token, so a key tile is read once for all of them, and the keys
// are dealt out in parts, one CTA each; a second kernel joins the parts' sums in order.
#include <algorithm>

#include "lm_attn_fwd.cuh"

namespace lm {

// ------------------------------------------------------------------ who sees whom
// The largest m with cu[m] <= t, 0 where there is none.
__device__ __forceinline__ int segment_of(const int32_t* cu, int n, int t) {
    int m = 0, over = n;
    while (m + 1 < over) {
        const int mid = (m + over) >> 1;
        if (cu[mid] <= t) m = mid;
        else over = mid;
    }
    return m;
}
// A CTA takes a tile of queries, or one of keys.  What sees or is seen by nothing gets an empty interval at a place
// that keeps the ends from decreasing.
constexpr int kStaged = 2048;
__global__ void __launch_bounds__(kTile) cross_ranges_kernel(const __grid_constant__ lm_cross a, int Tq, int Tk, CrossTables out) {
    griddep_launch_dependents();
    griddep_wait();
    const int qtiles = (Tq + kTile - 1) / kTile, n = a.n_docs;
    const bool key = (int)blockIdx.x >= qtiles;
    const int tile = (int)blockIdx.x - (key ? qtiles : 0), t = tile * kTile + threadIdx.x, T = key ? Tk : Tq;
    const int32_t* cu = key ? a.cu_k : a.cu_q;
    __shared__ int32_t own[kStaged];
    if (n < kStaged) {  // (all loads at once, and the search's steps in shared memory)
        for (int i = threadIdx.x; i <= n; i += kTile) own[i] = cu[i];
        __syncthreads();
        cu = own;
    }
    bool seen = true;  // (rows past the end are zeros)
    if (t < T) {
        const int m = segment_of(cu, n, t);
        const int qs = clampi(a.cu_q[m], 0, Tq), qe = clampi(a.cu_q[m + 1], qs, Tq);
        const int ks = clampi(a.cu_k[m], 0, Tk), ke = clampi(a.cu_k[m + 1], ks, Tk);
        const int kl = ks + (a.k_len ? clampi(a.k_len[m], 0, ke - ks) : ke - ks);
        int2 r;
        if (key) r = t < ks ? make_int2(qs, qs) : t >= kl ? make_int2(qe, qe) : make_int2(qs, qe);
        else r = t < qs ? make_int2(ks, ks) : t >= qe ? make_int2(ke, ke) : make_int2(ks, kl);
        (key ? out.krange : out.qrange)[t] = r;
        seen = r.x < r.y;
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, seen);
    if ((threadIdx.x & 31) == 0) reinterpret_cast<uint32_t*>(key ? out.kseen : out.qseen)[tile * 4 + (threadIdx.x >> 5)] = bits;
}
cudaError_t launch_cross_ranges(const lm_cross& a, int64_t Tq, int64_t Tk, const CrossTables& t, cudaStream_t st) {
    const unsigned tiles = (unsigned)((Tq + kTile - 1) / kTile + (Tk + kTile - 1) / kTile);
    return launch_pdl(cross_ranges_kernel, dim3(tiles), dim3(kTile), 0, st, nullptr, 0, a, (int)Tq, (int)Tk, t);
}

__global__ void __launch_bounds__(256) fill_kernel(float* out, int64_t n, float v) {
    griddep_launch_dependents();
    griddep_wait();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) out[i] = v;
}
cudaError_t launch_fill(float* out, int64_t n, float v, cudaStream_t st) {
    return launch_pdl(fill_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, nullptr, 0, out, n, v);
}

// ------------------------------------------------------------------ few queries
FewPlan plan_few(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk) {
    const int group = hq / hk;
    FewPlan P{0, 0, 0};
    if (group > kTile || Tq == 0 || Tk == 0) return P;
    P.tokens = kTile / group;
    const int64_t items = (Tq + P.tokens - 1) / P.tokens * hk, tiles = (Tk + kTile - 1) / kTile;
    if (items * 2 > kCrossSms) return P;
    // each CTA has two accumulators, which take its tiles in turn
    P.splits = (int32_t)std::min<int64_t>(kCrossSms / items, (tiles + 1) / 2);
    P.parts = tiles > 1 ? 2 * P.splits : 1;
    return P;
}

// The parts' maxima (in units of log 2), sums and unnormalised rows to O and lse: a CTA a row, a warp every
// WARPS-th part, four dims a lane.
constexpr int kMostParts = 2 * kCrossSms, kAtOnce = 5;
template <bool CAP, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) cross_join_kernel(const __grid_constant__ AttnParams p) {
    __shared__ float2 part[kMostParts];
    __shared__ float4 sum[WARPS][32];
    __shared__ float sum_l[WARPS];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t rows = (int64_t)p.T * p.hq, row = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane * 4;
    // every part's m and l, in order over the lanes (all warps do the same); a part that saw nothing has l = 0.
    // (Short loops: code that runs once is as slow as it is long.)
    const float2* ml = p.part_ml + row;
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int s = lane; s < p.parts; s += 32) {
        const float2 v = ml[s * rows];
        if (warp == 0) part[s] = v;
        if (v.y != 0.f) m = fmaxf(m, v.x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* src = p.part_o + row * p.d + c;
#pragma unroll 1
    for (int s0 = warp; s0 < p.parts; s0 += WARPS * kAtOnce) {
        float4 v[kAtOnce];
        float x[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {  // (all asked for before the first is waited for)
            const int s = s0 + i * WARPS;
            const float2 q = s < p.parts ? part[s] : make_float2(0.f, 0.f);
            x[i] = q.y == 0.f ? 0.f : ex2(q.x - m);
            l += q.y == 0.f ? 0.f : q.y * x[i];
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x[i] != 0.f && c < p.d) v[i] = *reinterpret_cast<const float4*>(src + s * rows * p.d);  // (0: no row written, or too little to count)
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            o.x = fmaf(v[i].x, x[i], o.x), o.y = fmaf(v[i].y, x[i], o.y), o.z = fmaf(v[i].z, x[i], o.z), o.w = fmaf(v[i].w, x[i], o.w);
    }
    if (lane == 0) sum_l[warp] = l;
    sum[warp][lane] = o;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
        const float4 v = sum[w][lane];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
        l += sum_l[w];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (lane == 0) {
        const int64_t i = row / p.hq, h = row - i * p.hq;
        p.lse[h * p.T + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2 + (CAP ? p.cap : 0.f);
    }
    const float x[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    const uint32_t v0 = pack_bf16x2(x[0], x[1]), v1 = pack_bf16x2(x[2], x[3]);
    if (c < p.d) *reinterpret_cast<uint2*>(p.out + row * p.d + c) = make_uint2(v0, v1);
    if (p.out_lo && c < p.d16) {
        const uint32_t b[4] = {v0 & 0xFFFFu, v0 >> 16, v1 & 0xFFFFu, v1 >> 16};
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w |= (uint32_t)(bits_left(x[e], b[e]) & 255) << (8 * e);
        *reinterpret_cast<uint32_t*>(p.out_lo + row * p.d16 + c) = w;
    }
    if (!p.qrange) return;
    const float zero = fmaf(x[0], 0.f, fmaf(x[1], 0.f, fmaf(x[2], 0.f, x[3] * 0.f)));
    if (__any_sync(0xffffffffu, c < p.d && zero != zero)) {  // (another document's values?)
        const int i = (int)(row / p.hq);
        __syncwarp();
        if (!keys_of<ATTN_FEW>(p, i / p.rows * p.rows, p.rows).alike) own_row<CAP ? ATTN_CAP : ATTN_PLAIN, 4>(p, i, (int)(row % p.hq), 0);
    }
}

// ------------------------------------------------------------------ launches
template <int DP, int FORM>
static cudaError_t fwd_modes(const AttnParams& p, const FwdMaps& maps, int sms, cudaStream_t st) {
    return p.cap > 0.f ? launch_fwd<DP, ATTN_CAP, FORM>(p, maps, sms, st) : launch_fwd<DP, ATTN_PLAIN, FORM>(p, maps, sms, st);
}
template <int FORM>
static cudaError_t fwd_dims(const AttnParams& p, const FwdMaps& maps, int sms, cudaStream_t st) {
    return p.d <= 64 ? fwd_modes<64, FORM>(p, maps, sms, st) : fwd_modes<128, FORM>(p, maps, sms, st);
}

template <int WARPS>
static cudaError_t join(const AttnParams& p, int rows, cudaStream_t st) {
    const dim3 grid((unsigned)rows), block(WARPS * 32);
    return p.cap > 0.f ? launch_pdl(cross_join_kernel<true, WARPS>, grid, block, 0, st, nullptr, 0, p)
                       : launch_pdl(cross_join_kernel<false, WARPS>, grid, block, 0, st, nullptr, 0, p);
}

lm_status launch_cross_fwd(const AttnParams& given, int sms, cudaStream_t st) {
    FwdMaps maps;
    AttnParams p = given;
    const int group = p.hq / p.hk;
    const bool few = p.splits > 0;
    if (!few) p.rows = (int64_t)((p.T + 2 * kTile - 1) / (2 * kTile)) * p.hq * 2 <= sms ? kTile : 2 * kTile;
    const lm_heads q{p.q.p, p.q.ts, p.q.hs}, k{p.k.p, p.k.ts, p.k.hs}, v{p.v.p, p.v.ts, p.v.hs};
    lm_status s = few ? encode_heads(&maps.q, q, p.T, p.hq, p.d, p.rows, group) : encode_heads(&maps.q, q, p.T, p.hq, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps.k, k, p.Tk, p.hk, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps.v, v, p.Tk, p.hk, p.d, kTile);
    if (s != LM_OK) return s;
    cudaError_t e = few ? fwd_dims<ATTN_FEW>(p, maps, sms, st) : fwd_dims<ATTN_CROSS>(p, maps, sms, st);
    if (e == cudaSuccess && p.splits > 0 && p.parts > 1) {
        LaunchTag tag("cross.join", st);
        // eight warps a row where there are fewer rows than SMs (one token on 8192 states, 38 parts: 14.4 us for the call
        // instead of 15.4 with four), else four (2048 rows of 18 parts, most of them empty: 48 us instead of 50)
        const int rows = p.T * p.hq;  // (items are at most 76, of at most 128 rows)
        e = rows <= kCrossSms ? join<8>(p, rows, st) : join<4>(p, rows, st);
    }
    return e == cudaSuccess ? LM_OK : report_error(LM_ERR_CUDA, "cross attention forward launch: %s", cudaGetErrorString(e));
}

}  // namespace lm
