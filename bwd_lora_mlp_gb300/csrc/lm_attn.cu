// Attention over packed documents (include/lora_layer.h), forward and backward: one warp per row,
// the head's dimensions spread over its lanes.
//   forward   m, l, o updated key by key:  m' = max(m, s), o = o e^{m-m'} + e^{s-m'} v
//   backward  P = e^{s - lse}, dz = P (dO.v - delta) (1 - (u/cap)^2), delta = dO.O
// Bound by the five shuffles that join each dot product.
#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

constexpr int kPerLane = 4;  // d <= 128

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ------------------------------------------------------------------ who sees whom
__device__ __forceinline__ int clampi(int64_t v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : (int)v; }

__global__ void attn_ranges_kernel(lm_attn a, int T, TokRange* out) {
    const int t = blockIdx.x * blockDim.x + threadIdx.x;
    if (t >= T) return;
    int s = 0, e = T, pre = 0;
    bool in = true;
    if (a.cu_docs) {
        // the last document that begins at or before t and is not empty there: the largest m with cu[m] <= t
        int lo = 0, hi = a.n_docs;  // cu[lo] <= t < cu[hi] where t is inside
        while (lo + 1 < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.cu_docs[mid] <= t) lo = mid; else hi = mid;
        }
        s = clampi(a.cu_docs[lo], 0, T);
        e = clampi(a.cu_docs[lo + 1], 0, T);
        in = s <= t && t < e;
        if (in && a.prefix) pre = clampi(a.prefix[lo], 0, e - s);
    }
    TokRange r;
    if (!in) {  // padding: empty intervals at t, which keeps lo and hi non-decreasing over the tokens
        r.lo = r.hi = r.qlo = r.qhi = t;
    } else {
        const int W = a.window > 0 && a.window < T ? a.window : T;
        r.lo = max(s, t - W + 1);
        r.hi = a.causal ? min(max(t + 1, s + pre), t + W) : min(e, t + W);
        r.qlo = a.causal && t >= s + pre ? t : max(s, t - W + 1);
        r.qhi = min(e, t + W);
    }
    out[t] = r;
}

cudaError_t launch_attn_ranges(const lm_attn& a, int64_t T, TokRange* out, cudaStream_t st) {
    attn_ranges_kernel<<<(unsigned)((T + 255) / 256), 256, 0, st>>>(a, (int)T, out);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ one score
struct Lanes {
    float x[kPerLane];
};
__device__ __forceinline__ Lanes load_row(const uint16_t* p, int d, int lane) {
    Lanes r;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int c = lane + 32 * i;
        r.x[i] = c < d ? __uint_as_float((uint32_t)p[c] << 16) : 0.f;
    }
    return r;
}
__device__ __forceinline__ float dot(const Lanes& a, const Lanes& b) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) s += a.x[i] * b.x[i];
    return warp_sum(s);
}
// s from q.k, and du/dz
__device__ __forceinline__ float score(const AttnParams& p, float qk, float slope, int dist, float& bend) {
    float u = qk * p.scale;
    bend = 1.f;
    if (p.cap > 0.f) {
        const float t = tanhf(u / p.cap);
        u = p.cap * t;
        bend = 1.f - t * t;
    }
    return u - slope * (float)abs(dist);
}
__device__ __forceinline__ const uint16_t* row_of(const HeadsIn& t, int64_t tok, int64_t head) {
    return t.p + tok * t.ts + head * t.hs;
}
__device__ __forceinline__ void store_row(uint16_t* p, const Lanes& r, float f, int d, int lane) {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int c = lane + 32 * i;
        if (c < d) p[c] = (uint16_t)(pack_bf16x2(r.x[i] * f, 0.f) & 0xFFFFu);
    }
}

// The eight bits of a value's fp32 pattern that its bf16 rounding leaves out.
__device__ __forceinline__ int bits_left(float x) {
    const uint32_t hi = (pack_bf16x2(x, 0.f) & 0xFFFFu) << 16;
    return min((int32_t)(__float_as_uint(x) - hi) >> 8, 127);
}

// ------------------------------------------------------------------ forward
__global__ void __launch_bounds__(256) attn_fwd_kernel(const __grid_constant__ AttnParams p) {
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5), h = blockIdx.y, g = h / (p.hq / p.hk);
    if (i >= p.T) return;
    const TokRange r = p.rng[i];
    const Lanes q = load_row(row_of(p.q, i, h), p.d, lane);
    const float slope = p.slopes ? p.slopes[h] : 0.f;
    float m = -INFINITY, l = 0.f, bend;
    Lanes o{};
    for (int j = r.lo; j < r.hi; ++j) {
        const float s = score(p, dot(q, load_row(row_of(p.k, j, g), p.d, lane)), slope, i - j, bend);
        const Lanes v = load_row(row_of(p.v, j, g), p.d, lane);
        const float mn = fmaxf(m, s), f = expf(m - mn), e = expf(s - mn);
        l = l * f + e;
#pragma unroll
        for (int c = 0; c < kPerLane; ++c) o.x[c] = o.x[c] * f + e * v.x[c];
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int64_t at = ((int64_t)i * p.hq + h) * p.d;
    store_row(p.out + at, o, inv, p.d, lane);
    if (p.out_lo)
        for (int c = 0; c < kPerLane; ++c)
            if (lane + 32 * c < p.d) p.out_lo[at + lane + 32 * c] = (int8_t)bits_left(o.x[c] * inv);
    if (lane == 0) p.lse[(int64_t)h * p.T + i] = l > 0.f ? m + logf(l) : -INFINITY;
}

cudaError_t launch_attn_fwd(const AttnParams& p, cudaStream_t st) {
    attn_fwd_kernel<<<dim3((p.T + 7) / 8, p.hq), 256, 0, st>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ backward
// delta_i = dO_i . O_i; 0 where nothing is seen, whatever dO holds there
__global__ void __launch_bounds__(256) attn_delta_kernel(const __grid_constant__ AttnParams p, float* delta) {
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5), h = blockIdx.y;
    if (i >= p.T) return;
    const int64_t at = ((int64_t)i * p.hq + h) * p.d;
    Lanes o = load_row(p.O + at, p.d, lane);
    if (p.O_lo)
        for (int c = 0; c < kPerLane; ++c)
            if (lane + 32 * c < p.d) o.x[c] = __uint_as_float(__float_as_uint(o.x[c]) + ((int32_t)p.O_lo[at + lane + 32 * c] << 8));
    const float s = dot(load_row(row_of(p.dO, i, h), p.d, lane), o);
    if (lane == 0) delta[(int64_t)h * p.T + i] = s;
}

cudaError_t launch_attn_delta(const AttnParams& p, float* delta, cudaStream_t st) {
    attn_delta_kernel<<<dim3((p.T + 7) / 8, p.hq), 256, 0, st>>>(p, delta);
    return cudaGetLastError();
}

__global__ void __launch_bounds__(256) attn_dq_kernel(const __grid_constant__ AttnParams p) {
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5), h = blockIdx.y, g = h / (p.hq / p.hk);
    if (i >= p.T) return;
    const TokRange r = p.rng[i];
    const Lanes q = load_row(row_of(p.q, i, h), p.d, lane), dO = load_row(row_of(p.dO, i, h), p.d, lane);
    const float slope = p.slopes ? p.slopes[h] : 0.f;
    const float lse = p.lse_in[(int64_t)h * p.T + i], delta = p.delta[(int64_t)h * p.T + i];
    Lanes dq{};
    for (int j = r.lo; j < r.hi; ++j) {
        const Lanes k = load_row(row_of(p.k, j, g), p.d, lane);
        float bend;
        const float s = score(p, dot(q, k), slope, i - j, bend);
        const float dz = expf(s - lse) * (dot(dO, load_row(row_of(p.v, j, g), p.d, lane)) - delta) * bend;
#pragma unroll
        for (int c = 0; c < kPerLane; ++c) dq.x[c] += dz * k.x[c];
    }
    store_row(p.out + ((int64_t)i * p.hq + h) * p.d, dq, p.scale, p.d, lane);
}

cudaError_t launch_attn_dq(const AttnParams& p, cudaStream_t st) {
    attn_dq_kernel<<<dim3((p.T + 7) / 8, p.hq), 256, 0, st>>>(p);
    return cudaGetLastError();
}

__global__ void __launch_bounds__(256) attn_dkv_kernel(const __grid_constant__ AttnParams p) {
    const int lane = threadIdx.x & 31;
    const int j = blockIdx.x * 8 + (threadIdx.x >> 5), g = blockIdx.y, n = p.hq / p.hk;
    if (j >= p.T) return;
    const TokRange r = p.rng[j];
    const Lanes k = load_row(row_of(p.k, j, g), p.d, lane), v = load_row(row_of(p.v, j, g), p.d, lane);
    Lanes dk{}, dv{};
    for (int h = g * n; h < (g + 1) * n; ++h) {
        const float slope = p.slopes ? p.slopes[h] : 0.f;
        for (int i = r.qlo; i < r.qhi; ++i) {
            const Lanes q = load_row(row_of(p.q, i, h), p.d, lane), dO = load_row(row_of(p.dO, i, h), p.d, lane);
            float bend;
            const float s = score(p, dot(q, k), slope, i - j, bend);
            const float P = expf(s - p.lse_in[(int64_t)h * p.T + i]);
            const float dz = P * (dot(dO, v) - p.delta[(int64_t)h * p.T + i]) * bend;
#pragma unroll
            for (int c = 0; c < kPerLane; ++c) {
                dk.x[c] += dz * q.x[c];
                dv.x[c] += P * dO.x[c];
            }
        }
    }
    store_row(p.dK + ((int64_t)j * p.hk + g) * p.d, dk, p.scale, p.d, lane);
    store_row(p.dV + ((int64_t)j * p.hk + g) * p.d, dv, 1.f, p.d, lane);
}

cudaError_t launch_attn_dkv(const AttnParams& p, cudaStream_t st) {
    attn_dkv_kernel<<<dim3((p.T + 7) / 8, p.hk), 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace lm
