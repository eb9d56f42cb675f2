// Attention over packed documents (include/lora_layer.h): who sees whom, and the backward with one
// warp per row, the head's dimensions spread over its lanes.
//   P = e^{s - lse}, dz = P (dO.v - delta) (1 - (u/cap)^2), delta = dO.O
// Bound by the five shuffles that join each dot product.
#include "lm_attn.cuh"

namespace lm {

constexpr int kPerLane = 4;  // d <= 128

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ------------------------------------------------------------------ who sees whom
__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

__global__ void __launch_bounds__(256) attn_ranges_kernel(const __grid_constant__ lm_attn a, int T, TokRange* out) {
    griddep_launch_dependents();
    griddep_wait();
    const int t = blockIdx.x * blockDim.x + threadIdx.x;
    if (t >= T) return;
    // the document: the largest m with cu[m] <= t (empty documents before it are skipped)
    int m = 0, over = a.n_docs;
    while (m + 1 < over) {
        const int mid = (m + over) >> 1;
        if (a.cu_docs[mid] <= t) m = mid;
        else over = mid;
    }
    const int s = clampi(a.cu_docs[m], 0, T), e = clampi(a.cu_docs[m + 1], 0, T);
    TokRange r{t, t, t, t};  // padding: empty intervals at t, which keeps all four non-decreasing over the tokens
    if (s <= t && t < e) r = range_in(t, s, e, a.prefix ? clampi(a.prefix[m], 0, e - s) : 0, T, a.causal, a.window);
    out[t] = r;
}

cudaError_t launch_attn_ranges(const lm_attn& a, int64_t T, TokRange* out, cudaStream_t st) {
    return launch_pdl(attn_ranges_kernel, dim3((unsigned)((T + 255) / 256)), dim3(256), 0, st, nullptr, 0, a, (int)T, out);
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
    const TokRange r = tok_range(p, i);
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
    const TokRange r = tok_range(p, j);
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
