// Log probabilities of given tokens (include/lora_layer.h), with entropy and top alternatives.
//   m = max x,  S = sum e^{x-m},  w = sum e^{x-m} (x-m):  lse = m + log S,  H = log S - w / S
// One CTA per row, a pass for the maximum, one for the sums, and one for each alternative.
#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

constexpr int kLpThreads = 512;

__device__ __forceinline__ float logit(const LogprobParams& p, int64_t at) {
    return p.f32 ? static_cast<const float*>(p.logits)[at]
                 : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p.logits)[at] << 16);
}
__device__ __forceinline__ int64_t target_of(const LogprobParams& p, int64_t t) {
    const int64_t v = p.i64 ? static_cast<const int64_t*>(p.targets)[t] : static_cast<const int32_t*>(p.targets)[t];
    return v >= 0 && v < p.V ? v : -1;
}
// scale * logit, rounded by itself: forward and backward then take the same number, and what cancels
// in one cancels in the other
__device__ __forceinline__ float scaled(const LogprobParams& p, int64_t at) { return __fmul_rn(logit(p, at), p.scale); }
// Larger keys for larger logits; +0 and -0 are equal, every NaN is the largest.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
// (key, index) as one number: larger logit first, then the lower index
__device__ __forceinline__ uint64_t rank_of(float x, int64_t j) {
    return ((uint64_t)order_key(x) << 32) | (0xFFFFFFFFu - (uint32_t)j);
}

template <typename T, typename F>
__device__ T block_all(T x, F op) {
    __shared__ T part[kLpThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    T s = part[0];
    for (int i = 1; i < kLpThreads / 32; ++i) s = op(s, part[i]);
    return s;
}

__device__ __forceinline__ float max_nan(float a, float b) { return (a != a || a > b) ? a : b; }  // NaN wins

__global__ void __launch_bounds__(kLpThreads) logprob_fwd_kernel(const __grid_constant__ LogprobParams p) {
    const int64_t t = blockIdx.x, row = t * p.ld;
    float m = -INFINITY;
    for (int64_t j = threadIdx.x; j < p.V; j += kLpThreads) m = max_nan(scaled(p, row + j), m);
    m = block_all(m, [](float a, float b) { return max_nan(a, b); });
    const float m0 = m == -INFINITY ? 0.f : m;
    float S = 0.f, w = 0.f;
    for (int64_t j = threadIdx.x; j < p.V; j += kLpThreads) {
        const float x = scaled(p, row + j) - m0, e = expf(x);
        S += e;
        if (x != -INFINITY) w += e * x;
    }
    auto add = [](float a, float b) { return a + b; };
    S = block_all(S, add);
    w = block_all(w, add);
    const float lse = m == -INFINITY ? -INFINITY : m + logf(S);
    auto logp = [&](int64_t j) { return m == -INFINITY ? -INFINITY : scaled(p, row + j) - lse; };
    if (threadIdx.x == 0) {
        const int64_t at = target_of(p, t);
        p.lse[t] = lse;
        p.logp[t] = at < 0 ? 0.f : logp(at);
        if (p.entropy) p.entropy[t] = m == -INFINITY ? 0.f : logf(S) - w / S;
    }
    uint64_t last = ~0ull;
    for (int i = 0; i < p.k; ++i) {
        uint64_t best = 0;
        for (int64_t j = threadIdx.x; j < p.V; j += kLpThreads) {
            const uint64_t r = rank_of(logit(p, row + j), j);
            if (r < last && r > best) best = r;
        }
        last = block_all(best, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
        if (threadIdx.x == 0) {
            const uint32_t j = 0xFFFFFFFFu - (uint32_t)last;
            p.top_ids[t * p.k + i] = (int32_t)j;
            p.top_logp[t * p.k + i] = logp(j);
        }
    }
}

cudaError_t launch_logprob_fwd(const LogprobParams& p, cudaStream_t st) {
    logprob_fwd_kernel<<<(unsigned)p.T, kLpThreads, 0, st>>>(p);
    return cudaGetLastError();
}

__global__ void __launch_bounds__(kLpThreads) logprob_bwd_kernel(const __grid_constant__ LogprobParams p) {
    const int64_t t = blockIdx.x, row = t * p.ld, at = target_of(p, t);
    const float lse = p.lse_in[t], gH = p.dentropy ? p.dentropy[t] : 0.f, H = p.dentropy ? p.entropy_in[t] : 0.f;
    const float g = p.dlogp && at >= 0 ? p.dlogp[t] : 0.f;
    for (int64_t j = threadIdx.x; j < p.V; j += kLpThreads) {
        const float lp = scaled(p, row + j) - lse;
        const float e = expf(lp);
        float d = lse == -INFINITY || e == 0.f ? 0.f : -e * (g + gH * (lp + H));
        if (j == at && lse != -INFINITY) d += g;
        d *= p.scale;
        const int64_t o = t * p.ld_out + j;
        if (p.f32) static_cast<float*>(p.dlogits)[o] = d;
        else static_cast<uint16_t*>(p.dlogits)[o] = (uint16_t)(pack_bf16x2(d, 0.f) & 0xFFFFu);
    }
}

cudaError_t launch_logprob_bwd(const LogprobParams& p, cudaStream_t st) {
    logprob_bwd_kernel<<<(unsigned)p.T, kLpThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace lm
