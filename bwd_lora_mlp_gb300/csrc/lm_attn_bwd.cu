// Attention backward over packed documents: delta, and the launches of the other kernels (lm_attn_bwd.cuh).
#include "lm_attn_bwd.cuh"

namespace lm {

// ------------------------------------------------------------------ delta, and lse in the exponent's units
// A CTA takes 16 tokens and kDeltaHeads heads: 16 threads a token, 8 dims each, all heads' loads in flight at
// once.  The results lie by head, so they are exchanged and leave 16 tokens at a time.  Tokens that see
// nothing get zeros, whatever dO holds.  (8192 tokens, 32 heads of 128: 33 us, 5.0 TB/s; a token and head at a
// time, the results scattered, 37.)
constexpr int kDeltaHeads = 4;
__global__ void __launch_bounds__(256) attn_delta_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ lm_attn a_,
                                                         float* ndelta, float* nlse, TokRange* rng) {
    __shared__ float s_delta[kDeltaHeads][16], s_nlse[kDeltaHeads][16];
    griddep_launch_dependents();
    griddep_wait();
    if ((int)blockIdx.y * kDeltaHeads >= p.hq) {  // one row of CTAs more than the heads need: who sees whom
        const int t = (int)(blockIdx.x * blockDim.x + threadIdx.x);
        if (t < p.T) rng[t] = range_of(a_, t, p.T);
        return;
    }
    const int sub = threadIdx.x & 15, mine = threadIdx.x >> 4;
    const int t0 = (int)blockIdx.x * 16, t = t0 + mine, h0 = (int)blockIdx.y * kDeltaHeads;
    float lse[kDeltaHeads];
    uint4 a[kDeltaHeads], b[kDeltaHeads];
    uint2 lo[kDeltaHeads];
#pragma unroll
    for (int r = 0; r < kDeltaHeads; ++r) {
        const int h = h0 + r;
        a[r] = b[r] = make_uint4(0, 0, 0, 0);
        lo[r] = make_uint2(0, 0);
        lse[r] = -INFINITY;
        if (t >= p.T || h >= p.hq) continue;
        lse[r] = p.lse_in[(int64_t)h * p.T + t];
        if (sub * 8 >= p.d) continue;
        const int64_t row = (int64_t)t * p.hq + h;
        a[r] = *reinterpret_cast<const uint4*>(p.dO.p + (int64_t)t * p.dO.ts + (int64_t)h * p.dO.hs + sub * 8);
        b[r] = *reinterpret_cast<const uint4*>(p.O + row * p.d + sub * 8);
        if (p.O_lo) lo[r] = *reinterpret_cast<const uint2*>(p.O_lo + row * p.d16 + sub * 8);
    }
#pragma unroll
    for (int r = 0; r < kDeltaHeads; ++r) {
        const bool sees = lse[r] > -INFINITY || lse[r] != lse[r];
        const uint32_t av[4] = {a[r].x, a[r].y, a[r].z, a[r].w}, bv[4] = {b[r].x, b[r].y, b[r].z, b[r].w};
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t ob = e & 1 ? bv[e >> 1] & 0xFFFF0000u : bv[e >> 1] << 16;
            const int more = (int)(int8_t)((e < 4 ? lo[r].x : lo[r].y) >> (8 * (e & 3)));
            s += (e & 1 ? bf16hi(av[e >> 1]) : bf16lo(av[e >> 1])) * __uint_as_float(ob + (uint32_t)(more * 256));
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (sub == 0) {
            s_delta[r][mine] = sees ? -s : 0.f;
            s_nlse[r][mine] = sees ? (p.cap - lse[r]) * kLog2e : 0.f;  // (the cap: exponents)
        }
    }
    __syncthreads();
    const int r = mine % kDeltaHeads, which = mine / kDeltaHeads;
    if (which < 2 && h0 + r < p.hq)
        (which ? nlse : ndelta)[(int64_t)(h0 + r) * p.Tp + t0 + sub] = which ? s_nlse[r][sub] : s_delta[r][sub];
}

cudaError_t launch_attn_delta(const AttnParams& p, const lm_attn& a, float* ndelta, float* nlse, TokRange* rng, cudaStream_t st) {
    // (Tp: whole 128-token tiles)
    const dim3 grid((unsigned)(p.Tp / 16), (unsigned)((p.hq + kDeltaHeads - 1) / kDeltaHeads + (rng ? 1 : 0)));
    return launch_pdl(attn_delta_kernel, grid, dim3(256), 0, st, nullptr, 0, p, a, ndelta, nlse, rng);
}

template <int DP>
cudaError_t launch_mode(int mode, const AttnParams& p, const BwdMaps& maps, int sms, cudaStream_t st) {
    switch (mode) {
        case ATTN_PLAIN: return launch_both<DP, ATTN_PLAIN, ATTN_SELF>(p, maps, sms, st);
        case ATTN_BIAS: return launch_both<DP, ATTN_BIAS, ATTN_SELF>(p, maps, sms, st);
        case ATTN_CAP: return launch_both<DP, ATTN_CAP, ATTN_SELF>(p, maps, sms, st);
        default: return launch_both<DP, ATTN_CAP_BIAS, ATTN_SELF>(p, maps, sms, st);
    }
}

lm_status launch_attn_bwd(const AttnParams& p, int sms, cudaStream_t st) {
    BwdMaps maps;
    const lm_status s = encode_bwd(p, &maps);
    if (s != LM_OK) return s;
    const int mode = (p.slopes ? ATTN_BIAS : 0) | (p.cap > 0.f ? ATTN_CAP : 0);
    const cudaError_t e = p.d <= 64 ? launch_mode<64>(mode, p, maps, sms, st) : launch_mode<128>(mode, p, maps, sms, st);
    return e == cudaSuccess ? LM_OK : report_error(LM_ERR_CUDA, "attn backward launch: %s", cudaGetErrorString(e));
}

}  // namespace lm
