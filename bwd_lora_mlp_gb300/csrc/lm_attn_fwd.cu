// Attention forward over packed documents: the kernel's launches (lm_attn_fwd.cuh).
#include "lm_attn_fwd.cuh"

namespace lm {

template <int DP>
cudaError_t launch_mode(int mode, const AttnParams& p, const FwdMaps& maps, int sms, cudaStream_t st) {
    switch (mode) {
        case ATTN_PLAIN: return launch_fwd<DP, ATTN_PLAIN, ATTN_SELF>(p, maps, sms, st);
        case ATTN_BIAS: return launch_fwd<DP, ATTN_BIAS, ATTN_SELF>(p, maps, sms, st);
        case ATTN_CAP: return launch_fwd<DP, ATTN_CAP, ATTN_SELF>(p, maps, sms, st);
        default: return launch_fwd<DP, ATTN_CAP_BIAS, ATTN_SELF>(p, maps, sms, st);
    }
}

lm_status launch_attn_fwd(const AttnParams& given, int sms, cudaStream_t st) {
    FwdMaps maps;
    AttnParams p = given;
    // One query tile an item where the SMs take all of them at once (512 tokens, 32 heads: 19.5 us, 20.8 with two;
    // 1024 tokens, 16 heads of 64 dims: 24.1 and 26.0)
    p.rows = (int64_t)((p.T + 2 * kTile - 1) / (2 * kTile)) * p.hq * 2 <= sms ? kTile : 2 * kTile;
    const lm_heads q{p.q.p, p.q.ts, p.q.hs}, k{p.k.p, p.k.ts, p.k.hs}, v{p.v.p, p.v.ts, p.v.hs};
    lm_status s = encode_heads(&maps.q, q, p.T, p.hq, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps.k, k, p.T, p.hk, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps.v, v, p.T, p.hk, p.d, kTile);
    if (s != LM_OK) return s;
    // without slopes the factor of the scores goes into the exponent and has to be positive (the maximum of s c
    // is c max s); the cap's is
    const int mode = (p.slopes || !(p.scale > 0.f || p.cap > 0.f) ? ATTN_BIAS : 0) | (p.cap > 0.f ? ATTN_CAP : 0);
    const cudaError_t e = p.d <= 64 ? launch_mode<64>(mode, p, maps, sms, st) : launch_mode<128>(mode, p, maps, sms, st);
    return e == cudaSuccess ? LM_OK : report_error(LM_ERR_CUDA, "attn forward launch: %s", cudaGetErrorString(e));
}

}  // namespace lm
