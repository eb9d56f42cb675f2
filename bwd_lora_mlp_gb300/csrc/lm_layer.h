// Host-side declarations of the layer operators (include/lora_layer.h): kernel parameters, the
// launchers, and what lm_api.cu lends to the other translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lora_layer.h"

namespace lm {

// ---- from lm_api.cu
lm_status report_error(lm_status s, const char* fmt, ...);
// LM_OK on a device of compute capability 10.3; its SM count.  Fetches the tensor-map encoder.
lm_status device_ready(int* sms);
// 3D bf16 tensor map over (d, heads, tokens): box 64 x 1 x rows, 128-byte swizzle; reads outside give 0
lm_status encode_heads(CUtensorMap* m, const lm_heads& t, int64_t T, int heads, int d, int rows);
// An event pair around the kernel launched inside its lifetime, when tracing is on.
class LaunchTag {
  public:
    LaunchTag(const char* tag, cudaStream_t st);
    ~LaunchTag();
    LaunchTag(const LaunchTag&) = delete;
    LaunchTag& operator=(const LaunchTag&) = delete;

  private:
    void* scope_;
};

// ---- attention
// The interval of keys [lo, hi) that a query sees and of queries [qlo, qhi) that see a key, per token.
struct TokRange {
    int32_t lo, hi, qlo, qhi;
};
struct HeadsIn {
    const uint16_t* p;
    int64_t ts, hs;
};
struct AttnParams {
    int32_t T, hq, hk, d, d16;  // d16: d rounded up to 16
    float scale, cap;
    const float* slopes;
    const TokRange* rng;   // T entries, or null: one document
    int32_t causal, window;
    const int32_t* cu_docs;
    int32_t n_docs;
    HeadsIn q, k, v, dO;
    const uint16_t* O;
    const int8_t* O_lo;
    const float* lse_in;
    const float *ndelta, *nlse;  // -dO.O and -lse log2 e, rows of Tp
    int32_t Tp;                 // T rounded up to whole tiles
    int32_t rows;               // forward: queries of an item, 256 or 128
    uint16_t* out;         // O, or dQ
    int8_t* out_lo;
    float* lse;
    uint16_t *dK, *dV;
    int32_t* err;
    uint64_t wait_ns;
    int32_t starve;        // kernels whose loaders ask for nothing (attn_debug_inject)
};
enum AttnKernel : int { K_ATTN_FWD = 1, K_ATTN_DKV = 2, K_ATTN_DQ = 4 };
cudaError_t launch_attn_ranges(const lm_attn& a, int64_t T, TokRange* out, cudaStream_t st);
lm_status launch_attn_fwd(const AttnParams& p, int sms, cudaStream_t st);
// rng: the table of who sees whom is written too
cudaError_t launch_attn_delta(const AttnParams& p, const lm_attn& a, float* ndelta, float* nlse, TokRange* rng, cudaStream_t st);
lm_status launch_attn_bwd(const AttnParams& p, int sms, cudaStream_t st);

// ---- addnorm
struct AddNormParams {
    int64_t T;
    int32_t d;
    const void *h, *dh_out;
    const uint16_t *y, *dx;
    const void *w_in, *w_post, *gate;
    float alpha, eps, w_offset;
    bool h_f32, w_f32;
    void *h_out, *dh;
    uint16_t *x, *dy;
    float *rstd_y, *rstd_h;              // written by the forward
    const float *rstd_y_in, *rstd_h_in;  // read by the backward
    float *dw_in, *dw_post, *dgate;
    float* part;                         // backward: partial sums
};
size_t addnorm_part_bytes(int64_t T, int64_t d);
cudaError_t launch_addnorm_fwd(const AddNormParams& p, cudaStream_t st);
cudaError_t launch_addnorm_bwd(const AddNormParams& p, cudaStream_t st);

// ---- logprob
struct LogprobParams {
    int64_t T, V, ld, ld_out;
    const void* logits;
    bool f32, i64;
    const void* targets;
    float scale;
    int32_t k;
    float *logp, *entropy, *lse;
    int32_t* top_ids;
    float* top_logp;
    const float *lse_in, *entropy_in, *dlogp, *dentropy;
    void* dlogits;
};
constexpr int kMaxTop = 32;
cudaError_t launch_logprob_fwd(const LogprobParams& p, cudaStream_t st);
cudaError_t launch_logprob_bwd(const LogprobParams& p, cudaStream_t st);

}  // namespace lm
