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
// 3D bf16 tensor map over (d, heads, tokens): box 64 x box_heads x rows, 128-byte swizzle; reads outside give 0
lm_status encode_heads(CUtensorMap* m, const lm_heads& t, int64_t T, int heads, int d, int rows, int box_heads = 1);
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
    int32_t Tk;                 // keys (T, but for cross attention)
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
    int32_t rows;               // forward: queries of an item, 256 or 128 (few queries: tokens of a tile)
    // cross attention; null: every query sees every key.  By token, and by tile the rows that see or are seen at all
    const int2 *qrange, *krange;
    const uint4 *qseen, *kseen;
    int32_t splits, parts;      // few queries: CTAs that share the keys; parts that are joined, T x hq rows each
    float* part_o;
    float2* part_ml;
    int32_t kparts, qparts;     // cross attention backward: CTAs that share a key tile, parts of a query tile's keys
    float *part_dkv, *part_dq;  // their sums: [part][dV, dK][Tk][hk][d], [part][T][hq][d]
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

// ---- cross attention
// GB300's SMs, not asked of the device: a workspace's size has to be known on a host without one, and parts, whose sums
// are joined in order, are the same everywhere.
constexpr int kCrossSms = 152;
struct CrossTables {
    int2 *qrange, *krange;
    uint4 *qseen, *kseen;
};
cudaError_t launch_cross_ranges(const lm_cross& a, int64_t Tq, int64_t Tk, const CrossTables& t, cudaStream_t st);
// the form for few queries: CTAs that share the keys of a query tile, the parts that they leave (1: the result itself)
// and the tile's tokens; splits 0: the other form
struct FewPlan {
    int32_t splits, parts, tokens;
};
FewPlan plan_few(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk);
// the backward's parts (1: none), of a call with `docs` documents (1: without), and the most that any such call has
struct BwdParts {
    int32_t k, q;
};
BwdParts plan_parts(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk, int32_t d, int32_t docs);
BwdParts most_parts(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk);
cudaError_t launch_fill(float* out, int64_t n, float v, cudaStream_t st);
lm_status launch_cross_fwd(const AttnParams& p, int sms, cudaStream_t st);
lm_status launch_cross_bwd(const AttnParams& p, int sms, cudaStream_t st);

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

// ---- qkrope
// The query heads, or the key heads: what is read (x, and backward dy) and written (y: the result, or dx).
struct RopeSide {
    const uint16_t *x, *dy;
    uint16_t* y;
    int64_t x_ts, x_hs, dy_ts, dy_hs, y_ts, y_hs;
    const void* w;
    float* dw;
    int32_t heads;
    int32_t parts, per_part;  // (from here on: the launcher's) warps of a token, heads of a warp
    int32_t blocks;           // CTAs
};
struct QkRopeParams {
    int64_t T;
    int32_t d, rot, axes;
    const float* inv_freq;
    const void* pos;
    const int32_t* axis;
    bool pos_i64, w_f32, norm, interleaved;
    float factor, eps, w_offset;
    RopeSide q, k;
    float* part;
    int32_t vec, lanes;  // the launcher's: dims of a vector, lanes of a head
};
size_t qkrope_part_bytes(int d);
cudaError_t launch_qkrope(QkRopeParams p, bool backward, cudaStream_t st);

// ---- distill
struct DistillParams {
    int64_t T, V, ld, ld_out;
    const void* logits;
    bool f32, i64, t64, v_f32, rest;
    int32_t K;
    const void *ids, *values, *targets;
    float scale;
    float *kl, *logp, *lse;
    float* saved;  // T x 8
    const float *dkl, *dlogp;
    void* dlogits;
};
constexpr int kMaxEntries = 128;
cudaError_t launch_distill_fwd(const DistillParams& p, cudaStream_t st);
cudaError_t launch_distill_bwd(const DistillParams& p, cudaStream_t st);

}  // namespace lm
