// Who sees whom in attention over packed documents (include/lora_layer.h), as a table per token.
#include "lm_attn.cuh"

namespace lm {

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

}  // namespace lm
