// Who sees whom in attention over packed documents (include/lora_layer.h), as a table per token, for the
// forward; the backward's is written by its first kernel (lm_attn_bwd.cu).  (Documents searched for where
// they are wanted instead: two launches less, but 14 documents in 8192 tokens 529 -> 556 us.)
#include "lm_attn.cuh"

namespace lm {

__global__ void __launch_bounds__(256) attn_ranges_kernel(const __grid_constant__ lm_attn a, int T, TokRange* out) {
    griddep_launch_dependents();
    griddep_wait();
    const int t = blockIdx.x * blockDim.x + threadIdx.x;
    if (t < T) out[t] = range_of(a, t, T);
}

cudaError_t launch_attn_ranges(const lm_attn& a, int64_t T, TokRange* out, cudaStream_t st) {
    return launch_pdl(attn_ranges_kernel, dim3((unsigned)((T + 255) / 256)), dim3(256), 0, st, nullptr, 0, a, (int)T, out);
}

}  // namespace lm
