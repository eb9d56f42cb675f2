// What the kernels over rows of logits share: a pass over a row in 16-byte vectors, and what is NaN or
// largest in a batch of them; a row of a CTA, or of a cluster's CTAs.
#pragma once

#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

constexpr int kThreads = 256;
constexpr int kMaxCluster = 8;
constexpr float kL2e = 1.4426950408889634f;

__device__ __forceinline__ float lp_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool F32>
struct Row {
    static constexpr int kVec = F32 ? 4 : 8;  // logits of 16 bytes
    const char* p;
    __device__ __forceinline__ float at(int64_t j) const {
        if (F32) return reinterpret_cast<const float*>(p)[j];
        return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[j] << 16);
    }
    // elements before the first 16-byte boundary at or after element j
    __device__ __forceinline__ int64_t head(int64_t j) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p + j * (F32 ? 4 : 2)) & 15;
        return a ? (int64_t)((16 - a) / (F32 ? 4 : 2)) : 0;
    }
};

// f(v, index of vector 0, whole vectors from there on) over [j0, j1) in batches of U whole vectors of a thread of N
// (vector u lies u N vectors on), the next batch loading meanwhile, and one(x, index) for the single elements before the
// first and after the last 16-byte boundary.  In two steps: the first batch's loads are under way from the
// beginning, run(f, one) does the rest.
template <int U, bool F32, int N>
struct Scan {
    static constexpr int W = Row<F32>::kVec;
    const Row<F32> row;
    int64_t j0, j1, a;  // a: the first boundary
    int nv;
    const char* base;
    uint4 next[U];
    __device__ __forceinline__ Scan(const Row<F32>& row_, int64_t j0_, int64_t j1_) : row(row_), j0(j0_), j1(j1_) {
        a = min(j1, j0 + row.head(j0));
        nv = (int)((j1 - a) / W);
        base = row.p + a * (F32 ? 4 : 2);
        load(threadIdx.x);
    }
    __device__ __forceinline__ void load(int v) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * N < nv) next[u] = *reinterpret_cast<const uint4*>(base + (int64_t)(v + u * N) * 16);
    }
    template <typename F, typename G>
    __device__ __forceinline__ void run(F f, G one) {
        for (int v = threadIdx.x; v < nv; v += U * N) {
            uint32_t w[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) w[u][0] = next[u].x, w[u][1] = next[u].y, w[u][2] = next[u].z, w[u][3] = next[u].w;
            if (v + (U - 1) * N >= nv)  // (the last batch of some threads: what is not there counts nothing)
#pragma unroll
                for (int u = 1; u < U; ++u)
                    if (v + u * N >= nv)
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[u][e] = F32 ? 0xFF800000u : 0xFF80FF80u;
            load(v + U * N);
            f(w, a + (int64_t)v * W, nv - v);
        }
        const int64_t b = a + (int64_t)nv * W;
        const int64_t j = threadIdx.x < W ? j0 + threadIdx.x : b + (threadIdx.x - W);
        if (threadIdx.x < 2 * W && (threadIdx.x < W ? j < a : j < j1)) one(row.at(j), j);
    }
};
template <int U, bool F32, typename F, typename G>
__device__ __forceinline__ void scan(const Row<F32>& row, int64_t j0, int64_t j1, F f, G one) {
    Scan<U, F32, kThreads>(row, j0, j1).run(f, one);
}
// logit e of a vector
template <bool F32>
__device__ __forceinline__ float logit(const uint32_t (&w)[4], int e) {
    return F32 ? __uint_as_float(w[e % 4]) : e & 1 ? bf16hi(w[e / 2 % 4]) : bf16lo(w[e / 2 % 4]);
}

// Running softmax sums; max_nan keeps a NaN: a maximum that is one stays one, and the sums with it.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// the same of two pairs of bf16
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// the largest logit of a batch (NaN if there is one)
template <int U, bool F32>
__device__ __forceinline__ float largest(const uint32_t (&w)[U][4]) {
    if (F32) {
        float big = __uint_as_float(w[0][0]);
#pragma unroll
        for (int i = 1; i < 4 * U; ++i) big = max_nan(big, __uint_as_float(w[i / 4][i % 4]));
        return big;
    }
    uint32_t big = w[0][0];
#pragma unroll
    for (int i = 1; i < 4 * U; ++i) big = max2_nan(big, w[i / 4][i % 4]);
    return max_nan(bf16lo(big), bf16hi(big));
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// this CTA's shared variable at the same place in CTA 0 of the cluster
template <typename T>
__device__ __forceinline__ void st_first(T* p, T v) {
    const uint32_t a = map_to_rank(smem_u32(p), 0);
    if constexpr (sizeof(T) == 8) asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"((uint64_t)v) : "memory");
    else asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(a), "r"(__float_as_uint(v)) : "memory");
}

}  // namespace lm
