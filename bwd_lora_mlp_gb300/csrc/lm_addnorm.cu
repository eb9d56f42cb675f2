// Residual add with the norms before and after a block (include/lora_layer.h).
//   forward   n = y r_y w_post,  h' = h + alpha gate n,  x = h' r_h w_in,   r_a = rsqrt(mean a^2 + eps)
//   backward  g = dh' + r_h (dx w_in - h' r_h^2 mean(dx w_in h')),  dh = g,  dn = alpha gate g,
//             dy = r_y (dn w_post - y r_y^2 mean(dn w_post y)),
//             dw_in = sum dx h' r_h,  dw_post = sum dn y r_y,  dgate = sum alpha g n
// One CTA per row; the sums over tokens by one CTA per 32 columns and a share of the rows, joined
// in a fixed order.  Bound by memory.
#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

constexpr int kThreads = 256;
constexpr int kRowShares = 64;  // row shares of the column sums

__device__ __forceinline__ float ld_any(const void* p, int64_t i, bool f32) {
    return f32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}
__device__ __forceinline__ void st_any(void* p, int64_t i, bool f32, float v) {
    if (f32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
}

__device__ float block_sum(float x) {
    __shared__ float part[kThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    return s;
}

struct RowMath {
    const AddNormParams& p;
    int64_t at;   // the row's first element
    float ry;
    __device__ float weight(const void* w, int c) const { return ld_any(w, c, p.w_f32) + p.w_offset; }
    __device__ float gain(int c) const { return p.gate ? p.alpha * ld_any(p.gate, c, p.w_f32) : p.alpha; }
    __device__ float y(int c) const { return ld_any(p.y, at + c, false); }
    __device__ float normed(int c) const { return p.w_post ? y(c) * ry * weight(p.w_post, c) : y(c); }
    __device__ float sum(int c) const {
        const float h = ld_any(p.h, at + c, p.h_f32);
        return p.y ? h + gain(c) * normed(c) : h;
    }
};

__global__ void __launch_bounds__(kThreads) addnorm_fwd_kernel(const __grid_constant__ AddNormParams p) {
    const int64_t t = blockIdx.x;
    RowMath R{p, t * p.d, 0.f};
    if (p.w_post) {
        float s = 0.f;
        for (int c = threadIdx.x; c < p.d; c += kThreads) s += R.y(c) * R.y(c);
        R.ry = rsqrtf(block_sum(s) / p.d + p.eps);
        if (threadIdx.x == 0) p.rstd_y[t] = R.ry;
    }
    float s = 0.f;
    for (int c = threadIdx.x; c < p.d; c += kThreads) {
        const float v = R.sum(c);
        s += v * v;
        if (p.y) st_any(p.h_out, R.at + c, p.h_f32, v);
    }
    if (!p.w_in) return;
    const float rh = rsqrtf(block_sum(s) / p.d + p.eps);
    if (threadIdx.x == 0) p.rstd_h[t] = rh;
    for (int c = threadIdx.x; c < p.d; c += kThreads) st_any(p.x, R.at + c, false, R.sum(c) * rh * R.weight(p.w_in, c));
}

cudaError_t launch_addnorm_fwd(const AddNormParams& p, cudaStream_t st) {
    addnorm_fwd_kernel<<<(unsigned)p.T, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

// the row's mean(dx w_in h') goes to part[t] for the column sums, which form g again
__global__ void __launch_bounds__(kThreads) addnorm_bwd_kernel(const __grid_constant__ AddNormParams p) {
    const int64_t t = blockIdx.x;
    RowMath R{p, t * p.d, p.w_post ? p.rstd_y_in[t] : 0.f};
    float mh = 0.f, rh = 0.f;
    if (p.w_in) {
        rh = p.rstd_h_in[t];
        for (int c = threadIdx.x; c < p.d; c += kThreads)
            mh += ld_any(p.dx, R.at + c, false) * R.weight(p.w_in, c) * R.sum(c);
        mh = block_sum(mh) / p.d;
        if (threadIdx.x == 0) p.part[t] = mh;
    }
    auto grad = [&](int c) {
        float g = p.dh_out ? ld_any(p.dh_out, R.at + c, p.h_f32) : 0.f;
        if (p.w_in) g += rh * (ld_any(p.dx, R.at + c, false) * R.weight(p.w_in, c) - R.sum(c) * rh * rh * mh);
        return g;
    };
    float my = 0.f;
    if (p.w_post) {
        for (int c = threadIdx.x; c < p.d; c += kThreads) my += grad(c) * R.gain(c) * R.weight(p.w_post, c) * R.y(c);
        my = block_sum(my) / p.d;
    }
    for (int c = threadIdx.x; c < p.d; c += kThreads) {
        const float g = grad(c);
        st_any(p.dh, R.at + c, p.h_f32, g);
        if (!p.y) continue;
        float dn = g * R.gain(c);
        if (p.w_post) dn = R.ry * (dn * R.weight(p.w_post, c) - R.y(c) * R.ry * R.ry * my);
        st_any(p.dy, R.at + c, false, dn);
    }
}

__global__ void __launch_bounds__(kThreads) addnorm_columns_kernel(const __grid_constant__ AddNormParams p) {
    __shared__ float sm[3][8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float a[3] = {0.f, 0.f, 0.f};
    for (int64_t t = blockIdx.y * 8 + w; t < p.T; t += 8 * kRowShares) {
        RowMath R{p, t * p.d, p.w_post ? p.rstd_y_in[t] : 0.f};
        float g = p.dh_out ? ld_any(p.dh_out, R.at + c, p.h_f32) : 0.f;
        if (p.w_in) {
            const float dx = ld_any(p.dx, R.at + c, false), rh = p.rstd_h_in[t], s = R.sum(c);
            g += rh * (dx * R.weight(p.w_in, c) - s * rh * rh * p.part[t]);
            a[0] += dx * s * rh;
        }
        if (p.w_post) a[1] += g * R.gain(c) * R.y(c) * R.ry;
        if (p.gate) a[2] += p.alpha * g * R.normed(c);
    }
    for (int k = 0; k < 3; ++k) sm[k][w][lane] = a[k];
    __syncthreads();
    if (w < 3) {
        float s = 0.f;
        for (int i = 0; i < 8; ++i) s += sm[w][i][lane];
        p.part[p.T + ((int64_t)blockIdx.y * 3 + w) * p.d + c] = s;
    }
}

__global__ void __launch_bounds__(kThreads) addnorm_join_kernel(const __grid_constant__ AddNormParams p) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= p.d) return;
    float* out[3] = {p.dw_in, p.dw_post, p.dgate};
    for (int k = 0; k < 3; ++k) {
        if (!out[k]) continue;
        float s = 0.f;
        for (int i = 0; i < kRowShares; ++i) s += p.part[p.T + ((int64_t)i * 3 + k) * p.d + c];
        out[k][c] = s;
    }
}

size_t addnorm_part_bytes(int64_t T, int64_t d) { return (size_t)(T + (int64_t)kRowShares * 3 * d) * 4; }

cudaError_t launch_addnorm_bwd(const AddNormParams& p, cudaStream_t st) {
    addnorm_bwd_kernel<<<(unsigned)p.T, kThreads, 0, st>>>(p);
    if (p.dw_in || p.dw_post || p.dgate) {
        addnorm_columns_kernel<<<dim3(p.d / 32, kRowShares), kThreads, 0, st>>>(p);
        addnorm_join_kernel<<<(p.d + kThreads - 1) / kThreads, kThreads, 0, st>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace lm
