// Residual add with the norms before and after a block (include/lora_layer.h).
//   forward   n = y r_y w_post,  h' = h + alpha gate n,  x = h' r_h w_in,   r_a = rsqrt(mean a^2 + eps)
//   backward  g = dh' + r_h (dx w_in - h' r_h^2 mean(dx w_in h')),  dh = g,  dn = alpha gate g,
//             dy = r_y (dn w_post - y r_y^2 mean(dn w_post y)),
//             dw_in = sum dx h' r_h,  dw_post = sum dn y r_y,  dgate = sum alpha g n
// Bound by memory: every tensor of the row is read and written once.  A thread holds 8 neighbouring
// values of a row (16 for d > 8192), so the row stays in registers between its two means, and a row
// takes as many warps as that needs; small rows share a CTA.  The backward's CTAs stay and walk the
// rows with a stride, adding the three sums over tokens in shared memory, each thread for its own
// columns of its row group (in registers they cost the CTA a quarter of its threads); a second kernel
// joins the CTAs' sums in order.
#include <algorithm>

#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

constexpr int kFwdCta = 512;    // threads a forward CTA aims at (at least one row)
constexpr int kBwdCta = 1024;   // the backward's: one CTA per SM, 64 registers a thread
constexpr int kBwdGrid = 152;

struct Vec8 {
    float v[8];
};
template <bool F32>
__device__ __forceinline__ Vec8 load8(const void* p, int64_t i) {
    Vec8 r;
    if (F32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4);
        r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w, r.v[4] = b.x, r.v[5] = b.y, r.v[6] = b.z, r.v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        r.v[0] = bf16lo(a.x), r.v[1] = bf16hi(a.x), r.v[2] = bf16lo(a.y), r.v[3] = bf16hi(a.y);
        r.v[4] = bf16lo(a.z), r.v[5] = bf16hi(a.z), r.v[6] = bf16lo(a.w), r.v[7] = bf16hi(a.w);
    }
    return r;
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const Vec8& r) {
    if (F32) {
        float* q = static_cast<float*>(p) + i;
        *reinterpret_cast<float4*>(q) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
        *reinterpret_cast<float4*>(q + 4) = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
            make_uint4(pack_bf16x2(r.v[0], r.v[1]), pack_bf16x2(r.v[2], r.v[3]), pack_bf16x2(r.v[4], r.v[5]),
                       pack_bf16x2(r.v[6], r.v[7]));
    }
}

// The threads of one row: `warps` warps of the CTA, group `grp`, with a barrier of their own.
struct RowGroup {
    int warps, grp, lane_in_row;
    float* red;  // [2][32] floats of the CTA's shared memory, by warp
    int buf;

    // sum over the row's threads, the same in all of them; the additions' order is fixed
    __device__ __forceinline__ float sum(float x) {
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (warps == 1) return x;
        const int lane = threadIdx.x & 31, w0 = grp * warps;
        float* r = red + buf * 32;
        buf ^= 1;  // (the next sum's writes do not meet this one's reads: its barrier lies between)
        if (lane == 0) r[threadIdx.x >> 5] = x;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(warps * 32) : "memory");
        x = lane < warps ? r[w0 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    }
};

// d -> warps of a row, rows of a CTA
struct RowPlan {
    int nv, warps, rows, threads;
};
static RowPlan plan_rows(int d, int cta) {
    RowPlan P;
    P.nv = d > 8192 ? 2 : 1;
    P.warps = (d / 8 + 32 * P.nv - 1) / (32 * P.nv);
    P.rows = std::min(15, std::max(1, cta / (32 * P.warps)));  // (a barrier each, besides the CTA's)
    P.threads = P.rows * P.warps * 32;
    return P;
}

template <bool W32>
__device__ __forceinline__ Vec8 weight8(const AddNormParams& p, const void* w, int c) {
    Vec8 r = load8<W32>(w, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] += p.w_offset;
    return r;
}

template <int NV, bool H32, bool W32>
__global__ void __launch_bounds__(1024) addnorm_fwd_kernel(const __grid_constant__ AddNormParams p, int warps, int rows) {
    __shared__ float red[2 * 32];
    griddep_launch_dependents();
    griddep_wait();
    RowGroup R{warps, (int)(threadIdx.x >> 5) / warps, 0, red, 0};
    R.lane_in_row = (int)threadIdx.x - R.grp * warps * 32;
    const int64_t t = (int64_t)blockIdx.x * rows + R.grp;
    if (t >= p.T) return;  // (all of the row's threads)
    const int64_t at = t * p.d;
    const float inv_d = 1.f / (float)p.d;
    Vec8 h[NV], y[NV];
    bool on[NV];
    int c[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        c[k] = (R.lane_in_row + k * warps * 32) * 8;
        on[k] = c[k] < p.d;
        h[k] = y[k] = Vec8{};
        if (on[k]) {
            h[k] = load8<H32>(p.h, at + c[k]);
            if (p.y) y[k] = load8<false>(p.y, at + c[k]);
        }
    }
    if (p.y) {
        float ry = 1.f;
        if (p.w_post) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(y[k].v[e], y[k].v[e], s);
            ry = rsqrtf(fmaf(R.sum(s), inv_d, p.eps));
            if (R.lane_in_row == 0) p.rstd_y[t] = ry;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on[k]) {
                Vec8 n = y[k];
                if (p.w_post) {
                    const Vec8 w = weight8<W32>(p, p.w_post, c[k]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) n.v[e] = n.v[e] * ry * w.v[e];
                }
                if (p.gate) {
                    const Vec8 g = load8<W32>(p.gate, c[k]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) n.v[e] *= g.v[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) h[k].v[e] = fmaf(p.alpha, n.v[e], h[k].v[e]);
                store8<H32>(p.h_out, at + c[k], h[k]);
            }
    }
    if (!p.w_in) return;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(h[k].v[e], h[k].v[e], s);
    const float rh = rsqrtf(fmaf(R.sum(s), inv_d, p.eps));
    if (R.lane_in_row == 0) p.rstd_h[t] = rh;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (on[k]) {
            const Vec8 w = weight8<W32>(p, p.w_in, c[k]);
            Vec8 x;
#pragma unroll
            for (int e = 0; e < 8; ++e) x.v[e] = h[k].v[e] * rh * w.v[e];
            store8<false>(p.x, at + c[k], x);
        }
}

// Sums over tokens: [row group][dw_in, dw_post, dgate][half of 8 columns][vector of the row] float4, so
// that neighbouring lanes touch neighbouring 16 bytes.
struct TokenSums {
    float4* base;
    int nvec;  // vectors of a row group's threads
    __device__ __forceinline__ float4* at(int grp, int which, int half, int v) const {
        return base + ((size_t)(grp * 3 + which) * 2 + half) * nvec + v;
    }
    __device__ __forceinline__ void add(int grp, int which, int v, const Vec8& x) const {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float4* p = at(grp, which, half, v);
            float4 a = *p;
            a.x += x.v[4 * half], a.y += x.v[4 * half + 1], a.z += x.v[4 * half + 2], a.w += x.v[4 * half + 3];
            *p = a;
        }
    }
};

template <int NV, bool H32, bool W32, bool SUMS>
__global__ void __launch_bounds__(1024, 1)
    addnorm_bwd_kernel(const __grid_constant__ AddNormParams p, int warps, int rows) {
    __shared__ float red[2 * 32];
    extern __shared__ float4 sums_raw[];
    griddep_launch_dependents();
    RowGroup R{warps, (int)(threadIdx.x >> 5) / warps, 0, red, 0};
    R.lane_in_row = (int)threadIdx.x - R.grp * warps * 32;
    const float inv_d = 1.f / (float)p.d;
    const TokenSums A{sums_raw, warps * 32 * NV};
    if (SUMS) {
        for (int i = threadIdx.x; i < rows * 6 * A.nvec; i += blockDim.x) sums_raw[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        __syncthreads();
    }
    griddep_wait();
    for (int64_t t = (int64_t)blockIdx.x * rows + R.grp; t < p.T; t += (int64_t)gridDim.x * rows) {
        const int64_t at = t * p.d;
        const float ry = p.w_post ? p.rstd_y_in[t] : 1.f, rh = p.w_in ? p.rstd_h_in[t] : 0.f;
        Vec8 s[NV], n[NV], u[NV], g[NV];  // h', N(y) (or y), dx w_in, gradient
        float acc = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (R.lane_in_row + k * warps * 32) * 8;
            s[k] = n[k] = u[k] = g[k] = Vec8{};
            if (c < p.d) {
                s[k] = load8<H32>(p.h, at + c);
                if (p.dh_out) g[k] = load8<H32>(p.dh_out, at + c);
                if (p.y) n[k] = load8<false>(p.y, at + c);
                if (p.w_in) u[k] = load8<false>(p.dx, at + c);
                if (p.y) {
                    Vec8 add = n[k];
                    if (p.w_post) {
                        const Vec8 w = weight8<W32>(p, p.w_post, c);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            n[k].v[e] *= ry;  // y r_y
                            add.v[e] = n[k].v[e] * w.v[e];
                        }
                    }
                    if (p.gate) {
                        const Vec8 q = load8<W32>(p.gate, c);
#pragma unroll
                        for (int e = 0; e < 8; ++e) add.v[e] *= q.v[e];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[k].v[e] = fmaf(p.alpha, add.v[e], s[k].v[e]);
                }
                if (p.w_in) {
                    const Vec8 w = weight8<W32>(p, p.w_in, c);
                    Vec8 x;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        s[k].v[e] *= rh;  // h' r_h
                        x.v[e] = u[k].v[e] * s[k].v[e];
                        u[k].v[e] *= w.v[e];
                        acc = fmaf(x.v[e], w.v[e], acc);
                    }
                    if (SUMS && p.dw_in) A.add(R.grp, 0, c >> 3, x);
                }
            }
        }
        if (p.w_in) {
            const float m = R.sum(acc) * inv_d;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) g[k].v[e] = fmaf(rh, fmaf(-s[k].v[e], m, u[k].v[e]), g[k].v[e]);
        }
        acc = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (R.lane_in_row + k * warps * 32) * 8;
            if (c < p.d) {
                store8<H32>(p.dh, at + c, g[k]);
                if (p.y) {
                    Vec8 w;
                    if (p.w_post) w = weight8<W32>(p, p.w_post, c);
                    if (p.gate) {
                        const Vec8 q = load8<W32>(p.gate, c);
                        Vec8 x;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float ag = p.alpha * g[k].v[e];
                            x.v[e] = p.w_post ? ag * n[k].v[e] * w.v[e] : ag * n[k].v[e];
                            g[k].v[e] = ag * q.v[e];  // dn
                        }
                        if (SUMS && p.dgate) A.add(R.grp, 2, c >> 3, x);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[k].v[e] *= p.alpha;
                    }
                    if (p.w_post) {
                        Vec8 x;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x.v[e] = g[k].v[e] * n[k].v[e];
                            g[k].v[e] *= w.v[e];
                            acc = fmaf(x.v[e], w.v[e], acc);
                        }
                        if (SUMS && p.dw_post) A.add(R.grp, 1, c >> 3, x);
                    }
                }
            }
        }
        if (!p.y) continue;
        const float m = p.w_post ? R.sum(acc) * inv_d : 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (R.lane_in_row + k * warps * 32) * 8;
            if (c < p.d) {
                if (p.w_post)
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[k].v[e] = ry * fmaf(-n[k].v[e], m, g[k].v[e]);
                store8<false>(p.dy, at + c, g[k]);
            }
        }
    }
    if (SUMS) {  // the row groups' sums in order, to part[CTA][3][d]
        __syncthreads();
        for (int i = threadIdx.x; i < 3 * (p.d >> 2); i += blockDim.x) {
            const int which = i / (p.d >> 2), c4 = i - which * (p.d >> 2);
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int grp = 0; grp < rows; ++grp) {
                const float4 q = *A.at(grp, which, c4 & 1, c4 >> 1);
                s.x += q.x, s.y += q.y, s.z += q.z, s.w += q.w;
            }
            *reinterpret_cast<float4*>(p.part + ((int64_t)blockIdx.x * 3 + which) * p.d + 4 * c4) = s;
        }
    }
}

// The sum over `n` partial rows of 32 columns: 8 threads a column take every eighth row, then join.
__global__ void __launch_bounds__(256) addnorm_join_kernel(const __grid_constant__ AddNormParams p, int n) {
    __shared__ float sm[8][32];
    griddep_launch_dependents();
    griddep_wait();
    float* outs[3] = {p.dw_in, p.dw_post, p.dgate};
    float* out = outs[blockIdx.y];
    if (!out) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float* part = p.part + (int64_t)blockIdx.y * p.d + c;
    float s = 0.f;
#pragma unroll 4
    for (int i = w; i < n; i += 8) s += part[(int64_t)i * 3 * p.d];
    sm[w][lane] = s;
    __syncthreads();
    if (w == 0) {
        for (int i = 1; i < 8; ++i) s += sm[i][lane];
        out[c] = s;
    }
}

static int bwd_grid(int64_t T, const RowPlan& P) { return (int)std::min<int64_t>(kBwdGrid, (T + P.rows - 1) / P.rows); }
size_t addnorm_part_bytes(int64_t T, int64_t d) {
    return (size_t)bwd_grid(T, plan_rows((int)d, kBwdCta)) * 3 * (size_t)d * 4;
}

template <int NV, bool H32, bool W32>
static cudaError_t fwd_launch(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    return launch_pdl(addnorm_fwd_kernel<NV, H32, W32>, dim3((unsigned)((p.T + P.rows - 1) / P.rows)), dim3(P.threads), 0, st,
                      nullptr, 0, p, P.warps, P.rows);
}
template <int NV, bool H32, bool W32>
static cudaError_t bwd_launch(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    const unsigned grid = (unsigned)bwd_grid(p.T, P);
    if (!(p.dw_in || p.dw_post || p.dgate))
        return launch_pdl(addnorm_bwd_kernel<NV, H32, W32, false>, dim3(grid), dim3(P.threads), 0, st, nullptr, 0, p, P.warps,
                          P.rows);
    const int smem = P.rows * 6 * P.warps * 32 * NV * (int)sizeof(float4);
    auto kernel = addnorm_bwd_kernel<NV, H32, W32, true>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_pdl(kernel, dim3(grid), dim3(P.threads), smem, st, nullptr, 0, p, P.warps, P.rows);
    if (e == cudaSuccess)
        e = launch_pdl(addnorm_join_kernel, dim3((unsigned)(p.d / 32), 3), dim3(256), 0, st, nullptr, 0, p, (int)grid);
    return e;
}
template <int NV>
static cudaError_t fwd_types(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    if (p.h_f32) return p.w_f32 ? fwd_launch<NV, true, true>(p, P, st) : fwd_launch<NV, true, false>(p, P, st);
    return p.w_f32 ? fwd_launch<NV, false, true>(p, P, st) : fwd_launch<NV, false, false>(p, P, st);
}
template <int NV>
static cudaError_t bwd_types(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    if (p.h_f32) return p.w_f32 ? bwd_launch<NV, true, true>(p, P, st) : bwd_launch<NV, true, false>(p, P, st);
    return p.w_f32 ? bwd_launch<NV, false, true>(p, P, st) : bwd_launch<NV, false, false>(p, P, st);
}

cudaError_t launch_addnorm_fwd(const AddNormParams& p, cudaStream_t st) {
    const RowPlan P = plan_rows(p.d, kFwdCta);
    return P.nv == 1 ? fwd_types<1>(p, P, st) : fwd_types<2>(p, P, st);
}
cudaError_t launch_addnorm_bwd(const AddNormParams& p, cudaStream_t st) {
    const RowPlan P = plan_rows(p.d, kBwdCta);
    return P.nv == 1 ? bwd_types<1>(p, P, st) : bwd_types<2>(p, P, st);
}

}  // namespace lm
