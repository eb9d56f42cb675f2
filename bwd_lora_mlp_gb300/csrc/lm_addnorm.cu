// Residual add with the norms before and after a block (include/lora_layer.h).
//   forward   n = y r_y w_post,  h' = h + alpha gate n,  x = h' r_h w_in,   r_a = rsqrt(mean a^2 + eps)
//   backward  g = dh' + r_h (dx w_in - h' r_h^2 mean(dx w_in h')),  dh = g,  dn = alpha gate g,
//             dy = r_y (dn w_post - y r_y^2 mean(dn w_post y)),
//             dw_in = sum dx h' r_h,  dw_post = sum dn y r_y,  dgate = sum alpha g n
// Bound by memory: every tensor of the row is read and written once.  A thread holds 8 neighbouring
// values of a row (16 for d > 8192), so the row stays in registers between its two means, and a row
// takes as many warps as that needs; small rows share a CTA.  CTAs stay and walk the rows with a
// stride, each thread copying its own 16-byte pieces of the next rows to shared memory asynchronously:
// the reads of several rows are in flight while one is normalised (loaded when it was its turn, a
// 4096-wide row left the memory idle for two means and its stores: 78 us for 8192 rows, not KFWD).
// The backward is  adding the three sums over tokens in shared memory, each thread for its own
// columns of its row group (in registers they cost the CTA a quarter of its threads); a second kernel
// joins the CTAs' sums in order.
#include <algorithm>

#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

constexpr int kFwdCta = 512;    // threads a forward CTA aims at (at least one row)
constexpr int kBwdCta = 512;    // the backward's (at least one row): one CTA per SM
// Rows on their way: as many as the shared memory holds beside a first-level cache for the weights.
constexpr int fwd_stages(int nv, bool h32) { return nv == 2 && h32 ? 2 : 3; }
constexpr int bwd_stages(int nv, bool h32, int threads) { return nv == 2 ? 1 : threads <= 512 ? 3 : h32 ? 1 : 2; }
constexpr int kSms = 152;

struct Vec8 {
    float v[8];
};
__device__ __forceinline__ void unpack8(const uint4& a, Vec8& r) {
    r.v[0] = bf16lo(a.x), r.v[1] = bf16hi(a.x), r.v[2] = bf16lo(a.y), r.v[3] = bf16hi(a.y);
    r.v[4] = bf16lo(a.z), r.v[5] = bf16hi(a.z), r.v[6] = bf16lo(a.w), r.v[7] = bf16hi(a.w);
}
template <bool F32>
__device__ __forceinline__ Vec8 load8(const void* p, int64_t i) {
    Vec8 r;
    if (F32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4);
        r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w, r.v[4] = b.x, r.v[5] = b.y, r.v[6] = b.z, r.v[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i), r);
    }
    return r;
}
// A thread's pieces of rows on their way: slot [stage][piece][thread] of 16 bytes, written and read by
// the same thread, so no barrier is needed between the copy and its use.
__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool F32>
__device__ __forceinline__ void copy8(uint4* slot, int step, const void* p, int64_t i) {
    const char* src = static_cast<const char*>(p) + i * (F32 ? 4 : 2);
    copy16(slot, src);
    if (F32) copy16(slot + step, src + 16);
}
template <bool F32>
__device__ __forceinline__ Vec8 take8(const uint4* slot, int step) {
    Vec8 r;
    if (F32) {
        const float4 a = *reinterpret_cast<const float4*>(slot), b = *reinterpret_cast<const float4*>(slot + step);
        r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w, r.v[4] = b.x, r.v[5] = b.y, r.v[6] = b.z, r.v[7] = b.w;
    } else {
        unpack8(*slot, r);
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
    constexpr int kHp = H32 ? 2 : 1, kPieces = NV * (kHp + 1), kStages = fwd_stages(NV, H32);
    __shared__ float red[2 * 32];
    extern __shared__ uint4 pieces[];  // [stage][piece][thread]
    griddep_launch_dependents();
    griddep_wait();
    RowGroup R{warps, (int)(threadIdx.x >> 5) / warps, 0, red, 0};
    R.lane_in_row = (int)threadIdx.x - R.grp * warps * 32;
    const int step = blockDim.x;
    const int64_t stride = (int64_t)gridDim.x * rows;
    const float inv_d = 1.f / (float)p.d;
    auto ask = [&](int64_t t, int stage) {
        if (t < p.T) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (R.lane_in_row + k * warps * 32) * 8;
                uint4* slot = pieces + (stage * kPieces + k * (kHp + 1)) * step + threadIdx.x;
                if (c < p.d) {
                    copy8<H32>(slot, step, p.h, t * p.d + c);
                    if (p.y) copy8<false>(slot + kHp * step, step, p.y, t * p.d + c);
                }
            }
        }
        copies_commit();  // (a group a turn, empty ones too: the wait below counts them)
    };
    int64_t t = (int64_t)blockIdx.x * rows + R.grp;
#pragma unroll
    for (int i = 0; i < kStages; ++i) ask(t + i * stride, i);
    for (int stage = 0; t < p.T; t += stride, stage = stage + 1 == kStages ? 0 : stage + 1) {
        const int64_t at = t * p.d;
        copies_wait<kStages - 1>();
        Vec8 h[NV], y[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint4* slot = pieces + (stage * kPieces + k * (kHp + 1)) * step + threadIdx.x;
            h[k] = y[k] = Vec8{};
            if ((R.lane_in_row + k * warps * 32) * 8 < p.d) {
                h[k] = take8<H32>(slot, step);
                if (p.y) y[k] = take8<false>(slot + kHp * step, step);
            }
        }
        ask(t + kStages * stride, stage);  // (the pieces are in registers)
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
            for (int k = 0; k < NV; ++k) {
                const int c = (R.lane_in_row + k * warps * 32) * 8;
                if (c < p.d) {
                    Vec8 n = y[k];
                    if (p.w_post) {
                        const Vec8 w = weight8<W32>(p, p.w_post, c);
#pragma unroll
                        for (int e = 0; e < 8; ++e) n.v[e] = n.v[e] * ry * w.v[e];
                    }
                    if (p.gate) {
                        const Vec8 g = load8<W32>(p.gate, c);
#pragma unroll
                        for (int e = 0; e < 8; ++e) n.v[e] *= g.v[e];
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[k].v[e] = fmaf(p.alpha, n.v[e], h[k].v[e]);
                    store8<H32>(p.h_out, at + c, h[k]);
                }
            }
        }
        if (!p.w_in) continue;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(h[k].v[e], h[k].v[e], s);
        const float rh = rsqrtf(fmaf(R.sum(s), inv_d, p.eps));
        if (R.lane_in_row == 0) p.rstd_h[t] = rh;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (R.lane_in_row + k * warps * 32) * 8;
            if (c < p.d) {
                const Vec8 w = weight8<W32>(p, p.w_in, c);
                Vec8 x;
#pragma unroll
                for (int e = 0; e < 8; ++e) x.v[e] = h[k].v[e] * rh * w.v[e];
                store8<false>(p.x, at + c, x);
            }
        }
    }
}

template <int NV, bool H32, bool W32, bool SUMS, int MOST>
__global__ void __launch_bounds__(MOST, 1)
    addnorm_bwd_kernel(const __grid_constant__ AddNormParams p, int warps, int rows) {
    __shared__ float red[2 * 32];
    extern __shared__ uint4 smem_pieces[];  // [stage][piece][thread]
    griddep_launch_dependents();
    griddep_wait();
    RowGroup R{warps, (int)(threadIdx.x >> 5) / warps, 0, red, 0};
    R.lane_in_row = (int)threadIdx.x - R.grp * warps * 32;
    const float inv_d = 1.f / (float)p.d;
    constexpr int kHp = H32 ? 2 : 1, kPieces = NV * (2 * kHp + 2), kStages = bwd_stages(NV, H32, MOST);
    const int step = blockDim.x;
    uint4* pieces = smem_pieces + threadIdx.x;
    Vec8 a_in[NV], a_post[NV], a_gate[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) a_in[k] = a_post[k] = a_gate[k] = Vec8{};
    auto slot_of = [&](int stage, int k) { return pieces + (stage * kPieces + k * (2 * kHp + 2)) * step; };
    auto ask = [&](int64_t t, int stage) {
        if (t < p.T) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (R.lane_in_row + k * warps * 32) * 8;
                uint4* slot = slot_of(stage, k);
                if (c < p.d) {
                    copy8<H32>(slot, step, p.h, t * p.d + c);
                    if (p.dh_out) copy8<H32>(slot + kHp * step, step, p.dh_out, t * p.d + c);
                    if (p.y) copy8<false>(slot + 2 * kHp * step, step, p.y, t * p.d + c);
                    if (p.w_in) copy8<false>(slot + (2 * kHp + 1) * step, step, p.dx, t * p.d + c);
                }
            }
        }
        copies_commit();
    };
    const int64_t stride = (int64_t)gridDim.x * rows;
    int64_t t = (int64_t)blockIdx.x * rows + R.grp;
#pragma unroll
    for (int i = 0; i < kStages; ++i) ask(t + i * stride, i);
    for (int stage = 0; t < p.T; t += stride, stage = stage + 1 == kStages ? 0 : stage + 1) {
        const int64_t at = t * p.d;
        const float ry = p.w_post ? p.rstd_y_in[t] : 1.f, rh = p.w_in ? p.rstd_h_in[t] : 0.f;
        Vec8 s[NV], n[NV], u[NV], g[NV];  // h', y r_y (or y), dx w_in, gradient
        float acc = 0.f;
        copies_wait<kStages - 1>();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint4* slot = slot_of(stage, k);
            s[k] = n[k] = u[k] = g[k] = Vec8{};
            if ((R.lane_in_row + k * warps * 32) * 8 < p.d) {
                s[k] = take8<H32>(slot, step);
                if (p.dh_out) g[k] = take8<H32>(slot + kHp * step, step);
                if (p.y) n[k] = take8<false>(slot + 2 * kHp * step, step);
                if (p.w_in) u[k] = take8<false>(slot + (2 * kHp + 1) * step, step);
            }
        }
        ask(t + kStages * stride, stage);  // (this row's pieces are in registers)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (R.lane_in_row + k * warps * 32) * 8;
            if (c < p.d) {
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
                    if (SUMS)
#pragma unroll
                        for (int e = 0; e < 8; ++e) a_in[k].v[e] += x.v[e];
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
                        if (SUMS)
#pragma unroll
                            for (int e = 0; e < 8; ++e) a_gate[k].v[e] += x.v[e];
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
                        if (SUMS)
#pragma unroll
                            for (int e = 0; e < 8; ++e) a_post[k].v[e] += x.v[e];
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
        float4* join = reinterpret_cast<float4*>(smem_pieces);  // [row group][3][half of 8 columns][vector]
        const int nvec = warps * 32 * NV;
        copies_wait<0>();
        __syncthreads();  // (the pieces are done with)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float4* q = join + ((R.grp * 3) * 2 + half) * nvec + R.lane_in_row + k * warps * 32;
                q[0] = *reinterpret_cast<float4*>(&a_in[k].v[4 * half]);
                q[2 * nvec] = *reinterpret_cast<float4*>(&a_post[k].v[4 * half]);
                q[4 * nvec] = *reinterpret_cast<float4*>(&a_gate[k].v[4 * half]);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 3 * (p.d >> 2); i += blockDim.x) {
            const int which = i / (p.d >> 2), c4 = i - which * (p.d >> 2);
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int grp = 0; grp < rows; ++grp) {
                const float4 q = join[((grp * 3 + which) * 2 + (c4 & 1)) * nvec + (c4 >> 1)];
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

static int bwd_grid(int64_t T, const RowPlan& P) { return (int)std::min<int64_t>(kSms, (T + P.rows - 1) / P.rows); }
size_t addnorm_part_bytes(int64_t T, int64_t d) {
    return (size_t)bwd_grid(T, plan_rows((int)d, kBwdCta)) * 3 * (size_t)d * 4;
}

template <typename K>
static cudaError_t launch_rows(K kernel, int grid, const RowPlan& P, size_t smem, const AddNormParams& p, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return e == cudaSuccess ? launch_pdl(kernel, dim3(grid), dim3(P.threads), smem, st, nullptr, 0, p, P.warps, P.rows) : e;
}
template <int NV, bool H32, bool W32>
static cudaError_t fwd_launch(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    const size_t smem = (size_t)fwd_stages(NV, H32) * NV * (H32 ? 3 : 2) * P.threads * 16;
    const int resident = P.threads <= 512 ? 2 * kSms : kSms;  // (64 registers a thread at most)
    const int grid = (int)std::min<int64_t>(resident, (p.T + P.rows - 1) / P.rows);
    return launch_rows(addnorm_fwd_kernel<NV, H32, W32>, grid, P, smem, p, st);
}
template <int NV, bool H32, bool W32, int MOST>
static cudaError_t bwd_launch(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    const int grid = bwd_grid(p.T, P);
    const size_t pieces = (size_t)bwd_stages(NV, H32, MOST) * NV * (H32 ? 6 : 4) * P.threads * 16;
    if (!(p.dw_in || p.dw_post || p.dgate))
        return launch_rows(addnorm_bwd_kernel<NV, H32, W32, false, MOST>, grid, P, pieces, p, st);
    const size_t join = (size_t)NV * 6 * P.threads * 16;
    cudaError_t e = launch_rows(addnorm_bwd_kernel<NV, H32, W32, true, MOST>, grid, P, std::max(pieces, join), p, st);
    if (e == cudaSuccess)
        e = launch_pdl(addnorm_join_kernel, dim3((unsigned)(p.d / 32), 3), dim3(256), 0, st, nullptr, 0, p, grid);
    return e;
}
template <int NV>
static cudaError_t fwd_types(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    if (p.h_f32) return p.w_f32 ? fwd_launch<NV, true, true>(p, P, st) : fwd_launch<NV, true, false>(p, P, st);
    return p.w_f32 ? fwd_launch<NV, false, true>(p, P, st) : fwd_launch<NV, false, false>(p, P, st);
}
template <int NV, int MOST>
static cudaError_t bwd_types(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    if (p.h_f32) return p.w_f32 ? bwd_launch<NV, true, true, MOST>(p, P, st) : bwd_launch<NV, true, false, MOST>(p, P, st);
    return p.w_f32 ? bwd_launch<NV, false, true, MOST>(p, P, st) : bwd_launch<NV, false, false, MOST>(p, P, st);
}

cudaError_t launch_addnorm_fwd(const AddNormParams& p, cudaStream_t st) {
    const RowPlan P = plan_rows(p.d, kFwdCta);
    return P.nv == 1 ? fwd_types<1>(p, P, st) : fwd_types<2>(p, P, st);
}
cudaError_t launch_addnorm_bwd(const AddNormParams& p, cudaStream_t st) {
    const RowPlan P = plan_rows(p.d, kBwdCta);
    if (P.nv == 2) return bwd_types<2, 1024>(p, P, st);
    return P.threads <= 512 ? bwd_types<1, 512>(p, P, st) : bwd_types<1, 1024>(p, P, st);
}

}  // namespace lm
