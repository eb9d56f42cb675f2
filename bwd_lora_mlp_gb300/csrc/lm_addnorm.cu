// Residual add with the norms before and after a block (include/lora_layer.h).
//   forward   n = y r_y w_post,  h' = h + alpha gate n,  x = h' r_h w_in,   r_a = rsqrt(mean a^2 + eps)
//   backward  g = dh' + r_h (dx w_in - h' r_h^2 mean(dx w_in h')),  dh = g,  dn = alpha gate g,
//             dy = r_y (dn w_post - y r_y^2 mean(dn w_post y)),
//             dw_in = sum dx h' r_h,  dw_post = sum dn y r_y,  dgate = sum alpha g n
// Bound by memory as long as a row's arithmetic takes less than its bytes: each tensor of the row is
// read and written once.  A thread holds 8 or 16 columns, the same ones for every row its CTA walks, so the
// row stays in registers between its two means, and the backward's weights and its three sums over tokens
// are registers too (up to 4096 columns).  Each thread copies its own 16-byte pieces of the next rows to
// shared memory asynchronously, so reads are in flight while a row is normalised.  Small rows share a
// CTA; its row groups join their sums at its end and a second kernel joins the CTAs', both in order.
// Measured: 8192 x 4096 with all of it, forward 51 us, 5.3 TB/s (0.78 of the copy rate), backward 88 us,
// 4.6 TB/s (0.67); 3001 x 8192 with an fp32 stream 63 and 104 us (4.7 and 4.2 TB/s).  What is left is the
// two means a row, a barrier each.  (Weights and sums in shared memory: 1000 bytes of it moved per thread
// and row, its pipe as busy as the memory, 108 us for the 8192 x 4096 backward.)
#include <algorithm>

#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

// GB300's, not asked of the device: a workspace's size has to be known on a host without one, and the sums over
// tokens, by CTA, are the same bits everywhere.
constexpr int kSms = 152;

// A row takes `warps` warps, each thread NV vectors of 8 columns; a CTA holds `rows` of them.
struct RowPlan {
    int nv, warps, rows, threads;
};
// 512 threads, or what one row needs (at most 1024); `one`: the widest row with one vector a thread
static RowPlan plan_rows(int d, int one) {
    RowPlan P;
    P.nv = d > one ? 2 : 1;
    P.warps = (d / 8 + 32 * P.nv - 1) / (32 * P.nv);
    P.rows = std::min(15, std::max(1, 512 / (32 * P.warps)));  // (a barrier each, besides the CTA's)
    P.threads = P.rows * P.warps * 32;
    return P;
}
// Two vectors a thread halve what the means cost per column.  The forward has registers for it: 8192 x 4096
// 61 us with one, 51 with two; at 2048 columns one vector is already a CTA of two rows.  The backward's
// weights and sums do not fit then: 88 us with one, 139 with two; it takes two only where one does not fit.
constexpr int kFwdOne = 2048, kBwdOne = 4096;
// Rows on their way: as many as the shared memory holds beside a first-level cache for the weights that
// are not in registers.  (8192 x 4096 forward: 51 us with two, 56 with three and less cache.)
constexpr int fwd_stages(int nv, int most) { return nv == 1 ? 3 : most <= 512 ? 2 : 1; }
constexpr int bwd_stages(int nv, bool h32, int most) { return nv == 1 ? 3 : most <= 512 && !h32 ? 2 : 1; }

// ------------------------------------------------------------------ eight columns, as pairs
struct F8 {
    float2 v[4];
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ F8 zeros() { return F8{{both(0.f), both(0.f), both(0.f), both(0.f)}}; }
__device__ __forceinline__ F8 unpack8(const uint4& a) {
    return F8{{make_float2(bf16lo(a.x), bf16hi(a.x)), make_float2(bf16lo(a.y), bf16hi(a.y)),
               make_float2(bf16lo(a.z), bf16hi(a.z)), make_float2(bf16lo(a.w), bf16hi(a.w))}};
}
__device__ __forceinline__ F8 from4(const float4& a, const float4& b) {
    return F8{{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}
// eight values of a vector or a row, plus an offset
__device__ __forceinline__ F8 weight8(const void* w, int64_t c, bool f32, float offset) {
    F8 r;
    if (f32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
        r = from4(q[0], q[1]);
    } else {
        r = unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) r.v[e] = __fadd2_rn(r.v[e], both(offset));
    return r;
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const F8& r) {
    if (F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(r.v[0].x, r.v[0].y, r.v[1].x, r.v[1].y);
        q[1] = make_float4(r.v[2].x, r.v[2].y, r.v[3].x, r.v[3].y);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
            make_uint4(pack_bf16x2(r.v[0].x, r.v[0].y), pack_bf16x2(r.v[1].x, r.v[1].y), pack_bf16x2(r.v[2].x, r.v[2].y),
                       pack_bf16x2(r.v[3].x, r.v[3].y));
    }
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
__device__ __forceinline__ F8 take8(const uint4* slot, int step) {
    if (F32) return from4(*reinterpret_cast<const float4*>(slot), *reinterpret_cast<const float4*>(slot + step));
    return unpack8(*slot);
}

// ------------------------------------------------------------------ the threads of one row
struct RowGroup {
    int warps, grp, lane;  // lane: of the row's threads
    float *mine, *all;     // this warp's slot and this lane's warp's: [2][32] floats of the CTA, by warp
    bool has;

    __device__ __forceinline__ RowGroup(int warps_, float* red) : warps(warps_) {
        const int warp = (int)threadIdx.x >> 5, in_warp = (int)threadIdx.x & 31;
        grp = warp / warps;
        lane = (int)threadIdx.x - grp * warps * 32;
        mine = red + warp;
        has = in_warp < warps;
        all = red + grp * warps + (has ? in_warp : 0);
    }
    // sum over the row's threads, the same in all of them; the additions' order is fixed.  A row's two sums
    // use buffer 0 and 1, and rows with one sum alternate: a buffer is written again a barrier after its
    // last read
    __device__ __forceinline__ float sum(float2 q, int buf) {
        float x = q.x + q.y;
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (warps == 1) return x;
        if ((threadIdx.x & 31) == 0) mine[buf * 32] = x;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(warps * 32) : "memory");
        x = has ? all[buf * 32] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x;
    }
};

template <int NV, bool H32, bool W32, int MOST>
__global__ void __launch_bounds__(MOST, 1024 / MOST)
    addnorm_fwd_kernel(const __grid_constant__ AddNormParams p, int warps, int rows) {
    constexpr int kHp = H32 ? 2 : 1, kPieces = kHp + 1, kStages = fwd_stages(NV, MOST);
    __shared__ float red[2 * 32];
    extern __shared__ uint4 smem_raw[];  // [stage][vector][piece][thread]
    griddep_launch_dependents();
    griddep_wait();
    RowGroup R(warps, red);
    const int step = blockDim.x;
    const float inv_d = 1.f / (float)p.d;
    uint4* pieces = smem_raw + threadIdx.x;
    int c[NV];
    bool on[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) c[k] = (R.lane + k * warps * 32) * 8;
#pragma unroll
    for (int k = 0; k < NV; ++k) on[k] = c[k] < p.d;
    const int64_t stride = (int64_t)gridDim.x * rows, hop = stride * p.d;
    int64_t t = (int64_t)blockIdx.x * rows + R.grp;
    int64_t next = t * p.d + c[0];  // the first element that is asked for next
    auto ask = [&](int64_t t, int stage) {
        if (t < p.T) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (on[k]) {
                    uint4* slot = pieces + (stage * NV + k) * kPieces * step;
                    const int64_t i = next + k * warps * 256;
                    copy8<H32>(slot, step, p.h, i);
                    if (p.y) copy8<false>(slot + kHp * step, step, p.y, i);
                }
        }
        next += hop;
        copies_commit();  // (a group a turn, empty ones too: the wait below counts them)
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) ask(t + i * stride, i);
    const int flip = (p.y && p.w_post) && p.w_in ? 0 : 1;  // (one sum a row)
    int buf = 0;
    int64_t at = t * p.d - hop;
    for (int stage = 0; t < p.T; t += stride, stage = stage + 1 == kStages ? 0 : stage + 1) {
        at += hop;
        copies_wait<kStages - 1>();
        F8 h[NV], y[NV];
        float2 sq = both(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on[k]) {
                const uint4* slot = pieces + (stage * NV + k) * kPieces * step;
                h[k] = take8<H32>(slot, step);
                if (p.y) {
                    y[k] = take8<false>(slot + kHp * step, step);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sq = __ffma2_rn(y[k].v[e], y[k].v[e], sq);
                }
            }
        ask(t + kStages * stride, stage);  // (the pieces are in registers)
        buf ^= flip;
        if (p.y) {
            float ry = 1.f;
            if (p.w_post) {
                ry = rsqrtf(fmaf(R.sum(sq, buf), inv_d, p.eps));
                if (R.lane == 0) p.rstd_y[t] = ry;
            }
            const float2 ry2 = both(ry);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (on[k]) {
                    if (p.w_post) {
                        const F8 w = weight8(p.w_post, c[k], W32, p.w_offset);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[k].v[e] = __fmul2_rn(__fmul2_rn(y[k].v[e], ry2), w.v[e]);
                    }
                    if (p.gate) {
                        const F8 w = weight8(p.gate, c[k], W32, 0.f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[k].v[e] = __fmul2_rn(y[k].v[e], w.v[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[k].v[e] = __ffma2_rn(both(p.alpha), y[k].v[e], h[k].v[e]);
                    store8<H32>(p.h_out, at + c[k], h[k]);
                }
        }
        if (!p.w_in) continue;
        sq = both(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on[k])
#pragma unroll
                for (int e = 0; e < 4; ++e) sq = __ffma2_rn(h[k].v[e], h[k].v[e], sq);
        const float rh = rsqrtf(fmaf(R.sum(sq, buf ^ 1), inv_d, p.eps));
        if (R.lane == 0) p.rstd_h[t] = rh;
        const float2 rh2 = both(rh);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on[k]) {
                const F8 w = weight8(p.w_in, c[k], W32, p.w_offset);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[k].v[e] = __fmul2_rn(__fmul2_rn(h[k].v[e], rh2), w.v[e]);
                store8<false>(p.x, at + c[k], h[k]);
            }
    }
}

// ------------------------------------------------------------------ backward
// Sums over tokens of a CTA's rows to part[CTA][wanted sum][d].  POST: y is normed; GATE: it is gated.  W32
// (the weights' type) counts where the weights are read row by row, NV == 2.
template <int NV, bool H32, bool W32, bool POST, bool GATE, int MOST>
__global__ void __launch_bounds__(MOST, 1) addnorm_bwd_kernel(const __grid_constant__ AddNormParams p, int warps, int rows) {
    constexpr int kHp = H32 ? 2 : 1, kPieces = 2 * kHp + 2, kStages = bwd_stages(NV, H32, MOST);
    constexpr bool KEEP = NV == 1;
    const bool w32 = KEEP ? p.w_f32 : W32;
    __shared__ float red[2 * 32];
    extern __shared__ uint4 smem_raw[];
    griddep_launch_dependents();
    griddep_wait();
    RowGroup R(warps, red);
    const int step = blockDim.x;
    const float inv_d = 1.f / (float)p.d;
    const float2 alpha = both(p.alpha);
    uint4* pieces = smem_raw + threadIdx.x;
    int c[NV];
    bool on[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) c[k] = (R.lane + k * warps * 32) * 8;
    F8 w_post[NV], ag[NV], w_in[NV], a_in[NV], a_post[NV], a_gate[NV];
    auto weights_y = [&](int k) {
        if (POST) w_post[k] = weight8(p.w_post, c[k], w32, p.w_offset);
        if (GATE) {
            ag[k] = weight8(p.gate, c[k], w32, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) ag[k].v[e] = __fmul2_rn(ag[k].v[e], alpha);
        }
    };
    auto weight_in = [&](int k) {
        if (p.w_in) w_in[k] = weight8(p.w_in, c[k], w32, p.w_offset);
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        on[k] = c[k] < p.d;
        a_in[k] = a_post[k] = a_gate[k] = zeros();
        if (KEEP && on[k]) {
            weight_in(k);
            weights_y(k);
        }
    }
    auto slot_of = [&](int stage, int k) { return pieces + (stage * NV + k) * kPieces * step; };
    const int64_t stride = (int64_t)gridDim.x * rows, hop = stride * p.d;
    int64_t t = (int64_t)blockIdx.x * rows + R.grp;
    int64_t next = t * p.d + c[0];  // the first element that is asked for next
    auto ask = [&](int64_t t, int stage) {
        if (t < p.T) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (on[k]) {
                    uint4* slot = slot_of(stage, k);
                    const int64_t i = next + k * warps * 256;
                    copy8<H32>(slot, step, p.h, i);
                    if (p.dh_out) copy8<H32>(slot + kHp * step, step, p.dh_out, i);
                    if (p.y) copy8<false>(slot + 2 * kHp * step, step, p.y, i);
                    if (p.w_in) copy8<false>(slot + (2 * kHp + 1) * step, step, p.dx, i);
                }
        }
        next += hop;
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) ask(t + i * stride, i);
    float ry_next = 1.f, rh_next = 0.f;
    auto rstds = [&](int64_t t) {
        if (t >= p.T) return;
        if (POST) ry_next = p.rstd_y_in[t];
        if (p.w_in) rh_next = p.rstd_h_in[t];
    };
    rstds(t);
    const int flip = POST && p.w_in ? 0 : 1;  // (one sum a row)
    int buf = 0;
    int64_t at = t * p.d - hop;
    for (int stage = 0; t < p.T; t += stride, stage = stage + 1 == kStages ? 0 : stage + 1) {
        at += hop;
        const float2 ry = both(ry_next), rh = both(rh_next);
        rstds(t + stride);
        F8 s[NV], n[NV], u[NV], g[NV];  // h' r_h, y r_y (or y), dx w_in, gradient
        float2 acc = both(0.f);
        copies_wait<kStages - 1>();
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on[k]) {
                const uint4* slot = slot_of(stage, k);
                s[k] = take8<H32>(slot, step);
                if (p.y) {
                    if (!KEEP) weights_y(k);
                    n[k] = take8<false>(slot + 2 * kHp * step, step);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (POST) n[k].v[e] = __fmul2_rn(n[k].v[e], ry);
                        const float2 add = POST ? __fmul2_rn(n[k].v[e], w_post[k].v[e]) : n[k].v[e];
                        s[k].v[e] = __ffma2_rn(GATE ? ag[k].v[e] : alpha, add, s[k].v[e]);
                    }
                }
                if (p.w_in) {
                    if (!KEEP) weight_in(k);
                    u[k] = take8<false>(slot + (2 * kHp + 1) * step, step);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[k].v[e] = __fmul2_rn(s[k].v[e], rh);
                        a_in[k].v[e] = __ffma2_rn(u[k].v[e], s[k].v[e], a_in[k].v[e]);
                        u[k].v[e] = __fmul2_rn(u[k].v[e], w_in[k].v[e]);
                        acc = __ffma2_rn(u[k].v[e], s[k].v[e], acc);
                    }
                }
                if (p.dh_out) g[k] = take8<H32>(slot + kHp * step, step);
                else g[k] = zeros();
            }
        ask(t + kStages * stride, stage);  // (this row's pieces are in registers)
        buf ^= flip;
        if (p.w_in) {
            const float2 m = both(-R.sum(acc, buf) * inv_d);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (on[k])
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        g[k].v[e] = __ffma2_rn(rh, __ffma2_rn(m, s[k].v[e], u[k].v[e]), g[k].v[e]);
        }
        acc = both(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on[k]) {
                store8<H32>(p.dh, at + c[k], g[k]);
                if (p.y) {
                    if (!KEEP) weights_y(k);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (GATE)
                            a_gate[k].v[e] =
                                __ffma2_rn(g[k].v[e], POST ? __fmul2_rn(n[k].v[e], w_post[k].v[e]) : n[k].v[e], a_gate[k].v[e]);
                        g[k].v[e] = __fmul2_rn(g[k].v[e], GATE ? ag[k].v[e] : alpha);  // dn
                        if (POST) {
                            a_post[k].v[e] = __ffma2_rn(g[k].v[e], n[k].v[e], a_post[k].v[e]);
                            g[k].v[e] = __fmul2_rn(g[k].v[e], w_post[k].v[e]);
                            acc = __ffma2_rn(g[k].v[e], n[k].v[e], acc);
                        }
                    }
                    if (!POST) store8<false>(p.dy, at + c[k], g[k]);
                }
            }
        if (POST) {
            const float2 m = both(-R.sum(acc, buf ^ 1) * inv_d);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (on[k]) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) g[k].v[e] = __fmul2_rn(ry, __ffma2_rn(m, n[k].v[e], g[k].v[e]));
                    store8<false>(p.dy, at + c[k], g[k]);
                }
        }
    }
    const int s_post = p.dw_in ? 1 : 0, s_gate = s_post + (p.dw_post ? 1 : 0), nsums = s_gate + (p.dgate ? 1 : 0);
    if (!nsums) return;
    // the row groups' sums in order
    float4* join = reinterpret_cast<float4*>(smem_raw);  // [row group][sum][half of 8 columns][vector]
    const int nvec = warps * 32 * NV;
    copies_wait<0>();
    __syncthreads();  // (the pieces are done with)
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        auto put = [&](int which, const F8& a, float f) {
            float4* q = join + (R.grp * nsums + which) * 2 * nvec + R.lane + k * warps * 32;
            q[0] = make_float4(a.v[0].x * f, a.v[0].y * f, a.v[1].x * f, a.v[1].y * f);
            q[nvec] = make_float4(a.v[2].x * f, a.v[2].y * f, a.v[3].x * f, a.v[3].y * f);
        };
        if (p.dw_in) put(0, a_in[k], 1.f);
        if (p.dw_post) put(s_post, a_post[k], 1.f);
        if (p.dgate) put(s_gate, a_gate[k], p.alpha);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nsums * (p.d >> 2); i += blockDim.x) {
        const int which = i / (p.d >> 2), c4 = i - which * (p.d >> 2);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int grp = 0; grp < rows; ++grp) {
            const float4 q = join[((grp * nsums + which) * 2 + (c4 & 1)) * nvec + (c4 >> 1)];
            s.x += q.x, s.y += q.y, s.z += q.z, s.w += q.w;
        }
        *reinterpret_cast<float4*>(p.part + ((int64_t)blockIdx.x * nsums + which) * p.d + 4 * c4) = s;
    }
}

// The sum over the CTAs' `n` partial rows of 32 columns: 8 threads a column take every eighth, then join.
struct JoinOut {
    float* out[3];
};
__global__ void __launch_bounds__(256) addnorm_join_kernel(const float* all, int d, int n, JoinOut outs) {
    __shared__ float sm[8][32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const float* part = all + (int64_t)blockIdx.y * d + c;
    float s = 0.f;
#pragma unroll 10
    for (int i = w; i < n; i += 8) s += part[(int64_t)i * gridDim.y * d];
    sm[w][lane] = s;
    __syncthreads();
    if (w == 0) {
        for (int i = 1; i < 8; ++i) s += sm[i][lane];
        outs.out[blockIdx.y][c] = s;
    }
}

// ------------------------------------------------------------------ launches
static int bwd_grid(int64_t T, const RowPlan& P) { return (int)std::min<int64_t>(kSms, (T + P.rows - 1) / P.rows); }
size_t addnorm_part_bytes(int64_t T, int64_t d) {
    return (size_t)bwd_grid(T, plan_rows((int)d, kBwdOne)) * 3 * (size_t)d * 4;
}

template <typename K>
static cudaError_t launch_rows(K kernel, int grid, const RowPlan& P, size_t smem, const AddNormParams& p, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return e == cudaSuccess ? launch_pdl(kernel, dim3(grid), dim3(P.threads), smem, st, nullptr, 0, p, P.warps, P.rows) : e;
}
template <int NV, bool H32, bool W32, int MOST>
static cudaError_t fwd_launch(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    const size_t smem = (size_t)fwd_stages(NV, MOST) * NV * (H32 ? 3 : 2) * P.threads * 16;
    const int grid = (int)std::min<int64_t>(1024 / MOST * kSms, (p.T + P.rows - 1) / P.rows);
    return launch_rows(addnorm_fwd_kernel<NV, H32, W32, MOST>, grid, P, smem, p, st);
}
template <int NV, int MOST>
static cudaError_t fwd_types(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    if (p.h_f32) return p.w_f32 ? fwd_launch<NV, true, true, MOST>(p, P, st) : fwd_launch<NV, true, false, MOST>(p, P, st);
    return p.w_f32 ? fwd_launch<NV, false, true, MOST>(p, P, st) : fwd_launch<NV, false, false, MOST>(p, P, st);
}
template <int NV, bool H32, bool W32, bool POST, bool GATE, int MOST>
static cudaError_t bwd_launch(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    const int grid = bwd_grid(p.T, P);
    JoinOut outs{};
    int nsums = 0;
    for (float* o : {p.dw_in, p.dw_post, p.dgate})
        if (o) outs.out[nsums++] = o;
    const size_t pieces = (size_t)bwd_stages(NV, H32, MOST) * NV * (H32 ? 6 : 4) * P.threads * 16;
    const size_t join = (size_t)nsums * NV * P.threads * 32;
    cudaError_t e = launch_rows(addnorm_bwd_kernel<NV, H32, W32, POST, GATE, MOST>, grid, P, std::max(pieces, join), p, st);
    if (e == cudaSuccess && nsums)
        e = launch_pdl(addnorm_join_kernel, dim3((unsigned)(p.d / 32), (unsigned)nsums), dim3(256), 0, st, nullptr, 0,
                       (const float*)p.part, p.d, grid, outs);
    return e;
}
template <int NV, bool H32, bool W32, int MOST>
static cudaError_t bwd_forms(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    if (p.w_post) return p.gate ? bwd_launch<NV, H32, W32, true, true, MOST>(p, P, st) : bwd_launch<NV, H32, W32, true, false, MOST>(p, P, st);
    return p.gate ? bwd_launch<NV, H32, W32, false, true, MOST>(p, P, st) : bwd_launch<NV, H32, W32, false, false, MOST>(p, P, st);
}
template <int NV, int MOST>
static cudaError_t bwd_types(const AddNormParams& p, const RowPlan& P, cudaStream_t st) {
    if constexpr (NV == 2)
        if (p.w_f32) return p.h_f32 ? bwd_forms<NV, true, true, MOST>(p, P, st) : bwd_forms<NV, false, true, MOST>(p, P, st);
    return p.h_f32 ? bwd_forms<NV, true, false, MOST>(p, P, st) : bwd_forms<NV, false, false, MOST>(p, P, st);
}

cudaError_t launch_addnorm_fwd(const AddNormParams& p, cudaStream_t st) {
    const RowPlan P = plan_rows(p.d, kFwdOne);
    if (P.nv == 2) return P.threads <= 512 ? fwd_types<2, 512>(p, P, st) : fwd_types<2, 1024>(p, P, st);
    return fwd_types<1, 512>(p, P, st);
}
cudaError_t launch_addnorm_bwd(const AddNormParams& p, cudaStream_t st) {
    const RowPlan P = plan_rows(p.d, kBwdOne);
    if (P.nv == 1) return bwd_types<1, 512>(p, P, st);
    return P.threads <= 512 ? bwd_types<2, 512>(p, P, st) : bwd_types<2, 1024>(p, P, st);
}

}  // namespace lm
