// Norms of query and key heads with the rotation by position in the same pass (include/lora_layer.h).
//   n = x r w,  r = rsqrt(mean x^2 + eps);    (a, b) -> f (a cos - b sin, b cos + a sin)
//   backward: g the rotation's transpose of dy,  dw = sum g x r,  dx = r (g w - x r^2 mean(g w x))
// A head is taken by up to 32 lanes, each two vectors of 8 (or 4) dims that hold whole pairs, so the rotation
// needs no other lane and a mean a few shuffles.  A warp takes one token: its angles serve all of the token's
// heads.  The angle's whole turns have to go before it is rounded: a frequency becomes a 64-bit fraction of a
// turn, and position times that, modulo 2^64, is the angle's place in its turn to 2^-33 of one for positions
// up to 2^31.  Queries and keys have CTAs of their own, so the backward's weights and sums over tokens are one
// set of registers; a second kernel joins the CTAs' sums in order.
#include <algorithm>

#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

constexpr int kRopeThreads = 256, kRopeWarps = kRopeThreads / 32;
constexpr int kRopeSms = 152;  // GB300's: a workspace's size has to be known on a host without one
// heads of a lane whose loads are in flight at once
constexpr int kFwdHeads = 4, kBwdHeads = 2;

// f / (2 pi) as a fraction of a turn in units of 2^-64, whole turns left out.  f = m 2^e with a 24-bit m; 1 / (2 pi)
// to 128 bits.
__device__ __forceinline__ uint64_t turn_of(float f) {
    constexpr uint64_t kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;
    const uint32_t b = __float_as_uint(f), ex = b >> 23 & 255u;
    const uint64_t m = ex ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
    const int k = 150 - (int)(ex ? ex : 1u);  // f = m 2^-k
    const uint64_t w0 = m * kLo, c = __umul64hi(m, kLo), lo = m * kHi;
    const uint64_t w1 = lo + c, w2 = __umul64hi(m, kHi) + (w1 < lo);  // m / (2 pi) = w2 w1 . w0 (units of 2^-64 from w1 on)
    uint64_t t;
    if (k <= -64) t = 0;
    else if (k < 0) t = w1 << -k | w0 >> (64 + k);
    else if (k == 0) t = w1;
    else if (k < 64) t = w1 >> k | w2 << (64 - k);
    else t = k < 128 ? w2 >> (k - 64) : 0;
    return b >> 31 ? 0 - t : t;
}

template <int VEC>
struct Vec {
    uint32_t r[VEC / 2];
    __device__ __forceinline__ void load(const uint16_t* p) {
        if (VEC == 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            r[0] = v.x, r[1] = v.y, r[VEC / 2 - 2] = v.z, r[VEC / 2 - 1] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            r[0] = v.x, r[1] = v.y;
        }
    }
    __device__ __forceinline__ void store(uint16_t* p) const {
        if (VEC == 8) *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[VEC / 2 - 2], r[VEC / 2 - 1]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
    }
};

// A lane's 2 VEC dims of a head: pair e is (a[e], b[e]).
template <int VEC>
struct Dims {
    float a[VEC], b[VEC];
    // the two vectors hold the pairs' first and second dims, or (inter) whole pairs
    __device__ __forceinline__ void from(const Vec<VEC>& u, const Vec<VEC>& v, bool inter) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (inter) {
                const uint32_t w = e < VEC / 2 ? u.r[e % (VEC / 2)] : v.r[e % (VEC / 2)];
                a[e] = bf16lo(w), b[e] = bf16hi(w);
            } else {
                a[e] = e & 1 ? bf16hi(u.r[e / 2]) : bf16lo(u.r[e / 2]);
                b[e] = e & 1 ? bf16hi(v.r[e / 2]) : bf16lo(v.r[e / 2]);
            }
        }
    }
    __device__ __forceinline__ void to(Vec<VEC>& u, Vec<VEC>& v, bool inter) const {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            u.r[i] = inter ? pack_bf16x2(a[i], b[i]) : pack_bf16x2(a[2 * i], a[2 * i + 1]);
            v.r[i] = inter ? pack_bf16x2(a[VEC / 2 + i], b[VEC / 2 + i]) : pack_bf16x2(b[2 * i], b[2 * i + 1]);
        }
    }
};

// What a lane is to its heads: which of them (of `hpw` a warp), which dims.
template <int VEC, bool INTER>
struct Place {
    int sub, hpw;     // head of the warp's
    bool on, turns;   // this lane has dims; they are rotated
    int at[2];        // first dims of its two vectors
    int pair;         // its first pair
    bool inter;
    __device__ __forceinline__ explicit Place(const QkRopeParams& p) {
        const int lane = threadIdx.x & 31, j = lane & (p.lanes - 1), nr = p.rot / (2 * VEC);
        sub = lane / p.lanes;
        hpw = 32 / p.lanes;
        on = j * 2 * VEC < p.d;
        turns = j < nr;
        inter = INTER || !turns;  // (dims that are not rotated: any two)
        pair = j * VEC;
        at[0] = inter ? j * 2 * VEC : j * VEC;
        at[1] = inter ? at[0] + VEC : p.rot / 2 + j * VEC;
    }
    // dim of pair e's first and second
    __device__ __forceinline__ int first(int e) const { return INTER || !turns ? at[0] + 2 * e : at[0] + e; }
    __device__ __forceinline__ int second(int e) const { return INTER || !turns ? at[0] + 2 * e + 1 : at[1] + e; }
};

// cos and sin of a lane's pairs for one token, times the factor.
template <int VEC>
struct Turns {
    uint64_t f[VEC];
    int axis[VEC];
    float c[VEC], s[VEC];
    template <bool INTER>
    __device__ __forceinline__ void frequencies(const QkRopeParams& p, const Place<VEC, INTER>& at) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            f[e] = at.turns ? turn_of(p.inv_freq[at.pair + e]) : 0;
            axis[e] = at.turns && p.axis ? min(max(p.axis[at.pair + e], 0), p.axes - 1) : 0;
        }
    }
    __device__ __forceinline__ static int64_t position(const QkRopeParams& p, int axis, int64_t t) {
        if (!p.pos) return t;
        const int64_t i = axis * p.T + t;
        return p.pos_i64 ? static_cast<const int64_t*>(p.pos)[i] : static_cast<const int32_t*>(p.pos)[i];
    }
    __device__ __forceinline__ void at_token(const QkRopeParams& p, bool turns, int64_t t) {
        if (!turns) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) c[e] = 1.f, s[e] = 0.f;
            return;
        }
        const int64_t one = p.axis ? 0 : position(p, 0, t);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const uint64_t turn = (uint64_t)(p.axis ? position(p, axis[e], t) : one) * f[e];
            // within half a turn of zero, where the fast sine's absolute error is below 2^-21
            __sincosf((float)(int32_t)(turn >> 32) * 1.4629180792671596e-9f, &s[e], &c[e]);
            c[e] *= p.factor;
            s[e] *= p.factor;
        }
    }
};
template <int VEC, bool INTER>
__device__ __forceinline__ void weights_of(const QkRopeParams& p, const RopeSide& S, const Place<VEC, INTER>& at, float (&wa)[VEC],
                                           float (&wb)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        wa[e] = wb[e] = 1.f;
        if (S.w && at.on) {
            const int i = at.first(e), j = at.second(e);
            if (p.w_f32) wa[e] = static_cast<const float*>(S.w)[i], wb[e] = static_cast<const float*>(S.w)[j];
            else wa[e] = bf16lo(static_cast<const uint16_t*>(S.w)[i]), wb[e] = bf16lo(static_cast<const uint16_t*>(S.w)[j]);
            wa[e] += p.w_offset, wb[e] += p.w_offset;
        }
    }
}
// over the lanes of a head, the same in all of them
__device__ __forceinline__ float head_sum(float x, int lanes) {
    for (int o = lanes >> 1; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int VEC, bool NORM, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2) qkrope_fwd_kernel(const __grid_constant__ QkRopeParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const bool keys = (int)blockIdx.x >= p.q.blocks;
    const RopeSide& S = keys ? p.k : p.q;
    const Place<VEC, INTER> at(p);
    Turns<VEC> turn;
    turn.frequencies(p, at);
    float wa[VEC], wb[VEC];
    if (NORM) weights_of(p, S, at, wa, wb);
    const float inv_d = 1.f / (float)p.d;
    const int64_t items = p.T * S.parts, step = (int64_t)S.blocks * kRopeWarps;
    const int batch = at.hpw * kFwdHeads;
    for (int64_t item = (int64_t)((int)blockIdx.x - (keys ? p.q.blocks : 0)) * kRopeWarps + (threadIdx.x >> 5); item < items; item += step) {
        const int64_t t = item / S.parts;
        const int part = (int)(item - t * S.parts);
        const int h0 = part * S.per_part, h1 = min(S.heads, h0 + S.per_part);
        turn.at_token(p, at.turns, t);
        const uint16_t* x = S.x + t * S.x_ts;
        uint16_t* y = S.y + t * S.y_ts;
        for (int h = h0 + at.sub; h - at.sub < h1; h += batch) {
            Vec<VEC> u[kFwdHeads][2];
#pragma unroll
            for (int i = 0; i < kFwdHeads; ++i) {
                const int hh = h + i * at.hpw;
                u[i][0] = u[i][1] = Vec<VEC>{};
                if (hh < h1 && at.on)
                    for (int v = 0; v < 2; ++v) u[i][v].load(x + hh * S.x_hs + at.at[v]);
            }
#pragma unroll
            for (int i = 0; i < kFwdHeads; ++i) {
                const int hh = h + i * at.hpw;
                Dims<VEC> n;
                n.from(u[i][0], u[i][1], at.inter);
                if (NORM) {
                    float sq = 0.f;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) sq = fmaf(n.a[e], n.a[e], fmaf(n.b[e], n.b[e], sq));
                    const float r = rsqrtf(fmaf(head_sum(sq, p.lanes), inv_d, p.eps));
#pragma unroll
                    for (int e = 0; e < VEC; ++e) n.a[e] *= r * wa[e], n.b[e] *= r * wb[e];
                }
                Dims<VEC> z;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    z.a[e] = n.a[e] * turn.c[e] - n.b[e] * turn.s[e];
                    z.b[e] = n.b[e] * turn.c[e] + n.a[e] * turn.s[e];
                }
                z.to(u[i][0], u[i][1], at.inter);
                if (hh < h1 && at.on)
                    for (int v = 0; v < 2; ++v) u[i][v].store(y + hh * S.y_hs + at.at[v]);
            }
        }
    }
}

template <int VEC, bool NORM, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2) qkrope_bwd_kernel(const __grid_constant__ QkRopeParams p) {
    __shared__ float join[kRopeWarps][256];
    griddep_launch_dependents();
    griddep_wait();
    const bool keys = (int)blockIdx.x >= p.q.blocks;
    const RopeSide& S = keys ? p.k : p.q;
    const Place<VEC, INTER> at(p);
    Turns<VEC> turn;
    turn.frequencies(p, at);
    float wa[VEC], wb[VEC], da[VEC], db[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) da[e] = db[e] = 0.f;
    if (NORM) weights_of(p, S, at, wa, wb);
    const float inv_d = 1.f / (float)p.d;
    const int64_t items = p.T * S.parts, step = (int64_t)S.blocks * kRopeWarps;
    const int batch = at.hpw * kBwdHeads;
    for (int64_t item = (int64_t)((int)blockIdx.x - (keys ? p.q.blocks : 0)) * kRopeWarps + (threadIdx.x >> 5); item < items; item += step) {
        const int64_t t = item / S.parts;
        const int part = (int)(item - t * S.parts);
        const int h0 = part * S.per_part, h1 = min(S.heads, h0 + S.per_part);
        turn.at_token(p, at.turns, t);
        const uint16_t* x = S.x + t * S.x_ts;
        const uint16_t* dy = S.dy + t * S.dy_ts;
        uint16_t* dx = S.y + t * S.y_ts;
        for (int h = h0 + at.sub; h - at.sub < h1; h += batch) {
            Vec<VEC> u[kBwdHeads][2], w[kBwdHeads][2];
#pragma unroll
            for (int i = 0; i < kBwdHeads; ++i) {
                const int hh = h + i * at.hpw;
                u[i][0] = u[i][1] = w[i][0] = w[i][1] = Vec<VEC>{};
                if (hh < h1 && at.on)
                    for (int v = 0; v < 2; ++v) {
                        w[i][v].load(dy + hh * S.dy_hs + at.at[v]);
                        if (NORM) u[i][v].load(x + hh * S.x_hs + at.at[v]);
                    }
            }
#pragma unroll
            for (int i = 0; i < kBwdHeads; ++i) {
                const int hh = h + i * at.hpw;
                Dims<VEC> z, g;
                z.from(w[i][0], w[i][1], at.inter);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    g.a[e] = z.a[e] * turn.c[e] + z.b[e] * turn.s[e];
                    g.b[e] = z.b[e] * turn.c[e] - z.a[e] * turn.s[e];
                }
                if (NORM) {
                    Dims<VEC> n;
                    n.from(u[i][0], u[i][1], at.inter);
                    float sq = 0.f, dot = 0.f;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        sq = fmaf(n.a[e], n.a[e], fmaf(n.b[e], n.b[e], sq));
                        dot = fmaf(g.a[e] * wa[e], n.a[e], fmaf(g.b[e] * wb[e], n.b[e], dot));
                    }
                    for (int o = p.lanes >> 1; o; o >>= 1) {
                        sq += __shfl_xor_sync(0xffffffffu, sq, o);
                        dot += __shfl_xor_sync(0xffffffffu, dot, o);
                    }
                    const float r = rsqrtf(fmaf(sq, inv_d, p.eps)), m = dot * inv_d * r * r;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        da[e] = fmaf(g.a[e], n.a[e] * r, da[e]);
                        db[e] = fmaf(g.b[e], n.b[e] * r, db[e]);
                        g.a[e] = r * (g.a[e] * wa[e] - n.a[e] * m);
                        g.b[e] = r * (g.b[e] * wb[e] - n.b[e] * m);
                    }
                }
                g.to(w[i][0], w[i][1], at.inter);
                if (hh < h1 && at.on)
                    for (int v = 0; v < 2; ++v) w[i][v].store(dx + hh * S.y_hs + at.at[v]);
            }
        }
    }
    if (!NORM || !S.dw) return;
    // the heads of a warp, then the warps, in order
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        for (int o = p.lanes; o < 32; o <<= 1) {
            da[e] += __shfl_xor_sync(0xffffffffu, da[e], o);
            db[e] += __shfl_xor_sync(0xffffffffu, db[e], o);
        }
    if (at.sub == 0 && at.on)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            join[threadIdx.x >> 5][at.first(e)] = da[e];
            join[threadIdx.x >> 5][at.second(e)] = db[e];
        }
    __syncthreads();
    if ((int)threadIdx.x < p.d) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kRopeWarps; ++w) s += join[w][threadIdx.x];
        p.part[(int64_t)blockIdx.x * p.d + threadIdx.x] = s;
    }
}

// dw of queries (CTA 0) and keys (CTA 1): the sums of the CTAs' partial rows, eight interleaved and then joined.
__global__ void __launch_bounds__(1024) qkrope_join_kernel(const __grid_constant__ QkRopeParams p) {
    __shared__ float sm[1024];
    griddep_launch_dependents();
    griddep_wait();
    const RopeSide& S = blockIdx.y ? p.k : p.q;
    if (!S.dw) return;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    const float* part = p.part + (int64_t)(blockIdx.y ? p.q.blocks : 0) * p.d;
    float s = 0.f;
    if (c < p.d)
#pragma unroll 4
        for (int i = w; i < S.blocks; i += 32) s += part[(int64_t)i * p.d + c];
    sm[threadIdx.x] = s;
    __syncthreads();
    if (w == 0 && c < p.d) {
        for (int i = 1; i < 32; ++i) s += sm[i * 32 + threadIdx.x];
        S.dw[c] = s;
    }
}

// ------------------------------------------------------------------ launches
constexpr int kRopeCtas = 2;  // a SM
size_t qkrope_part_bytes(int d) { return (size_t)kRopeCtas * kRopeSms * d * 4; }

static void plan(QkRopeParams& p, int heads_at_once) {
    p.vec = p.d % 16 == 0 && p.rot % 16 == 0 ? 8 : 4;
    p.lanes = 1;
    while (p.lanes * 2 * p.vec < p.d) p.lanes *= 2;
    const int batch = 32 / p.lanes * heads_at_once, all = kRopeCtas * kRopeSms;
    const int hq = p.q.heads, hk = p.k.heads;
    for (RopeSide* S : {&p.q, &p.k}) {
        S->parts = S->per_part = 1;
        S->blocks = 0;
        if (!S->heads) continue;
        // a token's heads are shared among warps where there are fewer tokens than warps
        const int most = (S->heads + batch - 1) / batch;
        const int64_t warps = (int64_t)all * kRopeWarps * S->heads / (hq + hk);
        S->parts = (int)std::max<int64_t>(1, std::min<int64_t>(most, warps / std::max<int64_t>(1, p.T)));
        S->per_part = (most + S->parts - 1) / S->parts * batch;
        S->parts = (S->heads + S->per_part - 1) / S->per_part;
        const int share = S == &p.k && hq ? all - std::max(1, std::min(all - 1, (all * hq + (hq + hk) / 2) / (hq + hk)))
                                          : hk ? std::max(1, std::min(all - 1, (all * hq + (hq + hk) / 2) / (hq + hk))) : all;
        S->blocks = (int)std::min<int64_t>(share, (p.T * S->parts + kRopeWarps - 1) / kRopeWarps);
    }
}

template <int VEC, bool NORM, bool INTER>
static cudaError_t launch(const QkRopeParams& p, bool backward, cudaStream_t st) {
    const dim3 grid((unsigned)(p.q.blocks + p.k.blocks));
    if (!backward) return launch_pdl(qkrope_fwd_kernel<VEC, NORM, INTER>, grid, dim3(kRopeThreads), 0, st, nullptr, 0, p);
    cudaError_t e = launch_pdl(qkrope_bwd_kernel<VEC, NORM, INTER>, grid, dim3(kRopeThreads), 0, st, nullptr, 0, p);
    if (e == cudaSuccess && (p.q.dw || p.k.dw))
        e = launch_pdl(qkrope_join_kernel, dim3((unsigned)((p.d + 31) / 32), 2), dim3(1024), 0, st, nullptr, 0, p);
    return e;
}
template <int VEC>
static cudaError_t launch_forms(const QkRopeParams& p, bool backward, cudaStream_t st) {
    if (p.norm) return p.interleaved ? launch<VEC, true, true>(p, backward, st) : launch<VEC, true, false>(p, backward, st);
    return p.interleaved ? launch<VEC, false, true>(p, backward, st) : launch<VEC, false, false>(p, backward, st);
}
cudaError_t launch_qkrope(QkRopeParams p, bool backward, cudaStream_t st) {
    plan(p, backward ? kBwdHeads : kFwdHeads);
    return p.vec == 8 ? launch_forms<8>(p, backward, st) : launch_forms<4>(p, backward, st);
}

}  // namespace lm
