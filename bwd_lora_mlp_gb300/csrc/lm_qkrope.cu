// Norms of query and key heads with the rotation by position in the same pass (include/lora_layer.h).
//   n = x r w,  r = rsqrt(mean x^2 + eps);    (a, b) -> f (a cos - b sin, b cos + a sin)
//   backward: g the rotation's transpose of dy,  dw = sum g x r,  dx = r (g w - x r^2 mean(g w x))  (multiplied in this order:
//   r^3 overflows where a head and eps are tiny)
// A head is taken by up to 32 lanes, each two vectors of 8 (or 4) dims that hold whole pairs, so the rotation
// needs no other lane and a mean a few shuffles.  A warp takes one token at a time: its angles, formed by a lane each
// and exchanged in shared memory, serve all of the token's heads.  The next heads are on their way to shared memory
// meanwhile (each thread copies its own pieces: no barrier).  The angle's whole turns have to go before it is rounded: a
// frequency becomes a 64-bit fraction of a turn, and position times that, modulo 2^64, is the angle's place in its turn
// to 2^-33 of one for positions up to 2^31.  Queries and keys have CTAs of their own, so the backward's weights and
// sums over tokens are one set of registers; a second kernel joins the CTAs' sums in order.
// Bound by memory as far as its arithmetic lets it: 8192 tokens, 32 + 8 heads of 128 read from a fused buffer, 78 us a
// step in a graph, forward 30 (5.6 TB/s, 0.83 of the copy rate) and backward 49 (5.1); 16384 tokens 140 us, 5.9 TB/s.
// (Heads loaded to registers four at a time by the lane and the angles formed by every lane for itself: 116 and 205.)
#include <algorithm>

#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

constexpr int kRopeThreads = 256, kRopeWarps = kRopeThreads / 32;
constexpr int kRopeSms = 152;  // GB300's: a workspace's size has to be known on a host without one
// Heads of a lane at a step (two forward: two chains of shuffles and reciprocal roots at a time; the backward has
// registers for one), steps on their way, CTAs an SM.  (Three or more steps, or three CTAs of fewer registers, are no
// faster: 16384 tokens 154 us a step against 146 before positions came ahead, too.)
constexpr int kFwdHeads = 2, kFwdStages = 2, kBwdStages = 2, kFwdCtas = 2, kBwdCtas = 2;
static_assert(2 * kFwdHeads * kFwdStages * kRopeThreads * 16 + kRopeWarps * 2048 <= 48 * 1024 &&
              4 * kBwdStages * kRopeThreads * 16 + kRopeWarps * 2048 <= 48 * 1024, "more shared memory has to be asked for");
// Items a warp has at least, where tokens have parts enough (4097 tokens of 24 heads of 80, CTAs by heads: 24.5 us; with 16, 26.6).
constexpr int kTurns = 4;
static_assert(kFwdStages < 4 && kBwdStages < 4, "a place of positions would be written while it is read");

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

// A lane's 2 VEC dims of a head: pair e is (a, b)[e], kept two to a register pair.
template <int VEC>
struct Dims {
    float2 a[VEC / 2], b[VEC / 2];
    // its two vectors (u first) hold the pairs' first and second dims, or (inter) whole pairs
    __device__ __forceinline__ void from(const uint32_t (&u)[VEC], bool inter) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const uint32_t x = inter ? u[2 * i] : u[i], y = inter ? u[2 * i + 1] : u[VEC / 2 + i];
            a[i] = inter ? make_float2(bf16lo(x), bf16lo(y)) : make_float2(bf16lo(x), bf16hi(x));
            b[i] = inter ? make_float2(bf16hi(x), bf16hi(y)) : make_float2(bf16lo(y), bf16hi(y));
        }
    }
    __device__ __forceinline__ void to(uint32_t (&u)[VEC], bool inter) const {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const uint32_t x = inter ? pack_bf16x2(a[i].x, b[i].x) : pack_bf16x2(a[i].x, a[i].y);
            const uint32_t y = inter ? pack_bf16x2(a[i].y, b[i].y) : pack_bf16x2(b[i].x, b[i].y);
            u[inter ? 2 * i : i] = x;
            u[inter ? 2 * i + 1 : VEC / 2 + i] = y;
        }
    }
};
__device__ __forceinline__ float2 both2(float x) { return make_float2(x, x); }

// What a lane is to its heads: which of them (of `hpw` a warp), which dims.  The lanes' first vectors lie next to each
// other, and so do their second ones: 32 bytes of neighbouring dims a lane would ask for every sector twice
// (16384 tokens in neighbouring pairs: forward 76 us, backward 133).
template <int VEC, bool INTER>
struct Place {
    int sub, hpw;     // head of the warp's
    bool on;          // this lane has dims
    int at[2];        // first dims of its two vectors
    bool turns[2];    // pairs [0, VEC / 2) and the others are rotated, by the angles from pair[0] and from pair[1] on
    int pair[2];
    __device__ __forceinline__ explicit Place(const QkRopeParams& p) {
        const int lane = threadIdx.x & 31;
        sub = lane / p.lanes;
        hpw = 32 / p.lanes;
        const int j = lane - sub * p.lanes;
        on = j * 2 * VEC < p.d && sub < hpw;
        if (INTER) {
            at[0] = j * VEC;
            at[1] = p.d / 2 + j * VEC;
            for (int v = 0; v < 2; ++v) {
                turns[v] = at[v] < p.rot;
                pair[v] = at[v] / 2;
            }
        } else {
            const bool in = j * 2 * VEC < p.rot;  // (dims that are not rotated: the halves of what is left)
            at[0] = in ? j * VEC : p.rot / 2 + j * VEC;
            at[1] = in ? p.rot / 2 + j * VEC : p.d / 2 + j * VEC;
            turns[0] = turns[1] = in;
            pair[0] = j * VEC;
            pair[1] = j * VEC + VEC / 2;
        }
    }
    // dims of pair e's first and second
    __device__ __forceinline__ int first(int e) const { return INTER ? at[e / (VEC / 2)] + 2 * (e % (VEC / 2)) : at[0] + e; }
    __device__ __forceinline__ int second(int e) const { return INTER ? first(e) + 1 : at[1] + e; }
};

// A warp's way through its (token, part of the heads) items, `heads` at a step.  The same in all of its lanes, and made
// so in the compiler's eyes too.  (Items fit 32 bits: the tokens do, and only few tokens have parts.)
struct Walk {
    uint32_t item, t;
    int h, h1;  // the step's first head, and the part's end
    uint32_t n; // items begun before this one
    __device__ __forceinline__ Walk(const RopeSide& S, int first_block) {
        item = __shfl_sync(0xffffffffu, (blockIdx.x - first_block) * kRopeWarps + (threadIdx.x >> 5), 0);
        n = 0;
        begin(S);
    }
    __device__ __forceinline__ bool more(const QkRopeParams& p, const RopeSide& S) const { return item < (uint32_t)p.T * (uint32_t)S.parts; }
    __device__ __forceinline__ void begin(const RopeSide& S) {
        t = item;
        h = 0;
        h1 = S.heads;
        if (S.parts > 1) {
            t = item / (uint32_t)S.parts;
            h = (int)(item - t * (uint32_t)S.parts) * S.per_part;
            h1 = min(S.heads, h + S.per_part);
        }
    }
    // true: the next item has begun
    __device__ __forceinline__ bool next(const RopeSide& S, int heads) {
        h += heads;
        if (h < h1) return false;
        item += (uint32_t)S.blocks * kRopeWarps;
        ++n;
        begin(S);
        return true;
    }
    __device__ __forceinline__ int64_t at(int64_t ts, int64_t hs) const { return (int64_t)t * ts + (int64_t)h * hs; }
};

// The positions of a warp's coming items: copied ahead with their first heads, an axis a lane.  (Read where they are
// needed, they were waited for at every item: 16384 tokens 146 us a step, 143 so; 4097 with three axes 28, 24.5 so.)  Four
// items are on their way at most.
constexpr int kPosAxes = 32, kPosItems = 4;
struct Positions {
    char* slots;  // the warp's
    __device__ __forceinline__ explicit Positions(char* mine) : slots(mine) {}
    __device__ __forceinline__ static bool ahead(const QkRopeParams& p) { return p.pos && p.axes <= kPosAxes; }
    __device__ __forceinline__ void ask(const QkRopeParams& p, const Walk& A) const {
        const int a = threadIdx.x & 31;
        if (!ahead(p) || a >= p.axes) return;
        const uint32_t dst = smem_u32(slots + ((A.n % kPosItems) * kPosAxes + a) * 8);
        const int64_t i = (int64_t)a * p.T + A.t;
        if (p.pos_i64)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(static_cast<const int64_t*>(p.pos) + i) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(static_cast<const int32_t*>(p.pos) + i) : "memory");
    }
    __device__ __forceinline__ int64_t at(const QkRopeParams& p, const Walk& W, int axis) const {
        if (!p.pos) return W.t;
        if (!ahead(p)) {
            const int64_t i = (int64_t)axis * p.T + W.t;
            return p.pos_i64 ? static_cast<const int64_t*>(p.pos)[i] : static_cast<const int32_t*>(p.pos)[i];
        }
        const char* q = slots + ((W.n % kPosItems) * kPosAxes + axis) * 8;
        return p.pos_i64 ? *reinterpret_cast<const int64_t*>(q) : *reinterpret_cast<const int32_t*>(q);
    }
};

// The angles of a token, once for the warp: each lane forms up to four pairs' cosines and sines (times the factor)
// and leaves them in shared memory, where lanes of every head find theirs.
struct Angles {
    uint64_t f[4];
    int axis[4];
    float *c, *s;  // the warp's, 128 each
    __device__ __forceinline__ Angles(const QkRopeParams& p, float* mine) : c(mine), s(mine + 128) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = (threadIdx.x & 31) + 32 * i;
            const bool on = e < p.rot / 2;
            f[i] = on ? turn_of(p.inv_freq[e]) : 0;
            axis[i] = on && p.axis ? min(max(p.axis[e], 0), p.axes - 1) : 0;
        }
    }
    __device__ __forceinline__ void at_token(const QkRopeParams& p, const Positions& pos, const Walk& W) {
        __syncwarp();  // (the last token's have been read; this one's positions are there)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = (threadIdx.x & 31) + 32 * i;
            if (32 * i >= p.rot / 2) break;
            const uint64_t turn = (uint64_t)pos.at(p, W, axis[i]) * f[i];
            // within half a turn of zero, where the fast sine's absolute error is below 2^-21
            float sn, cs;
            __sincosf((float)(int32_t)(turn >> 32) * 1.4629180792671596e-9f, &sn, &cs);
            if (e < p.rot / 2) c[e] = cs * p.factor, s[e] = sn * p.factor;
        }
        __syncwarp();
    }
    template <int VEC, bool INTER>
    __device__ __forceinline__ void take(const Place<VEC, INTER>& at, float2 (&cc)[VEC / 2], float2 (&ss)[VEC / 2], float2 (&ns)[VEC / 2]) const {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const int v = i / (VEC / 4), e = at.pair[v] + 2 * (i % (VEC / 4));
            cc[i] = at.turns[v] ? *reinterpret_cast<const float2*>(c + e) : make_float2(1.f, 1.f);
            ss[i] = at.turns[v] ? *reinterpret_cast<const float2*>(s + e) : make_float2(0.f, 0.f);
            ns[i] = make_float2(-ss[i].x, -ss[i].y);
        }
    }
};
template <int VEC, bool INTER>
__device__ __forceinline__ void weights_of(const QkRopeParams& p, const RopeSide& S, const Place<VEC, INTER>& at,
                                           float2 (&wa)[VEC / 2], float2 (&wb)[VEC / 2]) {
    auto w = [&](int i) {
        if (!S.w || !at.on) return 1.f;
        return p.w_offset + (p.w_f32 ? static_cast<const float*>(S.w)[i] : bf16lo(static_cast<const uint16_t*>(S.w)[i]));
    };
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        wa[i] = make_float2(w(at.first(2 * i)), w(at.first(2 * i + 1)));
        wb[i] = make_float2(w(at.second(2 * i)), w(at.second(2 * i + 1)));
    }
}

// A thread's pieces of heads on their way: slot [stage][vector][thread], written and read by the same thread, so
// no barrier is needed between the copy and its use.
template <int VEC>
struct Pieces {
    static constexpr int kBytes = VEC * 2;  // of a vector
    char* slots;
    __device__ __forceinline__ explicit Pieces(void* smem) : slots(static_cast<char*>(smem) + threadIdx.x * kBytes) {}
    __device__ __forceinline__ char* slot(int i) const { return slots + i * (kRopeThreads * kBytes); }
    __device__ __forceinline__ void ask(int i, const uint16_t* src) const {
        if (VEC == 8) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot(i))), "l"(src) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(slot(i))), "l"(src) : "memory");
    }
    // lanes without dims count nothing in their head's sums
    __device__ __forceinline__ void clear(int n) const {
        for (int i = 0; i < n; ++i) {
            if constexpr (VEC == 8) *reinterpret_cast<uint4*>(slot(i)) = make_uint4(0, 0, 0, 0);
            else *reinterpret_cast<uint2*>(slot(i)) = make_uint2(0, 0);
        }
    }
    // vectors i and i + 1
    __device__ __forceinline__ void take(int i, uint32_t (&u)[VEC]) const {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            if constexpr (VEC == 8) {
                const uint4 x = *reinterpret_cast<const uint4*>(slot(i + v));
                u[4 * v] = x.x, u[4 * v + 1] = x.y, u[4 * v + 2] = x.z, u[4 * v + 3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(slot(i + v));
                u[2 * v] = x.x, u[2 * v + 1] = x.y;
            }
        }
    }
};
template <int VEC>
__device__ __forceinline__ void store_vecs(uint16_t* dst, int gap, const uint32_t (&u)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4*>(dst + gap) = make_uint4(u[4], u[5], u[6], u[7]);
    } else {
        *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[1]);
        *reinterpret_cast<uint2*>(dst + gap) = make_uint2(u[2], u[3]);
    }
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_for() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float rsqrt_fast(float x) {  // (2^-22.9 of itself; x at least eps, which is no subnormal)
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int VEC, bool NORM, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kFwdCtas) qkrope_fwd_kernel(const __grid_constant__ QkRopeParams p) {
    extern __shared__ uint4 smem[];
    __shared__ __align__(16) float angles[kRopeWarps][256];
    __shared__ __align__(8) char coming[kRopeWarps][kPosItems * kPosAxes * 8];
    griddep_launch_dependents();
    griddep_wait();
    const bool keys = (int)blockIdx.x >= p.q.blocks;
    const RopeSide& S = keys ? p.k : p.q;
    const Place<VEC, INTER> at(p);
    const Pieces<VEC> pieces(smem);
    const Positions pos(coming[threadIdx.x >> 5]);
    Walk W(S, keys ? p.q.blocks : 0);
    if (!W.more(p, S)) return;
    Walk A = W;  // asks kFwdStages steps ahead
    const int heads = kFwdHeads * at.hpw, gap = at.at[1] - at.at[0];
    const uint16_t* x = S.x + at.sub * S.x_hs + at.at[0];
    uint16_t* y = S.y + at.sub * S.y_hs + at.at[0];
    const int64_t x_step = at.hpw * S.x_hs, y_step = at.hpw * S.y_hs;
    bool fresh_ask = true;
    auto ask = [&](int stage) {
        if (A.more(p, S)) {
            const uint16_t* src = x + A.at(S.x_ts, S.x_hs);
#pragma unroll
            for (int i = 0; i < kFwdHeads; ++i)
                if (at.on && A.h + i * at.hpw + at.sub < A.h1) {
                    pieces.ask((stage * kFwdHeads + i) * 2, src + i * x_step);
                    pieces.ask((stage * kFwdHeads + i) * 2 + 1, src + i * x_step + gap);
                }
            if (fresh_ask) pos.ask(p, A);
            fresh_ask = A.next(S, heads);
        }
        commit();  // (a group a turn, empty ones too: the wait below counts them)
    };
    if (!at.on) pieces.clear(2 * kFwdHeads * kFwdStages);
#pragma unroll
    for (int i = 0; i < kFwdStages; ++i) ask(i);
    Angles angle(p, angles[threadIdx.x >> 5]);
    float2 wa[VEC / 2], wb[VEC / 2], c[VEC / 2], s[VEC / 2], ns[VEC / 2];
    if (NORM) weights_of(p, S, at, wa, wb);
    const float inv_d = 1.f / (float)p.d;
    bool fresh = true;
    for (int stage = 0; W.more(p, S); stage = stage + 1 == kFwdStages ? 0 : stage + 1) {
        wait_for<kFwdStages - 1>();
        if (fresh) {
            angle.at_token(p, pos, W);
            angle.take(at, c, s, ns);
        }
        uint32_t u[kFwdHeads][VEC];
#pragma unroll
        for (int i = 0; i < kFwdHeads; ++i) pieces.take((stage * kFwdHeads + i) * 2, u[i]);
        ask(stage);
        float r[kFwdHeads];
        if (NORM) {
#pragma unroll
            for (int i = 0; i < kFwdHeads; ++i) {
                Dims<VEC> n;
                n.from(u[i], INTER);
                float2 sq = both2(0.f);
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) sq = __ffma2_rn(n.a[e], n.a[e], __ffma2_rn(n.b[e], n.b[e], sq));
                r[i] = sq.x + sq.y;
            }
            for (int o = p.lanes >> 1; o; o >>= 1)
#pragma unroll
                for (int i = 0; i < kFwdHeads; ++i) r[i] += __shfl_xor_sync(0xffffffffu, r[i], o);
        }
        uint16_t* dst = y + W.at(S.y_ts, S.y_hs);
#pragma unroll
        for (int i = 0; i < kFwdHeads; ++i) {
            Dims<VEC> n, z;
            n.from(u[i], INTER);
            if (NORM) {
                const float2 r2 = both2(rsqrt_fast(fmaf(r[i], inv_d, p.eps)));
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    n.a[e] = __fmul2_rn(n.a[e], __fmul2_rn(r2, wa[e]));
                    n.b[e] = __fmul2_rn(n.b[e], __fmul2_rn(r2, wb[e]));
                }
            }
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                z.a[e] = __ffma2_rn(n.a[e], c[e], __fmul2_rn(n.b[e], ns[e]));
                z.b[e] = __ffma2_rn(n.b[e], c[e], __fmul2_rn(n.a[e], s[e]));
            }
            z.to(u[i], INTER);
            if (at.on && W.h + i * at.hpw + at.sub < W.h1) store_vecs<VEC>(dst + i * y_step, gap, u[i]);
        }
        fresh = W.next(S, heads);
    }
}

template <int VEC, bool NORM, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kBwdCtas) qkrope_bwd_kernel(const __grid_constant__ QkRopeParams p) {
    constexpr int kTensors = NORM ? 4 : 2;  // vectors of a head: dy, and for the norm x
    extern __shared__ uint4 smem[];
    __shared__ __align__(16) float angles[kRopeWarps][256];  // (in the end the warps' sums)
    __shared__ __align__(8) char coming[kRopeWarps][kPosItems * kPosAxes * 8];
    griddep_launch_dependents();
    griddep_wait();
    const bool keys = (int)blockIdx.x >= p.q.blocks;
    const RopeSide& S = keys ? p.k : p.q;
    const Place<VEC, INTER> at(p);
    const Pieces<VEC> pieces(smem);
    const Positions pos(coming[threadIdx.x >> 5]);
    Walk W(S, keys ? p.q.blocks : 0);
    Walk A = W;
    const int gap = at.at[1] - at.at[0];
    const uint16_t* dy = S.dy + at.sub * S.dy_hs + at.at[0];
    const uint16_t* x = NORM ? S.x + at.sub * S.x_hs + at.at[0] : nullptr;
    uint16_t* dx = S.y + at.sub * S.y_hs + at.at[0];
    bool fresh_ask = true;
    auto ask = [&](int stage) {
        if (A.more(p, S)) {
            if (at.on && A.h + at.sub < A.h1) {
                const uint16_t* src = dy + A.at(S.dy_ts, S.dy_hs);
                pieces.ask(kTensors * stage, src);
                pieces.ask(kTensors * stage + 1, src + gap);
                if (NORM) {
                    src = x + A.at(S.x_ts, S.x_hs);
                    pieces.ask(kTensors * stage + 2, src);
                    pieces.ask(kTensors * stage + 3, src + gap);
                }
            }
            if (fresh_ask) pos.ask(p, A);
            fresh_ask = A.next(S, at.hpw);
        }
        commit();
    };
    if (!at.on) pieces.clear(kTensors * kBwdStages);
#pragma unroll
    for (int i = 0; i < kBwdStages; ++i) ask(i);
    Angles angle(p, angles[threadIdx.x >> 5]);
    float2 wa[VEC / 2], wb[VEC / 2], c[VEC / 2], s[VEC / 2], ns[VEC / 2], da[VEC / 2], db[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) da[i] = db[i] = both2(0.f);
    if (NORM) weights_of(p, S, at, wa, wb);
    const float inv_d = 1.f / (float)p.d;
    bool fresh = true;
    for (int stage = 0; W.more(p, S); stage = stage + 1 == kBwdStages ? 0 : stage + 1) {
        wait_for<kBwdStages - 1>();
        if (fresh) {
            angle.at_token(p, pos, W);
            angle.take(at, c, s, ns);
        }
        const bool mine = at.on && W.h + at.sub < W.h1;
        uint32_t u[VEC];
        Dims<VEC> g, n;
        pieces.take(kTensors * stage, u);
        n.from(u, INTER);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            g.a[i] = __ffma2_rn(n.a[i], c[i], __fmul2_rn(n.b[i], s[i]));
            g.b[i] = __ffma2_rn(n.b[i], c[i], __fmul2_rn(n.a[i], ns[i]));
        }
        if (NORM) {
            pieces.take(kTensors * stage + 2, u);
            n.from(u, INTER);
        }
        ask(stage);
        if (NORM) {
            // t = g x, whose sums with r are dw's
            float2 sq = both2(0.f), dot = both2(0.f);
            Dims<VEC> t;
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                sq = __ffma2_rn(n.a[i], n.a[i], __ffma2_rn(n.b[i], n.b[i], sq));
                t.a[i] = __fmul2_rn(g.a[i], n.a[i]);
                t.b[i] = __fmul2_rn(g.b[i], n.b[i]);
                dot = __ffma2_rn(t.a[i], wa[i], __ffma2_rn(t.b[i], wb[i], dot));
            }
            float q = sq.x + sq.y, dt = dot.x + dot.y;
            for (int o = p.lanes >> 1; o; o >>= 1) {
                q += __shfl_xor_sync(0xffffffffu, q, o);
                dt += __shfl_xor_sync(0xffffffffu, dt, o);
            }
            const float r = rsqrt_fast(fmaf(q, inv_d, p.eps));
            const float2 r2 = both2(r), m = both2(-dt * inv_d * r * r);
            if (mine)  // (a slot that no copy came to holds anything)
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    da[i] = __ffma2_rn(t.a[i], r2, da[i]);
                    db[i] = __ffma2_rn(t.b[i], r2, db[i]);
                }
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                g.a[i] = __fmul2_rn(__ffma2_rn(n.a[i], m, __fmul2_rn(g.a[i], wa[i])), r2);
                g.b[i] = __fmul2_rn(__ffma2_rn(n.b[i], m, __fmul2_rn(g.b[i], wb[i])), r2);
            }
        }
        g.to(u, INTER);
        if (mine) store_vecs<VEC>(dx + W.at(S.y_ts, S.y_hs), gap, u);
        fresh = W.next(S, at.hpw);
    }
    if (!NORM || !S.dw) return;
    // the heads of a warp, then the warps, in order
    float* join = angles[threadIdx.x >> 5];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        float a = e & 1 ? da[e / 2].y : da[e / 2].x, b = e & 1 ? db[e / 2].y : db[e / 2].x;
        for (int o = p.lanes; o < 32; o <<= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (at.sub == 0 && at.on) {
            join[at.first(e)] = a;
            join[at.second(e)] = b;
        }
    }
    __syncthreads();
    if ((int)threadIdx.x < p.d) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kRopeWarps; ++w) x += angles[w][threadIdx.x];
        p.part[(int64_t)blockIdx.x * p.d + threadIdx.x] = x;
    }
}

// dw of queries (y = 0) and keys (y = 1): the sums of the CTAs' partial rows, 32 of them interleaved and then joined in order.
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
size_t qkrope_part_bytes(int d) { return (size_t)kBwdCtas * kRopeSms * d * 4; }

static void plan(QkRopeParams& p, int ctas, int heads_at_once) {
    p.vec = p.d % 16 == 0 && p.rot % 16 == 0 ? 8 : 4;
    p.lanes = 1;
    while (p.lanes * 2 * p.vec < p.d) p.lanes *= 2;
    // Without a norm lanes have nothing to exchange, and need be no power of two: as many as have dims, where a warp then takes
    // more heads.  (8192 tokens of 16 + 16 heads of 72: 42 us a step instead of 49; 4097 of 20 + 4 of 80 with three axes 20.5
    // instead of 21.1.  With the norm, whose sums then take thirds and fifths of a head in turn, 32 + 8 heads of 96 took 90 us
    // instead of 75, of 80 the same.)
    const int dims = (p.d + 2 * p.vec - 1) / (2 * p.vec);
    if (!p.norm && 32 / dims > 32 / p.lanes) p.lanes = dims;
    const int at_once = 32 / p.lanes * heads_at_once, all = ctas * kRopeSms;
    // CTAs by what a token takes, its steps and half of one for its angles; at least one each.  (8192 tokens of 32 + 1
    // heads, a step: 68 us, by heads alone 79, a whole step for the angles 73; 64 + 8: 129, 137, 133.)
    auto cost = [&](const RopeSide& S) { return (S.heads + at_once - 1) / at_once * 2 + 1; };
    const int both = cost(p.q) + cost(p.k);
    const int of_q = p.k.heads ? std::max(1, std::min(all - 1, (all * cost(p.q) + both / 2) / both)) : all;
    for (RopeSide* S : {&p.q, &p.k}) {
        S->parts = S->per_part = 1;
        S->blocks = 0;
        if (!S->heads) continue;
        const int most = S == &p.q ? of_q : all - of_q;
        // a token's heads are shared among warps while a warp has fewer than kTurns items: the warps' last ones then end
        // at about the same time
        const int turns = (S->heads + at_once - 1) / at_once;
        const int64_t want = (int64_t)most * kRopeWarps * kTurns;
        S->parts = (int)std::max<int64_t>(1, std::min<int64_t>(turns, want / std::max<int64_t>(1, p.T)));
        S->per_part = (turns + S->parts - 1) / S->parts * at_once;
        S->parts = (S->heads + S->per_part - 1) / S->per_part;
        S->blocks = (int)std::min<int64_t>(most, (p.T * S->parts + kRopeWarps - 1) / kRopeWarps);
    }
}

template <typename K>
static cudaError_t launch_pieces(K kernel, int pieces, const QkRopeParams& p, cudaStream_t st) {
    const size_t smem = (size_t)pieces * kRopeThreads * p.vec * 2;  // (48 KB at most with the angles and positions: no attribute is needed)
    return launch_pdl(kernel, dim3((unsigned)(p.q.blocks + p.k.blocks)), dim3(kRopeThreads), smem, st, nullptr, 0, p);
}
template <int VEC, bool NORM, bool INTER>
static cudaError_t launch(const QkRopeParams& p, bool backward, cudaStream_t st) {
    if (!backward) return launch_pieces(qkrope_fwd_kernel<VEC, NORM, INTER>, 2 * kFwdHeads * kFwdStages, p, st);
    cudaError_t e = launch_pieces(qkrope_bwd_kernel<VEC, NORM, INTER>, (NORM ? 4 : 2) * kBwdStages, p, st);
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
    plan(p, backward ? kBwdCtas : kFwdCtas, backward ? 1 : kFwdHeads);
    return p.vec == 8 ? launch_forms<8>(p, backward, st) : launch_forms<4>(p, backward, st);
}

}  // namespace lm
