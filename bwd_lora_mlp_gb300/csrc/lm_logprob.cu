// Log probabilities of given tokens (include/lora_layer.h), with entropy and top alternatives.
//   m = max x,  S = sum e^{x-m},  w = sum e^{x-m} (x-m):  lse = m + log S,  H = log S - w / S
// Forward: one pass over the logits with running m, S, w per thread, joined over the CTA.  A row is
// one CTA's, or a cluster's of up to eight where there are fewer rows than the device holds CTAs, each
// taking a segment, joined through distributed shared memory.  The k alternatives: the k-th largest of
// the threads' own maxima bounds the k-th largest logit from below, so a second look (from L2) by the
// threads whose own maximum reaches the bound finds k of them among a few dozen; rows of equal logits
// (masked, flat) take another look or two.  Bound by memory:
// 4096 x 131072 bf16 171 us, 6.2 TB/s (0.92 of the copy rate); at 1000 x 50257 with five alternatives 42 us,
// 2.4 TB/s: 1000 rows on 608 CTA places, whose joins and second looks are as long as their passes.  (CTAs of 512
// threads: 176 and 51 us.)
// Backward: one pass, dx = scale (g 1[target] - p (g + gH (log p + H))): 4096 x 131072 372 us, 5.8 TB/s (0.85), as long
// as the two tensors' rows lie alike on 16 bytes; where they do not, elements go one by one: 1000 x 50257 read with
// a row stride of 50304 and written without gaps 304 us, with the same stride 45.
#include <algorithm>
#include <type_traits>

#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

constexpr int kThreads = 256;
constexpr int kMaxCluster = 8;
constexpr int kCand = 512;  // alternatives above the bound that fit (to place n of them takes n^2 / kThreads steps a thread)
constexpr float kL2e = 1.4426950408889634f;

__device__ __forceinline__ float lp_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ int64_t target_of(const LogprobParams& p, int64_t t) {
    const int64_t v = p.i64 ? static_cast<const int64_t*>(p.targets)[t] : static_cast<const int32_t*>(p.targets)[t];
    return v >= 0 && v < p.V ? v : -1;
}
// Larger keys for larger logits; +0 and -0 are equal, every NaN is the largest.  kNothing: that of -inf, the smallest.
constexpr uint32_t kNothing = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
// (key, index) as one number: larger logit first, then the lower index; 0 is none
__device__ __forceinline__ uint64_t rank_of(uint32_t key, uint32_t j) { return ((uint64_t)key << 32) | (0xFFFFFFFFu - j); }
__device__ __forceinline__ uint64_t rank_of(float x, uint32_t j) { return rank_of(order_key(x), j); }

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

// f(v, index of vector 0) over [j0, j1) in batches of U whole vectors of a thread (vector u lies
// u kThreads vectors on; n of them are there), the next batch loading meanwhile, and one(x, index) for
// the single elements before the first and after the last 16-byte boundary.
template <int U, bool F32, typename F, typename G>
__device__ __forceinline__ void scan(const Row<F32>& row, int64_t j0, int64_t j1, F f, G one) {
    constexpr int W = Row<F32>::kVec;
    const int64_t a = min(j1, j0 + row.head(j0));
    const int nv = (int)((j1 - a) / W);
    const char* base = row.p + a * (F32 ? 4 : 2);
    uint4 next[U];
    auto load = [&](int v) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v + u * kThreads < nv) next[u] = *reinterpret_cast<const uint4*>(base + (int64_t)(v + u * kThreads) * 16);
    };
    load(threadIdx.x);
    for (int v = threadIdx.x; v < nv; v += U * kThreads) {
        uint32_t w[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) w[u][0] = next[u].x, w[u][1] = next[u].y, w[u][2] = next[u].z, w[u][3] = next[u].w;
        if (v + (U - 1) * kThreads >= nv)  // (the last batch of some threads: what is not there counts nothing)
#pragma unroll
            for (int u = 1; u < U; ++u)
                if (v + u * kThreads >= nv)
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[u][e] = F32 ? 0xFF800000u : 0xFF80FF80u;
        load(v + U * kThreads);
        f(w, a + (int64_t)v * W, nv - v);
    }
    const int64_t b = a + (int64_t)nv * W;
    const int64_t j = threadIdx.x < W ? j0 + threadIdx.x : b + (threadIdx.x - W);
    if (threadIdx.x < 2 * W && (threadIdx.x < W ? j < a : j < j1)) one(row.at(j), j);
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
struct Sums {
    float m, S, w;
};
// The sums of the parts held by N neighbouring lanes (N a power of two), the same in all of them: the largest
// maximum first, every part brought to it once, then plain sums in a fixed order.
template <int N>
__device__ __forceinline__ Sums join(Sums s) {
    float m = s.m;
#pragma unroll
    for (int o = N / 2; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float d = fmaxf(s.m - m, -1e30f), f = lp_ex2(d * kL2e);  // (where f is 0, any finite d does)
    // w moves with the maximum: sum e^{x-m} (x-m); an empty part counts nothing (a NaN sum is not empty)
    const bool any = s.S != 0.f;
    s.w = any ? f * fmaf(s.S, d, s.w) : 0.f;
    s.S = any ? s.S * f : 0.f;
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
        s.S += __shfl_xor_sync(0xffffffffu, s.S, o);
        s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
    }
    if (m != m) s.S = s.w = m;
    s.m = m;
    return s;
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

struct LpShared {
    Sums warp[kThreads / 32];
    float seg[kMaxCluster][3];
    uint64_t cand[kCand];
    uint64_t best[kMaxCluster * kMaxTop];  // the segments' alternatives (in CTA 0: of all)
    uint64_t mine[kMaxTop];
    uint64_t red[kThreads / 32];
    int count;
    int ties[kThreads / 32];
    // what segment_top leaves for segment_top_ties
    const char* row;
    int64_t j0, j1;
    uint32_t own_max[kThreads];
};
__shared__ LpShared sm;  // (the functions below that are not inlined address it directly)

// The k-th largest of the threads' maxima, down to bit `to` (the bits below are 0), and how many reach it.
__device__ __forceinline__ uint32_t kth_largest(uint32_t own_max, int k, int to, int& reach) {
    uint32_t bound = 0;
    reach = kThreads;
#pragma unroll 1
    for (int bit = 31; bit >= to; --bit) {
        const uint32_t t = bound | (1u << bit);
        const int n = __syncthreads_count(own_max >= t);
        if (n >= k) bound = t, reach = n;
    }
    return bound;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return key & 0x80000000u ? __uint_as_float(key & 0x7FFFFFFFu) : __uint_as_float(~key);
}
// What is at or above `least` (or NaN), or only what is above it, to the candidates; their number, which may be
// more than fit.  `look`: this thread's largest is among them.  FEW: they are expected to fit, and whether they do
// is not looked at on the way (1000 x 50257 with five alternatives: 30 us without, 37 with that).
template <bool FEW, bool F32>
__device__ __forceinline__ int collect(const Row<F32>& row, int64_t j0, int64_t j1, float least, bool strict, bool look) {
    constexpr int W = Row<F32>::kVec;
    auto take = [&](float x, int64_t j) {
        if (x < least || (strict && x == least)) return;
        const int at = atomicAdd(&sm.count, 1);
        if (at < kCand) sm.cand[at] = rank_of(x, (uint32_t)j);
    };
    if (look) scan<4>(row, j0, j1, [&](const uint32_t (&w)[4][4], int64_t j, int n) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t one[1][4] = {{w[u][0], w[u][1], w[u][2], w[u][3]}};
            if (u * kThreads < n && !(largest<1, F32>(one) < least) && (FEW || *(volatile int*)&sm.count <= kCand))
#pragma unroll 1
                for (int64_t i = j + (int64_t)u * kThreads * W, end = i + W; i < end; ++i) take(row.at(i), i);
        }
    }, take);
    __syncthreads();
    return sm.count;
}
// The candidates' k best to sm.mine: each one's place is the number of better ones (whatever order they came in).
__device__ __forceinline__ void place_candidates(int n, int k) {
    for (int c = threadIdx.x; c < n; c += kThreads) {
        const uint64_t r = sm.cand[c];
        int place = 0;
        for (int q = 0; q < n; ++q) place += sm.cand[q] > r;
        if (place < k) sm.mine[place] = r;
    }
}

// The k best of [j0, j1) (fewer if it is shorter: the rest are 0) to sm.mine, best first.  False: more reach the
// bound than fit, and nothing is done.
template <bool F32>
__device__ __noinline__ bool segment_top(const Row<F32>& row, int64_t j0, int64_t j1, int k, uint32_t own_max) {
    const int tid = threadIdx.x;
    if (tid < kMaxTop) sm.mine[tid] = 0;
    if (tid == 0) sm.count = 0;
    // 16 bits of the k-th largest of the threads' maxima: a little below it (of a bf16 nothing lies between), a
    // bound as good where logits differ.  What reaches it is in a thread whose own largest does
    int reach;
    const uint32_t bound = kth_largest(own_max, k, 16, reach);
    // (of logits that differ k threads and a few more reach it)
    const bool alike = reach > kThreads * 3 / 4 && j1 - j0 > kThreads;
    const int n = alike ? kCand + 1 : collect<true>(row, j0, j1, logit_of(bound), false, own_max >= bound);
    if (n > kCand) {
        if (tid == 0) sm.row = row.p, sm.j0 = j0, sm.j1 = j1;
        sm.own_max[tid] = own_max;
        __syncthreads();
        return false;
    }
    place_candidates(n, k);
    __syncthreads();
    return true;
}

// The same where more reach the bound than fit: masked rows, flat ones, fp32 logits that differ in their low bits
// only.  The bound is made exact, a logit's own key; then what is above it are few, and the rest are equal to
// it, from the lowest index up.  (Where it works on comes through shared memory: kept in registers for a call that
// is seldom made, it cost the kernel spills.  20 alternatives, all but ten logits masked: 4 rows of 131072 bf16
// 15 us, 1000 of 50257 79; 11 and 36 unmasked, 67 and 940 with a search of the segment for each alternative.)
template <bool F32>
__device__ __noinline__ void segment_top_ties(int k) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Row<F32> row{sm.row};
    const int64_t j0 = sm.j0, j1 = sm.j1;
    const uint32_t own_max = sm.own_max[tid];
    int reach;
    const uint32_t bound = kth_largest(own_max, k, 0, reach);
    int n = kCand + 1;
    bool ties = false;
    for (int strict = F32 && bound != kNothing ? 0 : 1; strict < 2 && n > kCand; ++strict) {
        if (tid == 0) sm.count = 0;
        __syncthreads();
        n = collect<false>(row, j0, j1, logit_of(bound), strict, strict ? own_max > bound : own_max >= bound);
        __syncthreads();
        ties = strict;
    }
    if (n > kCand) {  // a few threads hold most of the largest: k searches of the segment
        uint64_t last = ~0ull;
        for (int i = 0; i < k; ++i) {
            uint64_t b = 0;
            for (int64_t j = j0 + tid; j < j1; j += kThreads) {
                const uint64_t r = rank_of(row.at(j), (uint32_t)j);
                if (r < last && r > b) b = r;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) b = max(b, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)b, o));
            __syncthreads();
            if (lane == 0) sm.red[warp] = b;
            __syncthreads();
            last = 0;
            for (int q = 0; q < kThreads / 32; ++q) last = max(last, sm.red[q]);
            if (tid == 0) sm.mine[i] = last;
        }
        __syncthreads();
        return;
    }
    place_candidates(n, k);
    int have = ties ? min(n, k) : k;
    for (int64_t j = j0; have < k && j < j1; j += kThreads) {
        const bool tie = j + tid < j1 && order_key(row.at(j + tid)) == bound;
        const uint32_t votes = __ballot_sync(0xffffffffu, tie);
        __syncthreads();
        if (lane == 0) sm.ties[warp] = __popc(votes);
        __syncthreads();
        int before = have, total = 0;
        for (int q = 0; q < kThreads / 32; ++q) {
            if (q < warp) before += sm.ties[q];
            total += sm.ties[q];
        }
        const int place = before + __popc(votes & ((1u << lane) - 1u));
        if (tie && place < k) sm.mine[place] = rank_of(bound, (uint32_t)(j + tid));
        have += total;
    }
    __syncthreads();
}

template <bool F32>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logprob_fwd_kernel(const __grid_constant__ LogprobParams p, int cluster) {
    griddep_launch_dependents();
    if (cluster > 1) cluster_arrive();  // (waited for where the CTAs write to the first one's shared memory)
    griddep_wait();
    const int64_t t = blockIdx.x / cluster;
    const int part = cluster > 1 ? (int)cluster_rank() : 0;
    const Row<F32> row{static_cast<const char*>(p.logits) + t * p.ld * (F32 ? 4 : 2)};
    // segments of whole 64-element stretches
    const int64_t len = ((p.V + cluster - 1) / cluster + 63) / 64 * 64;
    const int64_t j0 = min(p.V, part * len), j1 = min(p.V, j0 + len);
    constexpr int W = Row<F32>::kVec;
    Sums s{-INFINITY, 0.f, 0.f};
    float own = -INFINITY;  // the thread's largest logit (NaN the largest)
    const bool plain = p.scale == 1.f;
    auto rise = [&](float big) {  // the running maximum follows, and the sums with it
        const float d = fmaxf(s.m - big, -1e30f), f = s.m == -INFINITY ? 0.f : lp_ex2(d * kL2e);  // (f 0: no 0 x inf)
        s.w = s.S > 0.f ? f * fmaf(s.S, d, s.w) : 0.f;
        s.S *= f;
        s.m = max_nan(s.m, big);  // (a NaN comes here every time and stays)
    };
    constexpr int U = 4;
    scan<U>(row, j0, j1, [&](uint32_t (&w)[U][4], int64_t, int) {
        float big = largest<U, F32>(w);
        own = max_nan(big, own);
        if (!plain) big = __fmul_rn(big, p.scale);
        if (!(big <= s.m)) rise(big);  // (a NaN comes here too)
        if (s.m == -INFINITY) return;
        auto add = [&](auto is_easy) {
            constexpr bool EASY = decltype(is_easy)::value;
            float2 S2[2] = {make_float2(s.S, 0.f), make_float2(0.f, 0.f)}, w2[2] = {make_float2(s.w, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < W; e += 2) {
                    float2 x = make_float2(logit<F32>(w[u], e), logit<F32>(w[u], e + 1));
                    if (!EASY) x = __fmul2_rn(x, make_float2(p.scale, p.scale));
                    const float2 d = __fadd2_rn(x, make_float2(-s.m, -s.m));
                    const float2 q = __fmul2_rn(d, make_float2(kL2e, kL2e));
                    const float2 y = make_float2(lp_ex2(q.x), lp_ex2(q.y));
                    S2[u & 1] = __fadd2_rn(S2[u & 1], y);
                    // (0 x -inf is none: where y is 0, any finite number does)
                    w2[u & 1] = __ffma2_rn(y, EASY ? d : make_float2(fmaxf(d.x, -1e30f), fmaxf(d.y, -1e30f)), w2[u & 1]);
                }
            s.S = (S2[0].x + S2[0].y) + (S2[1].x + S2[1].y);
            s.w = (w2[0].x + w2[0].y) + (w2[1].x + w2[1].y);
        };
        // bf16 as they are, m of an ordinary size: -inf made the lowest number in pairs, its difference is finite
        if (!F32 && plain && fabsf(s.m) < 1e36f) {
#pragma unroll
            for (int i = 0; i < 4 * U; ++i) w[i / 4][i % 4] = max2_nan(w[i / 4][i % 4], 0xFF7FFF7Fu);
            add(std::true_type{});
        } else {
            add(std::false_type{});
        }
    }, [&](float x, int64_t) {
        own = max_nan(x, own);
        x = __fmul_rn(x, p.scale);
        if (!(x <= s.m)) rise(x);
        if (x == -INFINITY) return;
        const float y = lp_ex2((x - s.m) * kL2e);
        s.S += y;
        s.w = fmaf(y, fmaxf(x - s.m, -1e30f), s.w);
    });
    if (s.m != s.m) s.S = s.w = s.m;
    s = join<32>(s);
    if ((threadIdx.x & 31) == 0) sm.warp[threadIdx.x >> 5] = s;
    __syncthreads();
    s = join<kThreads / 32>(sm.warp[threadIdx.x & (kThreads / 32 - 1)]);
    if (p.k && !segment_top(row, j0, j1, p.k, order_key(own) & (j0 < j1 ? ~0u : 0u))) segment_top_ties<F32>(p.k);
    if (cluster > 1) {
        __syncwarp();
        cluster_wait();  // CTA 0 has started
        if (threadIdx.x == 0) {
            st_first(&sm.seg[part][0], s.m);
            st_first(&sm.seg[part][1], s.S);
            st_first(&sm.seg[part][2], s.w);
        }
        if (threadIdx.x < p.k) st_first(&sm.best[part * p.k + threadIdx.x], sm.mine[threadIdx.x]);
        __syncwarp();
        cluster_sync();
        if (part) return;
        const int i = threadIdx.x & (kMaxCluster - 1);
        s = i < cluster ? Sums{sm.seg[i][0], sm.seg[i][1], sm.seg[i][2]} : Sums{-INFINITY, 0.f, 0.f};
        s = join<kMaxCluster>(s);
        const int n = cluster * p.k;
        if (threadIdx.x < n) {
            const uint64_t r = sm.best[threadIdx.x];
            int place = 0;
            for (int q = 0; q < n; ++q) place += sm.best[q] > r;
            if (r && place < p.k) sm.mine[place] = r;
        }
        __syncthreads();
    }
    const bool empty = s.m == -INFINITY;
    const float lse = empty ? -INFINITY : s.m + logf(s.S);
    auto logp = [&](int64_t j) { return empty ? -INFINITY : __fmul_rn(row.at(j), p.scale) - lse; };
    if (threadIdx.x == 0) {
        const int64_t at = target_of(p, t);
        p.lse[t] = lse;
        p.logp[t] = at < 0 ? 0.f : logp(at);
        if (p.entropy) p.entropy[t] = empty ? 0.f : logf(s.S) - s.w / s.S;
    }
    if (threadIdx.x < p.k) {
        const uint32_t j = 0xFFFFFFFFu - (uint32_t)sm.mine[threadIdx.x];
        p.top_ids[t * p.k + threadIdx.x] = (int32_t)j;
        p.top_logp[t * p.k + threadIdx.x] = logp(j);
    }
}

template <bool F32>
static cudaError_t fwd_launch(const LogprobParams& p, cudaStream_t st) {
    // A CTA per row fills the 152 SMs from about four rows an SM on; with fewer, a row is shared, as long as
    // a CTA's segment keeps every thread a few vectors.  (4 rows of 131072 fp32, 20 alternatives: 8 CTAs a row
    // 15 us, 16 a row 21.)
    int c = 1;
    while (c < kMaxCluster && p.T * c * 2 <= 152 * 1024 / kThreads && p.V / (c * 2) >= kThreads * 8) c *= 2;
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim = {(unsigned)c, 1, 1};
    return launch_pdl(logprob_fwd_kernel<F32>, dim3((unsigned)(p.T * c)), dim3(kThreads), 0, st, &a, 1, p, c);
}
cudaError_t launch_logprob_fwd(const LogprobParams& p, cudaStream_t st) {
    return p.f32 ? fwd_launch<true>(p, st) : fwd_launch<false>(p, st);
}

// ------------------------------------------------------------------ backward
constexpr int kBwdThreads = 256;
constexpr int kBwdVecs = 8;  // 16-byte vectors of a thread: a CTA takes a stretch of 2048 of them
// e^x of this and of anything below is 0 in fp32; the factor beside it then stays finite for gradients up to 1e36
constexpr float kNoWeight = -128.f;

template <bool F32>
__global__ void __launch_bounds__(kBwdThreads) logprob_bwd_kernel(const __grid_constant__ LogprobParams p, unsigned per_row) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int W = Row<F32>::kVec;
    const int64_t t = blockIdx.x / per_row;
    const Row<F32> row{static_cast<const char*>(p.logits) + t * p.ld * (F32 ? 4 : 2)};
    char* out = static_cast<char*>(p.dlogits) + t * p.ld_out * (F32 ? 4 : 2);
    const int64_t at = target_of(p, t);
    const float lse = p.lse_in[t], gH = p.dentropy ? p.dentropy[t] : 0.f, H = p.dentropy ? p.entropy_in[t] : 0.f;
    const float g = p.dlogp && at >= 0 ? p.dlogp[t] : 0.f;
    const bool empty = lse == -INFINITY;
    const float k0 = -p.scale * fmaf(gH, H, g), k1 = -p.scale * gH, at_target = p.scale * g;
    // scale (-p (g + gH (log p + H))); where p = 0 any finite factor does
    auto soft = [&](float x) {
        const float lp = __fmul_rn(x, p.scale) - lse;
        return empty ? 0.f : lp_ex2(lp * kL2e) * fmaf(k1, fmaxf(lp, kNoWeight), k0);
    };
    auto grad = [&](float x, int64_t j) { return soft(x) + (j == at && !empty ? at_target : 0.f); };
    auto put = [&](int64_t j, float d) {
        if (F32) reinterpret_cast<float*>(out)[j] = d;
        else reinterpret_cast<uint16_t*>(out)[j] = (uint16_t)(pack_bf16x2(d, 0.f) & 0xFFFFu);
    };
    // stretches begin at the row's first 16-byte boundary; the first CTA also takes what is before it
    const int64_t a = min(p.V, row.head(0)), n = (int64_t)kBwdThreads * kBwdVecs * W;
    const int64_t s0 = a + (blockIdx.x - t * per_row) * n, s1 = min(p.V, s0 + n);
    if (s0 == a && threadIdx.x < a) put(threadIdx.x, grad(row.at(threadIdx.x), threadIdx.x));
    if (((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.p)) & 15) == 0) {
        uint4 raw[kBwdVecs];
#pragma unroll
        for (int u = 0; u < kBwdVecs; ++u) {
            const int64_t j = s0 + (u * kBwdThreads + threadIdx.x) * W;
            if (j + W <= s1) raw[u] = *reinterpret_cast<const uint4*>(row.p + j * (F32 ? 4 : 2));
        }
#pragma unroll
        for (int u = 0; u < kBwdVecs; ++u) {
            const int64_t j = s0 + (u * kBwdThreads + threadIdx.x) * W;
            if (j + W <= s1) {
                const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                float d[W];
#pragma unroll
                for (int e = 0; e < W; ++e)
                    d[e] = F32 ? __uint_as_float(w[e % 4]) : e & 1 ? bf16hi(w[e / 2 % 4]) : bf16lo(w[e / 2 % 4]);
                if (empty) {
#pragma unroll
                    for (int e = 0; e < W; ++e) d[e] = 0.f;
                } else {
#pragma unroll
                    for (int e = 0; e < W; e += 2) {
                        const float2 lp = __fadd2_rn(__fmul2_rn(make_float2(d[e], d[e + 1]), make_float2(p.scale, p.scale)),
                                                     make_float2(-lse, -lse));
                        const float2 q = __fmul2_rn(lp, make_float2(kL2e, kL2e));
                        const float2 c = __ffma2_rn(make_float2(k1, k1), make_float2(fmaxf(lp.x, kNoWeight), fmaxf(lp.y, kNoWeight)),
                                                    make_float2(k0, k0));
                        const float2 r = __fmul2_rn(make_float2(lp_ex2(q.x), lp_ex2(q.y)), c);
                        d[e] = r.x;
                        d[e + 1] = r.y;
                    }
                    if ((uint64_t)(at - j) < (uint64_t)W) {  // the target is one of these
#pragma unroll
                        for (int e = 0; e < W; ++e) d[e] += at - j == e ? at_target : 0.f;
                    }
                }
                uint4 v;
                if (F32) v = make_uint4(__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3]));
                else v = make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]), pack_bf16x2(d[W - 4], d[W - 3]),
                                    pack_bf16x2(d[W - 2], d[W - 1]));
                *reinterpret_cast<uint4*>(out + j * (F32 ? 4 : 2)) = v;
            } else {
                for (int64_t i = j; i < s1; ++i) put(i, grad(row.at(i), i));
            }
        }
    } else {  // the rows of the two tensors lie differently: element by element, at a seventh of the rate
        for (int64_t j = s0 + threadIdx.x; j < s1; j += kBwdThreads) put(j, grad(row.at(j), j));
    }
}

template <bool F32>
static cudaError_t bwd_launch(const LogprobParams& p, cudaStream_t st) {
    const int64_t n = (int64_t)kBwdThreads * kBwdVecs * Row<F32>::kVec;
    const int64_t per_row = (p.V + n - 1) / n;
    if (p.T * per_row > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_pdl(logprob_bwd_kernel<F32>, dim3((unsigned)(p.T * per_row)), dim3(kBwdThreads), 0, st, nullptr, 0, p,
                      (unsigned)per_row);
}
cudaError_t launch_logprob_bwd(const LogprobParams& p, cudaStream_t st) {
    return p.f32 ? bwd_launch<true>(p, st) : bwd_launch<false>(p, st);
}

}  // namespace lm
