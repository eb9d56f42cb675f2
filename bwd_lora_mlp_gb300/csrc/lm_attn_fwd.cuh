// Attention forward (include/lora_layer.h) on the tensor cores.
//
// One CTA per SM stays and takes items of 256 queries of one head as two tiles of 128, walking the
// 128-key tiles that any of them sees.  For each query tile w and key tile j:
//   S_w = Q_w K_j^T                              (tcgen05, both operands in shared memory)
//   P_w = 2^{S c - m}, l += row sums             (eight warps, a row over four lanes)
//   O_w += P_w V_j                               (tcgen05, P_w from tensor memory, where it replaces S_w)
// The two query tiles take turns: while the tensor cores work on one, the other's warps form its
// exponentials.  The first scores of the next item are formed while this one's rows are written.  The
// weights go to the tensor cores 64 keys at a time, so the second product starts half a tile early.
// The running maximum m follows the row only when it has grown by more than 8 (a factor 256 in the
// weights): the weights then stay below 2^8, exact in their scale, and O_w is rescaled a few times per
// row instead of once per key tile.  Sums are fp32.  P is rounded to bf16 for the second product; for
// query tiles with rows of few keys (below) what the rounding left out is multiplied too, as a second left
// operand in the other half of S_w's place: such rows have few other weights to average their error with,
// and the backward takes differences against their O.
// Shared memory (d = 128): 64 KB of queries and a ring of five 32 KB key and value tiles; tensor
// memory: S_0, S_1, O_0, O_1 of 128 columns each, all of it.
// Measured: 8192 causal tokens, 32 heads of 128 dims, 384 to 391 us (box to box), 1.43 to 1.41 PFLOP/s, 0.75 to
// 0.73 of the burst rate of the tensor cores; 4096 tokens with capped scores 185 us (three exponential-unit
// results a score instead of one; 212 with tanh formed by itself and the slopes' arithmetic in it).  What bounds
// it is the way scores -> maximum -> weights -> product: with one score tile a query tile the tensor cores wait
// for it, and a load or store of tensor memory takes 300 cycles while they multiply from shared memory, 90 while
// the left operand is in tensor memory.  With capped scores that way is longer, and no unit is full: the
// exponential unit is 49 % busy, the tensor cores 33 %, the warps wait for tensor memory first and for the
// exponential unit's queue next.  Eight warps with a whole row a thread instead of sixteen: 384 us
// too, but capped 234 against 212, packed documents 182 against 159, prefixes 97 against 80.  One CTA an
// item instead of CTAs that stay: capped 240 against 212.
#pragma once

#include "lm_attn.cuh"

namespace lm {

constexpr float kRescale = 8.f;
// Rows of fewer keys than this, and all rows with slopes (whose weights are those of their nearest keys),
// multiply what the rounding of their weights left out.  (dO.O's part of the error of dQ and dK goes with the
// sum of a row's squared weights: with rows of fewer than 128 keys only, they were 2.5e-3 to 2.7e-3 off in
// documents of some hundred tokens and with slopes, now 2.4e-3.  O itself, rounded to bf16, is 1.66e-3 off in rows
// with the low bits and 2.3e-3 without.  Twice as many keys here would bring rows of 512 to 1023 keys to the former,
// dQ and dK by less than 3 %: 2.40e-3 and 2.37e-3 to 2.37e-3 and 2.36e-3 at 1024 tokens.  A step of 8192 tokens in 14
// documents takes 512 us instead of 507; with 1024 here it takes 518, and one of 2048 tokens 166 instead of 161.)
// (The form for few queries always does: it waits for memory, and takes 15.4 us with them where it took 14.4, 48.9 for
// 48.0; O is then 1.66e-3 off instead of 1.96e-3 and 2.15e-3.)
constexpr int kFewKeys = 512;
// Sixteen softmax warps and a warpgroup for the loader's and the issuer's: 640 threads start with 96
// registers each.
constexpr int kFwdThreads = 640, kFwdMath = 16, kFwdMathRegs = 104, kFwdIssueRegs = 64;
static_assert(4 * kFwdMathRegs + kFwdIssueRegs <= 5 * 96, "a register split above the launch's total waits forever");

// (few queries: one query tile, and the list of the key tiles that a CTA takes)
constexpr int kFewTiles = 4096 + 64;
template <int DP, int FORM>
struct FwdCfg {
    static constexpr uint32_t kTileBytes = (DP / 64) * kBoxBytes;
    static constexpr int kSlots = DP == 128 ? 5 : 8, kQTiles = FORM == ATTN_FEW ? 1 : 2;
    static constexpr int kHead = FORM == ATTN_FEW ? (2048 + kFewTiles * 2 + 1023) / 1024 * 1024 : 2048;
    static constexpr int kSmem = 1024 + kHead + (kQTiles + kSlots) * kTileBytes;
};

struct FwdMaps {
    CUtensorMap q, k, v;
};

// the key tiles [j0, j1) that the queries of a tile may see
struct TileSpan {
    int j0, j1;
    int lo_max, hi_min;  // keys in [lo_max, hi_min) are seen by every row
    __device__ __forceinline__ bool any() const { return j1 > j0; }
    __device__ __forceinline__ bool hides(int j) const { return j * kTile < lo_max || (j + 1) * kTile > hi_min; }
    __device__ __forceinline__ bool has(int j) const { return j >= j0 && j < j1; }
    // some row may see few keys: what its weights' rounding left out is multiplied too
    template <int MODE>
    __device__ __forceinline__ bool few_keys() const { return biased(MODE) || hi_min - lo_max < kFewKeys; }
};
template <int FORM>
__device__ __forceinline__ TileSpan key_tiles(const AttnParams& p, int q0, int tokens) {
    if (q0 >= p.T) return TileSpan{0, 0, 0, 0};
    const TokRange a = query_range<FORM>(p, q0), b = query_range<FORM>(p, min(q0 + tokens, p.T) - 1);
    if (b.hi <= a.lo) return TileSpan{0, 0, 0, 0};
    return TileSpan{a.lo / kTile, (b.hi + kTile - 1) / kTile, b.lo, a.hi};
}
// Item k of this CTA: the heavier items first (under a causal mask the last queries see the most keys),
// dealt out forwards and backwards in turn, so that every CTA gets about the same work.
// In the form for few queries an item is one tile of queries of all heads of a group, and one of `splits` shares
// of the key tiles that it sees; h is its key/value head.
struct Item {
    int h, q0, part;
    TileSpan span[2];
    int J0, J1;
    bool valid;
};
template <int FORM>
__device__ __forceinline__ Item item_of(const AttnParams& p, int k) {
    const int nqb = (p.T + p.rows - 1) / p.rows, G = (int)gridDim.x;
    const int idx = k & 1 ? (k + 1) * G - 1 - (int)blockIdx.x : k * G + (int)blockIdx.x;
    Item it;
    it.part = 0;
    if constexpr (FORM == ATTN_FEW) {  // (one a CTA)
        it.valid = k == 0;
        it.h = (int)blockIdx.x % p.hk;
        it.part = (int)blockIdx.x / p.hk % p.splits;
        it.q0 = (int)blockIdx.x / p.hk / p.splits * p.rows;
        it.span[0] = it.span[1] = it.valid ? key_tiles<FORM>(p, it.q0, p.rows) : TileSpan{0, 0, 0, 0};
        it.J0 = it.span[0].j0;
        it.J1 = it.span[0].j1;
        return it;
    }
    it.valid = idx < nqb * p.hq;
    it.h = idx % p.hq;
    it.q0 = (nqb - 1 - idx / p.hq) * p.rows;
    it.span[0] = it.span[1] = TileSpan{0, 0, 0, 0};
    it.J0 = it.J1 = 0;
    if (it.valid) {
        it.span[0] = key_tiles<FORM>(p, it.q0, kTile);
        if (p.rows > kTile) it.span[1] = key_tiles<FORM>(p, it.q0 + kTile, kTile);
        it.J0 = it.span[0].any() ? it.span[0].j0 : it.span[1].j0;
        if (it.span[1].any()) it.J0 = min(it.J0, it.span[1].j0);
        it.J1 = max(it.span[0].j1, it.span[1].j1);
    }
    return it;
}
template <int FORM>
__device__ __forceinline__ int rounds_of(const AttnParams& p) {
    if (FORM == ATTN_FEW) return 1;
    const int n = (p.T + p.rows - 1) / p.rows * p.hq;
    return (n + (int)gridDim.x - 1) / (int)gridDim.x;
}

// The keys [lo, hi) that some query of an item sees (hi past every place where they end with the last one), and whether
// all of its queries see the same.
struct ItemKeys {
    int lo, hi;
    bool alike;
    // the rows of key tile j that are in there
    __device__ __forceinline__ uint4 of_tile(int j) const {
        const int a = lo - j * kTile, z = hi - j * kTile;
        if (a <= 0 && z >= kTile) return make_uint4(~0u, ~0u, ~0u, ~0u);
        return make_uint4(bits_between(a, z), bits_between(a - 32, z - 32), bits_between(a - 64, z - 64), bits_between(a - 96, z - 96));
    }
};
template <int FORM>
__device__ __forceinline__ ItemKeys keys_of(const AttnParams& p, int q0, int tokens) {
    const TokRange a = query_range<FORM>(p, q0), b = query_range<FORM>(p, min(q0 + tokens, p.T) - 1);
    return ItemKeys{a.lo, b.hi == p.Tk ? 1 << 30 : b.hi, a.lo == b.lo && a.hi == b.hi};
}

// The key tiles that a CTA takes, in order.
struct FewTiles {
    int n, first;          // first of them, or < 0: they are listed
    const uint16_t* list;
    __device__ __forceinline__ int operator[](int i) const { return first < 0 ? list[i] : first + i; }
};
// The CTA's share of the key tiles that its queries see.  With documents, tiles that nobody sees are left out (padded
// states), and the shares are of those that are left.  All threads come here; red: 64 ints of shared memory.
__device__ __forceinline__ FewTiles few_setup(const AttnParams& p, uint16_t* list, int* red) {
    constexpr int kWarps = kFwdThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Item it = item_of<ATTN_FEW>(p, 0);
    const int n = max(it.J1 - it.J0, 0);
    auto share = [&](int total, int part) { return total * part / p.splits; };  // (at most 2^13 tiles, 152 parts)
    if (!p.kseen) {
        const int a = share(n, it.part);
        return FewTiles{share(n, it.part + 1) - a, it.J0 + a, list};
    }
    const int len = ((n + kWarps - 1) / kWarps + 31) / 32 * 32, j0 = min(n, warp * len), j1 = min(n, j0 + len);
    auto seen = [&](int i) {
        if (i >= j1) return false;
        const uint4 b = p.kseen[it.J0 + i];
        return (b.x | b.y | b.z | b.w) != 0u;
    };
    int mine = 0;
    uint32_t last = 0;
    for (int i = j0; i < j1; i += 32) {
        last = __ballot_sync(0xffffffffu, seen(i + lane));
        mine += __popc(last);
    }
    if (lane == 0) red[warp] = mine;
    __syncthreads();
    int total = 0, at = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += red[w];
        total += red[w];
    }
    const int a = share(total, it.part), z = share(total, it.part + 1);
    for (int i = j0; i < j1; i += 32) {
        // (up to 640 tiles a warp has 32 of them, and knows)
        const uint32_t votes = len == 32 ? last : __ballot_sync(0xffffffffu, seen(i + lane));
        const bool on = votes >> lane & 1u;
        const int r = at + __popc(votes & ((1u << lane) - 1u));
        if (on && r >= a && r < z) list[r - a] = (uint16_t)(it.J0 + i + lane);
        at += __popc(votes);
    }
    __syncthreads();
    return FewTiles{z - a, -1, list};
}

// O of query i and head h again, from its own keys alone, by a warp: dims [c0, c0 + 32 N), N a lane.  Where the queries
// of an item are of several documents its products multiply the others' values by weights of 0, which leaves a NaN where
// such a value is not finite; the weights and their sums are of the query's own keys in any case.  So what is finite stands,
// and the rest is formed again and written where that is finite.  (Nothing but an infinity or NaN among
// the values comes here, so it is simple: a lane a key, then a lane N dims.  A batch of 64 sequences of 1024 states with one
// NaN 0.7 ms instead of 58 us; 4097 queries in nine documents, 32 heads, 3.5 ms instead of 97 us.)
template <int MODE, int N>
__device__ __forceinline__ void own_row(const AttnParams& p, int i, int h, int c0) {
    const int lane = threadIdx.x & 31, g = h / (p.hq / p.hk), c = c0 + lane * N;
    const float lse = p.lse[(int64_t)h * p.T + i];
    if (!(fabsf(lse) < INFINITY)) return;  // (it sees nothing, or its own scores are not finite)
    uint16_t* out = p.out + ((int64_t)i * p.hq + h) * p.d;
    bool open[N];
#pragma unroll
    for (int e = 0; e < N; ++e) open[e] = c + e < p.d && (out[c + e] & 0x7F80u) == 0x7F80u;
    const TokRange t = query_range<ATTN_CROSS>(p, i);
    const uint16_t *q = p.q.p + (int64_t)i * p.q.ts + (int64_t)h * p.q.hs, *k = p.k.p + (int64_t)g * p.k.hs, *v = p.v.p + (int64_t)g * p.v.hs;
    const float sc = capped(MODE) ? 2.f * kLog2e * p.scale / p.cap : p.scale * kLog2e, sx = capped(MODE) ? 2.f * p.cap * kLog2e : sc;
    float m = -INFINITY, l = 0.f, o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.f;
#pragma unroll 1
    for (int j0 = t.lo; j0 < t.hi; j0 += 32) {
        bool left = false;
#pragma unroll
        for (int e = 0; e < N; ++e) left |= open[e] && fabsf(o[e]) < INFINITY;
        if (!__any_sync(0xffffffffu, left)) return;  // its own values are not finite either
        float x = 0.f;
        if (j0 + lane < t.hi) {
            const uint16_t* kj = k + (int64_t)(j0 + lane) * p.k.ts;
#pragma unroll 1
            for (int b = 0; b < p.d; b += 8) {
                const uint4 a = *reinterpret_cast<const uint4*>(q + b), w = *reinterpret_cast<const uint4*>(kj + b);
                x = fmaf(bf16lo(a.x), bf16lo(w.x), fmaf(bf16hi(a.x), bf16hi(w.x), x));
                x = fmaf(bf16lo(a.y), bf16lo(w.y), fmaf(bf16hi(a.y), bf16hi(w.y), x));
                x = fmaf(bf16lo(a.z), bf16lo(w.z), fmaf(bf16hi(a.z), bf16hi(w.z), x));
                x = fmaf(bf16lo(a.w), bf16lo(w.w), fmaf(bf16hi(a.w), bf16hi(w.w), x));
            }
        }
        x = j0 + lane < t.hi ? (capped(MODE) ? cap_n(two(x * sc)).x : x) * sx : -INFINITY;
        float top = x;
#pragma unroll
        for (int b = 16; b; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
        if (top > m) {
            const float f = ex2(m - top);  // (0 for the first keys)
            m = top;
            l *= f;
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] *= f;
        }
        const float w = x == -INFINITY ? 0.f : ex2(x - m);
        l += w;
#pragma unroll 4
        for (int b = 0; b < 32; ++b) {
            const float wb = __shfl_sync(0xffffffffu, w, b);
            const uint16_t* vj = v + (int64_t)(j0 + b) * p.v.ts + c;
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (j0 + b < t.hi && c + e < p.d) o[e] = fmaf(wb, bf16lo(vj[e]), o[e]);
        }
    }
#pragma unroll
    for (int b = 16; b; b >>= 1) l += __shfl_xor_sync(0xffffffffu, l, b);
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (open[e] && fabsf(o[e]) < INFINITY) {
            const float y = o[e] / l;
            const uint32_t bits = pack_bf16x2(y, 0.f) & 0xFFFFu;
            out[c + e] = (uint16_t)bits;
            if (p.out_lo) p.out_lo[((int64_t)i * p.hq + h) * p.d16 + c + e] = (int8_t)bits_left(y, bits);
        }
}

template <int DP, int MODE, int FORM>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attn_fwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ FwdMaps maps) {
    using C = FwdCfg<DP, FORM>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + C::kSlots;
    uint64_t* qfull = empty + C::kSlots;  // [2] the item's queries are there
    uint64_t* qempty = qfull + 2;         // [2] and are done with
    uint64_t* sfull = qempty + 2;         // [2] scores ready
    uint64_t* pfull = sfull + 2;          // [2][2] weights of the first, of the last 64 keys written
    uint64_t* odone = pfull + 4;          // [2] the last product of the item done
    uint64_t* lready = odone + 2;         // [2][4] the quarter's row sums exchanged
    uint64_t* drain = lready + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* s_odd = s_abort + 1;  // an infinity or NaN was written (not SELF)
    uint4* s_seen = reinterpret_cast<uint4*>(smem + 768);   // [slot] the tile's keys that some query of the item sees (not SELF)
    uint64_t* clean = reinterpret_cast<uint64_t*>(smem + 896);  // [slot] and the others have been cleared
    uint16_t* s_tiles = reinterpret_cast<uint16_t*>(smem + 2048);  // (few queries) this CTA's key tiles
    float* s_inv = reinterpret_cast<float*>(smem + 1024);  // [2][128] 1 / l
    uint8_t* sq = smem + C::kHead;
    uint8_t* ring = sq + C::kQTiles * C::kTileBytes;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            // (a slot is free when its products are done, and when the clearing warp has been there: it looks at every fill of
            // every slot, and would miss one that the next had replaced)
            mbar_init(smem_u32(&empty[s]), FORM != ATTN_SELF && p.kseen ? 2 : 1);
            if (FORM != ATTN_SELF) mbar_init(smem_u32(&clean[s]), 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_u32(&qfull[w]), 1);
            mbar_init(smem_u32(&qempty[w]), 1);
            mbar_init(smem_u32(&sfull[w]), 1);
            mbar_init(smem_u32(&pfull[2 * w]), 8);
            mbar_init(smem_u32(&pfull[2 * w + 1]), 8);
            mbar_init(smem_u32(&odone[w]), 1);
            for (int q = 0; q < 4; ++q) mbar_init(smem_u32(&lready[4 * w + q]), 2);
        }
        mbar_init(smem_u32(drain), 1);
        *s_abort = *s_odd = 0;
        fence_mbar_init();
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
    }
    __syncwarp();
    if (warp == kFwdMath) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    const uint32_t tmem = (uint32_t)uni((int)*tmem_slot);
    const int rounds = rounds_of<FORM>(p), group = p.hq / p.hk;
    // few queries: this CTA's key tiles, of those that the query tile sees its share
    FewTiles mine{0, 0, nullptr};
    if constexpr (FORM == ATTN_FEW) mine = few_setup(p, s_tiles, reinterpret_cast<int*>(s_inv));
    const int tiles = mine.n;

    if (warp >= kFwdMath) {
        regs_down<kFwdIssueRegs>();
        if (warp == kFwdMath + 1) {  // ---------------- loader
            if (lane == 0) {
                bool ok = true;
                uint32_t n = 0, nq[2] = {0, 0};  // tiles and queries asked for
                // (which keys are seen is asked for a tile ahead: a wait for memory here is a wait of every tile's)
                uint4 seen = make_uint4(0, 0, 0, 0);
                ItemKeys keys{0, 0, true};
                auto look = [&](int j) {
                    if (FORM != ATTN_SELF && p.kseen) seen = p.kseen[j];
                };
                auto pair_of = [&](const Item& it, int j, int then, auto between) {  // K_j, then V_j
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t s = n % C::kSlots, ph = (n / C::kSlots) & 1u;
                        if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1u, s_abort, p.wait_ns)) return false;
                        if (FORM != ATTN_SELF && kv && p.kseen) {
                            const uint4 here = keys.of_tile(j);  // (values of other documents are zeros here)
                            s_seen[s] = make_uint4(seen.x & here.x, seen.y & here.y, seen.z & here.z, seen.w & here.w);
                            look(then);
                        }
                        mbar_expect_tx(smem_u32(&full[s]), C::kTileBytes);
                        for (int b = 0; b < DP / 64; ++b)
                            tma_load_3d(smem_u32(ring + s * C::kTileBytes + b * kBoxBytes), kv ? &maps.v : &maps.k,
                                        smem_u32(&full[s]), b * 64, FORM == ATTN_FEW ? it.h : it.h / group, j * kTile);
                        ++n;
                        if (kv == 0 && !between()) return false;
                    }
                    return true;
                };
                for (int k = p.starve & K_ATTN_FWD ? rounds : 0; ok && k < rounds; ++k) {
                    const Item it = item_of<FORM>(p, k);
                    auto query = [&](int w) {
                        if (FORM == ATTN_FEW ? tiles == 0 : !it.span[w].any()) return true;
                        if (!mbar_wait(smem_u32(&qempty[w]), (nq[w] & 1u) ^ 1u, s_abort, p.wait_ns)) return false;
                        const uint32_t bar = smem_u32(&qfull[w]);
                        // (few queries: a box of all heads of the group, rows of a token next to each other)
                        mbar_expect_tx(bar, FORM == ATTN_FEW ? (uint32_t)(DP / 64 * 128 * p.rows * group) : C::kTileBytes);
                        for (int b = 0; b < DP / 64; ++b)
                            tma_load_3d(smem_u32(sq + w * C::kTileBytes + b * kBoxBytes), &maps.q, bar, b * 64,
                                        FORM == ATTN_FEW ? it.h * group : it.h, it.q0 + w * kTile);
                        ++nq[w];
                        return true;
                    };
                    ok = query(0);  // then K, then the other queries: the first scores wait for what they need
                    if (FORM != ATTN_SELF && p.kseen && it.J0 < it.J1) keys = keys_of<FORM>(p, it.q0, p.rows);
                    if constexpr (FORM == ATTN_FEW) {
                        if (tiles > 0) look(mine[0]);
                        for (int i = 0; ok && i < tiles; ++i)
                            ok = pair_of(it, mine[i], mine[min(i + 1, tiles - 1)], [] { return true; });
                    } else {
                        if (it.J0 < it.J1) look(it.J0);
                        for (int j = it.J0; ok && j < it.J1; ++j)
                            ok = pair_of(it, j, min(j + 1, it.J1 - 1), [&] { return j != it.J0 || query(1); });
                    }
                }
                if (!ok) {
                    attn_error(p, 5, 1);
                    *s_abort = 1;
                }
                // nothing may land in shared memory after the CTA has gone
                volatile int never = 0;
                bool in = drain_fills(smem_u32(&full[0]), C::kSlots, n, p.wait_ns);
                for (int w = 0; w < 2; ++w)
                    if (nq[w]) in = mbar_wait(smem_u32(&qfull[w]), (nq[w] - 1u) & 1u, &never, p.wait_ns) && in;
                if (!in) attn_error(p, 5, 5);
            }
        } else if (warp == kFwdMath && elect_one()) {  // ---------------- tensor cores
            const int ksteps = (p.d + 15) / 16;
            const uint32_t ids = make_idesc_bf16(kTile, kTile, false, false);
            const uint32_t ido = make_idesc_bf16(kTile, ksteps * 16, false, true);  // V is [key][dim]: MN-major
            int in0 = 0, in1 = 0;
            if (FORM == ATTN_SELF) inside_tokens(p, in0, in1);
            bool ok = true;
            uint32_t n = 0, nt[2] = {0, 0}, nq[2] = {0, 0};  // ring position of K_{J0}; tiles, items of each query tile
            // V's rows that no query of the item sees are zeros
            auto values = [&](uint32_t nv) {
                uint64_t* bar = FORM != ATTN_SELF && p.kseen ? clean : full;
                return mbar_wait(smem_u32(&bar[nv % C::kSlots]), (nv / C::kSlots) & 1u, s_abort, p.wait_ns);
            };
            if constexpr (FORM == ATTN_FEW) {
                // O_w (+)= P_w V, and what the rounding of P left out; V at ring position nv; last: of this accumulator
                auto weighted = [&](int w, uint32_t nv, uint32_t parity, bool first, bool last) {
                    const uint32_t ts = tmem + w * kTile, to = tmem + 2 * kTile + w * DP;
                    const uint32_t sv = smem_u32(ring + (nv % C::kSlots) * C::kTileBytes);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (!mbar_wait(smem_u32(&pfull[2 * w + half]), parity, s_abort, p.wait_ns)) return false;
                        tc_fence_after();
                        const uint32_t a = ts + half * 32;
                        const uint32_t b = desc_cols(sv) + half * 512;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16_ts(to, a + kk * 8, desc(b + kk * 128), ido, first && !half && !kk ? 0u : 1u);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) umma_bf16_ts(to, a + 64 + kk * 8, desc(b + kk * 128), ido, 1u);
                        if (half && last) umma_commit(smem_u32(&odone[w]));
                    }
                    return true;
                };
                // tile i is accumulator i & 1's: the next tile's scores are formed while this one's weights are
                auto scores = [&](int i) {
                    const uint32_t nk = 2 * (uint32_t)i, sk = smem_u32(ring + (nk % C::kSlots) * C::kTileBytes);
                    if (!mbar_wait(smem_u32(&full[nk % C::kSlots]), (nk / C::kSlots) & 1u, s_abort, p.wait_ns)) return false;
                    tc_fence_after();
                    mma_rows<DP>(tmem + (i & 1) * kTile, desc_rows(smem_u32(sq)), desc_rows(sk), ksteps, ids);
                    umma_commit(smem_u32(&sfull[i & 1]));
                    umma_commit(smem_u32(&empty[nk % C::kSlots]));
                    return true;
                };
                if (tiles > 0) ok = mbar_wait(smem_u32(&qfull[0]), 0, s_abort, p.wait_ns) && scores(0);
                for (int i = 0; ok && i < tiles; ++i) {
                    const uint32_t nv = 2 * (uint32_t)i + 1;
                    ok = (i + 1 >= tiles || scores(i + 1)) && values(nv);
                    if (!ok) break;
                    tc_fence_after();
                    ok = weighted(i & 1, nv, (uint32_t)(i >> 1) & 1u, i < 2, i + 2 >= tiles);
                    if (ok) umma_commit(smem_u32(&empty[nv % C::kSlots]));
                }
            }
            Item next = item_of<FORM>(p, 0);
            for (int k = 0; FORM != ATTN_FEW && ok && k < rounds; ++k) {
                const Item it = next;
                next = item_of<FORM>(p, k + 1);
                if (it.J1 <= it.J0) continue;
                for (int j = it.J0; ok && j <= it.J1; ++j) {
                    const uint32_t nk = n + 2 * (uint32_t)(j - it.J0), nv = nk - 1;  // ring positions of K_j and V_{j-1}
                    const uint32_t sk = smem_u32(ring + (nk % C::kSlots) * C::kTileBytes);
                    const uint32_t sv = smem_u32(ring + (nv % C::kSlots) * C::kTileBytes);
                    if (j > it.J0) {
                        ok = values(nv);
                        if (!ok) break;
                        if (FORM == ATTN_SELF)
                            clear_padding(ring + (nv % C::kSlots) * C::kTileBytes, DP / 64, (j - 1) * kTile, in0, in1);
                    }
                    if (j < it.J1) {
                        ok = mbar_wait(smem_u32(&full[nk % C::kSlots]), (nk / C::kSlots) & 1u, s_abort, p.wait_ns);
                        if (!ok) break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t ts = tmem + w * kTile, to = tmem + 2 * kTile + w * DP;
                        const TileSpan& sp = it.span[w];
                        if (j > it.J0 && sp.has(j - 1)) {  // O_w += P_w V_{j-1}
                            const bool first = j - 1 == sp.j0, both = sp.few_keys<MODE>();
#pragma unroll
                            for (int half = 0; half < 2 && ok; ++half) {
                                ok = mbar_wait(smem_u32(&pfull[2 * w + half]), (nt[w] - 1u) & 1u, s_abort, p.wait_ns);
                                if (!ok) break;
                                tc_fence_after();
                                const uint32_t a = ts + half * 32;
                                const uint32_t b = desc_cols(sv) + half * 512;
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    umma_bf16_ts(to, a + kk * 8, desc(b + kk * 128), ido, first && !half && !kk ? 0u : 1u);
                                if (both) {
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        umma_bf16_ts(to, a + 64 + kk * 8, desc(b + kk * 128), ido, 1u);
                                }
                                if (half && j == sp.j1) umma_commit(smem_u32(&odone[w]));
                            }
                            if (!ok) break;
                        }
                        if (sp.has(j)) {  // S_w = Q_w K_j^T
                            if (j == sp.j0) {
                                ok = mbar_wait(smem_u32(&qfull[w]), nq[w] & 1u, s_abort, p.wait_ns);
                                if (!ok) break;
                                ++nq[w];
                                tc_fence_after();
                            }
                            mma_rows<DP>(ts, desc_rows(smem_u32(sq + w * C::kTileBytes)), desc_rows(sk), ksteps, ids);
                            umma_commit(smem_u32(&sfull[w]));
                            ++nt[w];
                            if (j + 1 == sp.j1) umma_commit(smem_u32(&qempty[w]));
                        }
                    }
                    if (!ok) break;
                    if (j > it.J0) umma_commit(smem_u32(&empty[nv % C::kSlots]));
                    if (j < it.J1) umma_commit(smem_u32(&empty[nk % C::kSlots]));
                }
                n += 2 * (uint32_t)(it.J1 - it.J0);
            }
            if (!ok) {
                attn_error(p, 5, 2);
                *s_abort = 1;
            }
            umma_commit(smem_u32(drain));
            volatile int never = 0;
            mbar_wait(smem_u32(drain), 0, &never, p.wait_ns);
        }
        if (FORM != ATTN_SELF && warp == kFwdMath + 2 && p.kseen) {  // ---------------- clears values that no query of the item sees
            bool ok = true;
            uint32_t n = 0;
            auto pair_of = [&] {
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const uint32_t s = n % C::kSlots;
                    if (!mbar_wait_warp(smem_u32(&full[s]), (n / C::kSlots) & 1u, s_abort, p.wait_ns)) return false;
                    if (kv) clear_unseen_warp(ring + s * C::kTileBytes, DP / 64, s_seen[s]);
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&clean[s]));
                        mbar_arrive(smem_u32(&empty[s]));
                    }
                }
                return true;
            };
            if constexpr (FORM == ATTN_FEW) {
                for (int i = 0; ok && i < tiles; ++i) ok = pair_of();
            } else {
                for (int k = 0; ok && k < rounds; ++k) {
                    const Item it = item_of<FORM>(p, k);
                    for (int j = it.J0; ok && j < it.J1; ++j) ok = pair_of();
                }
            }
            if (!ok && lane == 0) {
                attn_error(p, 5, 4);
                *s_abort = 1;
            }
        }
    } else {  // ---------------- softmax: 16 query rows a warp, two of them (and a quarter of each) a thread
        regs_up<kFwdMathRegs>();
        const int w = warp >> 3, quarter = warp & 3, sub = (warp >> 2) & 1;
        const int row0 = quarter * 32 + sub * 16 + (lane >> 2), c0 = 2 * (lane & 3);  // rows row0, row0 + 8
        const uint32_t half_lanes = (uint32_t)(quarter * 32 + sub * 16) << 16, all_lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tmem + half_lanes + w * kTile, to = tmem + half_lanes + 2 * kTile + w * DP;
        // scores in units of log 2: x cx, x the product or (capped) n; with slopes x is the score itself.  Capped
        // ones are short of the constant cap, which lse gets back
        const float c = capped(MODE) ? 2.f * kLog2e * p.scale / p.cap : p.scale * kLog2e;
        const float cs = capped(MODE) ? 2.f * p.cap * kLog2e : c;
        const float cx = biased(MODE) ? 1.f : cs;
        uint32_t nt = 0, nq = 0;
        bool ok = true;
        Item next = item_of<FORM>(p, 0);
        for (int k = 0; ok && k < rounds; ++k) {
            const Item it = next;
            next = item_of<FORM>(p, k + 1);
            if (!it.valid || (FORM != ATTN_FEW && w * kTile >= p.rows)) continue;
            const TileSpan sp = w ? it.span[1] : it.span[0];
            // token and head of a row of the tile (T for rows of no token)
            auto token_of = [&](int row) {
                if (FORM != ATTN_FEW) return it.q0 + w * kTile + row;  // (few: both accumulators are of the same queries)
                return row < p.rows * group ? it.q0 + row / group : p.T;
            };
            auto head_of = [&](int row) { return FORM != ATTN_FEW ? it.h : it.h * group + row % group; };
            const int i0 = it.q0 + w * kTile + row0;
            int lo[2] = {0, 0}, hi[2] = {0, 0};
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (token_of(row0 + 8 * r) < p.T) {
                    const TokRange t = query_range<FORM>(p, token_of(row0 + 8 * r));
                    lo[r] = t.lo - c0;  // (in terms of this lane's first column)
                    hi[r] = t.hi - c0;
                }
            const float slope = biased(MODE) && p.slopes ? p.slopes[it.h] * kLog2e : 0.f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // running maxima, this lane's sums of weights
            // one key tile; tiles with hidden keys have code of their own.  x[4 g + 2 r + e]: row r, key
            // 8 g + c0 + e of the tile
            auto tile = [&](int j, bool begun, auto hides, auto few) {
                constexpr bool HIDDEN = decltype(hides)::value, REST = decltype(few)::value;
                const int k0 = j * kTile;
                if (FORM == ATTN_FEW && HIDDEN) {  // none of the warp's rows sees any of these keys
                    const int a = k0 - c0, z = a + kTile;
                    if (!__any_sync(0xffffffffu, (lo[0] < z && hi[0] > a && lo[0] < hi[0]) || (lo[1] < z && hi[1] > a && lo[1] < hi[1]))) {
                        const uint32_t none[16] = {};
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            tmem_st_pairs16(ts + half * 32, none);
                            if (REST) tmem_st_pairs16(ts + 64 + half * 32, none);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(smem_u32(&pfull[2 * w]));
                            mbar_arrive(smem_u32(&pfull[2 * w + 1]));
                        }
                        return;
                    }
                }
                float x[64];
                tmem_ld_frag32<0>(ts, x);
                tmem_ld_frag32<32>(ts + 64, x);
                tmem_ld_wait_f32<0>(x);
                tmem_ld_wait_f32<32>(x);
                if (capped(MODE)) {
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        const float2 n = cap_n(__fmul2_rn(make_float2(x[e], x[e + 1]), two(c)));
                        x[e] = n.x;
                        x[e + 1] = n.y;
                    }
                }
                if (biased(MODE)) {
                    const float dist = (float)(i0 - k0 - c0);
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        x[e] = fmaf(-slope, fabsf(dist + (float)((e & 2) * 4 - (e >> 2) * 8 - (e & 1))), x[e] * cs);
                }
                if (HIDDEN) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        // (bits of this lane's keys: 8 g + e of the chunk's 32, from its first column on)
                        const uint32_t b0 = bits_between(lo[0] - k0 - 32 * b, hi[0] - k0 - 32 * b);
                        const uint32_t b1 = bits_between(lo[1] - k0 - 32 * b, hi[1] - k0 - 32 * b);
                        if (__all_sync(0xffffffffu, ((b0 & b1) | ~0x03030303u) == ~0u)) continue;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (!((e & 2 ? b1 : b0) >> ((e >> 2) * 8 + (e & 1)) & 1u)) x[b * 16 + e] = -INFINITY;
                    }
                }
                float top[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float a = fmaxf(x[2 * r], x[2 * r + 1]), b = fmaxf(x[32 + 2 * r], x[32 + 2 * r + 1]);
#pragma unroll
                    for (int g = 1; g < 8; ++g) {
                        a = fmaxf(fmaxf(a, x[4 * g + 2 * r]), x[4 * g + 2 * r + 1]);
                        b = fmaxf(fmaxf(b, x[32 + 4 * g + 2 * r]), x[32 + 4 * g + 2 * r + 1]);
                    }
                    top[r] = fmaxf(a, b);
                }
#pragma unroll
                for (int o = 1; o <= 2; ++o)
#pragma unroll
                    for (int r = 0; r < 2; ++r) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], o));
                bool grow[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    top[r] *= cx;
                    grow[r] = top[r] > m[r] + kRescale || (m[r] == -INFINITY && top[r] > -INFINITY);
                }
                if (__any_sync(0xffffffffu, grow[0] || grow[1])) {
                    float f[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        f[r] = !grow[r] ? 1.f : m[r] == -INFINITY ? 0.f : ex2(m[r] - top[r]);
                        l[r] *= f[r];
                        if (grow[r]) m[r] = top[r];
                    }
                    // the earlier tiles are in O since these scores are there: products end in the order they
                    // are issued
                    if (begun) {
#pragma unroll 1
                        for (int cc = 0; cc < DP; cc += 32) {
                            float o[16];
                            tmem_ld_frag16<0>(to + cc, o);
                            tmem_ld_wait16_f32<0>(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f[(e >> 1) & 1];
                            tmem_st_frag16(to + cc, o);
                        }
                        tmem_st_wait();
                    }
                }
                const float2 c2 = two(cx);
                const float2 mu[2] = {two(m[0] == -INFINITY ? 0.f : -m[0]), two(m[1] == -INFINITY ? 0.f : -m[1])};
                float2 s2[2] = {two(0.f), two(0.f)};
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // 64 keys at a time: their product may begin
                    uint32_t pk[16], rest[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const int r = (e >> 1) & 1;
                        const float2 y = __ffma2_rn(make_float2(x[half * 32 + e], x[half * 32 + e + 1]), c2, mu[r]);
                        const float2 q = make_float2(ex2(y.x), ex2(y.y));
                        s2[r] = __fadd2_rn(s2[r], q);
                        const uint32_t hi2 = pack_bf16x2(q.x, q.y);
                        pk[e >> 1] = hi2;
                        if (REST) rest[e >> 1] = pack_bf16x2(q.x - bf16lo(hi2), q.y - bf16hi(hi2));
                    }
                    tmem_st_pairs16(ts + half * 32, pk);
                    if (REST) tmem_st_pairs16(ts + 64 + half * 32, rest);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&pfull[2 * w + half]));
                }
                l[0] += s2[0].x + s2[0].y;
                l[1] += s2[1].x + s2[1].y;
            };
            auto step = [&](int j, bool begun, bool few) {
                if (!mbar_wait_warp(smem_u32(&sfull[w]), nt & 1u, s_abort, p.wait_ns)) return false;
                tc_fence_after();
                if (few) {
                    if (sp.hides(j)) tile(j, begun, std::true_type{}, std::true_type{});
                    else tile(j, begun, std::false_type{}, std::true_type{});
                } else if constexpr (!biased(MODE) && FORM != ATTN_FEW) {
                    if (sp.hides(j)) tile(j, begun, std::true_type{}, std::false_type{});
                    else tile(j, begun, std::false_type{}, std::false_type{});
                }
                return true;
            };
            if constexpr (FORM == ATTN_FEW) {
                for (int i = w; ok && i < tiles; i += 2, ++nt) ok = step(mine[i], i >= 2, true);
            } else {
                for (int j = sp.j0; ok && j < sp.j1; ++j, ++nt) ok = step(j, j > sp.j0, sp.few_keys<MODE>());
            }
            const bool any = FORM == ATTN_FEW ? w < tiles : sp.any();  // (uniform over the query tile's warps)
            if (!ok) break;
            // ---- the item's rows: sums over a row's four lanes, then 1 / l to the quarter's two warps
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                // (no weight at all: nothing is seen; a NaN sum is one, of O and of lse)
                if ((lane & 3) == 0) {
                    const int i = token_of(row0 + 8 * r), h = head_of(row0 + 8 * r);
                    s_inv[w * kTile + row0 + 8 * r] = l[r] == 0.f ? 0.f : 1.f / l[r];
                    if (i < p.T) {
                        if (FORM == ATTN_FEW && p.parts > 1)
                            p.part_ml[(int64_t)(2 * it.part + w) * p.T * p.hq + (int64_t)i * p.hq + h] = make_float2(m[r], l[r]);
                        else if (FORM != ATTN_FEW || w == 0)
                            p.lse[(int64_t)h * p.T + i] =
                                l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2 + (capped(MODE) ? p.cap : 0.f);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&lready[4 * w + quarter]));
            // (this barrier completes twice an item: the sums are there; both warps have read them)
            ok = mbar_wait_warp(smem_u32(&lready[4 * w + quarter]), 0, s_abort, p.wait_ns);
            if (!ok) break;
            const int row = quarter * 32 + lane, i = token_of(row), h = head_of(row);
            const float inv = s_inv[w * kTile + row];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&lready[4 * w + quarter]));
            if (any) {
                ok = mbar_wait_warp(smem_u32(&odone[w]), nq & 1u, s_abort, p.wait_ns);
                if (!ok) break;
                ++nq;
                tc_fence_after();
            }
            // each of the quarter's warps writes half of the dims, a thread one row of them
            const int64_t at = (int64_t)i * p.hq + h;
            uint16_t* out = p.out + at * p.d;
            int8_t* out_lo = p.out_lo ? p.out_lo + at * p.d16 : nullptr;
            const bool partial = FORM == ATTN_FEW && (p.parts > 1 || w);
            if (FORM == ATTN_FEW && p.parts > 1 && any) {  // unnormalised, in fp32; rows that saw nothing have l = 0 and are not read
                float* dst = p.part_o + ((int64_t)(2 * it.part + w) * p.T * p.hq + at) * p.d;
                const bool mine = i < p.T && inv != 0.f;
                if (__any_sync(0xffffffffu, mine))
#pragma unroll 1
                    for (int cc = sub * (DP / 2); cc < (sub + 1) * (DP / 2); cc += 16) {
                        uint32_t raw[16];
                        tmem_ld_x16(tmem + all_lanes + 2 * kTile + w * DP + cc, raw);
                        tmem_ld_wait16(raw);
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            if (mine && cc + e < p.d)
                                *reinterpret_cast<uint4*>(dst + cc + e) = make_uint4(raw[e], raw[e + 1], raw[e + 2], raw[e + 3]);
                    }
            }
#pragma unroll 1
            for (int cc = sub * (DP / 2); cc < (sub + 1) * (DP / 2) && !partial; cc += 16) {
                float o[16];
                if (any) {
                    uint32_t raw[16];
                    tmem_ld_x16(tmem + all_lanes + 2 * kTile + w * DP + cc, raw);
                    tmem_ld_wait16(raw);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = inv == 0.f ? 0.f : __uint_as_float(raw[e]) * inv;
                    if (FORM != ATTN_SELF && p.qrange && i < p.T) {
                        float zero = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) zero = fmaf(o[e], 0.f, zero);
                        if (zero != zero) *s_odd = 1;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0.f;
                }
                uint32_t v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
                if (i < p.T && cc < p.d) {
                    if ((p.d & 15) == 0) {
                        st_global_v8(out + cc, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
                    } else {  // (d = 8 modulo 16: rows lie on 16 bytes, and the last chunk is half there)
                        *reinterpret_cast<uint4*>(out + cc) = make_uint4(v[0], v[1], v[2], v[3]);
                        if (cc + 8 < p.d) *reinterpret_cast<uint4*>(out + cc + 8) = make_uint4(v[4], v[5], v[6], v[7]);
                    }
                    if (out_lo) {
                        int more[4];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int pair = (bits_left(o[2 * e], v[e] & 0xFFFFu) & 255) | (bits_left(o[2 * e + 1], v[e] >> 16) & 255) << 8;
                            if (e & 1) more[e >> 1] |= pair << 16;
                            else more[e >> 1] = pair;
                        }
                        *reinterpret_cast<int4*>(out_lo + cc) = make_int4(more[0], more[1], more[2], more[3]);
                    }
                }
            }
            tc_fence_before();  // (the next item's products may overwrite O once the weights say so)
            ok = mbar_wait_warp(smem_u32(&lready[4 * w + quarter]), 1, s_abort, p.wait_ns);
        }
        if (!ok && lane == 0) {
            attn_error(p, 5, 3);
            *s_abort = 1;
        }
        // at the end, when nothing waits for these warps: the rows of this one that are not finite
        __syncwarp();  // (lanes read what others of them wrote)
        if (FORM != ATTN_SELF && ok && __any_sync(0xffffffffu, *s_odd))
#pragma unroll 1
            for (int k = 0; k < rounds; ++k) {
                const Item it = item_of<FORM>(p, k);
                if (!it.valid || (FORM == ATTN_FEW ? w : w * kTile >= p.rows) || keys_of<FORM>(p, it.q0, p.rows).alike) continue;
#pragma unroll 1
                for (int row = quarter * 32; row < quarter * 32 + 32; ++row) {
                    const int i = FORM != ATTN_FEW ? it.q0 + w * kTile + row : row < p.rows * group ? it.q0 + row / group : p.T;
                    if (i < p.T) own_row<MODE, DP / 64>(p, i, FORM != ATTN_FEW ? it.h : it.h * group + row % group, sub * (DP / 2));
                }
            }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kFwdMath) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DP, int MODE, int FORM>
cudaError_t launch_fwd(const AttnParams& p, const FwdMaps& maps, int sms, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(attn_fwd_kernel<DP, MODE, FORM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               FwdCfg<DP, FORM>::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)((p.T + p.rows - 1) / p.rows) * (FORM == ATTN_FEW ? p.hk * p.splits : p.hq);
    const unsigned grid = (unsigned)(items < sms || FORM == ATTN_FEW ? items : sms);
    return launch_pdl(attn_fwd_kernel<DP, MODE, FORM>, dim3(grid), dim3(kFwdThreads), FwdCfg<DP, FORM>::kSmem, st, nullptr, 0, p, maps);
}

}  // namespace lm
