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
constexpr int kFewKeys = 512;
// Sixteen softmax warps and a warpgroup for the loader's and the issuer's: 640 threads start with 96
// registers each.
constexpr int kFwdThreads = 640, kFwdMath = 16, kFwdMathRegs = 104, kFwdIssueRegs = 64;
static_assert(4 * kFwdMathRegs + kFwdIssueRegs <= 5 * 96, "a register split above the launch's total waits forever");

template <int DP>
struct FwdCfg {
    static constexpr uint32_t kTileBytes = (DP / 64) * kBoxBytes;
    static constexpr int kSlots = DP == 128 ? 5 : 8;
    static constexpr int kSmem = 3 * 1024 + (2 + kSlots) * kTileBytes;
};

struct FwdMaps {
    CUtensorMap q, k, v;
};

// the key tiles [j0, j1) that the query rows [q0, q0 + 128) may see
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
__device__ __forceinline__ TileSpan key_tiles(const AttnParams& p, int q0) {
    if (q0 >= p.T) return TileSpan{0, 0, 0, 0};
    const TokRange a = tok_range(p, q0), b = tok_range(p, min(q0 + kTile, p.T) - 1);
    if (b.hi <= a.lo) return TileSpan{0, 0, 0, 0};
    return TileSpan{a.lo / kTile, (b.hi + kTile - 1) / kTile, b.lo, a.hi};
}
// Item k of this CTA: the heavier items first (under a causal mask the last queries see the most keys),
// dealt out forwards and backwards in turn, so that every CTA gets about the same work.
struct Item {
    int h, q0;
    TileSpan span[2];
    int J0, J1;
    bool valid;
};
__device__ __forceinline__ Item item_of(const AttnParams& p, int k) {
    const int nqb = (p.T + p.rows - 1) / p.rows, G = (int)gridDim.x;
    const int idx = k & 1 ? (k + 1) * G - 1 - (int)blockIdx.x : k * G + (int)blockIdx.x;
    Item it;
    it.valid = idx < nqb * p.hq;
    it.h = idx % p.hq;
    it.q0 = (nqb - 1 - idx / p.hq) * p.rows;
    it.span[0] = it.span[1] = TileSpan{0, 0, 0, 0};
    it.J0 = it.J1 = 0;
    if (it.valid) {
        it.span[0] = key_tiles(p, it.q0);
        if (p.rows > kTile) it.span[1] = key_tiles(p, it.q0 + kTile);
        it.J0 = it.span[0].any() ? it.span[0].j0 : it.span[1].j0;
        if (it.span[1].any()) it.J0 = min(it.J0, it.span[1].j0);
        it.J1 = max(it.span[0].j1, it.span[1].j1);
    }
    return it;
}
__device__ __forceinline__ int rounds_of(const AttnParams& p) {
    const int n = (p.T + p.rows - 1) / p.rows * p.hq;
    return (n + (int)gridDim.x - 1) / (int)gridDim.x;
}

template <int DP, int MODE>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attn_fwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ FwdMaps maps) {
    using C = FwdCfg<DP>;
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
    float* s_inv = reinterpret_cast<float*>(smem + 1024);  // [2][128] 1 / l
    uint8_t* sq = smem + 2048;
    uint8_t* ring = sq + 2 * C::kTileBytes;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
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
        *s_abort = 0;
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
    const int rounds = rounds_of(p), group = p.hq / p.hk;

    if (warp >= kFwdMath) {
        regs_down<kFwdIssueRegs>();
        if (warp == kFwdMath + 1) {  // ---------------- loader
            if (lane == 0) {
                bool ok = true;
                uint32_t n = 0, nq[2] = {0, 0};  // tiles and queries asked for
                for (int k = p.starve & K_ATTN_FWD ? rounds : 0; ok && k < rounds; ++k) {
                    const Item it = item_of(p, k);
                    auto query = [&](int w) {
                        if (!it.span[w].any()) return true;
                        if (!mbar_wait(smem_u32(&qempty[w]), (nq[w] & 1u) ^ 1u, s_abort, p.wait_ns)) return false;
                        const uint32_t bar = smem_u32(&qfull[w]);
                        mbar_expect_tx(bar, C::kTileBytes);
                        for (int b = 0; b < DP / 64; ++b)
                            tma_load_3d(smem_u32(sq + w * C::kTileBytes + b * kBoxBytes), &maps.q, bar, b * 64, it.h,
                                        it.q0 + w * kTile);
                        ++nq[w];
                        return true;
                    };
                    ok = query(0);  // then K, then the other queries: the first scores wait for what they need
                    for (int j = it.J0; ok && j < it.J1; ++j)
                        for (int kv = 0; kv < 2; ++kv) {
                            const uint32_t s = n % C::kSlots, ph = (n / C::kSlots) & 1u;
                            if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1u, s_abort, p.wait_ns)) {
                                ok = false;
                                break;
                            }
                            mbar_expect_tx(smem_u32(&full[s]), C::kTileBytes);
                            for (int b = 0; b < DP / 64; ++b)
                                tma_load_3d(smem_u32(ring + s * C::kTileBytes + b * kBoxBytes), kv ? &maps.v : &maps.k,
                                            smem_u32(&full[s]), b * 64, it.h / group, j * kTile);
                            ++n;
                            if (j == it.J0 && kv == 0 && !query(1)) {
                                ok = false;
                                break;
                            }
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
            int in0, in1;
            inside_tokens(p, in0, in1);
            bool ok = true;
            uint32_t n = 0, nt[2] = {0, 0}, nq[2] = {0, 0};  // ring position of K_{J0}; tiles, items of each query tile
            Item next = item_of(p, 0);
            for (int k = 0; ok && k < rounds; ++k) {
                const Item it = next;
                next = item_of(p, k + 1);
                if (it.J1 <= it.J0) continue;
                for (int j = it.J0; ok && j <= it.J1; ++j) {
                    const uint32_t nk = n + 2 * (uint32_t)(j - it.J0), nv = nk - 1;  // ring positions of K_j and V_{j-1}
                    const uint32_t sk = smem_u32(ring + (nk % C::kSlots) * C::kTileBytes);
                    const uint32_t sv = smem_u32(ring + (nv % C::kSlots) * C::kTileBytes);
                    if (j > it.J0) {
                        ok = mbar_wait(smem_u32(&full[nv % C::kSlots]), (nv / C::kSlots) & 1u, s_abort, p.wait_ns);
                        if (!ok) break;
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
        Item next = item_of(p, 0);
        for (int k = 0; ok && k < rounds; ++k) {
            const Item it = next;
            next = item_of(p, k + 1);
            if (!it.valid || w * kTile >= p.rows) continue;
            const TileSpan sp = w ? it.span[1] : it.span[0];
            const int i0 = it.q0 + w * kTile + row0;
            int lo[2] = {0, 0}, hi[2] = {0, 0};
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (i0 + 8 * r < p.T) {
                    const TokRange t = tok_range(p, i0 + 8 * r);
                    lo[r] = t.lo - c0;  // (in terms of this lane's first column)
                    hi[r] = t.hi - c0;
                }
            const float slope = biased(MODE) && p.slopes ? p.slopes[it.h] * kLog2e : 0.f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // running maxima, this lane's sums of weights
            // one key tile; tiles with hidden keys have code of their own.  x[4 g + 2 r + e]: row r, key
            // 8 g + c0 + e of the tile
            auto tile = [&](int j, auto hides, auto few) {
                constexpr bool HIDDEN = decltype(hides)::value, REST = decltype(few)::value;
                const int k0 = j * kTile;
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
                    if (j > sp.j0) {
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
            for (int j = sp.j0; j < sp.j1; ++j, ++nt) {
                ok = mbar_wait_warp(smem_u32(&sfull[w]), nt & 1u, s_abort, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                if (sp.few_keys<MODE>()) {
                    if (sp.hides(j)) tile(j, std::true_type{}, std::true_type{});
                    else tile(j, std::false_type{}, std::true_type{});
                } else if constexpr (!biased(MODE)) {
                    if (sp.hides(j)) tile(j, std::true_type{}, std::false_type{});
                    else tile(j, std::false_type{}, std::false_type{});
                }
            }
            if (!ok) break;
            // ---- the item's rows: sums over a row's four lanes, then 1 / l to the quarter's two warps
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                // (no weight at all: nothing is seen; a NaN sum is one, of O and of lse)
                if ((lane & 3) == 0) {
                    s_inv[w * kTile + row0 + 8 * r] = l[r] == 0.f ? 0.f : 1.f / l[r];
                    if (i0 + 8 * r < p.T)
                        p.lse[(int64_t)it.h * p.T + i0 + 8 * r] =
                            l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2 + (capped(MODE) ? p.cap : 0.f);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&lready[4 * w + quarter]));
            // (this barrier completes twice an item: the sums are there; both warps have read them)
            ok = mbar_wait_warp(smem_u32(&lready[4 * w + quarter]), 0, s_abort, p.wait_ns);
            if (!ok) break;
            const int row = quarter * 32 + lane, i = it.q0 + w * kTile + row;
            const float inv = s_inv[w * kTile + row];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&lready[4 * w + quarter]));
            if (sp.any()) {
                ok = mbar_wait_warp(smem_u32(&odone[w]), nq & 1u, s_abort, p.wait_ns);
                if (!ok) break;
                ++nq;
                tc_fence_after();
            }
            // each of the quarter's warps writes half of the dims, a thread one row of them
            const int64_t at = (int64_t)i * p.hq + it.h;
            uint16_t* out = p.out + at * p.d;
            int8_t* out_lo = p.out_lo ? p.out_lo + at * p.d16 : nullptr;
#pragma unroll 1
            for (int cc = sub * (DP / 2); cc < (sub + 1) * (DP / 2); cc += 16) {
                float o[16];
                if (sp.any()) {  // (uniform over the query tile's warps)
                    uint32_t raw[16];
                    tmem_ld_x16(tmem + all_lanes + 2 * kTile + w * DP + cc, raw);
                    tmem_ld_wait16(raw);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = inv == 0.f ? 0.f : __uint_as_float(raw[e]) * inv;
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
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kFwdMath) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DP, int MODE>
cudaError_t launch_fwd(const AttnParams& p, const FwdMaps& maps, int sms, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(attn_fwd_kernel<DP, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               FwdCfg<DP>::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)((p.T + p.rows - 1) / p.rows) * p.hq;
    const unsigned grid = (unsigned)(items < sms ? items : sms);
    return launch_pdl(attn_fwd_kernel<DP, MODE>, dim3(grid), dim3(kFwdThreads), FwdCfg<DP>::kSmem, st, nullptr, 0, p, maps);
}

template <int DP>
cudaError_t launch_mode(int mode, const AttnParams& p, const FwdMaps& maps, int sms, cudaStream_t st) {
    switch (mode) {
        case ATTN_PLAIN: return launch_fwd<DP, ATTN_PLAIN>(p, maps, sms, st);
        case ATTN_BIAS: return launch_fwd<DP, ATTN_BIAS>(p, maps, sms, st);
        case ATTN_CAP: return launch_fwd<DP, ATTN_CAP>(p, maps, sms, st);
        default: return launch_fwd<DP, ATTN_CAP_BIAS>(p, maps, sms, st);
    }
}

lm_status launch_attn_fwd(const AttnParams& given, int sms, cudaStream_t st) {
    FwdMaps maps;
    AttnParams p = given;
    // One query tile an item where the SMs take all of them at once (512 tokens, 32 heads: 19.5 us, 20.8 with two;
    // 1024 tokens, 16 heads of 64 dims: 24.1 and 26.0)
    p.rows = (int64_t)((p.T + 2 * kTile - 1) / (2 * kTile)) * p.hq * 2 <= sms ? kTile : 2 * kTile;
    const lm_heads q{p.q.p, p.q.ts, p.q.hs}, k{p.k.p, p.k.ts, p.k.hs}, v{p.v.p, p.v.ts, p.v.hs};
    lm_status s = encode_heads(&maps.q, q, p.T, p.hq, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps.k, k, p.T, p.hk, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps.v, v, p.T, p.hk, p.d, kTile);
    if (s != LM_OK) return s;
    // without slopes the factor of the scores goes into the exponent and has to be positive (the maximum of s c
    // is c max s); the cap's is
    const int mode = (p.slopes || !(p.scale > 0.f || p.cap > 0.f) ? ATTN_BIAS : 0) | (p.cap > 0.f ? ATTN_CAP : 0);
    const cudaError_t e = p.d <= 64 ? launch_mode<64>(mode, p, maps, sms, st) : launch_mode<128>(mode, p, maps, sms, st);
    return e == cudaSuccess ? LM_OK : report_error(LM_ERR_CUDA, "attn forward launch: %s", cudaGetErrorString(e));
}

}  // namespace lm
