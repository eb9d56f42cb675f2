// Attention backward (include/lora_layer.h) on the tensor cores: two passes over the score tiles,
// one per owner of the result, so that no sum crosses CTAs and every run gives the same bits.
//   P = 2^{x - lse log2 e},  dz = P (dO.v - delta) (1 - (u / cap)^2),  delta = dO.O
//   attn_dkv: a CTA owns 128 keys of one key/value head and walks the query tiles that see them,
//             over all query heads of the group:  dV += P^T dO,  dK += dz^T Q   (4 products a tile)
//   attn_dq:  a CTA owns 128 queries of one head and walks their key tiles:  dQ += dz K  (3 products)
// The scores and dO.v are formed in both, seven products of 128 x 128 x d where one pass with dQ
// summed by atomics would take five; in exchange there is no fp32 dQ in memory, nothing to clear
// and no order of arrival.  Scores are formed with the owned rows as tensor-memory lanes (S^T in
// attn_dkv), so P and dz go back to tensor memory as the left operand of the next product without
// crossing threads.
// P and dz are rounded to bf16, the type of the tensor cores' operands, and what that leaves out is not multiplied: dV is
// 2.35e-3 off (2-norm), dQ and dK 2.3e-3 to 2.6e-3, where fp32 products rounded once leave 1.66e-3.  To multiply the
// low bits as well would be three products more for seven.
// attn_dkv is bound by the way from one product to the next: S to P to the next S, whose place P takes,
// and the same for dP and dz; sixteen warps share each step, 32 columns a thread.  8192 causal tokens, 32
// query heads on 8 of 128 dims, by itself: 776 us, 1.42 PFLOP/s, 0.74 of the burst rate.  attn_dq has room for a
// second score tile and runs its three products at 0.92 of it, 470 us by itself.  Both are one launch, dQ's CTAs
// after the others: they fill what dK and dV's last items leave, 1222 us.  (14 documents: 196 and 139 by
// themselves, 302 together.)  In two launches a whole step of 700 tokens took 76 us against 60, of 5000 in 84
// documents 155 against 124.  These are times of single launches; step after step the 8192 tokens draw all of the
// board's power, and the lower clock takes the forward, delta and this launch from 1649 us together to 1763.
// Tried in attn_dkv: eight warps that form P and eight that form dz from its bf16 rounding, a tile apart,
// 699 us there, but dK's error 2.9e-3 against 2.4e-3, and 133 against 119 for capped prefixes, 62 against 58
// for a biased window; the same with P in f16 for dz, 748 and 208 against 192 for packed documents (788 for the kept
// form then); two groups of eight that take every other tile, 771 and 223; P and dz handed over in two halves, 897 (a store to tensor
// memory and its wait take 300 cycles while the tensor cores multiply from shared memory).  In attn_dq: one
// CTA an item instead of CTAs that stay, 479; K and V asked for in another order than they are used, 623.
#pragma once

#include "lm_attn.cuh"

namespace lm {

// Sixteen arithmetic warps (four warpgroups, a thread: one row, 32 columns) and a warpgroup for the
// loader's and the issuer's warps: 640 threads start with 96 registers each.
constexpr int kBwdThreads = 640, kBwdMath = 16, kBwdMathRegs = 104, kBwdIssueRegs = 64;
static_assert(4 * kBwdMathRegs + kBwdIssueRegs <= 5 * 96, "a register split above the launch's total waits forever");
constexpr int kQStages = 2;  // attn_dkv: query tiles, and dO tiles, in flight

// A = P or dz in tensor memory: each 32 columns of the tile packed at the first 16 of their place
__device__ __forceinline__ void mma_weights(uint32_t d, uint32_t t, uint32_t b, uint32_t idesc, bool first) {
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk)
        umma_bf16_ts(d, t + (uint32_t)((kk >> 1) * 32 + (kk & 1) * 8), desc(b + kk * 128), idesc, first && kk == 0 ? 0u : 1u);
}

struct ScoreMath {
    float c, cap2, slope;
};
template <int MODE>
__device__ __forceinline__ ScoreMath score_math(const AttnParams& p) {
    return ScoreMath{capped(MODE) ? 2.f * kLog2e * p.scale / p.cap : p.scale * kLog2e, 2.f * p.cap * kLog2e, 0.f};
}
// x - lse in units of log 2 for two neighbouring columns (nlse holds the constant cap of capped scores);
// bend = -1/4 du/dz.  dist: i - j of the first, and the second's is one more (STEP 1: the columns are queries)
// or one less (-1: keys).
template <int MODE, int STEP>
__device__ __forceinline__ float2 exponents(const ScoreMath& S, float2 qk, float dist, float2 nlse, float2& bend) {
    float2 y;
    if (capped(MODE)) {
        const float2 n = cap_n(__fmul2_rn(qk, two(S.c)));
        bend = __ffma2_rn(n, n, n);
        y = __ffma2_rn(n, two(S.cap2), nlse);
    } else {
        y = __ffma2_rn(qk, two(S.c), nlse);
    }
    if (biased(MODE)) {
        y.x = fmaf(-S.slope, fabsf(dist), y.x);
        y.y = fmaf(-S.slope, fabsf(dist + (float)STEP), y.y);
    }
    return y;
}
// what dz K and dz^T Q are multiplied by in the end
template <int MODE>
__device__ __forceinline__ float gradient_scale(const AttnParams& p) {
    return capped(MODE) ? -4.f * p.scale : p.scale;
}

struct BwdMaps {
    CUtensorMap q, k, v, dO, dK, dV;
};

// ------------------------------------------------------------------ dK, dV
template <int DP>
struct DkvCfg {
    static constexpr uint32_t kTileBytes = (DP / 64) * kBoxBytes;
    static constexpr uint32_t kRowBytes = kTile * 4;  // nlse, and -delta, of a query tile
    static constexpr int kSmem = 2048 + (2 + 2 * kQStages) * kTileBytes + kQStages * 2 * kRowBytes;
    // CTAs that may share a key tile: the others' sums have to fit where the query and dO tiles were
    static constexpr int kMaxSplit = DP == 128 ? 4 : 2;
    static_assert((kMaxSplit - 1) * (2 * (DP / 64) / kMaxSplit) * kTile * 64 * 4 <= 2 * kQStages * kTileBytes, "");
};

// SHARED: a cluster of `ctas` CTAs shares the key tile.
template <int DP, int MODE, bool SHARED, int FORM>
__device__ __forceinline__ void attn_dkv(const AttnParams& p, const BwdMaps& maps, int ctas) {
    const int split = SHARED ? ctas : 1;
    using C = DkvCfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* qfull = reinterpret_cast<uint64_t*>(smem);
    uint64_t* qempty = qfull + kQStages;
    uint64_t* ofull = qempty + kQStages;
    uint64_t* oempty = ofull + kQStages;
    uint64_t* kvfull = oempty + kQStages;
    uint64_t* sfull = kvfull + 1;   // S^T ready
    uint64_t* pfull = sfull + 1;    // P^T written
    uint64_t* dpfull = pfull + 1;   // dP^T ready
    uint64_t* dsfull = dpfull + 1;  // dz^T written
    uint64_t* drain = dsfull + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* s_bad = s_abort + 1;  // [4] a warp of the warpgroup gave up
    uint4* s_seen = reinterpret_cast<uint4*>(smem + 768);  // [stage] the tile's queries that see something (not SELF)
    uint8_t* sk = smem + 1024;
    uint8_t* sv = sk + C::kTileBytes;
    uint8_t* sq = sv + C::kTileBytes;
    uint8_t* so = sq + kQStages * C::kTileBytes;
    float* srow = reinterpret_cast<float*>(so + kQStages * C::kTileBytes);  // [stage][nlse, -delta][128]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (under a causal mask the first keys, seen by most, come first)
    // PARTS: `kparts` CTAs that are no cluster share a key tile; their sums are joined by another kernel
    constexpr bool kShares = SHARED || FORM == ATTN_PARTS;
    const int shares = SHARED ? split : FORM == ATTN_PARTS ? p.kparts : 1;
    const int item = (int)blockIdx.x / shares, rank = (int)blockIdx.x % shares;
    const int g = item % p.hk, n = p.hq / p.hk;

    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kQStages; ++s) {
            mbar_init(smem_u32(&qfull[s]), 1);
            mbar_init(smem_u32(&qempty[s]), 1);
            mbar_init(smem_u32(&ofull[s]), 1);
            mbar_init(smem_u32(&oempty[s]), 1);
        }
        mbar_init(smem_u32(kvfull), 1);
        mbar_init(smem_u32(sfull), 1);
        mbar_init(smem_u32(pfull), kBwdMath);
        mbar_init(smem_u32(dpfull), 1);
        mbar_init(smem_u32(dsfull), kBwdMath);
        mbar_init(smem_u32(drain), 1);
        *s_abort = s_bad[0] = s_bad[1] = s_bad[2] = s_bad[3] = 0;
        fence_mbar_init();
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
        tma_prefetch_map(&maps.dO);
    }
    __syncwarp();
    if (warp == kBwdMath) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    const uint32_t tmem = (uint32_t)uni((int)*tmem_slot);
    const uint32_t ts = tmem, tdp = tmem + kTile, tdv = tmem + 2 * kTile, tdk = tdv + DP;
    const int k0 = uni(item / p.hk * kTile);
    const TokRange rf = key_range<FORM>(p, k0), rl = key_range<FORM>(p, min(k0 + kTile, p.Tk) - 1);
    const int qt0 = uni(rf.qlo / kTile), nt = uni(rl.qhi > rf.qlo ? (rl.qhi + kTile - 1) / kTile - qt0 : 0);
    // (head of the group, query tile) pairs, heads outermost: this CTA's are [first, first + N)
    auto begin = [&](int r) { return (int)((int64_t)nt * n * r / shares); };
    const int first = kShares ? begin(rank) : 0, N = kShares ? begin(rank + 1) - first : nt * n;
    const int hh0 = kShares && nt ? first / nt : 0, qi0 = kShares && nt ? first % nt : 0;

    if (warp >= kBwdMath) {
        regs_down<kBwdIssueRegs>();
        if (warp == kBwdMath + 1) {  // ---------------- loader
            if (lane == 0 && N > 0 && !(p.starve & K_ATTN_DKV)) {
                bool ok = true;
                mbar_expect_tx(smem_u32(kvfull), 2 * C::kTileBytes);
                for (int b = 0; b < DP / 64; ++b) {
                    tma_load_3d(smem_u32(sk + b * kBoxBytes), &maps.k, smem_u32(kvfull), b * 64, g, k0);
                    tma_load_3d(smem_u32(sv + b * kBoxBytes), &maps.v, smem_u32(kvfull), b * 64, g, k0);
                }
                uint32_t it = 0, no = 0;  // query and dO tiles asked for
                // (which queries see something is asked for a tile ahead, as which keys are seen below)
                uint4 seen = make_uint4(0, 0, 0, 0);
                if (FORM != ATTN_SELF && p.qseen && N > 0) seen = p.qseen[qt0 + qi0];  // (none: qt0 may be past the last tile)
                for (int hh = hh0; ok && (kShares ? no < (uint32_t)N : hh < n); ++hh)
                    for (int qt = qt0 + (hh == hh0 ? qi0 : 0); qt < qt0 + nt && (!kShares || no < (uint32_t)N); ++qt) {
                        const int h = g * n + hh;
                        const uint32_t s = no % kQStages, ph = (no / kQStages) & 1u;
                        const uint32_t bq = smem_u32(&qfull[s]), bo = smem_u32(&ofull[s]);
                        if (!mbar_wait(smem_u32(&qempty[s]), ph ^ 1u, s_abort, p.wait_ns)) {
                            ok = false;
                            break;
                        }
                        if (FORM != ATTN_SELF && p.qseen) {
                            s_seen[s] = seen;
                            seen = p.qseen[qt + 1 < qt0 + nt ? qt + 1 : qt0];
                        }
                        mbar_expect_tx(bq, C::kTileBytes + 2 * C::kRowBytes);
                        for (int b = 0; b < DP / 64; ++b)
                            tma_load_3d(smem_u32(sq + s * C::kTileBytes + b * kBoxBytes), &maps.q, bq, b * 64, h, qt * kTile);
                        const int64_t row = (int64_t)h * p.Tp + qt * kTile;
                        bulk_load(smem_u32(srow + s * 2 * kTile), p.nlse + row, C::kRowBytes, bq);
                        bulk_load(smem_u32(srow + s * 2 * kTile + kTile), p.ndelta + row, C::kRowBytes, bq);
                        ++it;
                        if (!mbar_wait(smem_u32(&oempty[s]), ph ^ 1u, s_abort, p.wait_ns)) {
                            ok = false;
                            break;
                        }
                        mbar_expect_tx(bo, C::kTileBytes);
                        for (int b = 0; b < DP / 64; ++b)
                            tma_load_3d(smem_u32(so + s * C::kTileBytes + b * kBoxBytes), &maps.dO, bo, b * 64, h, qt * kTile);
                        ++no;
                    }
                if (!ok) {
                    attn_error(p, 6, 1);
                    *s_abort = 1;
                }
                volatile int never = 0;
                bool in = mbar_wait(smem_u32(kvfull), 0, &never, p.wait_ns);
                in = drain_fills(smem_u32(&qfull[0]), kQStages, it, p.wait_ns) && in;
                in = drain_fills(smem_u32(&ofull[0]), kQStages, no, p.wait_ns) && in;
                if (!in) attn_error(p, 6, 5);
            }
        } else if (warp == kBwdMath && elect_one()) {  // ---------------- tensor cores
            const int ksteps = (p.d + 15) / 16;
            const uint32_t ids = make_idesc_bf16(kTile, kTile, false, false);
            const uint32_t idd = make_idesc_bf16(kTile, ksteps * 16, false, true);  // Q and dO are [query][dim]: MN-major
            int in0 = 0, in1 = 0;
            if (FORM == ATTN_SELF) inside_tokens(p, in0, in1);
            // (a stage's word is there with its queries, which are waited for before its dO)
            auto clear = [&](uint8_t* tile, int it, uint32_t s) {
                if (FORM == ATTN_SELF) clear_padding(tile, DP / 64, (qt0 + (first + it) % nt) * kTile, in0, in1);
                else if (p.qseen) clear_unseen(tile, DP / 64, s_seen[s]);
            };
            bool ok = N <= 0 || mbar_wait(smem_u32(kvfull), 0, s_abort, p.wait_ns);
            auto scores = [&](int it) {  // S^T(it) = K Q^T
                const uint32_t s = (uint32_t)it % kQStages;
                if (!mbar_wait(smem_u32(&qfull[s]), ((uint32_t)it / kQStages) & 1u, s_abort, p.wait_ns)) return false;
                clear(sq + s * C::kTileBytes, it, s);
                tc_fence_after();
                mma_rows<DP>(ts, desc_rows(smem_u32(sk)), desc_rows(smem_u32(sq + s * C::kTileBytes)), ksteps, ids);
                umma_commit(smem_u32(sfull));
                return true;
            };
            auto dots = [&](int it) {  // dP^T(it) = V dO^T
                const uint32_t s = (uint32_t)it % kQStages;
                if (!mbar_wait(smem_u32(&ofull[s]), ((uint32_t)it / kQStages) & 1u, s_abort, p.wait_ns)) return false;
                clear(so + s * C::kTileBytes, it, s);
                tc_fence_after();
                mma_rows<DP>(tdp, desc_rows(smem_u32(sv)), desc_rows(smem_u32(so + s * C::kTileBytes)), ksteps, ids);
                umma_commit(smem_u32(dpfull));
                return true;
            };
            if (ok && N > 0) ok = scores(0) && dots(0);
            for (int it = 0; ok && it < N; ++it) {
                const uint32_t s = (uint32_t)it % kQStages;
                if (!mbar_wait(smem_u32(pfull), (uint32_t)it & 1u, s_abort, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                mma_weights(tdv, ts, desc_cols(smem_u32(so + s * C::kTileBytes)), idd, it == 0);
                umma_commit(smem_u32(&oempty[s]));
                if (it + 1 < N && !scores(it + 1)) {  // (P(it) has been read by then: products run in order)
                    ok = false;
                    break;
                }
                if (!mbar_wait(smem_u32(dsfull), (uint32_t)it & 1u, s_abort, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                mma_weights(tdk, tdp, desc_cols(smem_u32(sq + s * C::kTileBytes)), idd, it == 0);
                umma_commit(smem_u32(&qempty[s]));
                if (it + 1 < N && !dots(it + 1)) {
                    ok = false;
                    break;
                }
            }
            if (!ok) {
                attn_error(p, 6, 2);
                *s_abort = 1;
            }
            umma_commit(smem_u32(drain));
            volatile int never = 0;
            mbar_wait(smem_u32(drain), 0, &never, p.wait_ns);
        }
        __syncwarp();
        if (SHARED) {  // (the arithmetic warps' two meetings of the cluster)
            cluster_sync();
            cluster_sync();
        }
    } else {  // ---------------- arithmetic: one key row, 32 query columns per thread
        regs_up<kBwdMathRegs>();
        const int part = warp >> 2;
        const int k = k0 + (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tsw = ts + lanes + part * 32, tdpw = tdp + lanes + part * 32;
        TokRange r{0, 0, 0, 0};
        if (k < p.Tk) r = key_range<FORM>(p, k);
        ScoreMath S = score_math<MODE>(p);
        bool ok = true;
        // one query tile, its scores ready; tiles with hidden pairs have code of their own
        auto tile = [&](int it, const float* row, float dist, uint32_t bits, auto hides) {
            constexpr bool HIDDEN = decltype(hides)::value;
            float x[32];
            uint32_t pk[16];
            tmem_ld_f32<0>(tsw, x);
            const bool some = !HIDDEN || __any_sync(0xffffffffu, bits != 0u);
            tmem_ld_wait_f32<0>(x);
            if (some) {  // (a chunk that none of the warp's keys is seen from has no exponentials)
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 nl = *reinterpret_cast<const float4*>(row + e);
                    const float nls[4] = {nl.x, nl.y, nl.z, nl.w};
#pragma unroll
                    for (int f = 0; f < 4; f += 2) {
                        float2 bend = two(1.f);
                        const float2 y = exponents<MODE, 1>(S, make_float2(x[e + f], x[e + f + 1]), dist + (float)(e + f),
                                                            make_float2(nls[f], nls[f + 1]), bend);
                        float2 P = make_float2(ex2(y.x), ex2(y.y));
                        if (HIDDEN) {
                            if (!(bits >> (e + f) & 1u)) P.x = 0.f;
                            if (!(bits >> (e + f + 1) & 1u)) P.y = 0.f;
                        }
                        pk[(e + f) / 2] = pack_bf16x2(P.x, P.y);
                        if (capped(MODE)) P = __fmul2_rn(P, bend);
                        x[e + f] = P.x;
                        x[e + f + 1] = P.y;
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = 0u;
            }
            tmem_st_x16(tsw, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(pfull));
            if (!mbar_wait_warp(smem_u32(dpfull), (uint32_t)it & 1u, s_abort, p.wait_ns)) return false;
            tc_fence_after();
            if (some) {
                float y[32];
                tmem_ld_f32<0>(tdpw, y);
                tmem_ld_wait_f32<0>(y);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 dl = *reinterpret_cast<const float4*>(row + kTile + e);
                    const float dls[4] = {dl.x, dl.y, dl.z, dl.w};
#pragma unroll
                    for (int f = 0; f < 4; f += 2) {
                        float2 d = __fadd2_rn(make_float2(y[e + f], y[e + f + 1]), make_float2(dls[f], dls[f + 1]));
                        d = __fmul2_rn(d, make_float2(x[e + f], x[e + f + 1]));
                        if (HIDDEN) {  // (not 0 x what a padding key's dP holds)
                            if (!(bits >> (e + f) & 1u)) d.x = 0.f;
                            if (!(bits >> (e + f + 1) & 1u)) d.y = 0.f;
                        }
                        pk[(e + f) / 2] = pack_bf16x2(d.x, d.y);
                    }
                }
            }
            tmem_st_x16(tdpw, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(dsfull));
            return true;
        };
        int it = 0;
        for (int hh = hh0; ok && (kShares ? it < N : hh < n); ++hh) {
            if (biased(MODE)) S.slope = p.slopes[g * n + hh] * kLog2e;
            for (int qt = qt0 + (hh == hh0 ? qi0 : 0); qt < qt0 + nt && (!kShares || it < N); ++qt, ++it) {
                const int q0 = qt * kTile + part * 32;
                const float* row = srow + (it % kQStages) * 2 * kTile + part * 32;
                // every query of the tile sees every key of this one, or some pair is hidden
                const bool hidden = qt * kTile < rl.qlo || (qt + 1) * kTile > rf.qhi;
                const uint32_t bits = hidden ? bits_between(r.qlo - q0, r.qhi - q0) : ~0u;
                const float dist = (float)(q0 - k);
                // the query tile's rows (nlse, -delta) come with it; the scores are ready after it is
                if (!mbar_wait_warp(smem_u32(&qfull[it % kQStages]), ((uint32_t)it / kQStages) & 1u, s_abort, p.wait_ns) ||
                    !mbar_wait_warp(smem_u32(sfull), (uint32_t)it & 1u, s_abort, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // (a warp whose keys are seen from all of its columns has nothing to mask)
                ok = __all_sync(0xffffffffu, bits == ~0u) ? tile(it, row, dist, bits, std::false_type{})
                                                         : tile(it, row, dist, bits, std::true_type{});
                if (!ok) break;
            }
        }
        // DP / 64 warpgroups write dV, as many dK, a box of 64 dims each
        if (ok && N > 0) ok = mbar_wait_warp(smem_u32(drain), 0, s_abort, p.wait_ns);
        tc_fence_after();
        if (!ok && lane == 0) {
            attn_error(p, 6, 3);
            *s_abort = 1;
        }
        // (b's box, of 64 dims of dV or dK, is the (b % split)-th CTA's to write)
        constexpr int kBoxes = DP / 64;
        const int r128 = (warp & 3) * 32 + lane, b = part % kBoxes, owner = SHARED ? part % split : 0;
        const bool key = part >= kBoxes;
        const uint32_t acc = (key ? tdk : tdv) + lanes + b * 64;
        uint8_t* box = sk + part * kBoxBytes;  // (staged where the keys and values were)
        if (FORM == ATTN_PARTS && p.kparts > 1) {  // this share's sums, in fp32
            if (ok && part < 2 * kBoxes)
                store_dims_f32<64>(p.part_dkv + ((((int64_t)rank * 2 + (key ? 1 : 0)) * p.Tk + k) * p.hk + g) * p.d,
                                   (key ? tdk : tdv) + lanes, b * 64, p.d, key ? gradient_scale<MODE>(p) : 1.f, N > 0, k < p.Tk);
        } else if (!SHARED) {
            if (group_ok(ok, s_bad + part, 1 + part) && part < 2 * kBoxes) {
                stage_row(box, r128, acc, key ? gradient_scale<MODE>(p) : 1.f, N > 0);
                store_box(key ? &maps.dK : &maps.dV, box, b * 64, g, k0, 1 + part, r128 == 0);
            }
        } else {
            // Every CTA's products are done before sums arrive where its query tiles were, and all sums have
            // arrived before any CTA reads them or leaves.  A place holds 64 values of 128 rows, by peer and box.
            auto place = [&](int from, int to) {
                return sq + ((from - (from > to ? 1 : 0)) * (2 * kBoxes / split) + part / split) * (kTile * 64 * 4);
            };
            __syncwarp();
            cluster_sync();
            if (part < 2 * kBoxes && owner != rank && N > 0) {
                const uint32_t to = map_to_rank(smem_u32(place(rank, owner)), owner) + r128 * 16;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x[32];
                    tmem_ld_f32<0>(acc + c * 32, x);
                    tmem_ld_wait_f32<0>(x);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) st_peer4(to + (c * 8 + e / 4) * (kTile * 16), x[e], x[e + 1], x[e + 2], x[e + 3]);
                }
            }
            __syncwarp();
            cluster_sync();
            if (group_ok(ok, s_bad + part, 1 + part) && part < 2 * kBoxes && owner == rank) {
                const float f = key ? gradient_scale<MODE>(p) : 1.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // 16 dims: this CTA's and the others', in their order
                    float s[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[e] = 0.f;
                    for (int from = 0; from < split; ++from) {
                        if (begin(from + 1) == begin(from)) continue;
                        if (from == rank) {
                            uint32_t o[16];
                            tmem_ld_x16(acc + c * 16, o);
                            tmem_ld_wait16(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) s[e] += __uint_as_float(o[e]);
                        } else {
                            const float4* q = reinterpret_cast<const float4*>(place(from, rank)) + r128;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 v = q[(c * 4 + e) * kTile];
                                s[4 * e] += v.x, s[4 * e + 1] += v.y, s[4 * e + 2] += v.z, s[4 * e + 3] += v.w;
                            }
                        }
                    }
                    uint32_t v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = pack_bf16x2(s[2 * e] * f, s[2 * e + 1] * f);
                    stage_pairs(box, r128, c, v);
                }
                store_box(key ? &maps.dK : &maps.dV, box, b * 64, g, k0, 1 + part, r128 == 0);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kBwdMath) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ dQ
template <int DP>
struct DqCfg {
    static constexpr uint32_t kTileBytes = (DP / 64) * kBoxBytes;
    static constexpr int kKStages = 3, kVStages = 2;  // S runs one key tile ahead of dz, so K stays longer
    static constexpr int kSmem = 2048 + (2 + kKStages + kVStages) * kTileBytes;
};
// Item k of this CTA, 128 queries of one head: dealt out like the forward's (the heavier ones first,
// forwards and backwards in turn).  CTAs stay: the next item's operands load and its first scores are
// formed while this one's rows are written (10 thousand cycles an item otherwise, as much as five tiles).
struct DqItem {
    int h, q0, kt0, N;    // key tiles [kt0, kt0 + N) (PARTS: one of `qparts` parts of them)
    int part;
    int lo_max, hi_min;   // keys in [lo_max, hi_min) are seen by every row
    bool valid;
};
// This CTA's place among those that form dQ.
struct DqCtas {
    int at, of;
};
template <int FORM>
__device__ __forceinline__ DqItem dq_item(const AttnParams& p, const DqCtas& who, int k) {
    const int nqt = (p.T + kTile - 1) / kTile, parts = FORM == ATTN_PARTS ? p.qparts : 1;
    int idx = k & 1 ? (k + 1) * who.of - 1 - who.at : k * who.of + who.at, part = 0;
    if (FORM == ATTN_PARTS) {
        part = idx % parts;
        idx /= parts;
    }
    DqItem it{idx % p.hq, (nqt - 1 - idx / p.hq) * kTile, 0, 0, part, 0, 0, idx < nqt * p.hq};
    if (it.valid) {
        const TokRange rf = query_range<FORM>(p, it.q0), rl = query_range<FORM>(p, min(it.q0 + kTile, p.T) - 1);
        it.kt0 = rf.lo / kTile;
        it.N = rl.hi > rf.lo ? (rl.hi + kTile - 1) / kTile - it.kt0 : 0;
        if (FORM == ATTN_PARTS) {  // (at most 2^13 tiles and a few hundred parts)
            const int from = it.N * part / parts, to = it.N * (part + 1) / parts;
            it.kt0 += from;
            it.N = to - from;
        }
        it.lo_max = rl.lo;
        it.hi_min = rf.hi;
    }
    return it;
}

template <int DP, int MODE, int FORM>
__device__ __forceinline__ void attn_dq(const AttnParams& p, const BwdMaps& maps, const DqCtas& who) {
    using C = DqCfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* kfull = reinterpret_cast<uint64_t*>(smem);
    uint64_t* kempty = kfull + C::kKStages;
    uint64_t* vfull = kempty + C::kKStages;
    uint64_t* vempty = vfull + C::kVStages;
    uint64_t* qfull = vempty + C::kVStages;  // [2] the item's Q, dO
    uint64_t* qempty = qfull + 2;
    uint64_t* sfull = qempty + 2;    // [2] S ready
    uint64_t* dpfull = sfull + 2;    // dP ready
    uint64_t* dsfull = dpfull + 1;   // dz written (in place of S), dP read
    uint64_t* dqdone = dsfull + 1;   // the item's last product done
    uint64_t* drain = dqdone + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint4* s_seen = reinterpret_cast<uint4*>(smem + 768);  // [key stage] the tile's keys that somebody sees (not SELF)
    uint64_t* clean = reinterpret_cast<uint64_t*>(smem + 896);  // [key stage] and the others have been cleared
    uint8_t* sq = smem + 1024;
    uint8_t* so = sq + C::kTileBytes;
    uint8_t* sk = so + C::kTileBytes;
    uint8_t* sv = sk + C::kKStages * C::kTileBytes;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kKStages; ++s) {
            mbar_init(smem_u32(&kfull[s]), 1);
            mbar_init(smem_u32(&kempty[s]), 1);
            if (FORM != ATTN_SELF) mbar_init(smem_u32(&clean[s]), 1);
        }
        for (int s = 0; s < C::kVStages; ++s) {
            mbar_init(smem_u32(&vfull[s]), 1);
            mbar_init(smem_u32(&vempty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&qfull[s]), 1);
            mbar_init(smem_u32(&qempty[s]), 1);
            mbar_init(smem_u32(&sfull[s]), 1);
        }
        mbar_init(smem_u32(dpfull), 1);
        mbar_init(smem_u32(dsfull), kBwdMath);
        mbar_init(smem_u32(dqdone), 1);
        mbar_init(smem_u32(drain), 1);
        *s_abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
        tma_prefetch_map(&maps.dO);
    }
    __syncwarp();
    if (warp == kBwdMath) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    const uint32_t tmem = (uint32_t)uni((int)*tmem_slot);
    const uint32_t tdp = tmem + 2 * kTile, tdq = tmem + 3 * kTile;
    const int rounds = ((p.T + kTile - 1) / kTile * p.hq * (FORM == ATTN_PARTS ? p.qparts : 1) + who.of - 1) / who.of;

    if (warp >= kBwdMath) {
        regs_down<kBwdIssueRegs>();
        if (warp == kBwdMath + 1) {  // ---------------- loader
            if (lane == 0) {
                bool ok = true;
                uint32_t nk = 0, nv = 0, nq[2] = {0, 0};  // tiles asked for
                uint4 seen = make_uint4(0, 0, 0, 0);
                for (int r = p.starve & K_ATTN_DQ ? rounds : 0; ok && r < rounds; ++r) {
                    const DqItem it = dq_item<FORM>(p, who, r);
                    if (FORM != ATTN_SELF && p.kseen && it.N > 0) seen = p.kseen[it.kt0];
                    auto query = [&](int which) {  // Q, then dO
                        if (!mbar_wait(smem_u32(&qempty[which]), (nq[which] & 1u) ^ 1u, s_abort, p.wait_ns)) return false;
                        const uint32_t bar = smem_u32(&qfull[which]);
                        mbar_expect_tx(bar, C::kTileBytes);
                        for (int b = 0; b < DP / 64; ++b)
                            tma_load_3d(smem_u32((which ? so : sq) + b * kBoxBytes), which ? &maps.dO : &maps.q, bar, b * 64, it.h,
                                        it.q0);
                        ++nq[which];
                        return true;
                    };
                    for (int j = 0; ok && j < it.N; ++j)
                        for (int kv = 0; kv < 2; ++kv) {  // Q, K_0, dO, V_0, K_1, V_1, ...
                            if (j == 0 && !query(kv)) {
                                ok = false;
                                break;
                            }
                            uint32_t& n = kv ? nv : nk;
                            const uint32_t st = kv ? n % C::kVStages : n % C::kKStages;
                            const uint32_t ph = (kv ? n / C::kVStages : n / C::kKStages) & 1u;
                            const uint32_t bar = smem_u32(kv ? &vfull[st] : &kfull[st]);
                            if (!mbar_wait(smem_u32(kv ? &vempty[st] : &kempty[st]), ph ^ 1u, s_abort, p.wait_ns)) {
                                ok = false;
                                break;
                            }
                            if (FORM != ATTN_SELF && !kv && p.kseen) {
                                s_seen[st] = seen;
                                seen = p.kseen[it.kt0 + min(j + 1, it.N - 1)];
                            }
                            mbar_expect_tx(bar, C::kTileBytes);
                            for (int b = 0; b < DP / 64; ++b)
                                tma_load_3d(smem_u32((kv ? sv : sk) + st * C::kTileBytes + b * kBoxBytes), kv ? &maps.v : &maps.k, bar,
                                            b * 64, it.h / (p.hq / p.hk), (it.kt0 + j) * kTile);
                            ++n;
                        }
                }
                if (!ok) {
                    attn_error(p, 7, 1);
                    *s_abort = 1;
                }
                volatile int never = 0;
                bool in = drain_fills(smem_u32(&kfull[0]), C::kKStages, nk, p.wait_ns);
                in = drain_fills(smem_u32(&vfull[0]), C::kVStages, nv, p.wait_ns) && in;
                for (int s = 0; s < 2; ++s)
                    if (nq[s]) in = mbar_wait(smem_u32(&qfull[s]), (nq[s] - 1u) & 1u, &never, p.wait_ns) && in;
                if (!in) attn_error(p, 7, 5);
            }
        } else if (warp == kBwdMath && elect_one()) {  // ---------------- tensor cores
            const int ksteps = (p.d + 15) / 16;
            const uint32_t ids = make_idesc_bf16(kTile, kTile, false, false);
            const uint32_t idd = make_idesc_bf16(kTile, ksteps * 16, false, true);  // K is [key][dim]: MN-major
            int in0 = 0, in1 = 0;
            if (FORM == ATTN_SELF) inside_tokens(p, in0, in1);
            bool ok = true;
            uint32_t base = 0, items = 0;  // tiles and items with tiles before this one
            DqItem next = dq_item<FORM>(p, who, 0);
            for (int r = 0; ok && r < rounds; ++r) {
                const DqItem it = next;
                next = dq_item<FORM>(p, who, r + 1);
                if (it.N <= 0) continue;
                auto scores = [&](int j) {  // S(j) = Q K^T, in buffer t & 1
                    const uint32_t t = base + (uint32_t)j, s = t % C::kKStages;
                    uint64_t* there = FORM != ATTN_SELF && p.kseen ? clean : kfull;
                    if (!mbar_wait(smem_u32(&there[s]), (t / C::kKStages) & 1u, s_abort, p.wait_ns)) return false;
                    if (FORM == ATTN_SELF) clear_padding(sk + s * C::kTileBytes, DP / 64, (it.kt0 + j) * kTile, in0, in1);
                    tc_fence_after();
                    mma_rows<DP>(tmem + (t & 1u) * kTile, desc_rows(smem_u32(sq)), desc_rows(smem_u32(sk + s * C::kTileBytes)), ksteps,
                                 ids);
                    umma_commit(smem_u32(&sfull[t & 1u]));
                    if (j == it.N - 1) umma_commit(smem_u32(&qempty[0]));
                    return true;
                };
                auto dots = [&](int j) {  // dP(j) = dO V^T
                    const uint32_t t = base + (uint32_t)j, s = t % C::kVStages;
                    if (!mbar_wait(smem_u32(&vfull[s]), (t / C::kVStages) & 1u, s_abort, p.wait_ns)) return false;
                    tc_fence_after();
                    mma_rows<DP>(tdp, desc_rows(smem_u32(so)), desc_rows(smem_u32(sv + s * C::kTileBytes)), ksteps, ids);
                    umma_commit(smem_u32(dpfull));
                    umma_commit(smem_u32(&vempty[s]));
                    if (j == it.N - 1) umma_commit(smem_u32(&qempty[1]));
                    return true;
                };
                ok = mbar_wait(smem_u32(&qfull[0]), items & 1u, s_abort, p.wait_ns) && scores(0) &&
                     mbar_wait(smem_u32(&qfull[1]), items & 1u, s_abort, p.wait_ns) && dots(0) && (it.N < 2 || scores(1));
                for (int j = 0; ok && j < it.N; ++j) {
                    const uint32_t t = base + (uint32_t)j, s = t % C::kKStages;
                    if (!mbar_wait(smem_u32(dsfull), t & 1u, s_abort, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (j + 1 < it.N && !dots(j + 1)) {
                        ok = false;
                        break;
                    }
                    mma_weights(tdq, tmem + (t & 1u) * kTile, desc_cols(smem_u32(sk + s * C::kTileBytes)), idd, j == 0);
                    umma_commit(smem_u32(&kempty[s]));
                    if (j == it.N - 1) umma_commit(smem_u32(dqdone));
                    if (j + 2 < it.N && !scores(j + 2)) {
                        ok = false;
                        break;
                    }
                }
                base += (uint32_t)it.N;
                ++items;
            }
            if (!ok) {
                attn_error(p, 7, 2);
                *s_abort = 1;
            }
            umma_commit(smem_u32(drain));
            volatile int never = 0;
            mbar_wait(smem_u32(drain), 0, &never, p.wait_ns);
        }
        if (FORM != ATTN_SELF && warp == kBwdMath + 2 && p.kseen) {  // ---------------- clears keys that nobody sees
            bool ok = true;
            uint32_t t = 0;
            for (int r = 0; ok && r < rounds; ++r) {
                const DqItem it = dq_item<FORM>(p, who, r);
                for (int j = 0; ok && j < it.N; ++j, ++t) {
                    const uint32_t s = t % C::kKStages;
                    ok = mbar_wait_warp(smem_u32(&kfull[s]), (t / C::kKStages) & 1u, s_abort, p.wait_ns);
                    if (!ok) break;
                    clear_unseen_warp(sk + s * C::kTileBytes, DP / 64, s_seen[s]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&clean[s]));
                }
            }
            if (!ok && lane == 0) {
                attn_error(p, 7, 4);
                *s_abort = 1;
            }
        }
    } else {  // ---------------- arithmetic: one query row, 32 key columns per thread
        regs_up<kBwdMathRegs>();
        const int part = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        struct RowOf {
            int lo, hi;
            float nlse, ndelta;
        };
        auto row_of = [&](const DqItem& it) {
            RowOf r{0, 0, 0.f, 0.f};
            const int i = it.q0 + row;
            if (it.valid && i < p.T) {
                const TokRange t = query_range<FORM>(p, i);
                r.lo = t.lo;
                r.hi = t.hi;
                r.nlse = p.nlse[(int64_t)it.h * p.Tp + i];
                r.ndelta = p.ndelta[(int64_t)it.h * p.Tp + i];
            }
            return r;
        };
        ScoreMath S = score_math<MODE>(p);
        bool ok = true;
        uint32_t t = 0, items = 0;  // tiles; items with tiles
        DqItem next = dq_item<FORM>(p, who, 0);
        RowOf next_row = row_of(next);
        for (int r = 0; ok && r < rounds; ++r) {
            const DqItem it = next;
            const RowOf R = next_row;
            next = dq_item<FORM>(p, who, r + 1);
            next_row = row_of(next);
            if (!it.valid) continue;
            if (biased(MODE)) S.slope = p.slopes[it.h] * kLog2e;
            auto tile = [&](uint32_t tsw, float dist, uint32_t bits, auto hides) {
                constexpr bool HIDDEN = decltype(hides)::value;
                float x[32], y[32];
                uint32_t pk[16];
                tmem_ld_f32<0>(tsw, x);
                const bool some = !HIDDEN || __any_sync(0xffffffffu, bits != 0u);
                tmem_ld_wait_f32<0>(x);
                if (some) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float2 bend = two(1.f);
                        const float2 v = exponents<MODE, -1>(S, make_float2(x[e], x[e + 1]), dist - (float)e, two(R.nlse), bend);
                        float2 P = make_float2(ex2(v.x), ex2(v.y));
                        if (capped(MODE)) P = __fmul2_rn(P, bend);
                        x[e] = P.x;
                        x[e + 1] = P.y;
                    }
                }
                if (!mbar_wait_warp(smem_u32(dpfull), t & 1u, s_abort, p.wait_ns)) return false;
                tc_fence_after();
                if (some) {
                    tmem_ld_f32<0>(tdp + lanes + part * 32, y);
                    tmem_ld_wait_f32<0>(y);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float2 d = __fadd2_rn(make_float2(y[e], y[e + 1]), two(R.ndelta));
                        d = __fmul2_rn(d, make_float2(x[e], x[e + 1]));
                        if (HIDDEN) {
                            if (!(bits >> e & 1u)) d.x = 0.f;
                            if (!(bits >> (e + 1) & 1u)) d.y = 0.f;
                        }
                        pk[e / 2] = pack_bf16x2(d.x, d.y);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[e] = 0u;
                }
                tmem_st_x16(tsw, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(dsfull));
                return true;
            };
            for (int j = 0; j < it.N; ++j, ++t) {
                const uint32_t tsw = tmem + lanes + (t & 1u) * kTile + part * 32;
                const int kt = (it.kt0 + j) * kTile, k0 = kt + part * 32;
                const bool hidden = kt < it.lo_max || kt + kTile > it.hi_min;
                const float dist = (float)(it.q0 + row - k0);
                ok = mbar_wait_warp(smem_u32(&sfull[t & 1u]), (t >> 1) & 1u, s_abort, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t bits = hidden ? bits_between(R.lo - k0, R.hi - k0) : ~0u;
                // (a warp whose rows see all of its columns has nothing to mask)
                ok = __all_sync(0xffffffffu, bits == ~0u) ? tile(tsw, dist, bits, std::false_type{})
                                                         : tile(tsw, dist, bits, std::true_type{});
                if (!ok) break;
            }
            if (!ok) break;
            if (it.N > 0) {
                ok = mbar_wait_warp(smem_u32(dqdone), items & 1u, s_abort, p.wait_ns);
                if (!ok) break;
                ++items;
                tc_fence_after();
            }
            // each warpgroup a quarter of the dims, a thread one row of them
            const int i = it.q0 + row;
            if (FORM == ATTN_PARTS && p.qparts > 1)
                store_dims_f32<DP / 4>(p.part_dq + (((int64_t)it.part * p.T + i) * p.hq + it.h) * p.d, tdq + lanes, part * (DP / 4), p.d,
                                       gradient_scale<MODE>(p), it.N > 0, i < p.T);
            else store_dims<DP / 4>(p.out + ((int64_t)i * p.hq + it.h) * p.d, tdq + lanes, part * (DP / 4), p.d, gradient_scale<MODE>(p),
                               it.N > 0, i < p.T);
            tc_fence_before();  // (the next item's products may overwrite dQ once dz says so)
        }
        if (!ok && lane == 0) {
            attn_error(p, 7, 3);
            *s_abort = 1;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kBwdMath) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ launches
constexpr int kDqWaves = 4;
// One launch: the first `dkv` CTAs form dK and dV, the others dQ as SMs come free.
template <int DP, int MODE, bool SHARED, int FORM>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attn_bwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ BwdMaps maps, int ctas, int dkv) {
    if ((int)blockIdx.x < dkv) attn_dkv<DP, MODE, SHARED, FORM>(p, maps, ctas);
    else attn_dq<DP, MODE, FORM>(p, maps, DqCtas{(int)blockIdx.x - dkv, (int)gridDim.x - dkv});
}
template <int DP, int MODE, bool SHARED, int FORM>
cudaError_t launch_bwd(const AttnParams& p, const BwdMaps& maps, int items, int split, int dq, cudaStream_t st) {
    constexpr int kSmem = DkvCfg<DP>::kSmem > DqCfg<DP>::kSmem ? DkvCfg<DP>::kSmem : DqCfg<DP>::kSmem;
    const cudaError_t e =
        cudaFuncSetAttribute(attn_bwd_kernel<DP, MODE, SHARED, FORM>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim = {(unsigned)split, 1, 1};
    const unsigned grid = (unsigned)(items * split + (dq + split - 1) / split * split);
    LaunchTag tag("attn.bwd", st);
    return launch_pdl(attn_bwd_kernel<DP, MODE, SHARED, FORM>, dim3(grid), dim3(kBwdThreads), kSmem, st, &cluster, SHARED ? 1 : 0, p, maps,
                      split, items * split);
}
template <int DP, int MODE, int FORM>
cudaError_t launch_both(const AttnParams& p, const BwdMaps& maps, int sms, cudaStream_t st) {
    // A key tile is shared where there are fewer of them than SMs and the (head, query tile) pairs that see one
    // are many: down to 4 a CTA while the SMs take all CTAs at once, from 32 a CTA up to two CTAs an SM.  A join
    // costs about six pairs.  (32 query heads on 8, 128 dims: 512 tokens 35 -> 24 us with four CTAs a tile, 27 with
    // two; 1024 62 -> 39 with two, 44 with four; 2048 116 -> 68 with two, 104 with four; 8 heads on 1, 8192 tokens
    // 848 -> 207 with four.  16 heads on 16, 1024 tokens: 20 with one, 29 with two.)
    const int tiles = (p.T + kTile - 1) / kTile, items = (p.Tk + kTile - 1) / kTile * p.hk;  // (of queries; of keys)
    const int reach = p.window > 0 && p.window / kTile + 2 < tiles ? p.window / kTile + 2 : tiles;
    int split = 1;
    while (FORM != ATTN_PARTS && split < DkvCfg<DP>::kMaxSplit) {
        const int pairs = p.hq / p.hk * reach / split, after = items * split * 2;
        if (!(after <= sms && pairs >= 8) && !(after <= 2 * sms && pairs >= 32)) break;
        split *= 2;
    }
    // dQ's CTAs stay and take items, but a few an SM, as those that start late should have less to do (8192 tokens in
    // 14 documents: 506 us with four, 516 with one or two, 515 with eight)
    const int64_t dq_items = (int64_t)tiles * p.hq * (FORM == ATTN_PARTS ? p.qparts : 1);
    const int dq = (int)(dq_items < kDqWaves * sms ? dq_items : kDqWaves * sms);
    if constexpr (FORM != ATTN_PARTS) {
        if (split > 1) return launch_bwd<DP, MODE, true, FORM>(p, maps, items, split, dq, st);
    }
    return launch_bwd<DP, MODE, false, FORM>(p, maps, items * (FORM == ATTN_PARTS ? p.kparts : 1), 1, dq, st);
}

inline lm_status encode_bwd(const AttnParams& p, BwdMaps* maps) {
    const lm_heads q{p.q.p, p.q.ts, p.q.hs}, k{p.k.p, p.k.ts, p.k.hs}, v{p.v.p, p.v.ts, p.v.hs}, dO{p.dO.p, p.dO.ts, p.dO.hs};
    lm_status s = encode_heads(&maps->q, q, p.T, p.hq, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps->k, k, p.Tk, p.hk, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps->v, v, p.Tk, p.hk, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps->dO, dO, p.T, p.hq, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps->dK, lm_heads{p.dK, (int64_t)p.hk * p.d, p.d}, p.Tk, p.hk, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps->dV, lm_heads{p.dV, (int64_t)p.hk * p.d, p.d}, p.Tk, p.hk, p.d, kTile);
    return s;
}

}  // namespace lm
