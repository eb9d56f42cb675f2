// Attention forward (include/lora_layer.h) on the tensor cores.
//
// One CTA takes 256 queries of one head as two tiles of 128 and walks the 128-key tiles that any of
// them sees.  For each query tile w and key tile j:
//   S_w = Q_w K_j^T                              (tcgen05, both operands in shared memory)
//   P_w = 2^{S c - m}, l += row sums             (four warps, one thread per query row)
//   O_w += P_w V_j                               (tcgen05, P_w from tensor memory, where it replaces S_w)
// The two query tiles take turns: while the tensor cores work on one, the other's four warps form
// its exponentials, so neither waits for the other as long as 2 x 128 x d x 128 multiply-adds take
// longer than 128 x 128 exponentials with their loads, maxima, sums and packing.  The running
// maximum m follows the row only when it has grown by more than 8 (a factor 256 in the weights): the
// weights then stay below 2^8, exact in their scale, and O_w is rescaled a few times per row
// instead of once per key tile.  Sums are fp32.  P is rounded to bf16 for the second product; on tiles with
// hidden keys what the rounding left out is multiplied too (as a second left operand, in the other
// half of S_w's place): rows of few keys have no other weights to average their error with, and the
// backward takes differences against their O.  That is one more product on the tiles along the
// diagonal and at document ends; dQ of packed prefixes went from 2.51e-3 to 2.4e-3 of its norm off.
// Shared memory (d = 128): 64 KB of queries and a ring of five 32 KB key and value tiles; tensor
// memory: S_0, S_1, O_0, O_1 of 128 columns each.
#include "lm_attn.cuh"

namespace lm {

constexpr float kRescale = 8.f;

template <int DP>
struct FwdCfg {
    static constexpr uint32_t kTileBytes = (DP / 64) * kBoxBytes;
    static constexpr int kSlots = DP == 128 ? 5 : 8;
    static constexpr int kSmem = 2048 + (2 + kSlots) * kTileBytes;
};

struct FwdMaps {
    CUtensorMap q, k, v, o;
};

// the key tiles [j0, j1) that the query rows [q0, q0 + 128) may see
struct TileSpan {
    int j0, j1;
    int lo_max, hi_min;  // keys in [lo_max, hi_min) are seen by every row
    __device__ __forceinline__ bool hides(int j) const { return j * kTile < lo_max || (j + 1) * kTile > hi_min; }
};
__device__ __forceinline__ TileSpan key_tiles(const AttnParams& p, int q0) {
    if (q0 >= p.T) return TileSpan{0, 0, 0, 0};
    const TokRange a = tok_range(p, q0), b = tok_range(p, min(q0 + kTile, p.T) - 1);
    const int lo = uni(a.lo), hi = uni(b.hi);
    if (hi <= lo) return TileSpan{0, 0, 0, 0};
    return TileSpan{lo / kTile, (hi + kTile - 1) / kTile, uni(b.lo), uni(a.hi)};
}

template <int DP, int MODE>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_fwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ FwdMaps maps) {
    using C = FwdCfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + C::kSlots;
    uint64_t* qfull = empty + C::kSlots;
    uint64_t* sfull = qfull + 2;   // [2] scores ready
    uint64_t* pfull = sfull + 2;   // [2][2] weights of the first, of the last 64 keys written (and the scores read)
    uint64_t* hdone = pfull + 4;   // [2] the first half of a P V product done (once a tile)
    uint64_t* odone = hdone + 2;   // [2] the last product of the row tile done (once)
    uint64_t* drain = odone + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* s_bad = s_abort + 1;  // [2] a warp of the warpgroup gave up
    uint8_t* sq = smem + 1024;
    uint8_t* ring = sq + 2 * C::kTileBytes;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the longest rows first: under a causal mask the last queries see the most keys
    const int nqb = (p.T + 2 * kTile - 1) / (2 * kTile);
    const int h = (int)blockIdx.x % p.hq, q0 = (nqb - 1 - (int)blockIdx.x / p.hq) * 2 * kTile;
    const int g = h / (p.hq / p.hk);

    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_u32(&qfull[w]), 1);
            mbar_init(smem_u32(&sfull[w]), 1);
            mbar_init(smem_u32(&pfull[2 * w]), 4);
            mbar_init(smem_u32(&pfull[2 * w + 1]), 4);
            mbar_init(smem_u32(&hdone[w]), 1);
            mbar_init(smem_u32(&odone[w]), 1);
        }
        mbar_init(smem_u32(drain), 1);
        *s_abort = s_bad[0] = s_bad[1] = 0;
        fence_mbar_init();
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
        tma_prefetch_map(&maps.o);
    }
    __syncwarp();
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    const uint32_t tmem = (uint32_t)uni((int)*tmem_slot);
    const TileSpan span[2] = {key_tiles(p, q0), key_tiles(p, q0 + kTile)};
    int J0 = span[0].j0, J1 = span[0].j1;
    if (span[1].j1 > span[1].j0) {
        J0 = J1 > J0 ? min(J0, span[1].j0) : span[1].j0;
        J1 = max(J1, span[1].j1);
    }

    if (warp >= 8) {
        regs_down<kIssueRegs>();
        if (warp == 9) {  // ---------------- loader
            if (lane == 0 && J1 > J0) {
                bool ok = true;
                auto query = [&](int w) {
                    mbar_expect_tx(smem_u32(&qfull[w]), C::kTileBytes);
                    for (int b = 0; b < DP / 64; ++b)
                        tma_load_3d(smem_u32(sq + w * C::kTileBytes + b * kBoxBytes), &maps.q, smem_u32(&qfull[w]), b * 64, h,
                                    q0 + w * kTile);
                };
                query(0);  // then K: the first scores wait for these alone
                uint32_t n = 0;
                for (int j = J0; ok && j < J1; ++j)
                    for (int kv = 0; kv < 2; ++kv, ++n) {
                        const uint32_t s = n % C::kSlots, ph = (n / C::kSlots) & 1u;
                        if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1u, s_abort, p.wait_ns)) {
                            ok = false;
                            break;
                        }
                        mbar_expect_tx(smem_u32(&full[s]), C::kTileBytes);
                        for (int b = 0; b < DP / 64; ++b)
                            tma_load_3d(smem_u32(ring + s * C::kTileBytes + b * kBoxBytes), kv ? &maps.v : &maps.k,
                                        smem_u32(&full[s]), b * 64, g, j * kTile);
                        if (n == 0) query(1);
                    }
                if (!ok) {
                    attn_error(p, 5, 1);
                    *s_abort = 1;
                }
                // nothing may land in shared memory after the CTA has gone
                volatile int never = 0;
                bool in = mbar_wait(smem_u32(&qfull[0]), 0, &never, p.wait_ns);
                if (n > 0) in = mbar_wait(smem_u32(&qfull[1]), 0, &never, p.wait_ns) && in;
                if (!drain_fills(smem_u32(&full[0]), C::kSlots, n, p.wait_ns) || !in) attn_error(p, 5, 5);
            }
        } else if (warp == 8 && elect_one()) {  // ---------------- tensor cores
            const int ksteps = (p.d + 15) / 16;
            const uint32_t ids = make_idesc_bf16(kTile, kTile, false, false);
            const uint32_t ido = make_idesc_bf16(kTile, ksteps * 16, false, true);  // V is [key][dim]: MN-major
            int in0, in1;
            inside_tokens(p, in0, in1);
            bool ok = true;
            for (int j = J0; ok && j <= J1 && J1 > J0; ++j) {
                const uint32_t nk = 2 * (j - J0), nv = nk - 1;  // ring positions of K_j and V_{j-1}
                const uint32_t sk = smem_u32(ring + (nk % C::kSlots) * C::kTileBytes);
                const uint32_t sv = smem_u32(ring + (nv % C::kSlots) * C::kTileBytes);
                if (j > J0) {
                    ok = mbar_wait(smem_u32(&full[nv % C::kSlots]), (nv / C::kSlots) & 1u, s_abort, p.wait_ns);
                    if (!ok) break;
                    clear_padding(ring + (nv % C::kSlots) * C::kTileBytes, DP / 64, (j - 1) * kTile, in0, in1);
                }
                if (j < J1) {
                    ok = mbar_wait(smem_u32(&full[nk % C::kSlots]), (nk / C::kSlots) & 1u, s_abort, p.wait_ns);
                    if (!ok) break;
                }
                tc_fence_after();
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t ts = tmem + w * kTile, to = tmem + 2 * kTile + w * DP;
                    if (j > span[w].j0 && j <= span[w].j1) {  // O_w += P_w V_{j-1}
                        const uint32_t n = (uint32_t)(j - 1 - span[w].j0);
                        const bool hides = span[w].hides(j - 1);
#pragma unroll
                        for (int half = 0; half < 2 && ok; ++half) {
                            ok = mbar_wait(smem_u32(&pfull[2 * w + half]), n & 1u, s_abort, p.wait_ns);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t a = ts + half * 32;
                            const uint32_t b = desc_cols(sv) + half * 512;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_bf16_ts(to, a + kk * 8, desc(b + kk * 128), ido, (n || half || kk) ? 1u : 0u);
                            if (hides) {
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    umma_bf16_ts(to, a + 64 + kk * 8, desc(b + kk * 128), ido, 1u);
                            }
                            if (half == 0) umma_commit(smem_u32(&hdone[w]));
                            else if (j == span[w].j1) umma_commit(smem_u32(&odone[w]));
                        }
                        if (!ok) break;
                    }
                    if (j >= span[w].j0 && j < span[w].j1) {  // S_w = Q_w K_j^T
                        if (j == span[w].j0) {
                            ok = mbar_wait(smem_u32(&qfull[w]), 0, s_abort, p.wait_ns);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        mma_rows<DP>(ts, desc_rows(smem_u32(sq + w * C::kTileBytes)), desc_rows(sk), ksteps, ids);
                        umma_commit(smem_u32(&sfull[w]));
                    }
                }
                if (!ok) break;
                if (j > J0) umma_commit(smem_u32(&empty[nv % C::kSlots]));
                if (j < J1) umma_commit(smem_u32(&empty[nk % C::kSlots]));
            }
            if (!ok) {
                attn_error(p, 5, 2);
                *s_abort = 1;
            }
            umma_commit(smem_u32(drain));
            volatile int never = 0;
            mbar_wait(smem_u32(drain), 0, &never, p.wait_ns);
        }
    } else {  // ---------------- softmax: warpgroup w, one thread per query row
        regs_up<kMathRegs>();
        const int w = warp >> 2;
        const int i = q0 + w * kTile + (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + w * kTile, to = tmem + lanes + 2 * kTile + w * DP;
        TokRange r{0, 0, 0, 0};
        if (i < p.T) r = tok_range(p, i);
        const int j0 = span[w].j0, j1 = span[w].j1;
        const float slope = MODE != ATTN_PLAIN && p.slopes ? p.slopes[h] * kLog2e : 0.f;
        // scores in units of log 2: x = s c + bias (plain), or cap tanh(s scale / cap) log2 e + bias
        const float c = MODE == ATTN_CAP ? 2.f * kLog2e * p.scale / p.cap : p.scale * kLog2e;
        const float cap = p.cap * kLog2e;
        const float cx = MODE == ATTN_PLAIN ? c : 1.f;
        float m = -INFINITY, l = 0.f;  // running maximum, sum of weights
        bool ok = true;
        // 64 keys, one step of the running softmax; tiles with hidden keys have code of their own
        auto step = [&](int j, int half, float(&x)[64], auto hides) {
            constexpr bool HIDDEN = decltype(hides)::value;
            const int k0 = j * kTile + half * 64;
            if (MODE != ATTN_PLAIN) {
                const float dist = (float)(i - k0);
#pragma unroll
                for (int e = 0; e < 64; ++e) {
                    float v = x[e] * c;
                    if (MODE == ATTN_CAP) v = cap * tanh_from_2log2e(v);
                    x[e] = fmaf(-slope, fabsf(dist - (float)e), v);
                }
            }
            // on a tile with hidden keys most chunks of 32 keys are seen in full, or not at all, by all rows of
            // the warp: only the others are masked key by key, and chunks that nobody sees have no exponentials
            bool some[2] = {true, true};
            if (HIDDEN) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t bits = bits_between(r.lo - k0 - 32 * b, r.hi - k0 - 32 * b);
                    if (__all_sync(0xffffffffu, bits == ~0u)) continue;
                    some[b] = __any_sync(0xffffffffu, bits != 0u);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(bits >> e & 1u)) x[b * 32 + e] = -INFINITY;
                }
            }
            float mx[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                mx[b] = x[b * 16];
#pragma unroll
                for (int e = 1; e < 15; e += 2) mx[b] = fmaxf(fmaxf(mx[b], x[b * 16 + e]), x[b * 16 + e + 1]);
                mx[b] = fmaxf(mx[b], x[b * 16 + 15]);
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cx;
            const bool grow = top > m + kRescale || (m == -INFINITY && top > -INFINITY);
            if (__any_sync(0xffffffffu, grow)) {
                const float f = !grow ? 1.f : m == -INFINITY ? 0.f : ex2(m - top);
                if (j > j0 || half) {
                    // what was multiplied before this half is in O: earlier tiles since these scores are (products
                    // end in the order they are issued), and the tile's first half once it says so
                    if (half && !mbar_wait_warp(smem_u32(&hdone[w]), (uint32_t)(j - j0) & 1u, s_abort, p.wait_ns)) return false;
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < DP; cc += 16) {
                        uint32_t o[16];
                        tmem_ld_x16(to + cc, o);
                        tmem_ld_wait16(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st_x16(to + cc, o);
                    }
                    tmem_st_wait();
                }
                l *= f;
                if (grow) m = top;
            }
            const float2 c2 = two(cx), mu = two(m == -INFINITY ? 0.f : -m);
            float2 s2[2] = {two(0.f), two(0.f)};
            uint32_t pk[32], rest[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (HIDDEN && !some[b]) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[b * 16 + e] = rest[b * 16 + e] = 0u;
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 y = __ffma2_rn(make_float2(x[b * 32 + e], x[b * 32 + e + 1]), c2, mu);
                    const float2 q = make_float2(ex2(y.x), ex2(y.y));
                    s2[(e >> 1) & 1] = __fadd2_rn(s2[(e >> 1) & 1], q);
                    const uint32_t hi = pack_bf16x2(q.x, q.y);
                    pk[b * 16 + (e >> 1)] = hi;
                    if (HIDDEN) rest[b * 16 + (e >> 1)] = pack_bf16x2(q.x - bf16lo(hi), q.y - bf16hi(hi));
                }
            }
            tmem_st_x32(ts + half * 32, pk);
            if (HIDDEN) tmem_st_x32(ts + 64 + half * 32, rest);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&pfull[2 * w + half]));
            const float2 s = __fadd2_rn(s2[0], s2[1]);
            l += s.x + s.y;
            return true;
        };
        for (int j = j0; ok && j < j1; ++j) {
            ok = mbar_wait_warp(smem_u32(&sfull[w]), (uint32_t)(j - j0) & 1u, s_abort, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const bool hides = span[w].hides(j);
            float x0[64], x1[64];
            tmem_ld_f32<0>(ts, x0);
            tmem_ld_f32<32>(ts + 32, x0);
            tmem_ld_wait_f32<0>(x0);
            tmem_ld_wait_f32<32>(x0);
            tmem_ld_f32<0>(ts + 64, x1);  // on its way during the first half's arithmetic
            tmem_ld_f32<32>(ts + 96, x1);
            if (hides) {  // (the first half writes into the second's columns)
                tmem_ld_wait_f32<0>(x1);
                tmem_ld_wait_f32<32>(x1);
                ok = step(j, 0, x0, std::true_type{}) && step(j, 1, x1, std::true_type{});
            } else {
                ok = step(j, 0, x0, std::false_type{});
                tmem_ld_wait_f32<0>(x1);
                tmem_ld_wait_f32<32>(x1);
                ok = ok && step(j, 1, x1, std::false_type{});
            }
        }
        if (ok && j1 > j0) ok = mbar_wait_warp(smem_u32(&odone[w]), 0, s_abort, p.wait_ns);
        tc_fence_after();
        if (!ok && lane == 0) {
            attn_error(p, 5, 3);
            *s_abort = 1;
        }
        if (!group_ok(ok, s_bad + w, 1 + w)) {
            // (nothing is written)
        } else {
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const int row = (warp & 3) * 32 + lane;
            uint8_t* stage = sq + w * C::kTileBytes;  // (the queries have been read)
            int8_t* lo = p.out_lo ? p.out_lo + ((int64_t)i * p.hq + h) * p.d16 : nullptr;
#pragma unroll 1
            for (int cc = 0; cc < DP; cc += 16) {
                uint32_t o[16];
                if (j1 > j0) {  // (uniform over the warpgroup)
                    tmem_ld_x16(to + cc, o);
                    tmem_ld_wait16(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0;
                }
                uint32_t v[8];
                int more[4];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = inv > 0.f ? __uint_as_float(o[2 * e]) * inv : 0.f;
                    const float b = inv > 0.f ? __uint_as_float(o[2 * e + 1]) * inv : 0.f;
                    v[e] = pack_bf16x2(a, b);
                    const int two = (bits_left(a, v[e] & 0xFFFFu) & 255) | (bits_left(b, v[e] >> 16) & 255) << 8;
                    if (e & 1) more[e >> 1] |= two << 16;
                    else more[e >> 1] = two;
                }
                stage_pairs(stage + (cc / 64) * kBoxBytes, row, (cc & 63) / 16, v);
                if (lo && i < p.T && cc < p.d)
                    *reinterpret_cast<int4*>(lo + cc) = make_int4(more[0], more[1], more[2], more[3]);
            }
            if (q0 + w * kTile < p.T)  // (uniform over the warpgroup)
                for (int b = 0; b < DP / 64; ++b)
                    store_box(&maps.o, stage + b * kBoxBytes, b * 64, h, q0 + w * kTile, 1 + w, row == 0);
            if (i < p.T) p.lse[(int64_t)h * p.T + i] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 8) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DP, int MODE>
cudaError_t launch_fwd(const AttnParams& p, const FwdMaps& maps, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(attn_fwd_kernel<DP, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               FwdCfg<DP>::kSmem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((p.T + 2 * kTile - 1) / (2 * kTile)) * (unsigned)p.hq;
    return launch_pdl(attn_fwd_kernel<DP, MODE>, dim3(grid), dim3(kAttnThreads), FwdCfg<DP>::kSmem, st, nullptr, 0, p, maps);
}

lm_status launch_attn_fwd(const AttnParams& p, cudaStream_t st) {
    FwdMaps maps;
    const lm_heads q{p.q.p, p.q.ts, p.q.hs}, k{p.k.p, p.k.ts, p.k.hs}, v{p.v.p, p.v.ts, p.v.hs};
    lm_status s = encode_heads(&maps.q, q, p.T, p.hq, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps.k, k, p.T, p.hk, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps.v, v, p.T, p.hk, p.d, kTile);
    if (s == LM_OK) s = encode_heads(&maps.o, lm_heads{p.out, (int64_t)p.hq * p.d, p.d}, p.T, p.hq, p.d, kTile);
    if (s != LM_OK) return s;
    // the plain form folds the scale into the exponent and needs it positive (the maximum of s c is c max s)
    const int mode = p.cap > 0.f ? ATTN_CAP : p.slopes || !(p.scale > 0.f) ? ATTN_BIAS : ATTN_PLAIN;
    cudaError_t e;
    if (p.d <= 64)
        e = mode == ATTN_CAP    ? launch_fwd<64, ATTN_CAP>(p, maps, st)
            : mode == ATTN_BIAS ? launch_fwd<64, ATTN_BIAS>(p, maps, st)
                                : launch_fwd<64, ATTN_PLAIN>(p, maps, st);
    else
        e = mode == ATTN_CAP    ? launch_fwd<128, ATTN_CAP>(p, maps, st)
            : mode == ATTN_BIAS ? launch_fwd<128, ATTN_BIAS>(p, maps, st)
                                : launch_fwd<128, ATTN_PLAIN>(p, maps, st);
    return e == cudaSuccess ? LM_OK : report_error(LM_ERR_CUDA, "attn forward launch: %s", cudaGetErrorString(e));
}

}  // namespace lm
