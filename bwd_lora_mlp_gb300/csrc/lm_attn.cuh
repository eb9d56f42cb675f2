// What the attention kernels share: parameters, who sees whom, tensor-memory and TMA forms that the
// projection kernels do not use, and the score arithmetic.
#pragma once

#include <type_traits>

#include "lm_gemm.cuh"
#include "lm_layer.h"
#include "lm_ptx.cuh"

namespace lm {

constexpr int kTile = 128;             // queries and keys of a score tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// How scores are formed from q.k: bit 0 slopes, bit 1 the cap.  Without slopes the factor of the scores is
// part of the exponent's multiply-add.
enum AttnMode : int { ATTN_PLAIN = 0, ATTN_BIAS = 1, ATTN_CAP = 2, ATTN_CAP_BIAS = 3 };
constexpr bool biased(int mode) { return mode & 1; }
constexpr bool capped(int mode) { return mode & 2; }

// ---------------------------------------------------------------- who sees whom
__host__ __device__ inline TokRange range_in(int t, int s, int e, int pre, int T, int causal, int window) {
    const int W = window > 0 && window < T ? window : T;  // (T <= 2^20: no sum overflows)
    TokRange r;
    r.lo = s > t - W + 1 ? s : t - W + 1;
    r.hi = e;
    if (causal) r.hi = t + 1 > s + pre ? t + 1 : s + pre;
    if (r.hi > t + W) r.hi = t + W;
    r.qlo = causal && t >= s + pre ? t : r.lo;
    r.qhi = e < t + W ? e : t + W;
    return r;
}
__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }
__device__ __forceinline__ TokRange range_of(const lm_attn& a, int t, int T) {
    // the document: the largest m with cu[m] <= t (empty documents before it are skipped)
    int m = 0, over = a.n_docs;
    while (m + 1 < over) {
        const int mid = (m + over) >> 1;
        if (a.cu_docs[mid] <= t) m = mid;
        else over = mid;
    }
    const int s = clampi(a.cu_docs[m], 0, T), e = clampi(a.cu_docs[m + 1], 0, T);
    // padding: empty intervals at t, which keeps all four non-decreasing over the tokens
    if (t < s || t >= e) return TokRange{t, t, t, t};
    return range_in(t, s, e, a.prefix ? clampi(a.prefix[m], 0, e - s) : 0, T, a.causal, a.window);
}
// of token t < T: from the table, or (one document) from the masks themselves.  (Not by a read-only load: the
// kernel may have begun before the one that writes the table ended.)
__device__ __forceinline__ TokRange tok_range(const AttnParams& p, int t) {
    if (p.rng) {
        const int4 v = *(reinterpret_cast<const int4*>(p.rng) + t);
        return TokRange{v.x, v.y, v.z, v.w};
    }
    return range_in(t, 0, p.T, 0, p.T, p.causal, p.window);
}

// ---------------------------------------------------------------- errors
__device__ __forceinline__ void attn_error(const AttnParams& p, int family, int where) {
    if (p.err) {
        atomicExch(p.err, kErrTimeout);
        p.err[1] = where;
        p.err[2] = blockIdx.x;
        p.err[3] = family;
    }
}

// ---------------------------------------------------------------- TMA, TMEM
// The box of 64 dims x 1 head x rows tokens at (dim x, head y, token z).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}
// Four floats to another CTA's shared memory (an address of map_to_rank).
__device__ __forceinline__ void st_peer4(uint32_t addr, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T: A is 128 rows (lanes) x 16 K values packed two to a column.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// True in one lane of the warp.  The issuing role runs inside a branch on it: the compiler then knows
// that one thread is active and takes descriptors to the uniform registers directly.  Eight products
// of 64 cycles each are issued in 175 cycles this way, in 390 under `lane == 0` and in 470 to 620 with
// the whole warp running the loop and a predicate on each (measured alone; the second and third were
// slower than the tensor cores together with the role's waits, and bound every kernel here).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
// 32 columns of this thread's row into x[AT .. AT + 31].
template <int AT, int N>
__device__ __forceinline__ void tmem_ld_f32(uint32_t taddr, float (&x)[N]) {
    static_assert(AT + 32 <= N, "");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(x[AT + 0]), "=f"(x[AT + 1]), "=f"(x[AT + 2]), "=f"(x[AT + 3]), "=f"(x[AT + 4]), "=f"(x[AT + 5]), "=f"(x[AT + 6]), "=f"(x[AT + 7]),
          "=f"(x[AT + 8]), "=f"(x[AT + 9]), "=f"(x[AT + 10]), "=f"(x[AT + 11]), "=f"(x[AT + 12]), "=f"(x[AT + 13]), "=f"(x[AT + 14]), "=f"(x[AT + 15]),
          "=f"(x[AT + 16]), "=f"(x[AT + 17]), "=f"(x[AT + 18]), "=f"(x[AT + 19]), "=f"(x[AT + 20]), "=f"(x[AT + 21]), "=f"(x[AT + 22]), "=f"(x[AT + 23]),
          "=f"(x[AT + 24]), "=f"(x[AT + 25]), "=f"(x[AT + 26]), "=f"(x[AT + 27]), "=f"(x[AT + 28]), "=f"(x[AT + 29]), "=f"(x[AT + 30]), "=f"(x[AT + 31])
        : "r"(taddr));
}
// Waits for this thread's loads; carries the values so that no use of them moves before it.
template <int AT, int N>
__device__ __forceinline__ void tmem_ld_wait_f32(float (&x)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[AT + 0]), "+f"(x[AT + 1]), "+f"(x[AT + 2]), "+f"(x[AT + 3]), "+f"(x[AT + 4]), "+f"(x[AT + 5]), "+f"(x[AT + 6]), "+f"(x[AT + 7]),
                   "+f"(x[AT + 8]), "+f"(x[AT + 9]), "+f"(x[AT + 10]), "+f"(x[AT + 11]), "+f"(x[AT + 12]), "+f"(x[AT + 13]), "+f"(x[AT + 14]), "+f"(x[AT + 15]),
                   "+f"(x[AT + 16]), "+f"(x[AT + 17]), "+f"(x[AT + 18]), "+f"(x[AT + 19]), "+f"(x[AT + 20]), "+f"(x[AT + 21]), "+f"(x[AT + 22]), "+f"(x[AT + 23]),
                   "+f"(x[AT + 24]), "+f"(x[AT + 25]), "+f"(x[AT + 26]), "+f"(x[AT + 27]), "+f"(x[AT + 28]), "+f"(x[AT + 29]), "+f"(x[AT + 30]), "+f"(x[AT + 31])
                 :
                 : "memory");
}
template <int AT, int N>
__device__ __forceinline__ void tmem_ld_wait16_f32(float (&x)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[AT + 0]), "+f"(x[AT + 1]), "+f"(x[AT + 2]), "+f"(x[AT + 3]), "+f"(x[AT + 4]), "+f"(x[AT + 5]), "+f"(x[AT + 6]), "+f"(x[AT + 7]),
                   "+f"(x[AT + 8]), "+f"(x[AT + 9]), "+f"(x[AT + 10]), "+f"(x[AT + 11]), "+f"(x[AT + 12]), "+f"(x[AT + 13]), "+f"(x[AT + 14]), "+f"(x[AT + 15])
                 :
                 : "memory");
}
// The same with a row's columns over four lanes: 16 rows of the warp's quarter (taddr names the first,
// 0 or 16 of the 32), 8 columns a group of four values: lane T holds row T / 4, columns 2 (T % 4) and
// one more, then the same of row T / 4 + 8.  A row's maximum then takes two shuffles, and two warps share
// a quarter's rows instead of its columns.
template <int AT, int N>
__device__ __forceinline__ void tmem_ld_frag32(uint32_t taddr, float (&x)[N]) {
    static_assert(AT + 32 <= N, "");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(x[AT + 0]), "=f"(x[AT + 1]), "=f"(x[AT + 2]), "=f"(x[AT + 3]), "=f"(x[AT + 4]), "=f"(x[AT + 5]), "=f"(x[AT + 6]), "=f"(x[AT + 7]),
          "=f"(x[AT + 8]), "=f"(x[AT + 9]), "=f"(x[AT + 10]), "=f"(x[AT + 11]), "=f"(x[AT + 12]), "=f"(x[AT + 13]), "=f"(x[AT + 14]), "=f"(x[AT + 15]),
          "=f"(x[AT + 16]), "=f"(x[AT + 17]), "=f"(x[AT + 18]), "=f"(x[AT + 19]), "=f"(x[AT + 20]), "=f"(x[AT + 21]), "=f"(x[AT + 22]), "=f"(x[AT + 23]),
          "=f"(x[AT + 24]), "=f"(x[AT + 25]), "=f"(x[AT + 26]), "=f"(x[AT + 27]), "=f"(x[AT + 28]), "=f"(x[AT + 29]), "=f"(x[AT + 30]), "=f"(x[AT + 31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_frag16(uint32_t taddr, const float (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]),
        "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
        : "memory");
}
template <int AT, int N>
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, float (&x)[N]) {
    static_assert(AT + 16 <= N, "");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(x[AT + 0]), "=f"(x[AT + 1]), "=f"(x[AT + 2]), "=f"(x[AT + 3]), "=f"(x[AT + 4]), "=f"(x[AT + 5]), "=f"(x[AT + 6]), "=f"(x[AT + 7]),
          "=f"(x[AT + 8]), "=f"(x[AT + 9]), "=f"(x[AT + 10]), "=f"(x[AT + 11]), "=f"(x[AT + 12]), "=f"(x[AT + 13]), "=f"(x[AT + 14]), "=f"(x[AT + 15])
        : "r"(taddr));
}
// Packed pairs (bf16) of such groups: lane T holds the pair 2 (T % 4) of row T / 4, then of row T / 4 + 8.
__device__ __forceinline__ void tmem_st_pairs16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- products of one tile
// Shared-memory tile of 128 rows x dp dims: dp / 64 boxes of 128 rows x 128 bytes, 128-byte swizzle.
constexpr uint32_t kBoxBytes = kTile * 128;

// A value that is the same in the whole warp, made so in the compiler's eyes too.
__device__ __forceinline__ int uni(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Low descriptor word of a tile: start address and leading offset in units of 16 bytes; the high word
// holds the stride of 8-row groups (1024 bytes), the version and the 128-byte swizzle.  (In a cluster an
// address says which CTA's it is above the bits of its place.)
__device__ __forceinline__ uint32_t desc_at(uint32_t addr) { return (addr >> 4) & 0x3FFFu; }
__device__ __forceinline__ uint32_t desc_rows(uint32_t addr) { return desc_at(addr) | (1u << 16); }                // K-major
__device__ __forceinline__ uint32_t desc_cols(uint32_t addr) { return desc_at(addr) | ((kBoxBytes >> 4) << 16); }  // MN-major
__device__ __forceinline__ uint64_t desc(uint32_t lo) {
    constexpr uint64_t hi = (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32;
    return hi | lo;
}
// D = A B^T over the tiles' dims (both K-major), `steps` of at most DP / 16 K steps
template <int DP>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, int steps, uint32_t idesc) {
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
        const uint32_t off = (uint32_t)(kk >> 2) * (kBoxBytes >> 4) + (uint32_t)(kk & 3) * 2;
        if (kk < steps) umma_bf16(d, desc(a + off), desc(b + off), idesc, kk ? 1u : 0u);
    }
}

// rows of padding tokens hold anything: they are cleared where they would be a right operand (0 x NaN).
// The issuing thread does it by itself, about 2 us for a whole tile, every time that the tile is loaded; only
// tiles with tokens before the first document or after the last one have such rows.
__device__ __forceinline__ void clear_padding(uint8_t* tile, int boxes, int t0, int in0, int in1) {
    if (t0 >= in0 && t0 + kTile <= in1) return;
    for (int r = 0; r < kTile; ++r)
        if (t0 + r < in0 || t0 + r >= in1)
            for (int b = 0; b < boxes; ++b)
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4*>(tile + b * kBoxBytes + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
}
// Rows past the last token come as zeros, so the tokens that need no clearing end with the last tile.  (4097 causal
// tokens, 32 heads on 8 of 128 dims, a step: 502 us; 607 with those rows cleared too.)
__device__ __forceinline__ void inside_tokens(const AttnParams& p, int& in0, int& in1) {
    in0 = 0;
    in1 = p.Tp;
    if (p.cu_docs) {
        in0 = max(0, p.cu_docs[0]);
        if (p.cu_docs[p.n_docs] < p.T) in1 = p.cu_docs[p.n_docs];
    }
}

// ---------------------------------------------------------------- arithmetic
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Capped scores: tanh x = 1 + 2 n with n = -1 / (1 + e^{2x}), exact at both ends, and 1 - tanh^2 x =
// -4 (n + n^2).  The kernels work with n: the factors 2 cap and -4 go into multiplications that are there
// anyway, and the constant cap into lse.  Given 2 log2(e) x; n's absolute error is a few 2^-25.
__device__ __forceinline__ float2 cap_n(float2 x) {
    const float2 a = __ffma2_rn(make_float2(ex2(x.x), ex2(x.y)), make_float2(-1.f, -1.f), make_float2(-1.f, -1.f));
    return make_float2(rcp(a.x), rcp(a.y));
}
// Bit e set: column e of a chunk of 32 is in [a, z).
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t bits_between(int a, int z) { return bits_below(z) & ~bits_below(a); }
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }

// Register budgets of a CTA's warpgroups: what the loader's and the MMA warp's do not need goes to the
// arithmetic ones.
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
// Whether every warp of the warpgroup (barrier `id`) came through: a warp that gave up a wait sets the
// group's flag, and either all of the group go on to the epilogue's barriers or none does.
__device__ __forceinline__ bool group_ok(bool ok, volatile int* bad, int id) {
    if (!ok) *bad = 1;
    group_sync(id);
    return *bad == 0;
}
// Eight packed pairs (16 dims, the c-th of a box's four) of row r to a staged box: 128-byte swizzle.
__device__ __forceinline__ void stage_pairs(uint8_t* box, int r, int c, const uint32_t (&v)[8]) {
    uint8_t* row = box + r * 128;
    *reinterpret_cast<uint4*>(row + (((2 * c) ^ (r & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ (r & 7)) << 4)) = make_uint4(v[4], v[5], v[6], v[7]);
}
// The staged box of 128 tokens x 64 dims to (dim x, head y, token z): all 128 threads of the warpgroup
// come here after their writes, barrier `id` is theirs; rows past the tensor's end are not written.
// Rows leave as 128-byte lines (a thread storing its own row would touch a line per lane and chunk: the
// forward's epilogue took 5000 cycles of a CTA that way).
__device__ __forceinline__ void store_box(const CUtensorMap* map, const uint8_t* box, int x, int y, int z, int id, bool first) {
    fence_proxy_async_smem();
    group_sync(id);
    if (first) {
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(map)),
                     "r"(smem_u32(box)), "r"(x), "r"(y), "r"(z)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
    }
}
// N (a multiple of 16) dims from dim c0 on of this thread's accumulator row (at t), times f, to bf16 at
// dst.  `any` false: the accumulator was never written and the row is zero (uniform over the warp).
template <int N>
__device__ __forceinline__ void store_dims(uint16_t* dst, uint32_t t, int c0, int d, float f, bool any, bool mine) {
#pragma unroll
    for (int c = 0; c < N; c += 16) {
        uint32_t o[16], v[8];
        if (any) {
            tmem_ld_x16(t + c0 + c, o);
            tmem_ld_wait16(o);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = any ? pack_bf16x2(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f) : 0u;
        if (!mine || c0 + c >= d) continue;
        uint16_t* q = dst + c0 + c;
        if ((d & 15) == 0) {
            st_global_v8(q, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
        } else {  // (d = 8 modulo 16: rows lie on 16 bytes, and the last chunk is half there)
            *reinterpret_cast<uint4*>(q) = make_uint4(v[0], v[1], v[2], v[3]);
            if (c0 + c + 8 < d) *reinterpret_cast<uint4*>(q + 8) = make_uint4(v[4], v[5], v[6], v[7]);
        }
    }
}
// 64 dims of this thread's accumulator row (lane r of the warpgroup's 128), times f, to a staged box as
// bf16.  `any` false: the accumulator was never written and the row is zero (uniform over the warp).
__device__ __forceinline__ void stage_row(uint8_t* box, int r, uint32_t t, float f, bool any) {
    float x[64];
    if (any) {
        tmem_ld_f32<0>(t, x);
        tmem_ld_f32<32>(t + 32, x);
        tmem_ld_wait_f32<0>(x);
        tmem_ld_wait_f32<32>(x);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = any ? pack_bf16x2(x[c * 16 + 2 * e] * f, x[c * 16 + 2 * e + 1] * f) : 0u;
        stage_pairs(box, r, c, v);
    }
}

// The next eight bits of a value's fp32 pattern after its bf16 rounding, to the nearest (held to 127).
__device__ __forceinline__ int bits_left(float x, uint32_t bf16_bits) {
    return min(((int32_t)(__float_as_uint(x) - (bf16_bits << 16)) + 128) >> 8, 127);
}

}  // namespace lm
