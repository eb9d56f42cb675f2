// Cross attention backward (include/lora_layer.h): attention's own kernels (lm_attn_bwd.cuh) with the ranges and the clearing
// of lm_cross.cu, and their sums in parts where one CTA would walk long.
#include <algorithm>

#include "lm_attn_bwd.cuh"

namespace lm {

// ------------------------------------------------------------------ parts of the backward
// Few key tiles (short states under long texts) are shared by more CTAs than a cluster has, and few query tiles under many
// keys are split along them; the parts' sums are joined in order.  Both where what one CTA walks would be long beside
// what an SM has in all: a step is a pair of tiles.  (A training step in
// a graph, with parts and without: 12000 queries on 78 states, 4 heads on 1 of 64, 46 and 278 us; 3700 on 651 in documents 58 and
// 87; 160 on 27000, 40 heads on 8, 627 and 689.  The joins take 6 us of the first.)
static int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }
constexpr int kLeastPairs = 4, kLeastTiles = 16;  // (an item begins and ends for five tiles' time)
BwdParts most_parts(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk) {
    const int64_t qt = tiles_of(Tq), kt = tiles_of(Tk), qitems = qt * hq;
    if (!qt || !kt) return BwdParts{1, 1};
    const int64_t k = std::min<int64_t>(kCrossSms / (kt * hk), hq / hk * qt / kLeastPairs);
    const int64_t q = std::min<int64_t>((2 * kCrossSms + qitems - 1) / qitems, kt / kLeastTiles);
    return BwdParts{(int32_t)std::max<int64_t>(k, 1), (int32_t)std::max<int64_t>(q, 1)};
}
BwdParts plan_parts(int64_t Tq, int64_t Tk, int32_t hq, int32_t hk, int32_t d, int32_t docs) {
    const int64_t qt = tiles_of(Tq), kt = tiles_of(Tk);
    if (!qt || !kt) return BwdParts{1, 1};
    // with documents a tile has partners in its own alone, about
    const int64_t pairs = hq / hk * ((qt + docs - 1) / docs), row = (kt + docs - 1) / docs;
    const int64_t sm = (kt * hk * pairs + qt * hq * row) / kCrossSms + 1;  // steps of an SM
    const int cluster = d <= 64 ? 2 : 4;
    const BwdParts most = most_parts(Tq, Tk, hq, hk);
    BwdParts P{1, 1};
    if (pairs > 2 * cluster * sm) P.k = (int32_t)std::min<int64_t>(most.k, std::min(pairs / kLeastPairs, (pairs + sm - 1) / sm));
    if (P.k <= cluster) P.k = 1;
    if (2 * row > sm) P.q = (int32_t)std::max<int64_t>(1, std::min<int64_t>(most.q, row / kLeastTiles));
    return P;
}

// The sums over `parts` of rows of d values, to bf16: a row takes WARPS of a CTA's eight warps, four values a lane.  Rows
// from rows0 on go to dst1.
constexpr int kSumAtOnce = 5;
template <int WARPS>
__global__ void __launch_bounds__(256) cross_sum_kernel(const float* src, int64_t rows, int d, int parts, uint16_t* dst0, uint16_t* dst1,
                                                        int64_t rows0) {
    __shared__ float4 sum[8][32];
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane * 4, mine = warp % WARPS;
    const int64_t row = (int64_t)blockIdx.x * (8 / WARPS) + warp / WARPS;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows && c < d) {
        const float* p = src + row * d + c;
#pragma unroll 1
        for (int s0 = mine; s0 < parts; s0 += WARPS * kSumAtOnce) {
            float4 v[kSumAtOnce];
#pragma unroll
            for (int i = 0; i < kSumAtOnce; ++i) {
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s0 + i * WARPS < parts) v[i] = *reinterpret_cast<const float4*>(p + (s0 + i * WARPS) * rows * d);
            }
#pragma unroll
            for (int i = 0; i < kSumAtOnce; ++i) o.x += v[i].x, o.y += v[i].y, o.z += v[i].z, o.w += v[i].w;
        }
    }
    if (WARPS > 1) {
        sum[warp][lane] = o;
        __syncthreads();
        if (mine) return;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
            const float4 v = sum[warp + w][lane];
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
        }
    }
    if (row < rows && c < d) {
        uint16_t* dst = row < rows0 ? dst0 + row * d : dst1 + (row - rows0) * d;
        *reinterpret_cast<uint2*>(dst + c) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    }
}
static cudaError_t launch_sum(const float* src, int64_t rows, int d, int parts, uint16_t* dst0, uint16_t* dst1, int64_t rows0,
                              cudaStream_t st) {
    LaunchTag tag("cross.sum", st);
    if (parts >= 8)
        return launch_pdl(cross_sum_kernel<8>, dim3((unsigned)rows), dim3(256), 0, st, nullptr, 0, src, rows, d, parts, dst0, dst1, rows0);
    return launch_pdl(cross_sum_kernel<1>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, nullptr, 0, src, rows, d, parts, dst0,
                      dst1, rows0);
}

// ------------------------------------------------------------------ launches
template <int DP, int FORM>
static cudaError_t bwd_modes(const AttnParams& p, const BwdMaps& maps, int sms, cudaStream_t st) {
    return p.cap > 0.f ? launch_both<DP, ATTN_CAP, FORM>(p, maps, sms, st) : launch_both<DP, ATTN_PLAIN, FORM>(p, maps, sms, st);
}
template <int DP>
static cudaError_t bwd_forms(const AttnParams& p, const BwdMaps& maps, int sms, cudaStream_t st) {
    return p.kparts > 1 || p.qparts > 1 ? bwd_modes<DP, ATTN_PARTS>(p, maps, sms, st) : bwd_modes<DP, ATTN_CROSS>(p, maps, sms, st);
}
lm_status launch_cross_bwd(const AttnParams& p, int sms, cudaStream_t st) {
    BwdMaps maps;
    const lm_status s = encode_bwd(p, &maps);
    if (s != LM_OK) return s;
    cudaError_t e = p.d <= 64 ? bwd_forms<64>(p, maps, sms, st) : bwd_forms<128>(p, maps, sms, st);
    const int64_t krows = (int64_t)p.Tk * p.hk, qrows = (int64_t)p.T * p.hq;
    if (e == cudaSuccess && p.kparts > 1) e = launch_sum(p.part_dkv, 2 * krows, p.d, p.kparts, p.dV, p.dK, krows, st);
    if (e == cudaSuccess && p.qparts > 1) e = launch_sum(p.part_dq, qrows, p.d, p.qparts, p.out, nullptr, qrows, st);
    return e == cudaSuccess ? LM_OK : report_error(LM_ERR_CUDA, "cross attention backward launch: %s", cudaGetErrorString(e));
}

}  // namespace lm
