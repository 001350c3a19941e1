// Expert products of few rows, for gfx950: the weights are the traffic.
//
//   out[r,n] = act(sum_c x[r,c] W[e,n,c] + b[e,n]) + residual[r,n]
//
// One workgroup takes up to 16 rows of an expert and 16 outputs (32 weight
// rows when gated), its waves the blocks of k in turn; the sums are joined in
// LDS in a fixed order.  The tiled product's grid of 64 or 128 outputs a
// workgroup leaves most of the chip idle on one small product, and its waves
// wait at each step for one another: 16 x 4096 x 8192 takes 19.7 us here (3.4
// TB/s), 31.0 there.
#include "few_device.h"

namespace epget {
namespace {

template <int ACT, bool FP8>
__global__ __launch_bounds__(kFewThreads) void product_few_kernel(ProductArgs a) {
    constexpr bool GATED = act_gated(ACT);
    constexpr int FF = GATED ? 2 : 1;
    __shared__ int first[EP_MAX_EXPERTS + 1];
    __shared__ int wave_sum[kFewWaves];
    __shared__ f32x4 part[kFewWaves][FF][64];
    if (a.seg.E > 1) {
        tile_prefix<kFewThreads>(a.seg, 16, first, wave_sum);
    } else if (threadIdx.x < 2) {  // no sums over experts: a decode-sized product is mostly latency
        int64_t row0;
        first[threadIdx.x] = threadIdx.x ? (segment(a.seg, 0, &row0) + 15) / 16 : 0;
    }
    __syncthreads();
    const int lane = __lane_id(), li = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nf = (a.N + 15) / 16;
    const int64_t total = static_cast<int64_t>(first[a.seg.E]) * nf;
    const int64_t pitch = static_cast<int64_t>(a.C) * (FP8 ? 1 : 2);
    const int G = gridDim.x;
    for (int64_t round = 0; round * G < total; ++round) {
        const int64_t tile = tile_of(total, round, blockIdx.x, G);
        if (tile < 0) break;
        const int e = tile_expert(first, a.seg.E, static_cast<int>(tile / nf));
        const int f0 = __builtin_amdgcn_readfirstlane(first[e]);
        const int nt = __builtin_amdgcn_readfirstlane(first[e + 1]) - f0;
        int tt, ft;
        tile_in_expert(tile - static_cast<int64_t>(f0) * nf, nt, nf, &tt, &ft);
        int64_t row0;
        const int rows = segment(a.seg, e, &row0);
        const int n0 = ft * 16, t0 = tt * 16;
        const char *row[FF];
        const float *w_sf[FF];
        f32x4 acc[FF][1];
#pragma unroll
        for (int f = 0; f < FF; ++f) {
            const int64_t r = static_cast<int64_t>(e) * a.M + f * a.N + min(n0 + li, a.N - 1);
            row[f] = static_cast<const char *>(a.weight) + r * pitch;
            w_sf[f] = FP8 ? static_cast<const float *>(a.w_sf) +
                                (static_cast<int64_t>(e) * (a.M / 128) + (f * a.N + n0) / 128) * (a.C / 128)
                          : nullptr;
            acc[f][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const int64_t xr = row0 + min(t0 + li, rows - 1);
        const char *const col[1] = {static_cast<const char *>(a.x) + xr * pitch};
        const float *const x_sf[1] = {FP8 ? a.x_sf + xr * a.sf_ts : nullptr};
        // neighbouring tiles start at different blocks of k, so that they do
        // not all read the same piece of x at once (1.5 us of 14)
        accumulate_blocks<FP8, FP8>(acc, row, col, w_sf, x_sf, a.sf_hs, a.C, (wave + ft) % kFewWaves, kFewWaves, lg);
        const int tok = t0 + li, n = n0 + lg * 4;
#pragma unroll
        for (int f = 0; f < FF; ++f) part[wave][f][lane] = acc[f][0];
        __syncthreads();
        if (wave == 0 && tok < rows && n < a.N) {
            f32x4 v[1] = {sum_waves(&part[0][0][lane], FF * 64)};
            f32x4 u[1] = {GATED ? sum_waves(&part[0][FF - 1][lane], FF * 64) : v[0]};
            write_outputs<ACT>(a, e, row0 + tok, n, v, u);
        }
        __syncthreads();
    }
}

template <int ACT, bool FP8>
hipError_t launch_few(const ProductArgs &a, hipStream_t stream) {
    // no more workgroups than tiles there can be, each expert's last tile in part filled
    const int64_t tiles = (a.entries / 16 + min(static_cast<int64_t>(a.seg.E), a.entries)) * ((a.N + 15) / 16);
    const uint32_t grid = static_cast<uint32_t>(min(int64_t{512}, (tiles + 7) / 8 * 8));
    product_few_kernel<ACT, FP8><<<grid, kFewThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_product_few(const ProductArgs &a, bool fp8, hipStream_t stream) {
    switch (a.act) {
#define EP_ACT_CASE(A) \
    case A: return fp8 ? launch_few<A, true>(a, stream) : launch_few<A, false>(a, stream);
        EP_ACT_CASE(EP_ACT_NONE)
        EP_ACT_CASE(EP_ACT_RELU)
        EP_ACT_CASE(EP_ACT_GELU)
        EP_ACT_CASE(EP_ACT_SILU)
        EP_ACT_CASE(EP_ACT_SWIGLU)
        EP_ACT_CASE(EP_ACT_GEGLU)
#undef EP_ACT_CASE
        default: return hipErrorInvalidValue;
    }
}

}  // namespace epget
