// Products of a few tokens with a weight that is read once: the weight's
// rows go from memory straight to the matrix instruction's registers (its 16
// rows are weight rows, its 16 columns tokens), with no stop in LDS, and k is
// split over the waves of a workgroup in blocks of 128.  Shared by the
// few-token layer and the expert products of few rows.
#pragma once

#include <type_traits>

#include "product_device.h"

namespace epget {
namespace {

constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / 64;
constexpr int kBlockK = 128;  // k per block: one scale of an FP8 weight

// A block of one fragment of 16 weight rows, as it comes from memory: bf16 in
// four pieces of 8 k a lane (k = 32 q + 8 g), e4m3 in two of 16 (k = 64 q + 16 g).
// The weight is read once: its loads carry the non-temporal hint.
template <bool FP8>
struct WeightBlock {
    static constexpr int kPieces = FP8 ? 2 : 4;
    u32x4 v[kPieces];

    // row: this lane's row; b: the block; K: end of k, with zeros past it in a block that is not FULL
    template <bool FULL>
    __device__ __forceinline__ void load(const char *row, int b, int K, int lg) {
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int k = b * kBlockK + (FP8 ? 64 * q + 16 * lg : 32 * q + 8 * lg);
            const u32x4 *p = reinterpret_cast<const u32x4 *>(row + static_cast<int64_t>(k) * (FP8 ? 1 : 2));
            v[q] = FULL || k < K ? __builtin_nontemporal_load(p) : u32x4{0, 0, 0, 0};
        }
    }

    // bf16 operand of matrix instruction s (0..3) of the block; e4m3 codes are widened, which is exact.
    __device__ __forceinline__ bf16x8 operand(int s) const {
        if constexpr (!FP8) {
            return __builtin_bit_cast(bf16x8, v[s]);
        } else {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            bf16x8 o;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t c = v[s >> 1][(s & 1) * 2 + w];
                const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false);
                const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true);
                o[4 * w] = lo[0], o[4 * w + 1] = lo[1], o[4 * w + 2] = hi[0], o[4 * w + 3] = hi[1];
            }
            return o;
        }
    }
};

// The same block of 16 columns (tokens): column li, the k that the weight's
// lanes hold.  WFP8, XFP8: element types of the weight and of the column.
template <bool WFP8, bool XFP8>
struct ColumnBlock {
    static constexpr int kPieces = XFP8 ? 2 : 4;
    u32x4 v[kPieces];

    template <bool FULL>
    __device__ __forceinline__ void load(const char *col, int b, int K, int lg) {
#pragma unroll
        for (int s = 0; s < kPieces; ++s) {
            const int k = b * kBlockK + (XFP8 ? 64 * s + 16 * lg : WFP8 ? 64 * (s >> 1) + 16 * lg + 8 * (s & 1) : 32 * s + 8 * lg);
            const u32x4 *p = reinterpret_cast<const u32x4 *>(col + static_cast<int64_t>(k) * (XFP8 ? 1 : 2));
            v[s] = FULL || k < K ? *p : u32x4{0, 0, 0, 0};
        }
    }
};

// acc += the block's product, times scale where the weight is FP8.
template <bool WFP8, bool XFP8>
__device__ __forceinline__ void add_block(f32x4 &acc, const WeightBlock<WFP8> &w, const ColumnBlock<WFP8, XFP8> &x,
                                          float scale) {
    f32x4 d = WFP8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc;
    if constexpr (XFP8) {
        union Frag {
            u32x4 part[2];
            i32x8 all;
        } a, b;
#pragma unroll
        for (int q = 0; q < 2; ++q) a.part[q] = w.v[q], b.part[q] = x.v[q];
        // block scales of one (127 is 2^0): the fp32 scale follows in fp32
        d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.all, b.all, d, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
    } else {
#pragma unroll
        for (int s = 0; s < 4; ++s)
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.operand(s), __builtin_bit_cast(bf16x8, x.v[s]), d, 0, 0, 0);
    }
    if constexpr (WFP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(d[i], scale, acc[i]);
    } else {
        acc = d;
    }
}

// Loads blocks first, first + step, .. below n and adds each, one block's
// loads in flight while the one before is added.  T holds a block.
template <class T, class Load, class Add>
__device__ __forceinline__ void pipelined(int first, int step, int n, Load load, Add add) {
    int b = first;
    if (b >= n) return;
    T even, odd;
    load(even, b);
    for (;;) {
        if ((b += step) >= n) return add(even, b - step);
        load(odd, b);
        add(even, b - step);
        if ((b += step) >= n) return add(odd, b - step);
        load(even, b);
        add(odd, b - step);
    }
}

// acc[f][t] += W rows x columns over the blocks of k first, first + step, ..
template <bool WFP8, bool XFP8, int FF, int TF>
__device__ __forceinline__ void accumulate_blocks(f32x4 (&acc)[FF][TF], const char *const (&row)[FF],
                                                  const char *const (&col)[TF], const float *const (&w_sf)[FF],
                                                  const float *const (&x_sf)[TF], int64_t x_sf_step, int K, int first,
                                                  int step, int lg) {
    struct Block {
        WeightBlock<WFP8> w[FF];
        ColumnBlock<WFP8, XFP8> x[TF];
        float sw[FF], sx[TF];
    };
    auto load = [&](auto full, Block &o, int b) {
#pragma unroll
        for (int f = 0; f < FF; ++f) {
            o.w[f].template load<full()>(row[f], b, K, lg);
            if (WFP8) o.sw[f] = w_sf[f][b];
        }
#pragma unroll
        for (int t = 0; t < TF; ++t) {
            o.x[t].template load<full()>(col[t], b, K, lg);
            if (XFP8) o.sx[t] = x_sf[t][b * x_sf_step];
        }
    };
    auto add = [&](const Block &o, int) {
#pragma unroll
        for (int f = 0; f < FF; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t)
                add_block<WFP8, XFP8>(acc[f][t], o.w[f], o.x[t], XFP8 ? o.sw[f] * o.sx[t] : WFP8 ? o.sw[f] : 1.0f);
    };
    const int full = K / kBlockK;
    if constexpr (FF + TF <= 3) {
        pipelined<Block>(first, step, full, [&](Block &o, int b) { load(std::true_type{}, o, b); }, add);
    } else {
        // two blocks would take the registers of the second workgroup on a CU
        for (int b = first; b < full; b += step) {
            Block o;
            load(std::true_type{}, o, b);
            add(o, b);
        }
    }
    if (K % kBlockK && full % step == first) {
        Block o;
        load(std::false_type{}, o, full);
        add(o, full);
    }
}

// The sum over the waves of what each left in part[wave], in order.
__device__ __forceinline__ f32x4 sum_waves(const f32x4 *part, int stride) {
    f32x4 v = part[0];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += part[w * stride];
    return v;
}

}  // namespace
}  // namespace epget
