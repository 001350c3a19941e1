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

constexpr int weight_bits(int w) { return w == kBf16 ? 16 : w == kFp8 ? 8 : 4; }
// k per block: one scale of an FP8 weight, and a whole line of 128 bytes of a row at least
constexpr int block_k(int w) { return w == kFp4 ? 256 : 128; }
template <int W>
using Scale = std::conditional_t<W == kFp4, uint8_t, float>;

// A block of one fragment of 16 weight rows, as it comes from memory: bf16 in
// four pieces of 8 k a lane (k = 32 q + 8 g), e4m3 in two of 16 (k = 64 q + 16 g),
// e2m1 in two of 32 (k = 128 q + 32 g), each with a scale of its own.
// The weight is read once: its loads carry the non-temporal hint.
template <int W>
struct WeightBlock {
    static constexpr int kPieces = W == kBf16 ? 4 : 2;
    u32x4 v[kPieces];
    uint8_t e8[W == kFp4 ? kPieces : 1];  // scales of the pieces of an FP4 block

    // row: this lane's row; b: the block; K: end of k, with zeros past it in a block that is not FULL
    template <bool FULL>
    __device__ __forceinline__ void load(const char *row, int b, int K, int lg) {
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int k = b * block_k(W) + (W == kBf16 ? 32 * q + 8 * lg : W == kFp8 ? 64 * q + 16 * lg : 128 * q + 32 * lg);
            const u32x4 *p = reinterpret_cast<const u32x4 *>(row + static_cast<int64_t>(k) * weight_bits(W) / 8);
            v[q] = FULL || k < K ? __builtin_nontemporal_load(p) : u32x4{0, 0, 0, 0};
        }
    }

    template <bool FULL>
    __device__ __forceinline__ void load_scales(const uint8_t *sf, int b, int K, int lg) {
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int group = b * (block_k(W) / 32) + 4 * q + lg;
            e8[q] = FULL || group * 32 < K ? sf[group] : 127;
        }
    }

    // The e8m0 scale of a piece as fp32: 2^-127 is a subnormal number there.
    __device__ __forceinline__ float scale(int q) const {
        const uint32_t b = e8[q];
        return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
    }

    // bf16 operand of matrix instruction s of the block; codes are widened, which is exact.
    __device__ __forceinline__ bf16x8 operand(int s) const {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        if constexpr (W == kBf16) {
            return __builtin_bit_cast(bf16x8, v[s]);
        } else if constexpr (W == kFp4) {
            const uint32_t c = v[s >> 2][s & 3];
            const float f = scale(s >> 2);
            const bf16x2 o0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 0);
            const bf16x2 o1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 1);
            const bf16x2 o2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 2);
            const bf16x2 o3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 3);
            return bf16x8{o0[0], o0[1], o1[0], o1[1], o2[0], o2[1], o3[0], o3[1]};
        } else {
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
// lanes hold.  W: the weight's type; XFP8: whether the column is e4m3, else bf16.
template <int W, bool XFP8>
struct ColumnBlock {
    static constexpr int kPieces = XFP8 ? 2 : block_k(W) / 32;
    u32x4 v[kPieces];

    template <bool FULL>
    __device__ __forceinline__ void load(const char *col, int b, int K, int lg) {
#pragma unroll
        for (int s = 0; s < kPieces; ++s) {
            const int k = b * block_k(W) + (XFP8         ? 64 * s + 16 * lg
                                            : W == kFp4 ? 128 * (s >> 2) + 32 * lg + 8 * (s & 3)
                                            : W == kFp8 ? 64 * (s >> 1) + 16 * lg + 8 * (s & 1)
                                                        : 32 * s + 8 * lg);
            const u32x4 *p = reinterpret_cast<const u32x4 *>(col + static_cast<int64_t>(k) * (XFP8 ? 1 : 2));
            v[s] = FULL || k < K ? *p : u32x4{0, 0, 0, 0};
        }
    }
};

// acc += the block's product, times scale where the weight is FP8.
template <int W, bool XFP8>
__device__ __forceinline__ void add_block(f32x4 &acc, const WeightBlock<W> &w, const ColumnBlock<W, XFP8> &x,
                                          float scale) {
    f32x4 d = W == kFp8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc;
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
        for (int s = 0; s < block_k(W) / 32; ++s)
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.operand(s), __builtin_bit_cast(bf16x8, x.v[s]), d, 0, 0, 0);
    }
    if constexpr (W == kFp8) {
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
template <int W, bool XFP8, int FF, int TF>
__device__ __forceinline__ void accumulate_blocks(f32x4 (&acc)[FF][TF], const char *const (&row)[FF],
                                                  const char *const (&col)[TF], const Scale<W> *const (&w_sf)[FF],
                                                  const float *const (&x_sf)[TF], int64_t x_sf_step, int K, int first,
                                                  int step, int lg) {
    struct Block {
        WeightBlock<W> w[FF];
        ColumnBlock<W, XFP8> x[TF];
        float sw[FF], sx[TF];
    };
    auto load = [&](auto full, Block &o, int b) {
#pragma unroll
        for (int f = 0; f < FF; ++f) {
            o.w[f].template load<full()>(row[f], b, K, lg);
            if constexpr (W == kFp8) o.sw[f] = w_sf[f][b];
            if constexpr (W == kFp4) o.w[f].template load_scales<full()>(w_sf[f], b, K, lg);
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
                add_block<W, XFP8>(acc[f][t], o.w[f], o.x[t], XFP8 ? o.sw[f] * o.sx[t] : W == kFp8 ? o.sw[f] : 1.0f);
    };
    const int full = K / block_k(W);
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
    if (K % block_k(W) && full % step == first) {
        Block o;
        load(std::false_type{}, o, full);
        add(o, full);
    }
}

// Where the scales of weight row `row` lie, of M rows of K columns an expert: row m of expert e, whose block of 128
// rows an FP8 weight has one scale for.
template <int W>
__device__ __forceinline__ const Scale<W> *weight_scales(const void *sf, int e, int M, int m, int64_t row, int K) {
    if constexpr (W == kFp8)
        return static_cast<const float *>(sf) + (static_cast<int64_t>(e) * (M / 128) + m / 128) * (K / 128);
    else if constexpr (W == kFp4)
        return static_cast<const uint8_t *>(sf) + row * (K / 32);
    else
        return nullptr;
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
