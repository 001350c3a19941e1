// Parameters of the experts' products and of the few-token expert layer.
// Internal header; the public ABI is include/ep_get.h.
#pragma once

#include "ep_internal.h"

namespace epget {

// Weights as bf16, as e4m3 with one fp32 scale for 128 x 128, or as e2m1 with one e8m0 scale for 32 of a row: EP_WEIGHTS_*.
enum WeightType { kBf16, kFp8, kFp4 };

// Rows of the experts inside a receive buffer: expert e owns `count[e]` rows
// from row (e / L) * S + offset[e] on, as the layout places them, cut off at
// the end of its slice.  Null arrays: one expert that owns rows [0, dense).
struct Segments {
    const int32_t *count, *offset;
    int32_t E, L, dense;
    int64_t S;
};

// One grouped product and its epilogue.  Element sizes: 2 bytes (bf16), or 1
// (e4m3 codes with scales) for x and the weight of an FP8 product, or half a
// byte (e2m1) for the weight of an FP4 product.
struct ProductArgs {
    Segments seg;
    int32_t C, N, M;  // inputs, outputs, weight rows (N, or 2N when gated)
    int32_t act;
    const void *x, *weight;
    const float *x_sf;         // FP8 scales, else null
    const void *w_sf;          // fp32 or e8m0 scales, else null
    int64_t sf_ts, sf_hs;
    const float *bias;         // [E, M] or null
    const uint16_t *residual;  // or null
    uint16_t *pre;             // or null
    uint16_t *out;
    int64_t entries;           // T * K, the most rows there can be
    int64_t mean_rows;         // rows of an average expert, for the choice of the tile
};

struct ProductGradArgs {
    Segments seg;
    int32_t C, N, M, act;
    const uint16_t *dout, *pre, *x, *weight;
    uint16_t *dpre;  // gradient of the pre-activations: dout itself without an activation
    uint16_t *dx, *dweight;
    float *dweight_acc, *dbias, *partial;
    int64_t entries;
    int32_t splits;  // row ranges of an expert whose bias gradients are summed apart
    int64_t mean_rows;
};

// The layer for a few tokens.
struct TokensArgs {
    int32_t T, H, I, M, E, K, act;
    const uint16_t *x;
    const int32_t *idx;
    const float *w;
    const void *w1, *w2, *w1_sf, *w2_sf;
    const float *b1, *b2;
    const uint16_t *residual;
    uint16_t *out;
    int32_t *status;
    uint16_t *h;  // [T * K, I] hidden rows, scaled by their weights
    float *y;     // [T * K, H] rows of the entries before their sum, where the 4-bit layer keeps them
};

// Row ranges that each expert's rows are cut into for the elementwise pass of
// the backward call; the bias gradients are summed by range, then joined.
int32_t grad_row_ranges(int32_t E, int32_t N);

hipError_t launch_product_few(const ProductArgs &a, bool fp8, hipStream_t stream);
hipError_t launch_product(const ProductArgs &a, bool fp8, hipStream_t stream);
hipError_t launch_product_grad(const ProductGradArgs &a, hipStream_t stream);
hipError_t launch_tokens(const TokensArgs &a, bool fp8, hipStream_t stream);
hipError_t launch_product_fp4(const ProductArgs &a, hipStream_t stream);
// Bytes of TokensArgs::y, or 0 where it is not used.
int64_t tokens_fp4_rows_bytes(int32_t T, int32_t K, int32_t E, int32_t H, int32_t I);
hipError_t launch_tokens_fp4(const TokensArgs &a, hipStream_t stream);
hipError_t launch_combine_backward(const CopyParams &c, const uint16_t *dout, const uint16_t *y, const int32_t *slot,
                                   const float *w, uint16_t *dy, float *dw, hipStream_t stream);

}  // namespace epget
