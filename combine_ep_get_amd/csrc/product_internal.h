// Parameters of the experts' products and of the few-token expert layer.
// Internal header; the public ABI is include/ep_get.h.
#pragma once

#include "ep_internal.h"

namespace epget {

// Rows of the experts inside a receive buffer: expert e owns `count[e]` rows
// from row (e / L) * S + offset[e] on, as the layout places them, cut off at
// the end of its slice.  Null arrays: one expert that owns rows [0, dense).
struct Segments {
    const int32_t *count, *offset;
    int32_t E, L, dense;
    int64_t S;
};

// One grouped product and its epilogue.  Element sizes: 2 bytes (bf16), or 1
// (e4m3 codes with scales) for x and the weight of an FP8 product.
struct ProductArgs {
    Segments seg;
    int32_t C, N, M;  // inputs, outputs, weight rows (N, or 2N when gated)
    int32_t act;
    const void *x, *weight;
    const float *x_sf, *w_sf;  // FP8 scales, else null
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
    const void *w1, *w2;
    const float *w1_sf, *w2_sf, *b1, *b2;
    const uint16_t *residual;
    uint16_t *out;
    int32_t *status;
    uint16_t *h;  // [T * K, I] hidden rows, scaled by their weights
};

// Row ranges that each expert's rows are cut into for the elementwise pass of
// the backward call; the bias gradients are summed by range, then joined.
int32_t grad_row_ranges(int32_t E, int32_t N);

hipError_t launch_product_few(const ProductArgs &a, bool fp8, hipStream_t stream);
hipError_t launch_product(const ProductArgs &a, bool fp8, hipStream_t stream);
hipError_t launch_product_grad(const ProductGradArgs &a, hipStream_t stream);
hipError_t launch_tokens(const TokensArgs &a, bool fp8, hipStream_t stream);
hipError_t launch_combine_backward(const CopyParams &c, const uint16_t *dout, const uint16_t *y, const int32_t *slot,
                                   const float *w, uint16_t *dy, float *dw, hipStream_t stream);

}  // namespace epget
