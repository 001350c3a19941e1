// Device helpers shared by the experts' products and the few-token layer:
// activations, the segment walk, and matrix-instruction types.
#pragma once

#include "../../include/ep_get.h"
#include "device_common.h"
#include "product_internal.h"

namespace epget {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr bool act_gated(int act) { return act == EP_ACT_SWIGLU || act == EP_ACT_GEGLU; }

// sigmoid through the hardware's exp2 and reciprocal (each within an ulp or
// two of fp32, far below the bf16 rounding of what it enters).
__device__ __forceinline__ float sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}

// Phi, the normal distribution function.  Below -6 it is under 1e-9, where
// the difference 1 + erf would be rounded away: erfc keeps its digits.
__device__ __forceinline__ float normal_cdf(float v) { return 0.5f * erfcf(-0.70710678118654752f * v); }

// One-input activations (the gate's one for the gated ones), and their derivatives.
template <int ACT>
__device__ __forceinline__ float act_one(float v) {
    if constexpr (ACT == EP_ACT_RELU) return v > 0.0f ? v : (v != v ? v : 0.0f);
    if constexpr (ACT == EP_ACT_GELU || ACT == EP_ACT_GEGLU) return v * normal_cdf(v);
    if constexpr (ACT == EP_ACT_SILU || ACT == EP_ACT_SWIGLU) return v * sigmoid(v);
    return v;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float v) {
    if constexpr (ACT == EP_ACT_RELU) return v > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == EP_ACT_GELU || ACT == EP_ACT_GEGLU)
        return normal_cdf(v) + v * 0.3989422804014327f * __builtin_amdgcn_exp2f(-0.7213475204444817f * v * v);
    if constexpr (ACT == EP_ACT_SILU || ACT == EP_ACT_SWIGLU) {
        const float s = sigmoid(v);
        return s * (1.0f + v * (1.0f - s));
    }
    return 1.0f;
}

__device__ __forceinline__ u32x4 pack_bf16(const f32x4 (&v)[2]) {
    return u32x4{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]), pack_bf16x2(v[1][0], v[1][1]),
                 pack_bf16x2(v[1][2], v[1][3])};
}

// bf16 of 4 G neighbouring values, and back.
template <int G>
__device__ __forceinline__ void store_bf16(uint16_t *p, const f32x4 (&v)[G]) {
    if constexpr (G == 2)
        *reinterpret_cast<u32x4 *>(p) = pack_bf16(v);
    else
        *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3])};
}

template <int G>
__device__ __forceinline__ void add_bf16(f32x4 (&v)[G], const uint16_t *p) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const u32x2 r = reinterpret_cast<const u32x2 *>(p)[g];
        v[g] += f32x4{bf16_lo(r[0]), bf16_hi(r[0]), bf16_lo(r[1]), bf16_hi(r[1])};
    }
}

// Epilogue of the 4 G neighbouring outputs from n on of row r: v (and, gated,
// u) are their sums.
template <int ACT, int G>
__device__ __forceinline__ void write_outputs(const ProductArgs &a, int e, int64_t r, int n, f32x4 (&v)[G], f32x4 (&u)[G]) {
    constexpr bool GATED = act_gated(ACT);
    if (a.bias) {
        const f32x4 *b = reinterpret_cast<const f32x4 *>(a.bias + static_cast<int64_t>(e) * a.M + n);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            v[g] += b[g];
            if (GATED) u[g] += b[a.N / 4 + g];
        }
    }
    if (a.pre) {
        store_bf16(a.pre + r * a.M + n, v);
        if (GATED) store_bf16(a.pre + r * a.M + a.N + n, u);
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[g][i] = act_one<ACT>(v[g][i]);
            if (GATED) v[g][i] *= u[g][i];
        }
    if (a.residual) add_bf16(v, a.residual + r * a.N + n);
    store_bf16(a.out + r * a.N + n, v);
}

// Rows of expert e, from `row0` on; an expert whose rows run past its slice
// keeps those inside it (the layout gives the others no slot), and arrays
// that no layout wrote cannot lead outside the buffer.
__device__ __forceinline__ int segment(const Segments &s, int e, int64_t *row0) {
    if (!s.count) {
        *row0 = 0;
        return s.dense;
    }
    const int64_t off = max(s.offset[e], 0);
    *row0 = static_cast<int64_t>(e / s.L) * s.S + off;
    const int64_t left = s.S - off;
    return static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(s.count[e]), left)));
}

// The tiles of `rows_per_tile` rows of the experts before e, for all e in
// [0, E], into first[].  Called by a whole workgroup of NT threads, which may read
// first[] afterwards.
template <int NT>
__device__ __forceinline__ void tile_prefix(const Segments &s, int rows_per_tile, int *first, int *wave_sum) {
    constexpr int NW = NT / 64;
    const int per = (s.E + NT - 1) / NT;  // consecutive experts of a thread
    const int e0 = threadIdx.x * per, e1 = min(e0 + per, s.E);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        int64_t row0;
        sum += (segment(s, e, &row0) + rows_per_tile - 1) / rows_per_tile;
    }
    const int incl = wave_inclusive_sum(sum);
    if ((threadIdx.x & 63) == 63) wave_sum[threadIdx.x >> 6] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < NW; ++w)
        if (w < static_cast<int>(threadIdx.x >> 6)) before += wave_sum[w];
    for (int e = e0; e < e1; ++e) {
        first[e] = before;
        int64_t row0;
        before += (segment(s, e, &row0) + rows_per_tile - 1) / rows_per_tile;
    }
    if (e0 < s.E && e1 == s.E) first[s.E] = before;
    __syncthreads();
}

// The expert that owns row tile `t`: the last e with first[e] <= t.
__device__ __forceinline__ int tile_expert(const int *first, int E, int t) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Order of the tiles of one expert with `nt` row tiles and `nf` feature
// tiles: groups of up to kTileGroup row tiles, row tiles fastest, so that
// workgroups that run together share both operands' panels in L2.
constexpr int kTileGroup = 8;
__device__ __forceinline__ void tile_in_expert(int64_t idx, int nt, int nf, int *tt, int *ft) {
    const int64_t per_group = static_cast<int64_t>(kTileGroup) * nf;
    const int g = static_cast<int>(idx / per_group);
    const int rem = static_cast<int>(idx - g * per_group);
    const int gs = min(kTileGroup, nt - g * kTileGroup);
    *ft = rem / gs;
    *tt = g * kTileGroup + rem - *ft * gs;
}

// Tile that workgroup `wg` of G (a multiple of 8) takes in round `round`, or
// -1: workgroups go to the 8 XCDs in turn, and each XCD takes a run of
// consecutive tiles of the round, whose operands its L2 then holds once.
__device__ __forceinline__ int64_t tile_of(int64_t total, int64_t round, int wg, int G) {
    const int64_t left = total - round * G;
    const int64_t now = left < G ? left : G;
    const int64_t run = (now + 7) / 8;
    const int64_t k = wg >> 3, idx = (wg & 7) * run + k;
    return k < run && idx < now ? round * G + idx : -1;
}

}  // namespace
}  // namespace epget
