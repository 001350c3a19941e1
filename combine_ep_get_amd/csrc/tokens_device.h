// The epilogues that the few-token layers of every weight type share.  Lists
// holds the entries by expert: `entry`, numbers t * K + j, and `id`, the expert of each entry, -1 for none.  A token
// that names an expert twice keeps one entry, with the sum of both weights.
#pragma once

#include "few_device.h"

namespace epget {
namespace {

// h of this lane's column c of the entries and outputs n0 + 4 lg .. + 3.  It is rounded to bf16, the type of the second
// product's operands: beside the output's own rounding a second one of the same size, independent of it, so a layer without a
// residual is off by sqrt(2) times a single rounding (2.3e-3 of its norm against 64 bits, one rounding 1.7e-3).
template <int ACT, class Lists>
__device__ __forceinline__ void up_write(const TokensArgs &a, const Lists &l, int e, int c, int m, int s0, int n0,
                                         f32x4 v, f32x4 u) {
    const int n = n0 + (__lane_id() >> 4) * 4;
    if (c >= m || n >= a.I) return;
    const int en = l.entry[s0 + c], j0 = en - en % a.K;
    // the weight of the entry, and of the token's others on this expert
    float wt = 0.0f;
    for (int j = j0; j < j0 + a.K; ++j)
        if (l.id[j] == e) wt += a.w ? a.w[j] : 1.0f;
    if (a.b1) {
        const float *b = a.b1 + static_cast<int64_t>(e) * a.M + n;
        v += *reinterpret_cast<const f32x4 *>(b);
        if (act_gated(ACT)) u += *reinterpret_cast<const f32x4 *>(b + a.I);
    }
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = wt * (act_one<ACT>(v[i]) * (act_gated(ACT) ? u[i] : 1.0f));
    *reinterpret_cast<u32x2 *>(a.h + static_cast<int64_t>(en) * a.I + n) =
        u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
}

// The outputs of 16 FF channels from n0 on, from the waves' sums of every
// token: sums [wave][token][16 FF].  Called by the whole workgroup after a barrier.
template <int FF, int NT = kFewThreads, class Lists>
__device__ __forceinline__ void down_write(const TokensArgs &a, const Lists &l, const float *sums, int n0) {
    const int size = a.T * 16 * FF;  // floats of a wave's sums
    // four outputs of one token a thread
    for (int i = threadIdx.x; i < size / 4; i += NT) {
        const int tok = i / (4 * FF), n = n0 + (i - tok * (4 * FF)) * 4;
        if (n >= a.H) continue;
        f32x4 v = sum_waves<NT / 64>(reinterpret_cast<const f32x4 *>(sums) + i, size / 4);
        if (a.b2) {
            for (int j = 0; j < a.K; ++j) {
                const int en = tok * a.K + j, e = l.id[en];
                if (e < 0) continue;
                const float wt = a.w ? a.w[en] : 1.0f;
                v += wt * *reinterpret_cast<const f32x4 *>(a.b2 + static_cast<int64_t>(e) * a.H + n);
            }
        }
        const int64_t at = static_cast<int64_t>(tok) * a.H + n;
        if (a.residual) {
            const u32x2 r = *reinterpret_cast<const u32x2 *>(a.residual + at);
            v += f32x4{bf16_lo(r[0]), bf16_hi(r[0]), bf16_lo(r[1]), bf16_hi(r[1])};
        }
        *reinterpret_cast<u32x2 *>(a.out + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
}

}  // namespace
}  // namespace epget
