// What the few-token layers of every weight type share: the entries sorted by
// expert, and the epilogues.  Every workgroup sorts the entries for itself, in LDS: at
// most EP_MOE_TOKENS_MAX * EP_MAX_TOPK ids, which stay in L2.  A token that names
// an expert twice keeps one entry, with the sum of both weights.
#pragma once

#include "few_device.h"

namespace epget {
namespace {

constexpr int kMaxEntries = EP_MOE_TOKENS_MAX * EP_MAX_TOPK;
static_assert(kMaxEntries <= 65536 && EP_MAX_EXPERTS <= 32768, "entries are 16-bit numbers, ids signed ones");

struct EntryLists {
    int end[EP_MAX_EXPERTS];             // end of expert e's run in `entry` (its start is end[e - 1])
    uint16_t expert[kMaxEntries < EP_MAX_EXPERTS ? kMaxEntries : EP_MAX_EXPERTS];  // experts with entries, ascending
    int16_t id[kMaxEntries];             // expert of each entry, -1 for none
    uint16_t entry[kMaxEntries];         // t * K + j, by expert
    int wave_sum[kFewWaves];
    int experts;                         // number of experts with entries
    int bad;

    __device__ __forceinline__ int start(int e) const { return e ? end[e - 1] : 0; }
};

// Called by the whole workgroup; ends with a barrier.
template <int NT = kFewThreads, class Lists>
__device__ __forceinline__ void sort_entries(const TokensArgs &a, Lists &l) {
    const int n = a.T * a.K;
    for (int e = threadIdx.x; e < a.E; e += NT) l.end[e] = 0;
    if (threadIdx.x == 0) l.bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT) {
        const int e = a.idx[i];
        const bool ok = e >= 0 && e < a.E;
        l.id[i] = ok ? e : -1;
        if (!ok && e != -1) l.bad = 1;
    }
    __syncthreads();
    // an entry whose expert the token names before it is left out
    auto first_of_token = [&](int i) {
        const int e = l.id[i];
        bool keep = e >= 0;
        for (int j = i - i % a.K; j < i; ++j) keep = keep && l.id[j] != e;
        return keep;
    };
    for (int i = threadIdx.x; i < n; i += NT)
        if (first_of_token(i)) atomicAdd(&l.end[l.id[i]], 1);
    __syncthreads();
    // exclusive sums of the counts (low half) and of the experts with any (high half)
    const int per = (a.E + NT - 1) / NT;
    const int e0 = min(static_cast<int>(threadIdx.x) * per, a.E), e1 = min(e0 + per, a.E);
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += l.end[e] + (l.end[e] ? 1 << 16 : 0);
    const int incl = wave_inclusive_sum(sum);
    if ((threadIdx.x & 63) == 63) l.wave_sum[threadIdx.x >> 6] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < NT / 64; ++w)
        if (w < static_cast<int>(threadIdx.x >> 6)) before += l.wave_sum[w];
    for (int e = e0; e < e1; ++e) {
        const int c = l.end[e];
        l.end[e] = before & 0xFFFF;
        if (c) l.expert[before >> 16] = static_cast<uint16_t>(e);
        before += c + (c ? 1 << 16 : 0);
    }
    if (threadIdx.x == NT - 1) l.experts = before >> 16;
    __syncthreads();
    // the order inside a run is the hardware's: every entry is a column of
    // its own, whose result does not depend on its place
    for (int i = threadIdx.x; i < n; i += NT)
        if (first_of_token(i)) l.entry[atomicAdd(&l.end[l.id[i]], 1)] = static_cast<uint16_t>(i);
    __syncthreads();
}

// h of this lane's column c of the entries and outputs n0 + 4 lg .. + 3.
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
