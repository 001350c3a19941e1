// The whole expert layer for a few tokens, in two kernels, for gfx950.
//
//   up:   h[t,j,:] = bf16(w[t,j] * act(W1[e] x[t] + b1[e])),  e = idx[t,j]
//   down: out[t,:] = bf16(residual[t,:] + sum_j (W2[e] h[t,j,:] + w[t,j] b2[e]))
//
// Both are bound by the weights of the experts that some token names, each
// read once.  The weights go from memory straight to the matrix
// instruction's registers: its 16 rows are weight rows, its 16 columns
// tokens, and k is split over the waves of a workgroup in blocks of 128, so
// that no wave waits for another until the sums are joined in LDS, in a fixed
// order.  Scaling h by its weight lets the down product sum a token's
// experts with no further factors.  h is rounded to bf16, which the down
// product's matrix instruction takes; the layer of 128 tokens is off by 0.0023 of
// its size for it, where the rounding of the result alone gives 0.0017.
//
// Measured: one token of top-8 of 64 experts (7168 -> 2 x 2048 -> 7168, 705 MB) 147-156
// us, 128 tokens of top-8 of 256 (22 GB) 4.4 ms: 4.5-5.1 TB/s, where a large
// copy reaches 4.7 and a streaming read 5.2.  The down product's workgroups are
// H / 16: with fewer channels than 2048 they leave CUs idle (64 tokens of 1024
// channels 2.8 TB/s, of 128 0.5).
//
// Every workgroup first sorts the entries by expert in LDS: at most
// EP_MOE_TOKENS_MAX * EP_MAX_TOPK ids, which stay in L2.  A token that names an
// expert twice keeps one entry, with the sum of both weights.
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
__device__ __forceinline__ void sort_entries(const TokensArgs &a, EntryLists &l) {
    const int n = a.T * a.K;
    for (int e = threadIdx.x; e < a.E; e += kFewThreads) l.end[e] = 0;
    if (threadIdx.x == 0) l.bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kFewThreads) {
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
    for (int i = threadIdx.x; i < n; i += kFewThreads)
        if (first_of_token(i)) atomicAdd(&l.end[l.id[i]], 1);
    __syncthreads();
    // exclusive sums of the counts (low half) and of the experts with any (high half)
    const int per = (a.E + kFewThreads - 1) / kFewThreads;
    const int e0 = min(static_cast<int>(threadIdx.x) * per, a.E), e1 = min(e0 + per, a.E);
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += l.end[e] + (l.end[e] ? 1 << 16 : 0);
    const int incl = wave_inclusive_sum(sum);
    if ((threadIdx.x & 63) == 63) l.wave_sum[threadIdx.x >> 6] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < kFewWaves; ++w)
        if (w < static_cast<int>(threadIdx.x >> 6)) before += l.wave_sum[w];
    for (int e = e0; e < e1; ++e) {
        const int c = l.end[e];
        l.end[e] = before & 0xFFFF;
        if (c) l.expert[before >> 16] = static_cast<uint16_t>(e);
        before += c + (c ? 1 << 16 : 0);
    }
    if (threadIdx.x == kFewThreads - 1) l.experts = before >> 16;
    __syncthreads();
    // the order inside a run is the hardware's: every entry is a column of
    // its own, whose result does not depend on its place
    for (int i = threadIdx.x; i < n; i += kFewThreads)
        if (first_of_token(i)) l.entry[atomicAdd(&l.end[l.id[i]], 1)] = static_cast<uint16_t>(i);
    __syncthreads();
}

// up: items are (expert with entries, 16 outputs).  With enough items for
// every wave of the chip, a wave takes an item by itself and waits for no
// other; else a workgroup does, each wave a share of k, joined in LDS.
constexpr int kTokenCUs = 256;
// Items from which waves work alone: four waves on each of 256 CUs keep enough loads in flight
// (one token of 8 experts: 166 us with items shared by a workgroup, 147 alone).
constexpr int kWaveItems = 1024;

// This lane's sums of columns c0 .. c0 + 16 CF - 1 of expert e's entries and
// outputs n0 .. n0 + 15 (of both halves when gated) over a share of k.
template <bool FP8, int FF, int CF>
__device__ __forceinline__ void up_columns(const TokensArgs &a, const EntryLists &l, f32x4 (&acc)[FF][CF], int e, int c0,
                                           int m, int s0, int n0, int first, int step) {
    const int li = __lane_id() & 15, lg = __lane_id() >> 4;
    const int64_t pitch = static_cast<int64_t>(a.H) * (FP8 ? 1 : 2);
    const char *row[FF], *col[CF];
    const float *w_sf[FF], *none[CF];
#pragma unroll
    for (int f = 0; f < FF; ++f) {
        const int64_t r = static_cast<int64_t>(e) * a.M + f * a.I + min(n0 + li, a.I - 1);
        row[f] = static_cast<const char *>(a.w1) + r * pitch;
        w_sf[f] = FP8 ? a.w1_sf + (static_cast<int64_t>(e) * (a.M / 128) + (f * a.I + n0) / 128) * (a.H / 128) : nullptr;
    }
#pragma unroll
    for (int c = 0; c < CF; ++c) {
        const int en = l.entry[s0 + min(c0 + c * 16 + li, m - 1)];
        col[c] = reinterpret_cast<const char *>(a.x + static_cast<int64_t>(en / a.K) * a.H);
        none[c] = nullptr;
#pragma unroll
        for (int f = 0; f < FF; ++f) acc[f][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    accumulate_blocks<FP8, false>(acc, row, col, w_sf, none, 0, a.H, first, step, lg);
}

// h of this lane's column c of the entries and outputs n0 + 4 lg .. + 3.
template <int ACT>
__device__ __forceinline__ void up_write(const TokensArgs &a, const EntryLists &l, int e, int c, int m, int s0, int n0,
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

template <int ACT, bool FP8>
__global__ __launch_bounds__(kFewThreads) void tokens_up_kernel(TokensArgs a) {
    constexpr int FF = act_gated(ACT) ? 2 : 1;
    __shared__ EntryLists l;
    __shared__ f32x4 part[kFewWaves][FF][64];
    sort_entries(a, l);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = l.bad ? EP_ERR_BAD_EXPERT : EP_OK;
    const int lane = __lane_id(), li = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nf = (a.I + 15) / 16, items = l.experts * nf;
    const bool alone = items >= kWaveItems;
    const int G = gridDim.x;
    for (int item = alone ? blockIdx.x + wave * G : blockIdx.x; item < items; item += alone ? G * kFewWaves : G) {
        const int e = __builtin_amdgcn_readfirstlane(l.expert[item / nf]);
        const int n0 = (item % nf) * 16;
        const int s0 = __builtin_amdgcn_readfirstlane(l.start(e)), m = __builtin_amdgcn_readfirstlane(l.end[e]) - s0;
        for (int c0 = 0; c0 < m;) {
            if (alone && m - c0 > 16) {
                f32x4 acc[FF][2];
                up_columns<FP8, FF, 2>(a, l, acc, e, c0, m, s0, n0, 0, 1);
                up_write<ACT>(a, l, e, c0 + li, m, s0, n0, acc[0][0], acc[FF - 1][0]);
                up_write<ACT>(a, l, e, c0 + 16 + li, m, s0, n0, acc[0][1], acc[FF - 1][1]);
                c0 += 32;
                continue;
            }
            f32x4 acc[FF][1];
            up_columns<FP8, FF, 1>(a, l, acc, e, c0, m, s0, n0, alone ? 0 : wave, alone ? 1 : kFewWaves);
            if (!alone) {
#pragma unroll
                for (int f = 0; f < FF; ++f) part[wave][f][lane] = acc[f][0];
                __syncthreads();
                if (wave == 0)
#pragma unroll
                    for (int f = 0; f < FF; ++f) acc[f][0] = sum_waves(&part[0][f][lane], FF * 64);
                __syncthreads();
            }
            if (alone || wave == 0) up_write<ACT>(a, l, e, c0 + li, m, s0, n0, acc[0][0], acc[FF - 1][0]);
            c0 += 16;
        }
    }
}

// down: one workgroup for each 16 FF outputs, all experts.  Each wave takes
// whole experts in turn (shares of their k where there are fewer experts than waves): the
// columns are the expert's entries, and their sums are added to the
// wave's own sums of every token in LDS, which are joined at the end.  No
// wave waits for another before that.  sums: [wave][token][16 FF] floats.
template <bool FP8, int FF, int CF>
__device__ __forceinline__ void down_columns(const TokensArgs &a, const EntryLists &l, float *sums, int e, int c0, int m,
                                             int s0, int n0, int first, int step) {
    const int lane = __lane_id(), li = lane & 15, lg = lane >> 4;
    const int64_t pitch = static_cast<int64_t>(a.I) * (FP8 ? 1 : 2);
    const char *row[FF], *col[CF];
    const float *w_sf[FF], *none[CF];
    int tok[CF];
    f32x4 acc[FF][CF];
#pragma unroll
    for (int f = 0; f < FF; ++f) {
        const int n = min(n0 + f * 16 + li, a.H - 1);
        row[f] = static_cast<const char *>(a.w2) + (static_cast<int64_t>(e) * a.H + n) * pitch;
        w_sf[f] = FP8 ? a.w2_sf + (static_cast<int64_t>(e) * (a.H / 128) + min(n0 + f * 16, a.H - 1) / 128) * (a.I / 128) : nullptr;
    }
#pragma unroll
    for (int c = 0; c < CF; ++c) {
        const int en = l.entry[s0 + min(c0 + c * 16 + li, m - 1)];
        tok[c] = c0 + c * 16 + li < m ? en / a.K : -1;
        col[c] = reinterpret_cast<const char *>(a.h + static_cast<int64_t>(en) * a.I);
        none[c] = nullptr;
#pragma unroll
        for (int f = 0; f < FF; ++f) acc[f][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    accumulate_blocks<FP8, false>(acc, row, col, w_sf, none, 0, a.I, first, step, lg);
#pragma unroll
    for (int c = 0; c < CF; ++c) {
        if (tok[c] < 0) continue;
#pragma unroll
        for (int f = 0; f < FF; ++f) *reinterpret_cast<f32x4 *>(sums + tok[c] * (16 * FF) + f * 16 + lg * 4) += acc[f][c];
    }
}

// MANY: an expert may have more than 16 entries, for which the code takes the registers of
// a second workgroup on the CU.
template <bool FP8, int FF, bool MANY>
__global__ __launch_bounds__(kFewThreads, MANY ? 2 : 4) void tokens_down_kernel(TokensArgs a) {
    __shared__ EntryLists l;
    extern __shared__ __attribute__((aligned(16))) float sums[];
    sort_entries(a, l);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * FF;
    const int size = a.T * 16 * FF;  // floats of a wave's sums
    float *mine = sums + wave * size;
    for (int i = __lane_id() * 4; i < size; i += 256) *reinterpret_cast<f32x4 *>(mine + i) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int shares = l.experts >= kFewWaves ? 1 : l.experts ? kFewWaves / l.experts : 1;
    for (int u = wave; u < l.experts * shares; u += kFewWaves) {
        const int e = __builtin_amdgcn_readfirstlane(l.expert[u / shares]);
        const int s0 = __builtin_amdgcn_readfirstlane(l.start(e)), m = __builtin_amdgcn_readfirstlane(l.end[e]) - s0;
        for (int c0 = 0; c0 < m; c0 += 32) {
            if (!MANY || m - c0 <= 16)
                down_columns<FP8, FF, 1>(a, l, mine, e, c0, m, s0, n0, u % shares, shares);
            else
                down_columns<FP8, FF, 2>(a, l, mine, e, c0, m, s0, n0, u % shares, shares);
        }
    }
    __syncthreads();
    // four outputs of one token a thread
    for (int i = threadIdx.x; i < size / 4; i += kFewThreads) {
        const int tok = i / (4 * FF), n = n0 + (i - tok * (4 * FF)) * 4;
        if (n >= a.H) continue;
        f32x4 v = sum_waves(reinterpret_cast<const f32x4 *>(sums) + i, size / 4);
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

template <bool FP8>
hipError_t launch_up(const TokensArgs &a, hipStream_t stream) {
    const int64_t entries = static_cast<int64_t>(a.T) * a.K;
    const int64_t items = (entries < a.E ? entries : a.E) * ((a.I + 15) / 16);
    // one workgroup fits a CU's registers: no more, so that each sorts the entries once
    const uint32_t grid = static_cast<uint32_t>(items < 1 ? 1 : items < kTokenCUs ? items : kTokenCUs);
    switch (a.act) {
#define EP_ACT_CASE(A) \
    case A: tokens_up_kernel<A, FP8><<<grid, kFewThreads, 0, stream>>>(a); break;
        EP_ACT_CASE(EP_ACT_NONE)
        EP_ACT_CASE(EP_ACT_RELU)
        EP_ACT_CASE(EP_ACT_GELU)
        EP_ACT_CASE(EP_ACT_SILU)
        EP_ACT_CASE(EP_ACT_SWIGLU)
        EP_ACT_CASE(EP_ACT_GEGLU)
#undef EP_ACT_CASE
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <bool FP8>
hipError_t launch_down(const TokensArgs &a, hipStream_t stream) {
    // 32 outputs a workgroup where the tokens' sums leave a CU's LDS to one
    // workgroup or two anyway and 16 would take more than one workgroup a CU,
    // else 16.  The layer for 128 tokens with 16 and with 32: 256 experts of
    // 7168 x 2048 4602 and 4412 us, 128 of 4608 x 2048 1920 and 1767, but 256
    // of 4096 x 2048 2491 and 2981; in FP8 2708 and 2442, 1142 and 1026, 1389
    // and 1668.
    const int ff = a.T > 64 && a.H > 16 * kTokenCUs ? 2 : 1;
    const uint32_t grid = (a.H + 16 * ff - 1) / (16 * ff), lds = kFewWaves * a.T * 16 * ff * 4;
    static_assert(sizeof(EntryLists) + kFewWaves * EP_MOE_TOKENS_MAX * 16 * 2 * 4 <= 160 * 1024, "a CU's LDS");
    if (ff == 2)
        tokens_down_kernel<FP8, 2, true><<<grid, kFewThreads, lds, stream>>>(a);
    else if (a.T > 16)
        tokens_down_kernel<FP8, 1, true><<<grid, kFewThreads, lds, stream>>>(a);
    else
        tokens_down_kernel<FP8, 1, false><<<grid, kFewThreads, lds, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tokens(const TokensArgs &a, bool fp8, hipStream_t stream) {
    const hipError_t rc = fp8 ? launch_up<true>(a, stream) : launch_up<false>(a, stream);
    if (rc != hipSuccess || a.T == 0) return rc;
    return fp8 ? launch_down<true>(a, stream) : launch_down<false>(a, stream);
}

}  // namespace epget
