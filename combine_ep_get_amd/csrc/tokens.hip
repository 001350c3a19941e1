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
// experts in the accumulators themselves: a column is one token, and an
// expert that the token does not name multiplies zeros.
//
// Every workgroup first sorts the entries by expert in LDS: at most
// kMaxTokens * EP_MAX_TOPK ids, which stay in L2.  A token that names an
// expert twice keeps one entry, with the sum of both weights.
#include "product_device.h"

namespace epget {
namespace {

constexpr int kTokThreads = 512;
constexpr int kTokWaves = kTokThreads / 64;
constexpr int kMaxEntries = kMaxTokens * EP_MAX_TOPK;
constexpr int kBlockK = 128;  // k per block: one scale of an FP8 weight, four bf16 matrix instructions

struct EntryLists {
    int end[EP_MAX_EXPERTS];             // end of expert e's run in `entry` (its start is end[e - 1])
    uint16_t expert[kMaxEntries < EP_MAX_EXPERTS ? kMaxEntries : EP_MAX_EXPERTS];  // experts with entries, ascending
    int16_t id[kMaxEntries];             // expert of each entry, -1 for none
    uint16_t entry[kMaxEntries];         // t * K + j, by expert
    int wave_sum[kTokWaves];
    int experts;                         // number of experts with entries
    int bad;

    __device__ __forceinline__ int start(int e) const { return e ? end[e - 1] : 0; }
};

// Called by the whole workgroup; ends with a barrier.
__device__ __forceinline__ void sort_entries(const TokensArgs &a, EntryLists &l) {
    const int n = a.T * a.K;
    for (int e = threadIdx.x; e < a.E; e += kTokThreads) l.end[e] = 0;
    if (threadIdx.x == 0) l.bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kTokThreads) {
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
    for (int i = threadIdx.x; i < n; i += kTokThreads)
        if (first_of_token(i)) atomicAdd(&l.end[l.id[i]], 1);
    __syncthreads();
    // exclusive sums of the counts (low half) and of the experts with any (high half)
    const int per = (a.E + kTokThreads - 1) / kTokThreads;
    const int e0 = min(static_cast<int>(threadIdx.x) * per, a.E), e1 = min(e0 + per, a.E);
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += l.end[e] + (l.end[e] ? 1 << 16 : 0);
    const int incl = wave_inclusive_sum(sum);
    if ((threadIdx.x & 63) == 63) l.wave_sum[threadIdx.x >> 6] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < kTokWaves; ++w)
        if (w < static_cast<int>(threadIdx.x >> 6)) before += l.wave_sum[w];
    for (int e = e0; e < e1; ++e) {
        const int c = l.end[e];
        l.end[e] = before & 0xFFFF;
        if (c) l.expert[before >> 16] = static_cast<uint16_t>(e);
        before += c + (c ? 1 << 16 : 0);
    }
    if (threadIdx.x == kTokThreads - 1) l.experts = before >> 16;
    __syncthreads();
    // the order inside a run is the hardware's: every entry is a column of
    // its own, whose result does not depend on its place
    for (int i = threadIdx.x; i < n; i += kTokThreads)
        if (first_of_token(i)) l.entry[atomicAdd(&l.end[l.id[i]], 1)] = static_cast<uint16_t>(i);
    __syncthreads();
}

// A block of 128 k of one weight row fragment, as it comes from memory: bf16
// in four pieces of 8 k a lane (k = 32 q + 8 g), e4m3 in two of 16 (k = 64 q + 16 g).
template <bool FP8>
struct WeightBlock {
    static constexpr int kPieces = FP8 ? 2 : 4;
    u32x4 v[kPieces];

    // row: this lane's row; k0: first k; K: end of k (zeros past it)
    __device__ __forceinline__ void load(const char *row, int k0, int K, int lg) {
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
            const int k = k0 + (FP8 ? 64 * q + 16 * lg : 32 * q + 8 * lg);
            const char *p = row + static_cast<int64_t>(k) * (FP8 ? 1 : 2);
            v[q] = k < K ? __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p)) : u32x4{0, 0, 0, 0};
        }
    }

    // Operand of matrix instruction s (0..3) of the block.
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

// The bf16 operand of the same block: column li, the k that the weight's lanes hold.
template <bool FP8>
struct ColumnBlock {
    u32x4 v[4];
    __device__ __forceinline__ void load(const uint16_t *col, bool live, int k0, int K, int lg) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = k0 + (FP8 ? 64 * (s >> 1) + 16 * lg + 8 * (s & 1) : 32 * s + 8 * lg);
            v[s] = live && k < K ? *reinterpret_cast<const u32x4 *>(col + k) : u32x4{0, 0, 0, 0};
        }
    }
};

template <bool FP8>
__device__ __forceinline__ f32x4 block_product(const WeightBlock<FP8> &w, const ColumnBlock<FP8> &x, f32x4 c) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.operand(s), __builtin_bit_cast(bf16x8, x.v[s]), c, 0, 0, 0);
    return c;
}

// Adds the block's product to acc; an FP8 block's is scaled first.
template <bool FP8>
__device__ __forceinline__ void add_block(f32x4 &acc, const WeightBlock<FP8> &w, const ColumnBlock<FP8> &x, float scale) {
    if constexpr (FP8) {
        const f32x4 d = block_product<FP8>(w, x, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(d[i], scale, acc[i]);
    } else {
        acc = block_product<FP8>(w, x, acc);
    }
}

// up: items are (expert with entries, 16 outputs), one workgroup each in turn.
template <int ACT, bool FP8>
__global__ __launch_bounds__(kTokThreads) void tokens_up_kernel(TokensArgs a) {
    constexpr bool GATED = act_gated(ACT);
    constexpr int FF = GATED ? 2 : 1;
    __shared__ EntryLists l;
    __shared__ f32x4 part[kTokWaves][FF][64];
    sort_entries(a, l);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = l.bad ? EP_ERR_BAD_EXPERT : EP_OK;
    const int lane = __lane_id(), li = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nf = (a.I + 15) / 16, items = l.experts * nf;
    const int blocks = (a.H + kBlockK - 1) / kBlockK;
    const int64_t pitch = static_cast<int64_t>(a.H) * (FP8 ? 1 : 2);
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int e = __builtin_amdgcn_readfirstlane(l.expert[item / nf]);
        const int n0 = (item % nf) * 16;
        const int s0 = __builtin_amdgcn_readfirstlane(l.start(e)), m = __builtin_amdgcn_readfirstlane(l.end[e]) - s0;
        const char *row[FF];
        const float *scale[FF];
#pragma unroll
        for (int f = 0; f < FF; ++f) {
            const int64_t r = static_cast<int64_t>(e) * a.M + f * a.I + min(n0 + li, a.I - 1);
            row[f] = static_cast<const char *>(a.w1) + r * pitch;
            scale[f] = FP8 ? a.w1_sf + (static_cast<int64_t>(e) * (a.M / 128) + (f * a.I + n0) / 128) * (a.H / 128) : nullptr;
        }
        for (int c0 = 0; c0 < m; c0 += 16) {
            const int en = l.entry[s0 + min(c0 + li, m - 1)];
            const uint16_t *col = a.x + static_cast<int64_t>(en / a.K) * a.H;
            f32x4 acc[FF];
#pragma unroll
            for (int f = 0; f < FF; ++f) acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            for (int b = wave; b < blocks; b += kTokWaves) {
                WeightBlock<FP8> w[FF];
                ColumnBlock<FP8> x;
#pragma unroll
                for (int f = 0; f < FF; ++f) w[f].load(row[f], b * kBlockK, a.H, lg);
                x.load(col, true, b * kBlockK, a.H, lg);
#pragma unroll
                for (int f = 0; f < FF; ++f) add_block<FP8>(acc[f], w[f], x, FP8 ? scale[f][b] : 1.0f);
            }
#pragma unroll
            for (int f = 0; f < FF; ++f) part[wave][f][lane] = acc[f];
            __syncthreads();
            if (wave == 0) {
                f32x4 v[FF];
#pragma unroll
                for (int f = 0; f < FF; ++f) {
                    v[f] = part[0][f][lane];
#pragma unroll
                    for (int w = 1; w < kTokWaves; ++w) v[f] += part[w][f][lane];
                }
                const int n = n0 + lg * 4;
                if (c0 + li < m && n < a.I) {
                    // the weight of the entry, and of the token's others on this expert
                    float wt = 0.0f;
                    for (int j = en - en % a.K; j < en - en % a.K + a.K; ++j)
                        if (l.id[j] == e) wt += a.w ? a.w[j] : 1.0f;
#pragma unroll
                    for (int f = 0; f < FF; ++f)
                        if (a.b1) v[f] += *reinterpret_cast<const f32x4 *>(a.b1 + static_cast<int64_t>(e) * a.M + f * a.I + n);
                    float o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = wt * (act_one<ACT>(v[0][i]) * (GATED ? v[FF - 1][i] : 1.0f));
                    *reinterpret_cast<u32x2 *>(a.h + static_cast<int64_t>(en) * a.I + n) =
                        u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
                }
            }
            __syncthreads();
        }
    }
}

// down: one workgroup for each 16 outputs, all experts; TF fragments of 16 tokens.
template <bool FP8, int TF>
__global__ __launch_bounds__(kTokThreads) void tokens_down_kernel(TokensArgs a) {
    __shared__ EntryLists l;
    __shared__ f32x4 part[kTokWaves][64];
    sort_entries(a, l);
    const int lane = __lane_id(), li = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16;
    const int blocks = (a.I + kBlockK - 1) / kBlockK, units = l.experts * blocks;
    const int64_t pitch = static_cast<int64_t>(a.I) * (FP8 ? 1 : 2);
    f32x4 acc[TF];
#pragma unroll
    for (int t = 0; t < TF; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int u = wave; u < units; u += kTokWaves) {
        const int o = u / blocks, b = u - o * blocks;
        const int e = __builtin_amdgcn_readfirstlane(l.expert[o]);
        const int s0 = __builtin_amdgcn_readfirstlane(l.start(e)), s1 = __builtin_amdgcn_readfirstlane(l.end[e]);
        WeightBlock<FP8> w;
        w.load(static_cast<const char *>(a.w2) + (static_cast<int64_t>(e) * a.H + min(n0 + li, a.H - 1)) * pitch,
               b * kBlockK, a.I, lg);
        const float scale =
            FP8 ? a.w2_sf[(static_cast<int64_t>(e) * (a.H / 128) + n0 / 128) * (a.I / 128) + b] : 1.0f;
        int en[TF];
#pragma unroll
        for (int t = 0; t < TF; ++t) en[t] = -1;
        for (int s = s0; s < s1; ++s) {
            const int i = l.entry[s], tok = i / a.K;
#pragma unroll
            for (int t = 0; t < TF; ++t) en[t] = tok == t * 16 + li ? i : en[t];
        }
#pragma unroll
        for (int t = 0; t < TF; ++t) {
            if (__ballot(en[t] >= 0) == 0) continue;
            ColumnBlock<FP8> x;
            x.load(a.h + static_cast<int64_t>(max(en[t], 0)) * a.I, en[t] >= 0, b * kBlockK, a.I, lg);
            f32x4 sum = acc[t];
            add_block<FP8>(sum, w, x, scale);
            // a token that does not name the expert keeps its sum: zero times
            // a weight that is not finite is not zero
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = en[t] >= 0 ? sum[i] : acc[t][i];
        }
    }
#pragma unroll
    for (int t = 0; t < TF; ++t) {
        part[wave][lane] = acc[t];
        __syncthreads();
        const int tok = t * 16 + li, n = n0 + lg * 4;
        if (wave == 0 && tok < a.T && n < a.H) {
            f32x4 v = part[0][lane];
#pragma unroll
            for (int w = 1; w < kTokWaves; ++w) v += part[w][lane];
            if (a.b2) {
                for (int j = 0; j < a.K; ++j) {
                    const int i = tok * a.K + j, e = l.id[i];
                    if (e < 0) continue;
                    const float wt = a.w ? a.w[i] : 1.0f;
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
        __syncthreads();
    }
}

template <bool FP8>
hipError_t launch_up(const TokensArgs &a, hipStream_t stream) {
    const int64_t entries = static_cast<int64_t>(a.T) * a.K;
    const int64_t items = (entries < a.E ? entries : a.E) * ((a.I + 15) / 16);
    const uint32_t grid = static_cast<uint32_t>(items < 1 ? 1 : items < 1024 ? items : 1024);
    switch (a.act) {
#define EP_ACT_CASE(A) \
    case A: tokens_up_kernel<A, FP8><<<grid, kTokThreads, 0, stream>>>(a); break;
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
    const uint32_t grid = (a.H + 15) / 16;
    if (a.T <= 16)
        tokens_down_kernel<FP8, 1><<<grid, kTokThreads, 0, stream>>>(a);
    else if (a.T <= 32)
        tokens_down_kernel<FP8, 2><<<grid, kTokThreads, 0, stream>>>(a);
    else if (a.T <= 64)
        tokens_down_kernel<FP8, 4><<<grid, kTokThreads, 0, stream>>>(a);
    else
        tokens_down_kernel<FP8, 8><<<grid, kTokThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tokens(const TokensArgs &a, bool fp8, hipStream_t stream) {
    const hipError_t rc = fp8 ? launch_up<true>(a, stream) : launch_up<false>(a, stream);
    if (rc != hipSuccess || a.T == 0) return rc;
    return fp8 ? launch_down<true>(a, stream) : launch_down<false>(a, stream);
}

}  // namespace epget
