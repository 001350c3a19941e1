// Products and the few-token layer on MXFP4 weights, for gfx950: e2m1 codes with
// one e8m0 scale for 32 neighbours of a row, and bf16 tokens.
//
//   product: out[r,n] = act(sum_c x[r,c] W[e,n,c] + b[e,n]) + residual[r,n]
//   layer:   h[t,j,:] = bf16(w[t,j] * act(W1[e] x[t] + b1[e])),  e = idx[t,j]
//            out[t,:] = bf16(residual[t,:] + sum_j (W2[e] h[t,j,:] + w[t,j] b2[e]))
//
// Bound by the weights, each read once: 0.53 bytes a value.  A code and its scale
// are widened to bf16 by one instruction for two, exactly (infinite from 2^128
// on), and multiplied by the bf16 matrix instruction (its 16 rows are weight
// rows, its 16 columns tokens).
//
// The matrix instruction's lane l has row l % 16 of a fragment, and the address
// unit joins the accesses of neighbouring lanes only.  Loads in that order take
// it one access a lane; with weights of 4 bits that is the bound (92 % busy at 3.3
// TB/s).  And a load that asks for half a line leaves the next one waiting for
// the same line in the cache (2.8 TB/s).  So eight neighbouring lanes load a
// line of 128 bytes of a row, and the bytes go through LDS, a few KB of each wave's
// own, to the lanes that want them: a wave waits for no other.  The eight 16-byte
// pieces of a line are permuted there by bits of the row, on the side of the
// load's address, so that the writes are linear and the reads of 16 rows spread
// over the banks.
//
// A layer of 128 tokens over 256 experts of 7168 x 2048 takes 1240 to 1260 us in a call, 4.7 TB/s, the rate of a large
// copy; of one token and 8 experts 45 us (4.2).  100 rows of tokens by 128 experts of 4096 x 2 x 1408: 200 us, 4.0 TB/s.
#include <limits.h>

#include "tokens_device.h"

namespace epget {
namespace {

constexpr int kStageK = 256;  // k of a stage: a line of a weight's row, four of a column's

// Where piece `piece` of a line of row `row` of a fragment lies in LDS, and back.
__device__ __forceinline__ int place_of(int row, int piece) { return piece ^ (row & 7) ^ (row >> 3); }

// What a lane loads, and where it finds its operands.
struct Lanes {
    int row, piece;  // loads of lines: row % 8 of the fragment, piece of rows 0..7 (piece ^ 1 of rows 8..15)
    int li, lg;
    __device__ __forceinline__ Lanes() {
        const int l = __lane_id();
        row = l >> 3;
        piece = place_of(row, l & 7);
        li = l & 15;
        lg = l >> 4;
    }
};

// kStageK of FF fragments of 16 weight rows and of XC columns (8 or 16).
template <int FF, int XC>
struct Stage {
    static constexpr int kHalves = XC / 8;
    u32x4 w[FF][2], x[4][kHalves];
    uint32_t sf[FF];  // of row lane / 4, four scales from 4 (lane & 1) on
};

// Bases that a wave shares, and this lane's bytes from them.  A fragment's 16 rows are whole: sizes are multiples of 32.
// An expert's weight is at most 2^31 values, and the columns are at most 4096 rows of 2^16 values.
template <int FF, int XC>
struct Rows {
    const char *w[FF], *sf[FF], *x;
    uint32_t w_at[2], sf_at, x_at[XC / 8];
};

// The weights of stage b.  FULL: no k of it is past K, of which there are zeros.  ONCE: past the caches, for weights that no
// other wave reads soon.
template <bool FULL, bool ONCE, int FF, int XC>
__device__ __forceinline__ void load_weights(u32x4 (&w)[FF][2], uint32_t (&sf)[FF], const Rows<FF, XC> &r, int b, int K,
                                             const Lanes &ll) {
    const int64_t w_off = static_cast<int64_t>(b) * (kStageK / 2), sf_off = static_cast<int64_t>(b) * (kStageK / 32);
#pragma unroll
    for (int f = 0; f < FF; ++f) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 *p = reinterpret_cast<const u32x4 *>(r.w[f] + w_off + r.w_at[h]);
            w[f][h] = u32x4{0, 0, 0, 0};
            if (FULL || b * kStageK + (ll.piece ^ h) * 32 < K) w[f][h] = ONCE ? __builtin_nontemporal_load(p) : *p;
        }
        const char *p = r.sf[f] + sf_off + r.sf_at;
        if constexpr (FULL) {
            __builtin_memcpy(&sf[f], p, 4);  // at any address
        } else {
            const int k = b * kStageK + (__lane_id() & 1) * 128;
            sf[f] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (k + i * 32 < K) sf[f] |= uint32_t{static_cast<uint8_t>(p[i])} << 8 * i;
        }
    }
}

// Tiles of eight columns are for experts of which most have one tile; of sixteen an expert may have many, and each reads its
// weights again (dense, weights from memory: 128 x 7168 x 2 x 2048 26.3 us, past the caches 32.1, 64 rows 18.1 and 20.7; of
// one tile, 16 rows, 13.1 and 12.9).
template <bool FULL, int FF, int XC>
__device__ __forceinline__ void load_stage(Stage<FF, XC> &s, const Rows<FF, XC> &r, int b, int K, const Lanes &ll) {
    load_weights<FULL, XC == 8>(s.w, s.sf, r, b, K, ll);
    const char *x = r.x + static_cast<int64_t>(b) * (kStageK * 2);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int h = 0; h < XC / 8; ++h)
            s.x[u][h] = FULL || b * kStageK + u * 64 + (ll.piece ^ (h & 1)) * 8 < K
                            ? *reinterpret_cast<const u32x4 *>(x + u * 128 + r.x_at[h])
                            : u32x4{0, 0, 0, 0};
}

// The scale of this lane's codes of half q of a stage, from the lane that loaded it: e8m0 is fp32's exponent.
__device__ __forceinline__ float scale_of(uint32_t sf, int q, const Lanes &ll) {
    const uint32_t four = __builtin_amdgcn_ds_bpermute((ll.li * 4 + q) * 4, sf);
    return __uint_as_float((four >> 8 * ll.lg & 255) << 23);  // the conversion takes no other bits
}

// Eight codes as bf16.
__device__ __forceinline__ bf16x8 widened(uint32_t codes, float scale) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 o0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 o1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 o2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 o3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16x8{o0[0], o0[1], o1[0], o1[1], o2[0], o2[1], o3[0], o3[1]};
}

// Bytes of LDS of a wave: a stage's weights, and half of its k of one fragment of columns.
template <int FF, int XC>
constexpr int kScratch = FF * 2048 + XC / 8 * 2048;

// acc += the stage's products.  A lane's 16 bytes of a weight row are one scale's 32 codes, k = 128 q + 32 lg + 8 i + 0..7
// for matrix instruction i of half q, and the column's operand is read from the same k.
template <int FF, int XC>
__device__ __forceinline__ void use_stage(f32x4 (&acc)[FF], const Stage<FF, XC> &s, char *scratch, const Lanes &ll) {
    const int lane16 = __lane_id() * 16;
    char *xs = scratch + FF * 2048;
    const int xi = XC == 16 ? ll.li : ll.li & 7;  // eight columns are there twice
    const int w_row = (ll.li >> 3) * 1024 + (ll.li & 7) * 128;
    const int x_row = ((ll.lg >> 1) * (XC / 8) + (xi >> 3)) * 1024 + (xi & 7) * 128;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int f = 0; f < FF; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<u32x4 *>(scratch + (f * 2 + h) * 1024 + lane16) = s.w[f][h];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < XC / 8; ++h)
                *reinterpret_cast<u32x4 *>(xs + (u * (XC / 8) + h) * 1024 + lane16) = s.x[2 * q + u][h];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        bf16x8 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = *reinterpret_cast<const bf16x8 *>(xs + x_row + place_of(xi, (ll.lg & 1) * 4 + i) * 16);
#pragma unroll
        for (int f = 0; f < FF; ++f) {
            const int at = f * 2048 + w_row + place_of(ll.li, 4 * q + ll.lg) * 16;
            const u32x4 w = *reinterpret_cast<const u32x4 *>(scratch + at);
            const float scale = scale_of(s.sf[f], q, ll);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widened(w[i], scale), x[i], acc[f], 0, 0, 0);
        }
    }
}

// acc += W rows x columns over the stages first, first + step, ..; the loads of DEPTH stages are on their way.
template <int DEPTH, int FF, int XC>
__device__ __forceinline__ void accumulate(f32x4 (&acc)[FF], const Rows<FF, XC> &r, int K, int first, int step,
                                           char *scratch, const Lanes &ll) {
    const int full = K / kStageK;
    const int n = first < full ? (full - first + step - 1) / step : 0;  // whole stages
    const bool rest = K % kStageK && full % step == first;              // and stage n, in part past K
    Stage<FF, XC> s[DEPTH];
    auto load = [&](int i, int at) {
        if (at < n)
            load_stage<true>(s[i], r, first + at * step, K, ll);
        else if (at == n && rest)
            load_stage<false>(s[i], r, full, K, ll);
    };
    const int all = n + rest;
    int at = 0;  // the stage in s[0]
    if (n >= DEPTH) {
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) load_stage<true>(s[i], r, first + i * step, K, ll);
        for (; at + 2 * DEPTH <= n; at += DEPTH) {
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                use_stage(acc, s[i], scratch, ll);
                load_stage<true>(s[i], r, first + (at + i + DEPTH) * step, K, ll);
            }
        }
        // fewer than 2 DEPTH whole ones are left
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            use_stage(acc, s[i], scratch, ll);
            load(i, at + i + DEPTH);
        }
        at += DEPTH;
    } else {
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) load(i, i);
    }
#pragma unroll
    for (int i = 0; i < DEPTH; ++i)
        if (at + i < all) use_stage(acc, s[i], scratch, ll);
}

template <int FF>
__device__ __forceinline__ void clear(f32x4 (&acc)[FF]) {
#pragma unroll
    for (int f = 0; f < FF; ++f) acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

// r's weights: expert e's, of M rows of K columns, fragment f from row m on, rows 8..15 of it `half` further than they
// would be.
template <int FF, int XC>
__device__ __forceinline__ void set_weights(Rows<FF, XC> &r, const void *w, const void *sf, int e, int M, int K,
                                            const int (&m)[FF], const Lanes &ll, int half = 0) {
    const int row = __lane_id() >> 2;
    r.w_at[0] = ll.row * (K / 2) + ll.piece * 16;
    r.w_at[1] = (ll.row + 8 + half) * (K / 2) + (ll.piece ^ 1) * 16;
    r.sf_at = (row + (row >= 8 ? half : 0)) * (K / 32) + (__lane_id() & 1) * 4;
#pragma unroll
    for (int f = 0; f < FF; ++f) {
        const int64_t row = static_cast<int64_t>(e) * M + m[f];
        r.w[f] = static_cast<const char *>(w) + row * (K / 2);
        r.sf[f] = static_cast<const char *>(sf) + row * (K / 32);
    }
}

// The first product of either call works on items of FF fragments of weight
// rows, two for the layer: 16 outputs with a gate, 32 without.  `share` waves of a workgroup split
// k of one item between them, so that few items still fill the chip: items times
// waves an item up to kItemWaves.  Their sums are joined in LDS, in order.
// (2048 are all waves of the chip.  One token of 8 experts, 7168 x 2 x 2048: the layer takes 45.7 us, with up to 1024
// waves 62, with up to 4096 47.)
constexpr int kItemWaves = 2048;
constexpr int item_outputs(bool gated, int FF) { return gated ? 8 * FF : 16 * FF; }
__device__ __forceinline__ int waves_of_item(int64_t items) {
    int share = kFewWaves;
    while (share > 1 && items * share > kItemWaves) share >>= 1;
    return share;
}

template <int FF>
struct Part {
    f32x4 v[kFewWaves][FF][64];
};

// The sums of the waves of an item, on its first wave.  Called by the whole workgroup.
template <int FF>
__device__ __forceinline__ void join(f32x4 (&acc)[FF], Part<FF> &part, int wave, int share) {
    const int lane = __lane_id();
    if (share == 1) return;
#pragma unroll
    for (int f = 0; f < FF; ++f) part.v[wave][f][lane] = acc[f];
    __syncthreads();
    if (wave % share == 0) {
#pragma unroll
        for (int f = 0; f < FF; ++f)
            for (int w = 1; w < share; ++w) acc[f] += part.v[wave + w][f][lane];
    }
    __syncthreads();
}

// FF: fragments of an item.  One, where two would leave CUs idle, has the gates in its rows 0..7 and the other halves in
// rows 8..15 (1 x 7168 x 2 x 2048: 7.0 us, two 8.8; 64 x 7168 x 2 x 512:
// a call 10.7 and 13.3; where two keep all CUs busy, 64 x 7168 x 2 x 2048, 22.8 and 20.2).
template <int ACT, int FF, int XC>
__global__ __launch_bounds__(kFewThreads, 2) void product_fp4_kernel(ProductArgs a) {
    constexpr bool GATED = act_gated(ACT);
    constexpr int kOut = item_outputs(GATED, FF);
    __shared__ __attribute__((aligned(16))) char scratch[kFewWaves][kScratch<FF, XC>];
    __shared__ Part<FF> part;
    __shared__ int first[EP_MAX_EXPERTS + 1];
    __shared__ int wave_sum[kFewWaves];
    if (a.seg.E > 1) {
        tile_prefix<kFewThreads>(a.seg, XC, first, wave_sum);
    } else if (threadIdx.x < 2) {  // no sums over experts: a decode-sized product is mostly latency
        int64_t row0;
        first[threadIdx.x] = threadIdx.x ? (segment(a.seg, 0, &row0) + XC - 1) / XC : 0;
    }
    __syncthreads();
    const Lanes ll;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nf = a.N / kOut;
    const int64_t items = static_cast<int64_t>(first[a.seg.E]) * nf;
    const int share = waves_of_item(items), per = kFewWaves / share;
    for (int64_t g = blockIdx.x; g * per < items; g += gridDim.x) {
        const int64_t item = g * per + wave / share;
        f32x4 acc[FF];
        clear(acc);
        int e = 0, n0 = 0, t0 = 0, rows = 0;
        int64_t row0 = 0;
        if (item < items) {
            e = tile_expert(first, a.seg.E, static_cast<int>(item / nf));
            const int f0 = __builtin_amdgcn_readfirstlane(first[e]);
            const int nt = __builtin_amdgcn_readfirstlane(first[e + 1]) - f0;
            int tt, ft;
            tile_in_expert(item - static_cast<int64_t>(f0) * nf, nt, nf, &tt, &ft);
            rows = segment(a.seg, e, &row0);
            n0 = ft * kOut, t0 = tt * XC;
            Rows<FF, XC> r;
            int m[FF];
#pragma unroll
            for (int f = 0; f < FF; ++f) m[f] = n0 + f * (GATED ? a.N : 16);
            set_weights(r, a.weight, a.w_sf, e, a.M, a.C, m, ll, GATED && FF == 1 ? a.N - 8 : 0);
            r.x = reinterpret_cast<const char *>(static_cast<const uint16_t *>(a.x) + (row0 + t0) * a.C);
#pragma unroll
            for (int h = 0; h < XC / 8; ++h)
                r.x_at[h] = static_cast<uint32_t>(min(h * 8 + ll.row, rows - 1 - t0)) * a.C * 2 + (ll.piece ^ h) * 16;
            accumulate<2>(acc, r, a.C, wave % share, share, scratch[wave], ll);
        }
        join(acc, part, wave, share);
        if (item < items && wave % share == 0) {
            const int t = t0 + ll.li, n = n0 + ll.lg * 4;
            f32x4 v[1] = {acc[0]}, u[1] = {acc[FF - 1]};
            if (GATED && FF == 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) u[0][i] = __shfl_xor(u[0][i], 32);
            if (t >= rows || ll.li >= XC || (GATED && FF == 1 && ll.lg >= 2)) continue;
            write_outputs<ACT>(a, e, row0 + t, n, v, u);
            if (!GATED && FF == 2) write_outputs<ACT>(a, e, row0 + t, n + 16, u, u);
        }
    }
}

// Where experts have many columns each, the kernels above would take a weight through the matrix instructions' operands
// once for 16 of them, and each wave would load its own columns, four times the weight's bytes.  Here a workgroup of
// four waves works on up to 64 columns and 128 weight rows, 32 a wave; the waves' columns are the same, so each loads a
// quarter of their stage, 64 k of it, and all read it from LDS.  128 tokens, 8 of 32 experts of 4096 x 2 x 1408: 78 us
// instead of 133 (tiles of 32 columns: 82); 8 of 8 experts 45 instead of 95.  Bound by memory with two workgroups a CU,
// by the columns' way through LDS and the barriers with one.  More than two stages on their way: 58 to 60 us.
constexpr int kManyThreads = 256;
constexpr int kManyWaves = kManyThreads / 64;
constexpr int kManyColumns = 64;
constexpr int kManyShared = kManyColumns * kStageK * 2;  // bytes

// This lane's share of a stage: CF fragments of columns.
template <int CF>
struct ManyStage {
    u32x4 w[2][2], x[2 * CF];
    uint32_t sf[2];
};

template <bool FULL, int CF>
__device__ __forceinline__ void load_many(ManyStage<CF> &s, const Rows<2, kManyColumns> &r, int b, int K, int wave,
                                          const Lanes &ll) {
    load_weights<FULL, false>(s.w, s.sf, r, b, K, ll);
    const char *x = r.x + static_cast<int64_t>(b) * (kStageK * 2) + wave * 128;
#pragma unroll
    for (int h = 0; h < 2 * CF; ++h) {
        s.x[h] = u32x4{0, 0, 0, 0};
        if (FULL || b * kStageK + wave * 64 + (ll.piece ^ (h & 1)) * 8 < K) s.x[h] = *reinterpret_cast<const u32x4 *>(x + r.x_at[h]);
    }
}

// acc += W rows x columns; the loads of two stages are on their way.  Called by the whole workgroup.
template <int CF>
__device__ __forceinline__ void accumulate_many(f32x4 (&acc)[2][kManyColumns / 16], const Rows<2, kManyColumns> &r, int K,
                                                char *shared, char *scratch, int wave, const Lanes &ll) {
    const int full = K / kStageK, all = (K + kStageK - 1) / kStageK;
    const int lane16 = __lane_id() * 16;
    const int w_row = (ll.li >> 3) * 1024 + (ll.li & 7) * 128;
    const char *x_row = shared + (ll.lg >> 1) * (2 * CF * 1024) + w_row;
    ManyStage<CF> s[2];
    auto load = [&](ManyStage<CF> &d, int b) {
        if (b < full)
            load_many<true>(d, r, b, K, wave, ll);
        else if (b < all)
            load_many<false>(d, r, b, K, wave, ll);
    };
    auto step = [&](ManyStage<CF> &d, auto &&load_next) {
        __syncthreads();  // the stage before has been read
#pragma unroll
        for (int h = 0; h < 2 * CF; ++h) *reinterpret_cast<u32x4 *>(shared + (wave * 2 * CF + h) * 1024 + lane16) = d.x[h];
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h) *reinterpret_cast<u32x4 *>(scratch + (f * 2 + h) * 1024 + lane16) = d.w[f][h];
        const uint32_t sf[2] = {d.sf[0], d.sf[1]};
        load_next(d);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            u32x4 w[2];
            float scale[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int at = f * 2048 + w_row + place_of(ll.li, 4 * q + ll.lg) * 16;
                w[f] = *reinterpret_cast<const u32x4 *>(scratch + at);
                scale[f] = scale_of(sf[f], q, ll);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bf16x8 x[CF];
#pragma unroll
                for (int c = 0; c < CF; ++c)
                    x[c] = *reinterpret_cast<const bf16x8 *>(x_row + (2 * q * 2 * CF + c * 2) * 1024 +
                                                             place_of(ll.li, (ll.lg & 1) * 4 + i) * 16);
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const bf16x8 o = widened(w[f][i], scale[f]);
#pragma unroll
                    for (int c = 0; c < CF; ++c)
                        acc[f][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o, x[c], acc[f][c], 0, 0, 0);
                }
            }
        }
    };
    int b = 0;  // the stage in s[0]
    if (full >= 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            load_many<true>(s[i], r, i, K, wave, ll);
            __builtin_amdgcn_sched_barrier(0);  // in this order, as the loop below waits for them
        }
        for (; b + 4 <= full; b += 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) step(s[i], [&](ManyStage<CF> &d) { load_many<true>(d, r, b + i + 2, K, wave, ll); });
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) step(s[i], [&](ManyStage<CF> &d) { load(d, b + i + 2); });
        b += 2;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) load(s[i], i);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (b + i < all) step(s[i], [](ManyStage<CF> &) {});
}

__device__ __forceinline__ void accumulate_columns(f32x4 (&acc)[2][kManyColumns / 16], const Rows<2, kManyColumns> &r,
                                                   int columns, int K, char *shared, char *scratch, int wave,
                                                   const Lanes &ll) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int c = 0; c < kManyColumns / 16; ++c) acc[f][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (columns > 32)
        accumulate_many<4>(acc, r, K, shared, scratch, wave, ll);
    else
        accumulate_many<2>(acc, r, K, shared, scratch, wave, ll);
}

template <int ACT>
__global__ __launch_bounds__(kManyThreads, 2) void product_fp4_many_kernel(ProductArgs a) {
    constexpr bool GATED = act_gated(ACT);
    constexpr int kOut = item_outputs(GATED, 2), kGroup = kManyWaves * kOut;
    __shared__ __attribute__((aligned(16))) char shared[kManyShared], scratch[kManyWaves][4096];
    __shared__ int first[EP_MAX_EXPERTS + 1];
    __shared__ int wave_sum[kManyWaves];
    tile_prefix<kManyThreads>(a.seg, kManyColumns, first, wave_sum);
    const Lanes ll;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nf = (a.N + kGroup - 1) / kGroup;
    const int64_t items = static_cast<int64_t>(first[a.seg.E]) * nf;
    for (int64_t round = 0; round * gridDim.x < items; ++round) {
        const int64_t item = tile_of(items, round, blockIdx.x, gridDim.x);
        if (item < 0) break;
        const int e = tile_expert(first, a.seg.E, static_cast<int>(item / nf));
        const int f0 = __builtin_amdgcn_readfirstlane(first[e]);
        const int nt = __builtin_amdgcn_readfirstlane(first[e + 1]) - f0;
        int tt, ft;
        tile_in_expert(item - static_cast<int64_t>(f0) * nf, nt, nf, &tt, &ft);
        int64_t row0;
        const int rows = segment(a.seg, e, &row0), t0 = tt * kManyColumns;
        const int place = ft * kGroup + wave * kOut, n0 = min(place, a.N - kOut);
        Rows<2, kManyColumns> r;
        set_weights(r, a.weight, a.w_sf, e, a.M, a.C, {n0, GATED ? a.N + n0 : n0 + 16}, ll);
        r.x = reinterpret_cast<const char *>(static_cast<const uint16_t *>(a.x) + (row0 + t0) * a.C);
#pragma unroll
        for (int h = 0; h < kManyColumns / 8; ++h)
            r.x_at[h] = static_cast<uint32_t>(min(h * 8 + ll.row, rows - 1 - t0)) * a.C * 2 + (ll.piece ^ (h & 1)) * 16;
        f32x4 acc[2][kManyColumns / 16];
        accumulate_columns(acc, r, rows - t0, a.C, shared, scratch[wave], wave, ll);
        if (place != n0) continue;  // past the last output
#pragma unroll
        for (int c = 0; c < kManyColumns / 16; ++c) {
            const int t = t0 + c * 16 + ll.li;
            f32x4 v[1] = {acc[0][c]}, u[1] = {acc[1][c]};
            if (t < rows) {
                write_outputs<ACT>(a, e, row0 + t, n0 + ll.lg * 4, v, u);
                if (!GATED) write_outputs<ACT>(a, e, row0 + t, n0 + ll.lg * 4 + 16, u, u);
            }
        }
    }
}

// The entries by expert and their tiles, in LDS that the launch sizes.
struct Lists {
    int *start;                // entries of the experts before each
    int *begin, *first;        // the same, and tiles, of the experts with entries
    int *wave_sum;
    uint16_t *expert;          // the experts with entries, ascending
    uint16_t *entry;           // the entries by expert, ascending in each
    uint16_t *owner;           // number in `expert` of each tile
    uint16_t *rank;            // of an entry of a wave's among its expert's, kNone where it is left out
    int16_t *id;               // expert of each entry, -1 for none
    int &experts, &bad;
    static constexpr uint16_t kNone = 0xFFFF;
    static_assert(EP_MOE_TOKENS_MAX * EP_MAX_TOPK < kNone && EP_MAX_EXPERTS <= 32768,
                  "entries are 16-bit numbers, ids signed ones");

    static __host__ __device__ int most(const TokensArgs &a) { return a.E < a.T * a.K ? a.E : a.T * a.K; }
    static __host__ __device__ int bytes(const TokensArgs &a) {
        return (a.E * 4 + (most(a) + 1) * 8 + (2 * kFewWaves + 2) * 4 + most(a) * 2 + a.T * a.K * 8 + 15) / 16 * 16;
    }
    __device__ __forceinline__ Lists(const TokensArgs &a, char *p)
        : start(reinterpret_cast<int *>(p)), begin(start + a.E), first(begin + most(a) + 1), wave_sum(first + most(a) + 1),
          expert(reinterpret_cast<uint16_t *>(wave_sum + 2 * kFewWaves + 2)), entry(expert + most(a)), owner(entry + a.T * a.K),
          rank(owner + a.T * a.K), id(reinterpret_cast<int16_t *>(rank + a.T * a.K)), experts(wave_sum[2 * kFewWaves]),
          bad(wave_sum[2 * kFewWaves + 1]) {}

    // Fills them, tiles being of `width` entries at most.  An expert's entries are in ascending order, as they have to be
    // where several workgroups take tiles of them: each wave counts a run of tokens, up to 64 entries at a time, in a table
    // of its own in `space`, which nothing else uses meanwhile.  Called by the whole workgroup; ends with a barrier.
    template <int NT, int N>
    __device__ __forceinline__ void fill(const TokensArgs &a, int width, char (&space)[N]) {
        static_assert(N >= NT / 64 * EP_MAX_EXPERTS * 2, "a number of 16 bits for each wave and expert");
        const int n = a.T * a.K;
        if (n <= 64) {
            if (threadIdx.x < 64) fill_wave(a, width);
            __syncthreads();
            return;
        }
        constexpr int kWaves = NT / 64;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        uint16_t *counts = reinterpret_cast<uint16_t *>(space);
        uint16_t *mine = counts + wave * a.E;
        for (int i = threadIdx.x; i < kWaves * a.E; i += NT) counts[i] = 0;
        if (threadIdx.x == 0) bad = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += NT) {
            const int e = a.idx[i];
            const bool ok = e >= 0 && e < a.E;
            id[i] = static_cast<int16_t>(ok ? e : -1);
            if (!ok && e != -1) bad = 1;
        }
        __syncthreads();
        const int step = 64 - 64 % a.K, run = ((n + step - 1) / step + kWaves - 1) / kWaves * step;  // whole tokens
        auto each = [&](auto f) {  // entries of this wave, or -1
            for (int i = wave * run; i < min((wave + 1) * run, n); i += step) f(lane < step && i + lane < n ? i + lane : -1);
        };
        const uint64_t below = (uint64_t{1} << lane) - 1, token = below & ~((uint64_t{1} << (lane - lane % a.K)) - 1);
        each([&](int i) {
            const int e = i >= 0 ? id[i] : -1;
            uint64_t same = __ballot(e >= 0);
            for (int b = 0; (a.E - 1) >> b; ++b) {
                const uint64_t set = __ballot(e >> b & 1);
                same &= e >> b & 1 ? set : ~set;
            }
            // an entry whose expert the token names before it is left out
            const bool keep = e >= 0 && !(same & token);
            same &= __ballot(keep);
            const int before = __popcll(same & below);
            const int base = keep ? mine[e] : 0;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (keep && before == 0) mine[e] = static_cast<uint16_t>(base + __popcll(same));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (i >= 0) rank[i] = keep ? static_cast<uint16_t>(base + before) : kNone;
        });
        __syncthreads();
        // sums over the experts: entries (low half) and experts with any (high half), and tiles
        const int per = (a.E + NT - 1) / NT;
        const int e0 = min(static_cast<int>(threadIdx.x) * per, a.E), e1 = min(e0 + per, a.E);
        int sum = 0, tiles = 0;
        for (int e = e0; e < e1; ++e) {
            int m = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const int c = counts[w * a.E + e];
                counts[w * a.E + e] = static_cast<uint16_t>(m);
                m += c;
            }
            start[e] = m;
            sum += m + (m ? 1 << 16 : 0);
            tiles += (m + width - 1) / width;
        }
        const int all = wave_inclusive_sum(sum), all_tiles = wave_inclusive_sum(tiles);
        if (lane == 63) wave_sum[wave] = all, wave_sum[kFewWaves + wave] = all_tiles;
        __syncthreads();
        int before = all - sum, tile = all_tiles - tiles;
        for (int w = 0; w < wave; ++w) before += wave_sum[w], tile += wave_sum[kFewWaves + w];
        for (int e = e0; e < e1; ++e) {
            const int m = start[e], i = before >> 16;
            start[e] = before & 0xFFFF;
            if (m == 0) continue;
            expert[i] = static_cast<uint16_t>(e);
            begin[i] = start[e];
            first[i] = tile;
            for (int left = m; left > 0; left -= width) owner[tile++] = static_cast<uint16_t>(i);
            before += m + (1 << 16);
        }
        if (threadIdx.x == NT - 1) {
            experts = before >> 16;
            begin[experts] = before & 0xFFFF;
            first[experts] = tile;
        }
        __syncthreads();
        each([&](int i) {
            if (i >= 0 && rank[i] != kNone) entry[start[id[i]] + mine[id[i]] + rank[i]] = static_cast<uint16_t>(i);
        });
        __syncthreads();
    }

    // The same for up to 64 entries, one a lane of one wave: a decode batch waits for no other wave (a layer of one token
    // 46 to 48 us instead of 50).
    __device__ __forceinline__ void fill_wave(const TokensArgs &a, int width) {
        const int i = threadIdx.x, n = a.T * a.K;
        const int e = i < n ? a.idx[i] : -1;
        const bool ok = e >= 0 && e < a.E;
        const uint64_t wrong = __ballot(!ok && e != -1);
        uint64_t same = __ballot(ok);
        for (int b = 0; (a.E - 1) >> b; ++b) {
            const uint64_t set = __ballot(e >> b & 1);
            same &= e >> b & 1 ? set : ~set;
        }
        const uint64_t below = (uint64_t{1} << i) - 1, token = below & ~((uint64_t{1} << (i - i % a.K)) - 1);
        // an entry whose expert the token names before it is left out
        const bool keep = ok && !(same & token);
        const uint64_t kept = __ballot(keep);
        same &= kept;
        const int m = __popcll(same), rank = __popcll(same & below);
        const bool leads = keep && rank == 0;
        int i0 = 0, b0 = 0, f0 = 0, all = 0;  // experts, entries and tiles before this one's, and all tiles
        const uint64_t leaders = __ballot(leads);
        for (uint64_t left = leaders; left; left &= left - 1) {
            const int j = __ffsll(static_cast<unsigned long long>(left)) - 1;
            const int ej = __builtin_amdgcn_readlane(e, j), mj = __builtin_amdgcn_readlane(m, j);
            const int tj = (mj + width - 1) / width;
            if (ej < e) ++i0, b0 += mj, f0 += tj;
            all += tj;
        }
        if (i < n) id[i] = static_cast<int16_t>(ok ? e : -1);
        if (keep) entry[b0 + rank] = static_cast<uint16_t>(i);
        if (leads) {
            expert[i0] = static_cast<uint16_t>(e);
            begin[i0] = b0;
            first[i0] = f0;
            for (int t = 0; t * width < m; ++t) owner[f0 + t] = static_cast<uint16_t>(i0);
        }
        if (i == 0) {
            experts = __popcll(leaders);
            begin[experts] = __popcll(kept);
            first[experts] = all;
            bad = wrong != 0;
        }
    }
};

// The layer's two products as rows of the entries: the hidden rows, and what each entry adds to its token, in 32 bits.
template <int ACT>
struct UpRows {
    static constexpr bool kGated = act_gated(ACT), kFirst = true;
    static __host__ __device__ int outputs(const TokensArgs &a) { return a.I; }
    static __device__ int inputs(const TokensArgs &a) { return a.H; }
    static __device__ int weight_rows(const TokensArgs &a) { return a.M; }
    static __device__ const void *weight(const TokensArgs &a) { return a.w1; }
    static __device__ const void *scales(const TokensArgs &a) { return a.w1_sf; }
    static __device__ const uint16_t *x(const TokensArgs &a) { return a.x; }
    static __device__ int x_row(const TokensArgs &a, int entry) { return entry / a.K; }
    // Column c of an expert's m entries from s0 on, outputs n0 .. n0 + 15: v, and u of the gates' other halves or of the
    // next 16.
    static __device__ __forceinline__ void write(const TokensArgs &a, const Lists &l, int e, int c, int m, int s0, int n0,
                                                 f32x4 v, f32x4 u) {
        up_write<ACT>(a, l, e, c, m, s0, n0, v, u);
        if (!kGated) up_write<ACT>(a, l, e, c, m, s0, n0 + 16, u, u);
    }
};

struct DownRows {
    static constexpr bool kGated = false, kFirst = false;
    static __host__ __device__ int outputs(const TokensArgs &a) { return a.H; }
    static __device__ int inputs(const TokensArgs &a) { return a.I; }
    static __device__ int weight_rows(const TokensArgs &a) { return a.H; }
    static __device__ const void *weight(const TokensArgs &a) { return a.w2; }
    static __device__ const void *scales(const TokensArgs &a) { return a.w2_sf; }
    static __device__ const uint16_t *x(const TokensArgs &a) { return a.h; }
    static __device__ int x_row(const TokensArgs &, int entry) { return entry; }
    static __device__ __forceinline__ void write(const TokensArgs &a, const Lists &l, int, int c, int m, int s0, int n0,
                                                 f32x4 v, f32x4 u) {
        if (c >= m) return;
        float *y = a.y + static_cast<int64_t>(l.entry[s0 + c]) * a.H + n0 + (__lane_id() >> 4) * 4;
        *reinterpret_cast<f32x4 *>(y) = v;
        *reinterpret_cast<f32x4 *>(y + 16) = u;
    }
};

// Tile `tile` of `nf` tiles of outputs for each tile of up to XC entries.
struct EntryTile {
    int e, s0, m, c0, ft;  // expert, its first entry, its entries, the tile's first of them, tile of outputs
    __device__ __forceinline__ EntryTile(const Lists &l, int tile, int nf, int XC) {
        const int i = __builtin_amdgcn_readfirstlane(l.owner[tile / nf]);
        const int f0 = __builtin_amdgcn_readfirstlane(l.first[i]), nt = __builtin_amdgcn_readfirstlane(l.first[i + 1]) - f0;
        int tt;
        tile_in_expert(tile - f0 * nf, nt, nf, &tt, &ft);
        e = __builtin_amdgcn_readfirstlane(l.expert[i]);
        s0 = __builtin_amdgcn_readfirstlane(l.begin[i]);
        m = __builtin_amdgcn_readfirstlane(l.begin[i + 1]) - s0;
        c0 = tt * XC;
    }
    // Bytes of this lane's row h of the columns and its piece of a line.
    template <class Side>
    __device__ __forceinline__ uint32_t x_at(const TokensArgs &a, const Lists &l, int h, const Lanes &ll) const {
        const int row = Side::x_row(a, l.entry[s0 + min(c0 + h * 8 + ll.row, m - 1)]);
        return static_cast<uint32_t>(row) * Side::inputs(a) * 2 + (ll.piece ^ (h & 1)) * 16;
    }
};

// XC: columns of a tile of entries.
template <class Side, int XC>
__global__ __launch_bounds__(kFewThreads, 2) void tokens_rows_fp4_kernel(TokensArgs a) {
    constexpr int kOut = item_outputs(Side::kGated, 2);
    __shared__ __attribute__((aligned(16))) char scratch[kFewWaves * kScratch<2, XC>];
    __shared__ Part<2> part;
    extern __shared__ __attribute__((aligned(16))) char dynamic[];
    Lists l(a, dynamic);
    l.fill<kFewThreads>(a, XC, scratch);
    if (Side::kFirst && blockIdx.x == 0 && threadIdx.x == 0) *a.status = l.bad ? EP_ERR_BAD_EXPERT : EP_OK;
    const Lanes ll;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int N = Side::outputs(a), K = Side::inputs(a);
    const int nf = N / kOut, items = __builtin_amdgcn_readfirstlane(l.first[__builtin_amdgcn_readfirstlane(l.experts)]) * nf;
    const int share = waves_of_item(items), per = kFewWaves / share;
    for (int g = blockIdx.x; g * per < items; g += gridDim.x) {
        const int item = g * per + wave / share;
        f32x4 acc[2];
        clear(acc);
        const EntryTile t(l, min(item, items - 1), nf, XC);
        const int n0 = t.ft * kOut;
        if (item < items) {
            Rows<2, XC> r;
            set_weights(r, Side::weight(a), Side::scales(a), t.e, Side::weight_rows(a), K, {n0, n0 + (Side::kGated ? N : 16)}, ll);
            r.x = reinterpret_cast<const char *>(Side::x(a));
#pragma unroll
            for (int h = 0; h < XC / 8; ++h) r.x_at[h] = t.x_at<Side>(a, l, h, ll);
            accumulate<2>(acc, r, K, wave % share, share, scratch + wave * kScratch<2, XC>, ll);
        }
        join(acc, part, wave, share);
        if (item < items && wave % share == 0 && ll.li < XC)
            Side::write(a, l, t.e, t.c0 + ll.li, t.m, t.s0, n0, acc[0], acc[1]);
    }
}

template <class Side>
__global__ __launch_bounds__(kManyThreads, 2) void tokens_rows_fp4_many_kernel(TokensArgs a) {
    constexpr int kOut = item_outputs(Side::kGated, 2), kGroup = kManyWaves * kOut;
    __shared__ __attribute__((aligned(16))) char shared[kManyShared], scratch[kManyWaves][4096];
    extern __shared__ __attribute__((aligned(16))) char dynamic[];
    Lists l(a, dynamic);
    l.fill<kManyThreads>(a, kManyColumns, shared);
    if (Side::kFirst && blockIdx.x == 0 && threadIdx.x == 0) *a.status = l.bad ? EP_ERR_BAD_EXPERT : EP_OK;
    const Lanes ll;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int N = Side::outputs(a), K = Side::inputs(a);
    const int nf = (N + kGroup - 1) / kGroup;
    const int items = __builtin_amdgcn_readfirstlane(l.first[__builtin_amdgcn_readfirstlane(l.experts)]) * nf;
    for (int round = 0; round * static_cast<int>(gridDim.x) < items; ++round) {
        const int item = static_cast<int>(tile_of(items, round, blockIdx.x, gridDim.x));
        if (item < 0) break;
        const EntryTile t(l, item, nf, kManyColumns);
        const int place = t.ft * kGroup + wave * kOut, n0 = min(place, N - kOut);
        Rows<2, kManyColumns> r;
        set_weights(r, Side::weight(a), Side::scales(a), t.e, Side::weight_rows(a), K, {n0, n0 + (Side::kGated ? N : 16)}, ll);
        r.x = reinterpret_cast<const char *>(Side::x(a));
#pragma unroll
        for (int h = 0; h < kManyColumns / 8; ++h) r.x_at[h] = t.x_at<Side>(a, l, h, ll);
        f32x4 acc[2][kManyColumns / 16];
        accumulate_columns(acc, r, t.m - t.c0, K, shared, scratch[wave], wave, ll);
        if (place != n0) continue;  // past the last output
#pragma unroll
        for (int c = 0; c < kManyColumns / 16; ++c)
            Side::write(a, l, t.e, t.c0 + c * 16 + ll.li, t.m, t.s0, n0, acc[0][c], acc[1][c]);
    }
}

// down: one workgroup for each 16 outputs, all experts, each wave whole tiles
// of entries in turn, or shares of their k where there are fewer tiles than waves;
// the sums of every token are each wave's own in LDS, joined at the end.  One
// kernel, for few tiles.  (One stream of stages through all of a wave's tiles,
// with its loads ahead across the tiles' ends, takes more instructions a stage:
// a layer of 128 tokens over 256 experts 1340 us, 1270 without.)
template <int NT, int XC>
__global__ __launch_bounds__(NT, 2) void tokens_down_fp4_kernel(TokensArgs a) {
    constexpr int kWaves = NT / 64;
    __shared__ __attribute__((aligned(16))) char scratch[kWaves * kScratch<1, XC>];
    extern __shared__ __attribute__((aligned(16))) char dynamic[];
    Lists l(a, dynamic);
    float *sums = reinterpret_cast<float *>(dynamic + Lists::bytes(a));
    l.fill<NT>(a, XC, scratch);
    const Lanes ll;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16;
    const int size = a.T * 16;  // floats of a wave's sums
    float *mine = sums + wave * size;
    for (int i = __lane_id() * 4; i < size; i += 256) *reinterpret_cast<f32x4 *>(mine + i) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int tiles = __builtin_amdgcn_readfirstlane(l.first[__builtin_amdgcn_readfirstlane(l.experts)]);
    const int shares = tiles >= kWaves ? 1 : tiles ? kWaves / tiles : 1;
    for (int u = wave; u < tiles * shares; u += kWaves) {
        const int t = u / shares, i = __builtin_amdgcn_readfirstlane(l.owner[t]);
        const int e = __builtin_amdgcn_readfirstlane(l.expert[i]);
        const int c0 = (t - __builtin_amdgcn_readfirstlane(l.first[i])) * XC;
        const int s0 = __builtin_amdgcn_readfirstlane(l.begin[i]), m = __builtin_amdgcn_readfirstlane(l.begin[i + 1]) - s0;
        Rows<1, XC> r;
        set_weights(r, a.w2, a.w2_sf, e, a.H, a.I, {n0}, ll);
        r.x = reinterpret_cast<const char *>(a.h);
#pragma unroll
        for (int h = 0; h < XC / 8; ++h)
            r.x_at[h] = static_cast<uint32_t>(l.entry[s0 + min(c0 + h * 8 + ll.row, m - 1)]) * a.I * 2 + (ll.piece ^ h) * 16;
        f32x4 acc[1];
        clear(acc);
        accumulate<2>(acc, r, a.I, u - t * shares, shares, scratch + wave * kScratch<1, XC>, ll);
        if (c0 + ll.li < m && ll.li < XC) {
            const int tok = l.entry[s0 + c0 + ll.li] / a.K;
            *reinterpret_cast<f32x4 *>(mine + tok * 16 + ll.lg * 4) += acc[0];
        }
    }
    __syncthreads();
    down_write<1, NT>(a, l, sums, n0);
}

// The sums of DownRows' rows over the tokens, and what the layer adds to them: a workgroup has kJoinOutputs outputs of a
// token.
constexpr int kJoinThreads = 256, kJoinOutputs = kJoinThreads * 4;
__global__ __launch_bounds__(kJoinThreads) void tokens_join_fp4_kernel(TokensArgs a) {
    const int t = blockIdx.x, n = blockIdx.y * kJoinOutputs + threadIdx.x * 4, j = threadIdx.x & 63;
    const int64_t en = static_cast<int64_t>(t) * a.K;
    const int e = j < a.K ? a.idx[en + j] : -1;
    const bool ok = e >= 0 && e < a.E;
    bool keep = ok;  // the first of the token's entries with its expert has the sum of all
    for (int i = 0; i < a.K; ++i) {
        const int other = __builtin_amdgcn_readlane(e, i);
        keep = keep && (i >= j || other != e);
    }
    const uint64_t kept = __ballot(keep), valid = __ballot(ok);
    if (n >= a.H) return;
    const float *y = a.y + en * a.H + n;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < a.K; j0 += 4) {
        f32x4 r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (kept >> (j0 + i) & 1) r[i] = *reinterpret_cast<const f32x4 *>(y + static_cast<int64_t>(j0 + i) * a.H);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v += r[i];
    }
    if (a.b2) {
        for (uint64_t left = valid; left; left &= left - 1) {
            const int i = __ffsll(static_cast<unsigned long long>(left)) - 1;
            const float w = a.w ? a.w[en + i] : 1.0f;
            v += w * *reinterpret_cast<const f32x4 *>(a.b2 + static_cast<int64_t>(a.idx[en + i]) * a.H + n);
        }
    }
    const int64_t at = static_cast<int64_t>(t) * a.H + n;
    if (a.residual) {
        const u32x2 r = *reinterpret_cast<const u32x2 *>(a.residual + at);
        v += f32x4{bf16_lo(r[0]), bf16_hi(r[0]), bf16_lo(r[1]), bf16_hi(r[1])};
    }
    *reinterpret_cast<u32x2 *>(a.out + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

constexpr int kFp4Workgroups = 256;  // one a CU, which its registers fill

// Eight or sixteen columns a tile: sixteen where an expert has seven or more on average, of which many have more than
// eight.  Layers of 4096 x 2 x 1408, us with eight and with sixteen: 5 an expert, of 32 experts 98 and 105, of 128 307 and
// 322; 6: 103 and 107, 342 and 330; 7: 106 and 109, 370 and 340; 12 of 32 149 and 121.
bool wide_tiles(int64_t entries, int64_t E) { return entries >= 7 * E; }

template <int ACT, int FF, int XC>
hipError_t launch_items(const ProductArgs &a, int64_t tiles, hipStream_t stream) {
    const int64_t items = tiles * (a.N / item_outputs(act_gated(ACT), FF));
    product_fp4_kernel<ACT, FF, XC><<<min(items, int64_t{kFp4Workgroups}), kFewThreads, 0, stream>>>(a);
    return hipGetLastError();
}

// Whether it pays to share columns.  Us without and with it, products of 4096 x 2 x 1408: 7 columns an expert, of 32 experts
// 66 and 57, of 128 194 and 179; but 8 of 8 experts 20.8 and 23.5, for want of workgroups; 16 of 8 experts 36 and 23, of 4
// 17.4 and 22.8.  Layers over 32 experts, 32 tokens 112 and 98, 128 tokens 241 and 146.
bool many(int64_t entries, int64_t E, int64_t outputs, bool gated) {
    const int64_t group = kManyWaves * item_outputs(gated, 2);
    const int64_t items = max(entries / kManyColumns, min(E, entries)) * ((outputs + group - 1) / group);
    return (entries >= 7 * E && items >= 256) || (entries >= 16 * E && items >= 128);
}

// Whether the layer's second product leaves each entry's rows, which a third kernel sums: many tiles are better spread over
// the chip one by one than by outputs, of which there are too few for all CUs, or some more than one each.  Us of layers
// without and with it, of 2048 x 768: 2 tokens of 8 experts 25.1 and 25.1, 4 36.6 and 33.2, 64 tokens over 128 experts 106 and
// 80; of 4672 x 704 over 64 experts 101 and 85, over 256 450 and 360; of 4096 x 1408, with an output tile for each CU, over 64
// experts 134 and 138, over 128 289 and 285; a token of 8 experts 18.2 and 20.2.  Where outputs just fall short of that, 64
// tiles of 3200 x 1408 103 and 102, of 3232 110 and 112 (32 tiles 82 and 86, 89 and 92; 120 tiles 133 and 128, 144 and 139).
// Few tiles of a long k are as many where outputs are few.  A token of 8 experts, of 1024 channels, 64 stages 21.1 and 20.8, 80
// 24.2 and 22.8, 104 28.9 and 25.1; of 2048, 64 stages 23.9 and 24.6, 80 28.9 and 29.5, 104 34.5 and 33.5; of 2080, 104 stages
// 40.6 and 43.6.  Two or three tokens, 96 stages of 2048 channels 34.5 and 33.0, 37.1 and 35.7; of 2080 40.2 and 40.2, 42.7 and 41.4;
// 8 of 2880 x 2880 45.8 and 48.9.
bool rows_apart(int64_t entries, int64_t E, int64_t H, int64_t I) {
    const int64_t tiles = max(min(entries, E), entries / 16), stages = tiles * ((I + kStageK - 1) / kStageK);
    const bool even = H > 16 * 200 && H <= 16 * kFp4Workgroups;
    return many(entries, E, H, false) || tiles >= 128 || (!even && tiles >= 32) || (H <= 16 * 128 && stages >= 80);
}

template <int ACT, int XC>
hipError_t launch_rows(const ProductArgs &a, hipStream_t stream) {
    if (XC == 16 && many(a.entries, a.seg.E, a.N, act_gated(ACT))) {
        product_fp4_many_kernel<ACT><<<2 * kFp4Workgroups, kManyThreads, 0, stream>>>(a);
        return hipGetLastError();
    }
    const int64_t tiles = a.entries / XC + min(static_cast<int64_t>(a.seg.E), a.entries);  // each expert's last in part filled
    if (tiles * (a.N / item_outputs(act_gated(ACT), 2)) < kFp4Workgroups) return launch_items<ACT, 1, XC>(a, tiles, stream);
    return launch_items<ACT, 2, XC>(a, tiles, stream);
}

template <class Side, int XC>
hipError_t launch_tokens_rows(const TokensArgs &a, hipStream_t stream) {
    const int64_t entries = static_cast<int64_t>(a.T) * a.K, tiles = entries / XC + min(int64_t{a.E}, entries);
    const int64_t items = max(int64_t{1}, tiles * (Side::outputs(a) / item_outputs(Side::kGated, 2)));
    tokens_rows_fp4_kernel<Side, XC><<<min(items, int64_t{kFp4Workgroups}), kFewThreads, Lists::bytes(a), stream>>>(a);
    return hipGetLastError();
}

template <class Side>
hipError_t launch_side(const TokensArgs &a, hipStream_t stream) {
    const int64_t entries = static_cast<int64_t>(a.T) * a.K;
    if (many(entries, a.E, Side::outputs(a), Side::kGated)) {
        tokens_rows_fp4_many_kernel<Side><<<2 * kFp4Workgroups, kManyThreads, Lists::bytes(a), stream>>>(a);
        return hipGetLastError();
    }
    return wide_tiles(entries, a.E) ? launch_tokens_rows<Side, 16>(a, stream) : launch_tokens_rows<Side, 8>(a, stream);
}

template <int NT, int XC>
hipError_t launch_down(const TokensArgs &a, hipStream_t stream) {
    tokens_down_fp4_kernel<NT, XC><<<a.H / 16, NT, Lists::bytes(a) + NT / 64 * a.T * 16 * 4, stream>>>(a);
    return hipGetLastError();
}

// Eight waves a workgroup, or four where there are more workgroups than CUs, so that two fit one: one token of 7168
// channels and 8 experts 55.9 and 50.4 us, 9 tokens of 3424 channels 43.0 and 47.5.  Few tiles (rows_apart) are fewer than
// 2048 entries, whose lists, with the sums of 128 tokens and the waves' scratch, take 132 of a CU's 160 KB at most.
template <int XC>
hipError_t launch_down_rows(const TokensArgs &a, hipStream_t stream) {
    return a.H > 16 * kFp4Workgroups ? launch_down<256, XC>(a, stream) : launch_down<512, XC>(a, stream);
}

}  // namespace

hipError_t launch_product_fp4(const ProductArgs &a, hipStream_t stream) {
    const bool wide = wide_tiles(a.entries, a.seg.E);
    switch (a.act) {
#define EP_ACT_CASE(A) \
    case A: return wide ? launch_rows<A, 16>(a, stream) : launch_rows<A, 8>(a, stream);
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

int64_t tokens_fp4_rows_bytes(int32_t T, int32_t K, int32_t E, int32_t H, int32_t I) {
    const int64_t entries = static_cast<int64_t>(T) * K;
    return rows_apart(entries, E, H, I) ? entries * H * 4 : 0;
}

hipError_t launch_tokens_fp4(const TokensArgs &a, hipStream_t stream) {
    hipError_t rc = hipErrorInvalidValue;
    switch (a.act) {
#define EP_ACT_CASE(A) \
    case A: rc = launch_side<UpRows<A>>(a, stream); break;
        EP_ACT_CASE(EP_ACT_NONE)
        EP_ACT_CASE(EP_ACT_RELU)
        EP_ACT_CASE(EP_ACT_GELU)
        EP_ACT_CASE(EP_ACT_SILU)
        EP_ACT_CASE(EP_ACT_SWIGLU)
        EP_ACT_CASE(EP_ACT_GEGLU)
#undef EP_ACT_CASE
        default: break;
    }
    if (rc != hipSuccess || a.T == 0) return rc;
    const int64_t entries = static_cast<int64_t>(a.T) * a.K;
    if (rows_apart(entries, a.E, a.H, a.I)) {
        if ((rc = launch_side<DownRows>(a, stream)) != hipSuccess) return rc;
        const dim3 grid(a.T, (a.H + kJoinOutputs - 1) / kJoinOutputs);
        tokens_join_fp4_kernel<<<grid, kJoinThreads, 0, stream>>>(a);
        return hipGetLastError();
    }
    return wide_tiles(entries, a.E) ? launch_down_rows<16>(a, stream) : launch_down_rows<8>(a, stream);
}

}  // namespace epget
