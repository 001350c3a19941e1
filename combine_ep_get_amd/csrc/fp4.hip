// Products and the few-token layer on MXFP4 weights, for gfx950: e2m1 codes with
// one e8m0 scale for 32 neighbours of a row, and bf16 tokens.
//
//   product: out[r,n] = act(sum_c x[r,c] W[e,n,c] + b[e,n]) + residual[r,n]
//   layer:   h[t,j,:] = bf16(w[t,j] * act(W1[e] x[t] + b1[e])),  e = idx[t,j]
//            out[t,:] = bf16(residual[t,:] + sum_j (W2[e] h[t,j,:] + w[t,j] b2[e]))
//
// Bound by the weights, each read once: 0.53 bytes a value.  A code and its scale
// are widened to bf16 by one instruction for two, exactly, and multiplied by the
// bf16 matrix instruction (its 16 rows are weight rows, its 16 columns tokens).
//
// The matrix instruction's lane l has row l % 16 of a fragment, and the address
// unit joins the accesses of neighbouring lanes only.  Loads in that order take
// it one access a lane; with weights of 4 bits that is the bound (92 % busy at 3.3
// TB/s).  And a load that asks for half a line leaves the next one waiting for
// the same line in the cache (2.8 TB/s).  So eight neighbouring lanes load a
// line of 128 bytes of a row, and the bytes go through LDS, a few KB of each wave's
// own, to the lanes that want them: a wave waits for no other.  The eight 16-byte
// pieces of a line are permuted there by bits of the row, on the side of the
// load's address, so that neither the writes, linear, nor the reads have
// bank conflicts.
//
// A layer of 128 tokens over 256 experts of 7168 x 2048 takes 1260 us in a call, 4.7 TB/s, the rate of a large copy here;
// of one token and 8 experts 45 us (4.2).  100 rows of tokens by 128 experts of 4096 x 2 x 1408: 200 us, 4.0 TB/s.
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

// FULL: no k of the stage is past K, of which there are zeros.
template <bool FULL, int FF, int XC>
__device__ __forceinline__ void load_stage(Stage<FF, XC> &s, const Rows<FF, XC> &r, int b, int K, const Lanes &ll) {
    const int64_t w_off = static_cast<int64_t>(b) * (kStageK / 2), sf_off = static_cast<int64_t>(b) * (kStageK / 32);
    const char *x = r.x + static_cast<int64_t>(b) * (kStageK * 2);
#pragma unroll
    for (int f = 0; f < FF; ++f) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const char *p = r.w[f] + w_off;
            s.w[f][h] = FULL || b * kStageK + (ll.piece ^ h) * 32 < K
                            ? __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + r.w_at[h]))
                            : u32x4{0, 0, 0, 0};
        }
        const char *p = r.sf[f] + sf_off;
        if constexpr (FULL) {
            __builtin_memcpy(&s.sf[f], p + r.sf_at, 4);  // at any address
        } else {
            s.sf[f] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (b * kStageK + ((__lane_id() & 1) * 4 + i) * 32 < K) s.sf[f] |= uint32_t{static_cast<uint8_t>(p[r.sf_at + i])} << 8 * i;
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int h = 0; h < XC / 8; ++h)
            s.x[u][h] = FULL || b * kStageK + u * 64 + (ll.piece ^ h) * 8 < K
                            ? *reinterpret_cast<const u32x4 *>(x + u * 128 + r.x_at[h])
                            : u32x4{0, 0, 0, 0};
}

// Bytes of LDS of a wave: a stage's weights, and half of its k of one fragment of columns.
template <int FF, int XC>
constexpr int kScratch = FF * 2048 + XC / 8 * 2048;

// acc += the stage's products.  A lane's 16 bytes of a weight row are one scale's 32 codes, k = 128 q + 32 lg + 8 i + 0..7
// for matrix instruction i of half q, and the column's operand is read from the same k.
template <int FF, int XC>
__device__ __forceinline__ void use_stage(f32x4 (&acc)[FF], const Stage<FF, XC> &s, char *scratch, const Lanes &ll) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
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
            const u32x4 w = *reinterpret_cast<const u32x4 *>(scratch + f * 2048 + w_row + place_of(ll.li, 4 * q + ll.lg) * 16);
            // e8m0 is fp32's exponent; the conversion takes no other bits of its scale
            const uint32_t four = __builtin_amdgcn_ds_bpermute((ll.li * 4 + q) * 4, s.sf[f]);
            const float scale = __uint_as_float((four >> 8 * ll.lg & 255) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bf16x2 o0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], scale, 0);
                const bf16x2 o1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], scale, 1);
                const bf16x2 o2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], scale, 2);
                const bf16x2 o3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], scale, 3);
                const bf16x8 o = {o0[0], o0[1], o1[0], o1[1], o2[0], o2[1], o3[0], o3[1]};
                acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o, x[i], acc[f], 0, 0, 0);
            }
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

// The entries by expert and their tiles, in LDS that the launch sizes.
struct Lists {
    uint16_t *entry;           // the entries by expert, and room up to a multiple of eight
    uint16_t *owner;           // number in `expert` of each tile
    uint16_t *ordered;
    int16_t *id;               // expert of each entry, -1 for none
    int *end;                  // sort_entries' (by expert)
    int *begin, *first;        // entries and tiles of the experts (with entries) before each
    int *wave_sum;
    uint16_t *expert;          // the experts with entries, ascending
    int &experts, &bad;

    static __host__ __device__ int most(const TokensArgs &a) { return a.E < a.T * a.K ? a.E : a.T * a.K; }
    static __host__ __device__ int room(const TokensArgs &a) { return (a.T * a.K + 7) / 8 * 8; }
    static __host__ __device__ int bytes(const TokensArgs &a) {
        return (room(a) * 8 + a.E * 4 + (most(a) + 1) * 8 + (kFewWaves + 2) * 4 + most(a) * 2 + 15) / 16 * 16;
    }
    __device__ __forceinline__ Lists(const TokensArgs &a, char *p)
        : entry(reinterpret_cast<uint16_t *>(p)), owner(entry + room(a)), ordered(owner + room(a)),
          id(reinterpret_cast<int16_t *>(ordered + room(a))), end(reinterpret_cast<int *>(id + room(a))), begin(end + a.E),
          first(begin + most(a) + 1), wave_sum(first + most(a) + 1), expert(reinterpret_cast<uint16_t *>(wave_sum + kFewWaves + 2)),
          experts(wave_sum[kFewWaves]), bad(wave_sum[kFewWaves + 1]) {}

    // Fills them, tiles being of `width` entries at most.  ORDER: an expert's entries lie in ascending order, which they
    // have to where several workgroups take tiles of them.  Called by the whole workgroup; ends with a barrier.
    template <int NT, bool ORDER>
    __device__ __forceinline__ void fill(const TokensArgs &a, int width) {
        if (a.T * a.K <= 64) {
            if (threadIdx.x < 64) fill_wave(a, width);
            __syncthreads();
            return;
        }
        sort_entries<NT>(a, *this);
        const int per = (experts + NT - 1) / NT;
        const int i0 = min(static_cast<int>(threadIdx.x) * per, experts), i1 = min(i0 + per, experts);
        auto start = [&](int e) { return e ? end[e - 1] : 0; };
        int sum = 0;
        for (int i = i0; i < i1; ++i) sum += (end[expert[i]] - start(expert[i]) + width - 1) / width;
        const int incl = wave_inclusive_sum(sum);
        if ((threadIdx.x & 63) == 63) wave_sum[threadIdx.x >> 6] = incl;
        const int n = experts ? end[expert[experts - 1]] : 0;
        if (ORDER) {  // the sort leaves an expert's entries in the order of its atomics
            for (int p = threadIdx.x; p < n; p += NT) {
                const int v = entry[p], e = id[v], s = start(e), m = end[e] - s;
                int rank = p - s;
                if (m > width) {
                    rank = 0;
                    for (int q = s & ~7; q < s + m; q += 8) {
                        const u32x4 d = *reinterpret_cast<const u32x4 *>(entry + q);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            rank += q + i >= s && q + i < s + m && static_cast<int>(d[i / 2] >> 16 * (i & 1) & 0xFFFF) < v;
                    }
                }
                ordered[s + rank] = static_cast<uint16_t>(v);
            }
            entry = ordered;
        }
        __syncthreads();
        int before = incl - sum;
        for (int w = 0; w < NT / 64; ++w)
            if (w < static_cast<int>(threadIdx.x >> 6)) before += wave_sum[w];
        for (int i = i0; i < i1; ++i) {
            begin[i] = start(expert[i]);
            first[i] = before;
            for (int m = end[expert[i]] - begin[i]; m > 0; m -= width) owner[before++] = static_cast<uint16_t>(i);
        }
        if (threadIdx.x == NT - 1) first[experts] = before, begin[experts] = n;
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

// XC: columns of a tile of entries.
template <int ACT, int XC>
__global__ __launch_bounds__(kFewThreads, 2) void tokens_up_fp4_kernel(TokensArgs a) {
    constexpr bool GATED = act_gated(ACT);
    constexpr int kOut = item_outputs(GATED, 2);
    __shared__ __attribute__((aligned(16))) char scratch[kFewWaves][kScratch<2, XC>];
    __shared__ Part<2> part;
    extern __shared__ __attribute__((aligned(16))) char dynamic[];
    Lists l(a, dynamic);
    l.fill<kFewThreads, true>(a, XC);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = l.bad ? EP_ERR_BAD_EXPERT : EP_OK;
    const Lanes ll;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int experts = __builtin_amdgcn_readfirstlane(l.experts);
    const int nf = a.I / kOut, items = __builtin_amdgcn_readfirstlane(l.first[experts]) * nf;
    const int share = waves_of_item(items), per = kFewWaves / share;
    for (int g = blockIdx.x; g * per < items; g += gridDim.x) {
        const int item = g * per + wave / share;
        f32x4 acc[2];
        clear(acc);
        int e = 0, n0 = 0, c0 = 0, s0 = 0, m = 0;
        if (item < items) {
            const int i = __builtin_amdgcn_readfirstlane(l.owner[item / nf]);
            const int f0 = __builtin_amdgcn_readfirstlane(l.first[i]), nt = __builtin_amdgcn_readfirstlane(l.first[i + 1]) - f0;
            int tt, ft;
            tile_in_expert(item - f0 * nf, nt, nf, &tt, &ft);
            e = __builtin_amdgcn_readfirstlane(l.expert[i]);
            s0 = __builtin_amdgcn_readfirstlane(l.begin[i]), m = __builtin_amdgcn_readfirstlane(l.begin[i + 1]) - s0;
            n0 = ft * kOut, c0 = tt * XC;
            Rows<2, XC> r;
            set_weights(r, a.w1, a.w1_sf, e, a.M, a.H, {n0, GATED ? a.I + n0 : n0 + 16}, ll);
            r.x = reinterpret_cast<const char *>(a.x);
#pragma unroll
            for (int h = 0; h < XC / 8; ++h)
                r.x_at[h] = static_cast<uint32_t>(l.entry[s0 + min(c0 + h * 8 + ll.row, m - 1)] / a.K) * a.H * 2 + (ll.piece ^ h) * 16;
            accumulate<2>(acc, r, a.H, wave % share, share, scratch[wave], ll);
        }
        join(acc, part, wave, share);
        if (item < items && wave % share == 0 && ll.li < XC) {
            up_write<ACT>(a, l, e, c0 + ll.li, m, s0, n0, acc[0], acc[1]);
            if (!GATED) up_write<ACT>(a, l, e, c0 + ll.li, m, s0, n0 + 16, acc[1], acc[1]);
        }
    }
}

// down: one workgroup for each 16 outputs, all experts, each wave whole tiles
// of entries in turn, or shares of their k where there are fewer tiles than waves;
// the sums of every token are each wave's own in LDS, joined at the end.  (One
// stream of stages through all of a wave's tiles, with its loads ahead across the
// tiles' ends, takes more instructions a stage: 128 tokens of 256 experts 1340
// us, 1270 without.)
template <int NT, int XC>
__global__ __launch_bounds__(NT, 2) void tokens_down_fp4_kernel(TokensArgs a) {
    constexpr int kWaves = NT / 64;
    __shared__ __attribute__((aligned(16))) char scratch[kWaves][kScratch<1, XC>];
    extern __shared__ __attribute__((aligned(16))) char dynamic[];
    Lists l(a, dynamic);
    float *sums = reinterpret_cast<float *>(dynamic + Lists::bytes(a));
    l.fill<NT, false>(a, XC);  // a workgroup's own
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
        accumulate<2>(acc, r, a.I, u - t * shares, shares, scratch[wave], ll);
        if (c0 + ll.li < m && ll.li < XC) {
            const int tok = l.entry[s0 + c0 + ll.li] / a.K;
            *reinterpret_cast<f32x4 *>(mine + tok * 16 + ll.lg * 4) += acc[0];
        }
    }
    __syncthreads();
    down_write<1, NT>(a, l, sums, n0);
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

template <int ACT, int XC>
hipError_t launch_rows(const ProductArgs &a, hipStream_t stream) {
    const int64_t tiles = a.entries / XC + min(static_cast<int64_t>(a.seg.E), a.entries);  // each expert's last in part filled
    if (tiles * (a.N / item_outputs(act_gated(ACT), 2)) < kFp4Workgroups) return launch_items<ACT, 1, XC>(a, tiles, stream);
    return launch_items<ACT, 2, XC>(a, tiles, stream);
}

template <int ACT, int XC>
hipError_t launch_up(const TokensArgs &a, hipStream_t stream) {
    const int64_t entries = static_cast<int64_t>(a.T) * a.K, tiles = entries / XC + min(int64_t{a.E}, entries);
    const int64_t items = max(int64_t{1}, tiles * (a.I / item_outputs(act_gated(ACT), 2)));
    tokens_up_fp4_kernel<ACT, XC><<<min(items, int64_t{kFp4Workgroups}), kFewThreads, Lists::bytes(a), stream>>>(a);
    return hipGetLastError();
}

template <int NT, int XC>
hipError_t launch_down(const TokensArgs &a, hipStream_t stream) {
    tokens_down_fp4_kernel<NT, XC><<<a.H / 16, NT, Lists::bytes(a) + NT / 64 * a.T * 16 * 4, stream>>>(a);
    return hipGetLastError();
}

// Eight waves a workgroup, or four where there are more workgroups than CUs, so that two fit one: one token of 7168
// channels and 8 experts 55.9 and 50.4 us, 9 tokens of 3424 channels 43.0 and 47.5.  32 outputs a workgroup were no faster
// with 128 tokens (1275 and 1278 us).
template <int XC>
hipError_t launch_down_rows(const TokensArgs &a, hipStream_t stream) {
    const bool fits = Lists::bytes(a) + kFewWaves * (kScratch<1, XC> + a.T * 16 * 4) <= 160 * 1024;  // a CU's LDS
    return a.H > 16 * kFp4Workgroups || !fits ? launch_down<256, XC>(a, stream) : launch_down<512, XC>(a, stream);
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

hipError_t launch_tokens_fp4(const TokensArgs &a, hipStream_t stream) {
    hipError_t rc = hipErrorInvalidValue;
    const bool wide = wide_tiles(static_cast<int64_t>(a.T) * a.K, a.E);
    switch (a.act) {
#define EP_ACT_CASE(A) \
    case A: rc = wide ? launch_up<A, 16>(a, stream) : launch_up<A, 8>(a, stream); break;
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
    return wide ? launch_down_rows<16>(a, stream) : launch_down_rows<8>(a, stream);
}

}  // namespace epget
