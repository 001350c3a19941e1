// Grouped matrix products over the experts' rows, for gfx950.
//
//   forward      out[r,n] = act(sum_c x[r,c] W[e,n,c] + b[e,n]) + residual[r,n]
//   grad input   dx[r,c]  = sum_m dpre[r,m] W[e,m,c]
//   grad weight  dW[e,m,c] = sum_{r of e} dpre[r,m] x[r,c]
//
// All three are one tiled product D[feature, token] = sum_k P[feature, k]
// Q[token, k] on the matrix cores.  "Features" are the contiguous dimension
// of the result, so that a lane's four results of a 16x16 tile are four
// neighbours of one row: P is the weight (forward, grad input) or x (grad
// weight), Q is x or dpre; the tokens of grad weight are the weight's rows m.
// An operand whose rows are contiguous in k is read from LDS in 16-byte
// pieces; one whose rows are contiguous in the other dimension is read with
// the transposing LDS loads, so nothing is transposed in memory.
//
// Tiles come from global memory straight to LDS, 16 bytes a lane, in two
// buffers.  A lane always writes 16 bytes at lane * 16, so the swizzle that
// keeps LDS reads free of bank conflicts is applied to the address that the
// lane reads.  Rows past the segment or the operand's end are read as its
// last one (always in bounds) and never stored; a k that is no multiple of the
// step begins with a part step, through registers, with zeros in its other places.
//
// Bound by the matrix units and their power: 16384 x 7168 x 4096, with SwiGLU or
// without, takes 690-730 us (1.3-1.4 PFLOP/s; the library's plain product of
// that size 1.29-1.35), 30 us more with `pre` written, its gradients 710-760
// and 770-830 us, and in FP8 560-595 us (1.6-1.7 PFLOP/s).  With fewer rows
// the weights' traffic bounds it: 64 experts of 64 x 4096 x 4096 in 470-480 us (4.5-4.7 TB/s).
// A ring of four buffers of 32 k, three of them on their way, was no faster: what
// waits there is not the loads.  launch_sized chooses among three tile sizes.
#include <type_traits>

#include "product_device.h"

namespace epget {
namespace {

enum Mode { kForward, kGradInput, kGradWeight };

constexpr int kStepBytes = 128;  // of k per row and step: 64 bf16 or 128 e4m3
constexpr int kStepRows = 64;    // k rows per step of an operand contiguous in the other dimension

typedef __attribute__((address_space(3))) char lds_char;

// The lane, as a value that the compiler does not know to be the same
// everywhere: what is derived from it is computed where it is used instead of
// being kept through the k loop.  That loop's registers are all taken, and one
// address spilled in it is reloaded through the counter that the loads to
// LDS are waited for with (29 reloads a step cost the grad input 5 %).
__device__ __forceinline__ int fresh_lane() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// The operand tile of B rows (contiguous in k) or B columns (not: kStrided)
// in LDS, B * 128 bytes either way.  kWide (P): two fragments of 16 features
// share 32 neighbours, fragment f's row r being feature 8 (r / 4) + 4 (f & 1) +
// r % 4 of them, so that a lane's results of both are eight in a row.
template <int B, bool kStrided, bool kWide>
struct Tile {
    static constexpr int kPitch = kStrided ? B * 2 : kStepBytes;
    // Strided: 2^kShift chunks of 16 bytes move together (32 columns if wide,
    // else 16), their place permuted by bits of the row so that the 16 rows
    // that one transposing load touches lie evenly in the banks.
    static constexpr int kShift = kWide ? 2 : 1;
    static __device__ __forceinline__ int mix(int row) {
        const int key = kWide ? (row & 3) ^ (row >> 3 & 1) << 1 : (row & 3) | (row >> 3 & 3) << 2;
        return key & ((B >> (kShift + 3)) - 1);
    }

    // Row of the tile, and the 16-byte chunk of that row, that LDS byte `at` holds.
    static __device__ __forceinline__ void source(int at, int *row, int *chunk) {
        *row = at / kPitch;
        const int pos = (at % kPitch) / 16;
        *chunk = kStrided ? ((pos >> kShift) ^ mix(*row)) << kShift | (pos & ((1 << kShift) - 1)) : pos ^ (*row & 7);
    }

    // Fragments f and f + 1 (f even), k from 32 * ks on: lane l holds row l & 15
    // and k = (l >> 4) * 8 .. + 7.
    static __device__ __forceinline__ void pair(const char *lds, int lane, int f, int ks, bf16x8 &f0, bf16x8 &f1) {
        const int i = lane & 15, g = lane >> 4;
        if constexpr (kStrided) {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            union {
                s16x4 half[2];
                bf16x8 all;
            } u[2];
            // A load takes 4 rows of k and, of each, 4 columns a lane of four
            // lanes; lane i of 16 receives column i of the 4 rows.
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = g * 8 + (i >> 2);  // + 32 ks + 4 j, which mix does not see
                const char *at = lds + (row + 32 * ks + 4 * j) * kPitch;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = kWide ? (((f >> 1) ^ mix(row)) << 6) + (i & 3) * 16 + h * 8
                                        : (((f + h) ^ mix(row)) << 5) + (i & 3) * 8;
                    u[h].half[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(at + c));
                }
            }
            f0 = u[0].all;
            f1 = u[1].all;
        } else {
            const int chunk = ((ks * 4 + g) ^ (i & 7)) << 4;
            f0 = *reinterpret_cast<const bf16x8 *>(lds + (16 * f + i) * kPitch + chunk);
            f1 = *reinterpret_cast<const bf16x8 *>(lds + (16 * f + 16 + i) * kPitch + chunk);
        }
    }

    static __device__ __forceinline__ bf16x8 fragment(const char *lds, int lane, int f, int ks) {
        if constexpr (!kStrided)
            return *reinterpret_cast<const bf16x8 *>(lds + (16 * f + (lane & 15)) * kPitch +
                                                     (((ks * 4 + (lane >> 4)) ^ (lane & 7)) << 4));
        bf16x8 a, b;
        pair(lds, lane, f & ~1, ks, a, b);  // the reads of the other one are dropped
        return f & 1 ? b : a;
    }
};

// What a workgroup knows of one operand of its tile: the uniform base
// address, each lane's offsets from it, and the bytes from step to step.
template <int B, bool kStrided, bool kWide, int NW>
struct Operand {
    static constexpr int kLoads = B * kStepBytes / (NW * 1024);
    const char *base;
    uint32_t off[kLoads];
    int64_t step;

    static __device__ __forceinline__ int lds_at(int i) {
        return (i * NW + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 1024;
    }

    // The next step's tile.  The base is kept in scalar registers and opaque,
    // so that each load is one instruction of base and 32-bit offset; the
    // compiler would otherwise carry a 64-bit address a lane and load.
    template <int N = kLoads>
    __device__ __forceinline__ void load(char *lds) {
        asm volatile("" : "+s"(base));
#pragma unroll
        for (int i = 0; i < N; ++i)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(base + off[i]),
                                             (__attribute__((address_space(3))) void *)(lds + lds_at(i)), 16, 0, 0);
        base += step;
    }

    // A first step of `left` k only (bytes if contiguous in k, rows if not),
    // with zeros in its other places.
    __device__ __forceinline__ void load_part(char *lds, int left) {
        const int lane = fresh_lane();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = lds_at(i) + lane * 16;
            int row, chunk;
            Tile<B, kStrided, kWide>::source(at, &row, &chunk);
            u32x4 v = {0, 0, 0, 0};
            if ((kStrided ? row : chunk * 16) < left) v = *reinterpret_cast<const u32x4 *>(base + off[i]);
            *reinterpret_cast<u32x4 *>(lds + at) = v;
        }
        base += kStrided ? step / kStepRows * left : left;
    }
};

__device__ __forceinline__ void wait_loads_and_sync() {
    __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);  // this wave's loads to LDS have landed
    __syncthreads();
}

// The weight row that LDS row lr (fragment lr / 16) holds in the forward
// product.  With a gated activation the fragments alternate between the
// gate's rows and the other half's, so that one lane holds both values of an
// output.  Two fragments of outputs share 32 neighbours so that a lane's four
// of each, 8 lg + 4 j + 0..3, are eight in a row: they are stored as 16
// bytes, and the four lanes of a token as 64.
template <bool GATED>
__device__ __forceinline__ int weight_row(int lr, int n0, int N) {
    const int f = lr >> (GATED ? 5 : 4), r = lr & 15;
    const int n = min(n0 + (f >> 1) * 32 + (r >> 2) * 8 + (f & 1) * 4 + (r & 3), N - 1);
    return GATED && (lr >> 4 & 1) ? N + n : n;
}

// Calls f with the constant `live`, 1 to N.
template <int N, class F>
__device__ __forceinline__ void accumulate_fewer(int live, F &f) {
    if constexpr (N > 0) {
        if (live == N)
            f(std::integral_constant<int, N>{});
        else
            accumulate_fewer<N - 1>(live, f);
    }
}

template <int MODE, int ACT, bool FP8, int WF, int WT, int FF, int TF, class Args>
__global__ __launch_bounds__(64 * WF * WT, 2) void product_kernel(Args a) {
    constexpr int NT = 64 * WF * WT, NW = WF * WT;
    constexpr int BF = WF * FF * 16, BT = WT * TF * 16;
    constexpr bool kPs = MODE != kForward, kQs = MODE == kGradWeight;
    constexpr bool GATED = MODE == kForward && act_gated(ACT);
    constexpr int BN = GATED ? BF / 2 : BF;  // outputs of a tile
    constexpr int EL = FP8 ? 1 : 2;
    __shared__ __attribute__((aligned(1024))) char p0[BF * kStepBytes], q0[BT * kStepBytes];
    __shared__ __attribute__((aligned(1024))) char p1[BF * kStepBytes], q1[BT * kStepBytes];
    __shared__ int first[MODE == kGradWeight ? 1 : EP_MAX_EXPERTS + 1];
    __shared__ int wave_sum[NW];

    const int F = MODE == kForward ? a.N : a.C;  // features
    const int nf = (F + BN - 1) / BN;
    const int nt_w = (a.M + BT - 1) / BT;  // grad weight: row tiles of a weight
    int64_t total;
    if constexpr (MODE == kGradWeight) {
        total = static_cast<int64_t>(a.seg.E) * nt_w * nf;
    } else {
        tile_prefix<NT>(a.seg, BT, first, wave_sum);
        total = static_cast<int64_t>(first[a.seg.E]) * nf;
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wf = wave % WF, wt = wave / WF;
    const int G = gridDim.x;

    for (int64_t round = 0; round * G < total; ++round) {
        const int64_t tile = tile_of(total, round, blockIdx.x, G);
        if (tile < 0) break;
        int e, tt, ft;
        if constexpr (MODE == kGradWeight) {
            const int64_t per = static_cast<int64_t>(nt_w) * nf;
            e = static_cast<int>(tile / per);
            tile_in_expert(tile - e * per, nt_w, nf, &tt, &ft);
        } else {
            e = tile_expert(first, a.seg.E, static_cast<int>(tile / nf));
            const int f0 = __builtin_amdgcn_readfirstlane(first[e]);
            const int nt = __builtin_amdgcn_readfirstlane(first[e + 1]) - f0;
            tile_in_expert(tile - static_cast<int64_t>(f0) * nf, nt, nf, &tt, &ft);
        }
        int64_t row0;
        const int rows = segment(a.seg, e, &row0);
        const int n0 = ft * BN;  // first feature
        // The tokens are spread evenly over the tiles: each wave computes
        // `live` of its TF fragments of 16, the same number in all tiles.
        // Experts of 512 rows on average have 3 tiles of 256 as often as 2,
        // the third nearly empty.
        const int tokens = MODE == kGradWeight ? a.M : rows;
        const int tiles = (tokens + BT - 1) / BT;
        const int live = ((tokens + tiles - 1) / tiles + WT * 16 - 1) / (WT * 16);
        const int t0 = tt * live * (WT * 16);  // first token of the segment, or weight row
        if (t0 >= tokens) continue;            // rounded up, the tiles before hold all of them

        const int setup_lane = fresh_lane();
        Operand<BF, kPs, true, NW> p;
        Operand<BT, kQs, false, NW> q;
        int64_t k_total;  // in bytes, or in rows for grad weight
        if constexpr (MODE == kForward) {
            k_total = static_cast<int64_t>(a.C) * EL;
            p.base = static_cast<const char *>(a.weight) + static_cast<int64_t>(e) * a.M * a.C * EL;
            q.base = static_cast<const char *>(a.x) + (row0 + t0) * a.C * EL;
            p.step = q.step = kStepBytes;
        } else if constexpr (MODE == kGradInput) {
            k_total = static_cast<int64_t>(a.M) * 2;
            p.base = reinterpret_cast<const char *>(a.weight) + static_cast<int64_t>(e) * a.M * a.C * 2;
            q.base = reinterpret_cast<const char *>(a.dpre) + (row0 + t0) * a.M * 2;
            p.step = static_cast<int64_t>(kStepRows) * a.C * 2;
            q.step = kStepBytes;
        } else {
            k_total = rows;
            p.base = reinterpret_cast<const char *>(a.x) + row0 * a.C * 2;
            q.base = reinterpret_cast<const char *>(a.dpre) + row0 * a.M * 2;
            p.step = static_cast<int64_t>(kStepRows) * a.C * 2;
            q.step = static_cast<int64_t>(kStepRows) * a.M * 2;
        }
#pragma unroll
        for (int i = 0; i < p.kLoads; ++i) {
            int row, chunk;
            Tile<BF, kPs, true>::source(p.lds_at(i) + setup_lane * 16, &row, &chunk);
            if constexpr (kPs)  // rows of k, columns of features
                p.off[i] = static_cast<uint32_t>(row) * (a.C * 2) + min(n0 * 2 + chunk * 16, a.C * 2 - 16);
            else
                p.off[i] = static_cast<uint32_t>(weight_row<GATED>(row, n0, a.N)) * (a.C * EL) + chunk * 16;
        }
#pragma unroll
        for (int i = 0; i < q.kLoads; ++i) {
            int row, chunk;
            Tile<BT, kQs, false>::source(q.lds_at(i) + setup_lane * 16, &row, &chunk);
            if constexpr (kQs)
                q.off[i] = static_cast<uint32_t>(row) * (a.M * 2) + min(t0 * 2 + chunk * 16, a.M * 2 - 16);
            else
                q.off[i] = static_cast<uint32_t>(min(row, rows - 1 - t0)) * (MODE == kForward ? a.C * EL : a.M * 2) +
                           chunk * 16;
        }

        f32x4 acc[FF][TF];
#pragma unroll
        for (int f = 0; f < FF; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t) acc[f][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        // FP8: the scales of this wave's tokens (one a lane and fragment) and
        // features (one for each half: outputs are whole blocks of 128)
        const float *sf_row[TF], *sf_w[2] = {nullptr, nullptr};
        if constexpr (FP8) {
#pragma unroll
            for (int t = 0; t < TF; ++t)
                sf_row[t] = a.x_sf + (row0 + min(t0 + (wt * live + t) * 16 + (setup_lane & 15), rows - 1)) * a.sf_ts;
            const int kb = a.C / 128;
            // the wave's first output; past N in a tile's unused part
            const int nw = min(n0 + wf * (GATED ? FF * 8 : FF * 16), a.N - 1);
            sf_w[0] = a.w_sf + (static_cast<int64_t>(e) * (a.M / 128) + nw / 128) * kb;
            sf_w[1] = GATED ? sf_w[0] + static_cast<int64_t>(a.N / 128) * kb : sf_w[0];
        }
        struct Scales {
            float x[TF], w[2];
        } sa, sb;
        // The tokens' scales come four blocks at a time, a lane of each token
        // one of them (with a load a block, the lines that they lie in made half of the L2's
        // requests); a step takes its block's by permuting the lanes.
        float sx[TF], sx_next[TF];
        auto load_scales = [&](int s) {
            if constexpr (FP8) {
                const int at = min(s + (fresh_lane() >> 4), a.C / 128 - 1);
#pragma unroll
                for (int t = 0; t < TF; ++t) sx_next[t] = sf_row[t][at * a.sf_hs];
            }
        };
        auto read_scales = [&](Scales &to, int s) {
            if constexpr (FP8) {
                if ((s & 3) == 0) {
#pragma unroll
                    for (int t = 0; t < TF; ++t) sx[t] = sx_next[t];
                    load_scales(s + 4);
                }
                const int from = ((fresh_lane() & 15) + 16 * (s & 3)) * 4;
#pragma unroll
                for (int t = 0; t < TF; ++t)
                    to.x[t] = __int_as_float(__builtin_amdgcn_ds_bpermute(from, __float_as_int(sx[t])));
                typedef const __attribute__((address_space(4))) float *constant;  // read by the scalar unit
                to.w[0] = ((constant)sf_w[0])[s];
                to.w[1] = ((constant)sf_w[1])[s];
            }
        };

        const int lane = fresh_lane();
        auto accumulate = [&](auto live_fragments) {
            constexpr int TA = live_fragments();
            // A step is computed in phases of half of P's fragments, each with 32
            // k (bf16: four phases) or all 128 k (FP8: two).  Each phase's
            // fragments are read from LDS while the phase before it multiplies.
            constexpr int PF = FF / 2, KS = FP8 ? 2 : 1;
            union Frag {
                bf16x8 part[KS];
                i32x8 all;  // FP8
            };
            struct PFrags {
                Frag f[PF];
            } pa, pb;
            struct QFrags {
                Frag t[TF];
            } qa, qb;
            auto read_p = [&](PFrags &h, const char *pl, int ks, int half) {
#pragma unroll
                for (int f = 0; f < PF; f += 2)
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        Tile<BF, kPs, true>::pair(pl, lane, wf * FF + half * PF + f, FP8 ? k : ks, h.f[f].part[k],
                                                  h.f[f + 1].part[k]);
            };
            auto read_q = [&](QFrags &h, const char *ql, int ks) {
#pragma unroll
                for (int t = 0; t < TA; ++t)
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        h.t[t].part[k] = Tile<BT, kQs, false>::fragment(ql, lane, wt * TA + t, FP8 ? k : ks);
            };
            auto multiply = [&](const PFrags &pf, const QFrags &qf, const Scales &sc, int half) {
                if constexpr (FP8) {
                    // A block's products are scaled in fp32 while the matrix unit
                    // does the next fragment's: left to itself, the compiler waits for
                    // each product and scales it at once.  The instruction aligns a
                    // block's 128 products to the largest before it adds them (8.7e-5 of
                    // the sum of their magnitudes at most was lost); widened to bf16, which
                    // loses nothing, the codes would multiply at half the rate.
                    f32x4 d[2][TA];
#pragma unroll
                    for (int f = 0; f <= PF; ++f) {
#pragma unroll
                        for (int t = 0; t < TA; ++t) {
                            const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                            if (f < PF)  // block scales of one (127 is 2^0)
                                d[f & 1][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                    pf.f[f].all, qf.t[t].all, zero, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
                            if (f > 0) {
                                const float scale = sc.x[t] * sc.w[GATED ? (f - 1) & 1 : 0];
                                f32x4 &to = acc[half * PF + f - 1][t];
#pragma unroll
                                for (int r = 0; r < 4; ++r) to[r] = __builtin_fmaf(d[(f - 1) & 1][t][r], scale, to[r]);
                                __builtin_amdgcn_sched_barrier(0);
                            }
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } else {
#pragma unroll
                    for (int f = 0; f < PF; ++f)
#pragma unroll
                        for (int t = 0; t < TA; ++t)
                            acc[half * PF + f][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                pf.f[f].part[0], qf.t[t].part[0], acc[half * PF + f][t], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);  // phases stay apart: 16 % slower without
                }
            };

            // A part step comes first, if k is no multiple of the step.
            constexpr int kUnit = MODE == kGradWeight ? kStepRows : kStepBytes;
            const int full = static_cast<int>(k_total / kUnit);
            const int left = static_cast<int>(k_total - static_cast<int64_t>(full) * kUnit);
            // The loop takes two steps a round, one a buffer: an odd number of
            // steps has one of zeros before it, whose products pass while the
            // first loads are on their way.
            const int steps = full + (left > 0), pad = steps & 1, total_steps = steps + pad;
            auto fetch = [&](char *pl, char *ql) {
                p.load(pl);
                // the loads of the live rows: 8 a wave and load
                q.template load<kQs ? q.kLoads : (WT * TA * 2 + NW - 1) / NW>(ql);
            };
            // One step, with Q's first fragments in q0f: when every wave has read
            // all of this buffer and the next step's loads have landed, the loads
            // of the step after that start into this buffer, and the next step's
            // first fragments are read into q1f (FP8) or q0f during the last phase.
            auto step = [&](char *pl, char *ql, char *pn, char *qn, QFrags &q0f, QFrags &q1f, const Scales &sc, Scales &next,
                            int s, auto fetch_more, auto more) {
                if constexpr (more()) read_scales(next, s + 1 - pad);  // waited for with the loads to LDS
                read_p(pb, pl, 0, 1);
                multiply(pa, q0f, sc, 0);
                if constexpr (!FP8) {
                    read_q(q1f, ql, 1);
                    read_p(pa, pl, 1, 0);
                    multiply(pb, q0f, sc, 1);
                    read_p(pb, pl, 1, 1);
                    multiply(pa, q1f, sc, 0);
                }
                if constexpr (more()) {
                    wait_loads_and_sync();
                    if constexpr (fetch_more()) fetch(pl, ql);
                    read_q(FP8 ? q1f : q0f, qn, 0);
                    read_p(pa, pn, 0, 0);
                }
                multiply(pb, FP8 ? q0f : q1f, sc, 1);
            };
            constexpr std::true_type yes{};
            constexpr std::false_type no{};
            if (total_steps > 0) {
                __syncthreads();  // the previous tile's readers are done
                auto first_step = [&](char *pl, char *ql) {
                    if (left > 0) {
                        // k of grad input is bytes of dpre, rows of the weight
                        p.load_part(pl, MODE == kGradInput ? left / 2 : left);
                        q.load_part(ql, left);
                    } else {
                        fetch(pl, ql);
                    }
                };
                load_scales(0);
                if (pad) {
                    if constexpr (FP8) {
#pragma unroll
                        for (int t = 0; t < TF; ++t) sa.x[t] = 0.0f;
                        sa.w[0] = sa.w[1] = 0.0f;
                    }
                    p.load_part(p0, 0);
                    q.load_part(q0, 0);
                    first_step(p1, q1);
                    __syncthreads();
                } else {
                    first_step(p0, q0);
                    wait_loads_and_sync();
                    read_scales(sa, 0);
                    fetch(p1, q1);
                }
                read_q(qa, q0, 0);
                read_p(pa, p0, 0, 0);
                int s = 0;
                for (; s + 2 < total_steps; s += 2) {
                    step(p0, q0, p1, q1, qa, qb, sa, sb, s, yes, yes);
                    step(p1, q1, p0, q0, FP8 ? qb : qa, FP8 ? qa : qb, sb, sa, s + 1, yes, yes);
                }
                step(p0, q0, p1, q1, qa, qb, sa, sb, s, no, yes);
                step(p1, q1, p0, q0, FP8 ? qb : qa, FP8 ? qa : qb, sb, sa, s + 1, no, no);
            }
        };
        if (live == TF) {
            accumulate(std::integral_constant<int, TF>{});
        } else {
            accumulate_fewer<TF - 1>(live, accumulate);
        }

        // Epilogue: lane holds, of fragments (f, t) and (f + 1, t), token li
        // and eight neighbouring features.
        const int out_lane = fresh_lane(), li = out_lane & 15, lg = out_lane >> 4;
#pragma unroll
        for (int t = 0; t < TF; ++t) {
            const int tok = t0 + (wt * live + t) * 16 + li;
            if (t >= live || tok >= tokens) continue;
            if constexpr (MODE == kForward) {
                const int64_t r = row0 + tok;
#pragma unroll
                for (int f = 0; f < FF; f += GATED ? 4 : 2) {
                    const int n = n0 + (GATED ? (wf * FF + f) / 2 : wf * FF + f) * 16 + lg * 8;
                    if (n >= a.N) continue;
                    f32x4 v[2] = {acc[f][t], acc[f + (GATED ? 2 : 1)][t]};
                    f32x4 u[2] = {acc[f + 1][t], acc[f + (GATED ? 3 : 1)][t]};
                    write_outputs<ACT>(a, e, r, n, v, u);
                }
            } else {
                const int64_t at = (MODE == kGradInput ? row0 + tok : static_cast<int64_t>(e) * a.M + tok) * a.C;
#pragma unroll
                for (int f = 0; f < FF; f += 2) {
                    const int c = n0 + (wf * FF + f) * 16 + lg * 8;
                    if (c >= a.C) continue;
                    const f32x4 v[2] = {acc[f][t], acc[f + 1][t]};
                    if constexpr (MODE == kGradInput) {
                        store_bf16(a.dx + at + c, v);
                    } else {
                        // not read again soon: streamed past the caches that
                        // hold x and dpre (32 x 2816 x 4096 of 512 rows 487 -> 432 us)
                        if (a.dweight)
                            __builtin_nontemporal_store(pack_bf16(v), reinterpret_cast<u32x4 *>(a.dweight + at + c));
                        if (a.dweight_acc) {
                            f32x4 *to = reinterpret_cast<f32x4 *>(a.dweight_acc + at + c);
                            to[0] += v[0];
                            to[1] += v[1];
                        }
                    }
                }
            }
        }
    }
}

// dpre = dout * act'(pre), and the column sums of dpre in fp32, before it is
// rounded, for the bias gradient.  dpre is rounded to bf16 once, as the matrix
// instructions of both products take it (in fp32 they would run at a sixteenth of the rate
// and read twice the bytes); the gradients are off by 0.0023 of their size for it, where the
// rounding of the results alone gives 0.0017.  One workgroup takes a range of an
// expert's rows and 256 columns of dout: 32 lanes of 8 columns, 8 rows at a time.
constexpr int kGradColumns = 256;
constexpr int kGradRowLanes = 8;
// Workgroups aimed at, by cutting the experts' rows into ranges: with one
// range, the rows of a popular expert pass 8 at a time through 6 workgroups (161 us
// of a 1000-token batch's 485).
constexpr int kGradWorkgroups = 4096;

__device__ __forceinline__ void unpack8(const uint16_t *p, float v[8]) {
    const u32x4 u = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = bf16_lo(u[q]);
        v[2 * q + 1] = bf16_hi(u[q]);
    }
}

__device__ __forceinline__ void pack8(uint16_t *p, const float v[8]) {
    *reinterpret_cast<u32x4 *>(p) =
        u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

template <int ACT>
__global__ __launch_bounds__(256) void act_grad_kernel(ProductGradArgs a) {
    constexpr bool GATED = act_gated(ACT);
    constexpr int kHalves = GATED ? 2 : 1;
    __shared__ float sums[kGradRowLanes][kGradColumns];
    const int e = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
    int64_t row0;
    const int rows = segment(a.seg, e, &row0);
    const int per = (rows + a.splits - 1) / a.splits;
    const int r0 = static_cast<int>(min(static_cast<int64_t>(split) * per, static_cast<int64_t>(rows)));
    const int r1 = min(r0 + per, rows);
    const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int n = blockIdx.y * kGradColumns + lane * 8;
    float sum[kHalves][8] = {};
    if (n < a.N) {
        for (int r = r0 + rl; r < r1; r += kGradRowLanes) {
            const int64_t row = row0 + r;
            float d[8], v[8], u[8];
            unpack8(a.dout + row * a.N + n, d);
            if constexpr (ACT != EP_ACT_NONE) {
                unpack8(a.pre + row * a.M + n, v);
                if (GATED) unpack8(a.pre + row * a.M + a.N + n, u);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float slope = act_slope<ACT>(v[i]);
                    if (GATED) {
                        const float du = d[i] * act_one<ACT>(v[i]);
                        d[i] = d[i] * u[i] * slope;
                        u[i] = du;
                    } else {
                        d[i] *= slope;
                    }
                }
                pack8(a.dpre + row * a.M + n, d);
                if (GATED) pack8(a.dpre + row * a.M + a.N + n, u);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum[0][i] += d[i];
                if (GATED) sum[kHalves - 1][i] += u[i];
            }
        }
    }
    if (!a.dbias) return;
    const int col = blockIdx.y * kGradColumns + threadIdx.x;
    float *to = a.splits > 1 ? a.partial + static_cast<int64_t>(blockIdx.x) * a.M : a.dbias + static_cast<int64_t>(e) * a.M;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[rl][lane * 8 + i] = sum[h][i];
        __syncthreads();
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < kGradRowLanes; ++i) total += sums[i][threadIdx.x];
        if (col < a.N) to[h * a.N + col] = total;
    }
}

// dbias[e,m]: the row ranges' partial sums, in order.
__global__ __launch_bounds__(256) void bias_join_kernel(const float *__restrict__ partial, float *__restrict__ dbias,
                                                        int64_t n, int32_t M, int32_t splits) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t e = i / M, m = i - e * M;
    float sum = 0.0f;
    for (int s = 0; s < splits; ++s) sum += partial[(e * splits + s) * M + m];
    dbias[i] = sum;
}

constexpr int kCUs = 256;
// Tiles from which the larger sizes are taken.  Up to 128 tiles of 128 x 128 four
// times as many of 64 x 64 all run at once: 200 x 2048 x 2048 (32 tiles) takes 11.7 us
// and 19.0 in the larger, but 1280 x 2048 x 2048 (176) 32.8 and 24.0, in FP8 18.9
// either way; at the limit itself the forward product would still gain (500 x 4096
// x 4096: 34.7 and 41.0, FP8 22.3 and 30.9) and the weight gradient lose (16384 x
// 512 x 4096: 152 and 140).  256 x 256, one workgroup a CU, needs nearly a tile for
// each: 2048 x 2048 x 2048 takes 25.7 us in 128 x 128 and 44.5 in its 64 (counted as
// 72), grad input of 16384 x 4096 x 512 62.6 and 86.4 in 128, but 16384 x 7168 x
// 4096 841 and 690.
constexpr int kMediumTiles = 128, kLargeTiles = 192;

// Tiles of a product in the worst case, each expert's last one in part filled.
template <int MODE, class Args>
int64_t most_tiles(const Args &a, int64_t BF, int64_t BT) {
    const int64_t nf = ((MODE == kForward ? a.M : a.C) + BF - 1) / BF, E = a.seg.E;
    return nf * (MODE == kGradWeight ? E * ((a.M + BT - 1) / BT) : a.entries / BT + min(E, a.entries));
}

template <int MODE, int ACT, bool FP8, int WF, int WT, int FF, int TF, class Args>
hipError_t launch_tiled(const Args &a, hipStream_t stream) {
    // persistent workgroups: as many as the CUs' LDS holds (two buffers of both
    // tiles), and no more than there can be tiles
    constexpr int kPerCU = WF * WT > 4 ? 1 : 2;
    constexpr int BF = WF * FF * 16, BT = WT * TF * 16;
    const int64_t tiles = most_tiles<MODE>(a, BF, BT);
    const uint32_t grid = static_cast<uint32_t>(max(int64_t{8}, min(int64_t{kCUs * kPerCU}, (tiles + 7) / 8 * 8)));
    product_kernel<MODE, ACT, FP8, WF, WT, FF, TF><<<grid, 64 * WF * WT, 0, stream>>>(a);
    return hipGetLastError();
}

template <int MODE, int ACT, bool FP8, class Args>
hipError_t launch_sized(const Args &a, hipStream_t stream) {
    // 64 x 64 tiles where larger ones would leave most CUs idle
    if (most_tiles<MODE>(a, 128, 128) < kMediumTiles) return launch_tiled<MODE, ACT, FP8, 1, 4, 4, 1>(a, stream);
    if constexpr (FP8) {
        return launch_tiled<MODE, ACT, true, 2, 2, 4, 4>(a, stream);
    } else {
        // large tiles where the rows fill them and every CU has one: 64 experts of
        // 4096 x 4096 take 497 us in 128 x 128 and 515 in 256 x 256 with 128 rows each, 576 and
        // 534 with 160; the gradients of 32 experts of 4096 x 2816 146 and 137 (input),
        // 221 and 220 (weight) with 64
        if (a.mean_rows >= (MODE == kForward ? 160 : 64) && most_tiles<MODE>(a, 256, 256) >= kLargeTiles)
            return launch_tiled<MODE, ACT, false, 2, 4, 8, 4>(a, stream);
        return launch_tiled<MODE, ACT, false, 2, 2, 4, 4>(a, stream);
    }
}

template <bool FP8, class Args>
hipError_t launch_forward(const Args &a, hipStream_t stream) {
    switch (a.act) {
#define EP_ACT_CASE(A) \
    case A: return launch_sized<kForward, A, FP8>(a, stream);
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

}  // namespace

int32_t grad_row_ranges(int32_t E, int32_t N) {
    const int64_t groups = static_cast<int64_t>(E) * ((N + kGradColumns - 1) / kGradColumns);
    const int64_t s = (kGradWorkgroups + groups - 1) / groups;
    return static_cast<int32_t>(s < 1 ? 1 : s > 64 ? 64 : s);
}

// Which products take the kernel for few rows: up to 16 rows an expert on
// average and kFewTiles tiles of 128 weight rows in all, for which the tiled
// product starts too few workgroups (16 x 7168 x 2048, 16 tiles: 16.0 us
// against 28.2, in FP8 11.6 against 22.1; 16 x 4096 x 8192, 64 tiles: 19.7
// against 31.0, FP8 13.5 against 18.9).  From 65 to 96 tiles neither is ahead (+-40 %
// by the length of k); past that the tiled product is (16 x 4096 x 16256, 127
// tiles: 33.0 against 38.1), and more so where some experts have many rows, as
// every 16 of them read the weight again (128 experts of 7736 -> 3560, 8 rows on
// average by Zipf's law: 1128 us against 2211).
constexpr int kFewTiles = 64;
bool few_rows(const ProductArgs &a) {
    return a.mean_rows <= 16 && int64_t{a.seg.E} * ((a.M + 127) / 128) <= kFewTiles;
}

hipError_t launch_product(const ProductArgs &a, bool fp8, hipStream_t stream) {
    if (few_rows(a)) return launch_product_few(a, fp8, stream);
    return fp8 ? launch_forward<true>(a, stream) : launch_forward<false>(a, stream);
}

hipError_t launch_product_grad(const ProductGradArgs &a, hipStream_t stream) {
    if (a.act != EP_ACT_NONE || a.dbias) {
        const dim3 grid(a.seg.E * a.splits, (a.N + kGradColumns - 1) / kGradColumns);
        switch (a.act) {
#define EP_ACT_CASE(A) \
    case A: act_grad_kernel<A><<<grid, 256, 0, stream>>>(a); break;
            EP_ACT_CASE(EP_ACT_NONE)
            EP_ACT_CASE(EP_ACT_RELU)
            EP_ACT_CASE(EP_ACT_GELU)
            EP_ACT_CASE(EP_ACT_SILU)
            EP_ACT_CASE(EP_ACT_SWIGLU)
            EP_ACT_CASE(EP_ACT_GEGLU)
#undef EP_ACT_CASE
            default: return hipErrorInvalidValue;
        }
        const hipError_t rc = hipGetLastError();
        if (rc != hipSuccess) return rc;
    }
    if (a.dbias && a.splits > 1) {
        const int64_t n = static_cast<int64_t>(a.seg.E) * a.M;
        bias_join_kernel<<<static_cast<uint32_t>((n + 255) / 256), 256, 0, stream>>>(a.partial, a.dbias, n, a.M, a.splits);
        const hipError_t rc = hipGetLastError();
        if (rc != hipSuccess) return rc;
    }
    if (a.dx) {
        const hipError_t rc = launch_sized<kGradInput, EP_ACT_NONE, false>(a, stream);
        if (rc != hipSuccess) return rc;
    }
    if (a.dweight || a.dweight_acc) return launch_sized<kGradWeight, EP_ACT_NONE, false>(a, stream);
    return hipSuccess;
}

}  // namespace epget
