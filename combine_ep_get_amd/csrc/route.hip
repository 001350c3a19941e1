// The router, its balance loss and its gradient, for gfx950.
//
//   s[t,e]  softmax over e or sigmoid of the logits;  p[t,e] = s[t,e] / sum_e s[t,e]
//   idx[t]  the K experts of the greatest s + bias, w[t] their scores
//   losses  E / (K V^2) sum_e count_e sum_t p[t,e]  and  1/V sum_t lse[t]^2
//
// A token's logits are held by a group of L lanes of a wave, N a lane (16
// lanes up to 256 experts, so that a wave works on four tokens and a
// reduction over a token is four DPP moves); everything else follows from
// these registers, so the logits are read once.
//
// Small calls are one short kernel, or two where statistics are joined: 5 us each, of which 2 are a launch.  16384 tokens of
// 256 fp32 experts, whose logits' 17 MB take 3.6 us at the rate of a copy: the choice of 8 takes 9.8 us, by sigmoid and a
// bias 11.9, with statistics 16, and 5 to join them.  Those 16 us are 9 of instructions, and waits (56 % of the waves' cycles)
// for the rounds of the choice, each of which needs the one before, and for loads: a wave has its four tokens once, with
// one workgroup a CU, so nothing else covers them.  The gradient takes 10 to 11 us (7.2).  16384 tokens of 64 experts:
// statistics of given choices 5 and 5 us.
#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "../../include/ep_get.h"
#include "device_common.h"
#include "route_internal.h"

// Products and sums are joined where the code says so, and not as each kernel's
// surroundings suggest: the router's statistics are then those of the loss alone, bit for bit.
#pragma clang fp contract(off)

namespace epget {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;

// v of the lane CTRL names (row_ror:n is 0x120 + n: n lanes back in the row of 16)
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(dpp<CTRL>(__float_as_int(v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    return __hiloint2double(dpp<CTRL>(__double2hiint(v)), dpp<CTRL>(__double2loint(v)));
}

// v of the lane with the same place in the even and in the odd row of 16 (H = 16), or half of the wave (32).
template <int H>
__device__ __forceinline__ void both(uint32_t v, uint32_t *even, uint32_t *odd) {
    const auto t = [&] {
        if constexpr (H == 16)
            return __builtin_amdgcn_permlane16_swap(v, v, false, false);
        else
            return __builtin_amdgcn_permlane32_swap(v, v, false, false);
    }();
    *even = t[0], *odd = t[1];
}
template <int H, class V, class Op>
__device__ __forceinline__ V join_both(V v, Op op) {
    constexpr int W = sizeof(V) / 4;
    uint32_t u[W], even[W], odd[W];
    __builtin_memcpy(u, &v, sizeof(V));
#pragma unroll
    for (int i = 0; i < W; ++i) both<H>(u[i], even + i, odd + i);
    V a, b;
    __builtin_memcpy(&a, even, sizeof(V));
    __builtin_memcpy(&b, odd, sizeof(V));
    return op(a, b);
}

// Reduction over the group of L lanes; every lane gets the same result, since
// each step joins the same two values on both sides.
template <int L, class V, class Op>
__device__ __forceinline__ V group_reduce(V v, Op op) {
    v = op(v, dpp<0x128>(v));
    v = op(v, dpp<0x124>(v));
    v = op(v, dpp<0x122>(v));
    v = op(v, dpp<0x121>(v));
    if (L >= 32) v = join_both<16>(v, op);
    if (L >= 64) v = join_both<32>(v, op);
    return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
    return group_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ double group_max(double v) {
    return group_reduce<L>(v, [](double a, double b) { return fmax(a, b); });
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
    return group_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ int group_min(int v) {
    return group_reduce<L>(v, [](int a, int b) { return min(a, b); });
}

// Sums with the lanes 16 and 32 further on: every lane's with all lanes of its place in a group of S.
template <int S>
__device__ __forceinline__ float across_groups(float v) {
    auto add = [](float a, float b) { return a + b; };
    if (S <= 16) v = join_both<16>(v, add);
    if (S <= 32) v = join_both<32>(v, add);
    return v;
}

// The lane of a group, as a value that the compiler does not know to be the same for every token: addresses from it are made
// where they are used, and not held in registers through the loop over the tokens (199 of them in the gradient's).
template <int L>
__device__ __forceinline__ int lane_of_group() {
    int l = threadIdx.x & (L - 1);
    asm volatile("" : "+v"(l));
    return l;
}

__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The columns of a lane: runs of V neighbours, V values being 16 bytes where
// there are as many.  A wave also keeps its tokens' rows in LDS, value i of
// a lane at [i][lane], where any column of the lane's token is found.
template <bool BF16, int L, int N>
struct Columns {
    static constexpr int V = BF16 ? (N < 8 ? N : 8) : 4;
    static constexpr int B = BF16 ? 2 : 4;
    // column of value i of lane 0; that of lane l is l * V further
    static constexpr int at(int i) { return (i / V) * (L * V) + i % V; }
    static __device__ __forceinline__ int place(int column) {
        return (column / (L * V) * V + column % V) * 64 + (__lane_id() & ~(L - 1)) + column % (L * V) / V;
    }

    static __device__ __forceinline__ void keep(const float (&x)[N], float *kept) {
        wave_fence();
#pragma unroll
        for (int i = 0; i < N; ++i) kept[i * 64 + __lane_id()] = x[i];
        wave_fence();
    }

    // Logits of row `row`, -inf past the last column and where the token does not count (on).  wide: E is a multiple of V,
    // so that a run is one aligned load; else the row comes by way of `kept`.  All loads are made, of the row's last logits
    // in the place of those past it: a load that some lanes skip is waited for before the next.
    static __device__ __forceinline__ void load(float (&x)[N], const void *logits, int64_t row, int E, int l, bool wide,
                                                bool on, float *kept) {
        const char *base = static_cast<const char *>(logits) + row * E * B;
        if (wide) {
            uint32_t u[N * B / 4];
#pragma unroll
            for (int r = 0; r < N / V; ++r) {
                const char *p = base + min(l * V + at(r * V), E - V) * B;
                if constexpr (V * B == 16) {
                    const u32x4 d = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[r * 4 + i] = d[i];
                } else {
                    const u32x2 d = *reinterpret_cast<const u32x2 *>(p);
                    u[r * 2] = d[0], u[r * 2 + 1] = d[1];
                }
            }
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = !BF16 ? __uint_as_float(u[i]) : i & 1 ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]);
        } else {
            float v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const char *p = base + min(i * L + l, E - 1) * B;
                v[i] = BF16 ? bf16_lo(*reinterpret_cast<const uint16_t *>(p)) : *reinterpret_cast<const float *>(p);
            }
            wave_fence();
#pragma unroll
            for (int i = 0; i < N; ++i) kept[place(i * L + l)] = v[i];
            wave_fence();
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = kept[i * 64 + __lane_id()];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = on && l * V + at(i) < E ? x[i] : -INFINITY;
    }

    static __device__ __forceinline__ void store(const float (&x)[N], void *out, int64_t row, int E, int l, bool wide,
                                                 bool on, float *kept) {
        char *base = static_cast<char *>(out) + row * E * B;
        if (wide) {
            if (!on) return;
#pragma unroll
            for (int r = 0; r < N / V; ++r) {
                char *p = base + (l * V + at(r * V)) * B;
                if (l * V + at(r * V) >= E) continue;
                if constexpr (!BF16) {
                    *reinterpret_cast<f32x4 *>(p) = f32x4{x[r * V], x[r * V + 1], x[r * V + 2], x[r * V + 3]};
                } else {
#pragma unroll
                    for (int i = 0; i < V; i += 4)
                        *reinterpret_cast<u32x2 *>(p + i * B) =
                            u32x2{pack_bf16x2(x[r * V + i], x[r * V + i + 1]), pack_bf16x2(x[r * V + i + 2], x[r * V + i + 3])};
                }
            }
        } else {
            keep(x, kept);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = i * L + l;
                if (!on || c >= E) continue;
                const float v = kept[place(c)];
                if constexpr (BF16)
                    reinterpret_cast<uint16_t *>(base)[c] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
                else
                    reinterpret_cast<float *>(base)[c] = v;
            }
        }
    }
};

// exp(x) for x <= 0 or NaN, within two ulp: the hardware's exp2 of the rounded
// product, corrected by what the rounding dropped.
__device__ __forceinline__ float exp_down(float x) {
    const float c = __builtin_elementwise_maximum(x, -200.0f);  // -inf has no product's remainder; NaN stays
    const float t = c * 1.4426950408889634f;
    const float lo = __builtin_fmaf(c, 1.9259629911266175e-8f, __builtin_fmaf(c, 1.4426950408889634f, -t));
    const float r = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(r, lo * 0.6931471805599453f, r);
}

__device__ __forceinline__ float logistic(float x) { return 1.0f / (1.0f + expf(-x)); }

// sigmoid(x), with the reciprocal of the hardware (an ulp).
__device__ __forceinline__ float quick_logistic(float x, float *rcp) {
    const float t = exp_down(-fabsf(x));
    *rcp = __builtin_amdgcn_rcpf(1.0f + t);
    return (x >= 0.0f ? 1.0f : t) * *rcp;  // NaN by the reciprocal
}

// sigmoid(x) exp(-c) with c = min(top, 0), which no row of small logits takes to 0: e = exp(x - top).
__device__ __forceinline__ float sigmoid_numerator(float x, float e, float top) {
    float rcp;
    const float s = quick_logistic(x, &rcp);
    return top < 0.0f ? e * rcp : s;
}

// The softmax of a token's logits: e becomes exp(x - top).
struct Softmax {
    float top;  // greatest logit, 0 in a row without any above -inf
    float rcp;  // 1 / sum of e
    float lse;
    bool live;  // some logit is not -inf
};
template <int L, int N>
__device__ __forceinline__ Softmax softmax(const float (&x)[N], float (&e)[N]) {
    Softmax r;
    float m = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
    m = group_max<L>(m);
    r.top = m > -INFINITY ? m : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        e[i] = exp_down(x[i] - r.top);
        sum += e[i];
    }
    sum = group_sum<L>(sum);
    r.live = sum != 0.0f;  // NaN counts
    r.rcp = r.live ? 1.0f / sum : 0.0f;
    r.lse = r.live ? r.top + logf(sum) : 0.0f;
    return r;
}

enum RouteMode { kChoose, kChooseStats, kStats };

// Partial sums of the workgroups of a call.
struct Partials {
    int32_t *count;   // [G, E]
    float *prob;      // [G, E]
    double *z;        // [G]
    int32_t *tokens;  // [G]
    uint32_t *ticket;
};

__host__ __device__ __forceinline__ Partials partials(void *ws, int64_t G, int64_t E) {
    char *p = static_cast<char *>(ws);
    Partials o;
    o.ticket = reinterpret_cast<uint32_t *>(p);
    o.z = reinterpret_cast<double *>(p + 256);
    o.tokens = reinterpret_cast<int32_t *>(p + 256 + G * 8);
    o.count = o.tokens + G;
    o.prob = reinterpret_cast<float *>(o.count + G * E);
    return o;
}

// Sums over a wave, for its first lane.
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
    for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s);
    return v;
}

__device__ __forceinline__ void write_losses(const RouteArgs &a, double balance, double z, int tokens) {
    const double V = tokens > 0 ? tokens : 1;
    *a.token_count = tokens;
    a.losses[0] = static_cast<float>(balance * a.E / (a.K * V * V));
    a.losses[1] = static_cast<float>(z / V);
}

// The choice of K experts.  Each logit's rank is a key of 32 bits: the leading
// bits of the value that orders it, and below them the complement of its
// column, so that the greatest key is also the lowest column of equal values.
// The next smaller key is a subtraction and a maximum: for keys below `last`,
// key - last wraps to above all others.  Where the leading bits do not settle
// the order of two candidates, they are compared again exactly, and candidates
// are taken until the last one is settled against the next; a choice
// that a group's lanes do not suffice for is made exactly from the start.
// (Sixteen exact 64-bit scores a lane instead took 38 us for 16384 tokens of 256
// experts with sigmoid scores and a bias; this takes 16.)
template <int L, int N>
constexpr int kColumnBits = __builtin_ctz(L * N);

// Rises with v, which is no -0.
__device__ __forceinline__ uint32_t ordered_bits(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float ordered_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Whether keys without their columns, hi >= lo, leave open which value is greater.  Scores in 32 bits are off by 5 ulp of
// their sum with the bias at most, and by `off` where the bias cancels them.
template <bool BF16>
__device__ __forceinline__ bool unsettled(uint32_t hi, uint32_t lo, uint32_t unit, bool biased, float off) {
    if (lo == 0) return false;  // nothing to choose
    if (biased) return hi - lo < 2 * unit || !(ordered_value(hi) - ordered_value(lo) > off);
    return !BF16 && hi == lo;
}

// What orders an expert, exactly: its logit, or with a bias the sum in 64 bits.
struct ExactOrder {
    const float *bias;
    bool sigmoid;
    double top, sum;  // of the softmax
    __device__ __forceinline__ double operator()(float x, int column) const {
        if (!(x > -INFINITY)) return -INFINITY;
        if (!bias) return x;
        const double s = sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x))) : exp(x - top) / sum;
        const double v = s + bias[column];
        return v > -INFINITY ? v : -INFINITY;
    }
};

// The softmax's sum for it, of logits that each lane keeps in LDS, where it finds them by number.
template <int L, int N>
__device__ __forceinline__ double exact_sum(const float *mine, double top) {
    double sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < N; ++i) sum += exp(mine[i * 64] - top);
    return group_reduce<L>(sum, [](double u, double v) { return u + v; });
}

// The choice from exact values alone, on lane j of a group choice j.
template <class C, int L, int N>
__device__ __forceinline__ int choose_exactly(const ExactOrder &order, const float *mine, int E, int K, int l) {
    int pick = -1;
    uint32_t taken = 0;  // of this lane's logits
#pragma unroll 1
    for (int j = 0; j < K; ++j) {
        double best = -INFINITY;
        int at = 0, column = INT_MAX;
#pragma unroll 1
        for (int i = 0; i < N; ++i) {  // columns ascend
            const int c = l * C::V + (i / C::V) * (L * C::V) + i % C::V;
            const double v = c < E && !(taken >> i & 1) ? order(mine[i * 64], c) : -INFINITY;
            if (v > best) best = v, at = i, column = c;
        }
        const double top = group_max<L>(best);
        const int first = group_min<L>(best == top ? column : INT_MAX);
        if (column == first && first != INT_MAX) taken |= 1u << at;
        if (l == j) pick = first == INT_MAX ? -1 : first;
    }
    return pick;
}

// The choice of lane l from its keys: choice l of its group's token, or -1.  The logits are in `kept`.
template <bool BF16, int L, int N>
__device__ __forceinline__ int choose(const RouteArgs &a, const uint32_t (&key)[N], const Softmax &r, int l, float *kept) {
    using C = Columns<BF16, L, N>;
    constexpr uint32_t kLow = (1u << kColumnBits<L, N>) - 1;
    const int lane = __lane_id();
    const bool sigmoid = a.score == EP_SCORE_SIGMOID, biased = a.bias != nullptr;
    const float off = sigmoid ? 0x1p-20f : 0x1p-17f * r.rcp;
    uint32_t mine = 0, last = 0;
    int n = L;  // candidates of the group: up to one that is settled against the next
    int j = 0;
    for (;; ++j) {
        uint32_t far = key[0] - last;
#pragma unroll
        for (int i = 1; i < N; ++i) far = max(far, key[i] - last);
        far = static_cast<uint32_t>(group_reduce<L>(static_cast<int>(far), [](int u, int v) {
            return static_cast<int>(max(static_cast<uint32_t>(u), static_cast<uint32_t>(v)));
        }));
        // the first has no bound above it; none is left where the maximum is not below the last
        const uint32_t best = far + last, now = j == 0 || best < last ? best : 0;
        if (l == j) mine = now;
        if (j >= a.K) {
            if (n == L && !unsettled<BF16>(last & ~kLow, now & ~kLow, kLow + 1, biased, off)) n = j;
            if (__all(n != L) || j == L - 1) break;
        }
        last = now ? now : 1;  // 1 is below every key
    }
    const bool again = __any(n == L);
    int pick = l < n && mine != 0 ? static_cast<int>(kLow - (mine & kLow)) : -1;
    const uint32_t next = __shfl_down(mine, 1, L);
    const bool open = l + 1 < n && unsettled<BF16>(mine & ~kLow, next & ~kLow, kLow + 1, biased, off);
    if (!again && !__any(open || (l == 0 && n > a.K))) return l < a.K ? pick : -1;

    const ExactOrder order{a.bias, sigmoid, r.top, biased && !sigmoid ? exact_sum<L, N>(kept + lane, r.top) : 1.0};
    if (again) return choose_exactly<C, L, N>(order, kept + lane, a.E, a.K, l);
    double v = -INFINITY;
    if (pick >= 0) v = order(kept[C::place(pick)], pick);
    int rank = 0;
    for (int i = 0; i <= j; ++i) {
        const double other = __shfl(v, i, L);
        const int column = __shfl(pick, i, L);
        rank += other > v || (other == v && column < pick);
    }
    if (pick < 0) rank = l;  // empty ones stay behind
    pick = __builtin_amdgcn_ds_permute(((lane & ~(L - 1)) + rank) * 4, pick);
    return l < a.K ? pick : -1;
}

// The weight of this lane's choice (-1 none), of which val is the logit.
template <int L>
__device__ __forceinline__ float choice_weight(const RouteArgs &a, int pick, float val, const Softmax &r) {
    const bool sigmoid = a.score == EP_SCORE_SIGMOID;
    if (!a.normalise) {
        const float s = sigmoid ? logistic(val) : expf(val - r.top) * r.rcp;
        return pick >= 0 ? a.scale * s : 0.0f;
    }
    const float top = group_max<L>(pick >= 0 ? val : -INFINITY);
    const float e = expf(val - top);
    const float w = pick >= 0 ? (sigmoid ? sigmoid_numerator(val, e, top) : e) : 0.0f;
    const float sum = group_sum<L>(w);
    return pick >= 0 ? a.scale * (w / sum) : 0.0f;
}

// Workgroups that gather statistics are large, so that few leave partial sums (16384 tokens, 8 of 256 experts: 18.6 us;
// of four waves 21.7).
template <int MODE, int L, int N>
constexpr int kThreads = MODE != kChoose && L * N <= 256 ? 1024 : kRouteThreads;

template <bool BF16, int L, int N, int MODE>
__global__ __launch_bounds__((kThreads<MODE, L, N>)) void route_kernel(RouteArgs a) {
    using C = Columns<BF16, L, N>;
    constexpr int kWaves = kThreads<MODE, L, N> / 64;
    constexpr int kTokens = 64 / L;  // of a wave
    constexpr bool STATS = MODE != kChoose, CHOOSE = MODE != kStats;
    constexpr uint32_t kLow = (1u << kColumnBits<L, N>) - 1;
    __shared__ float kept[kWaves][64 * N];
    __shared__ float bias[CHOOSE ? L * N : 1];
    __shared__ int count[STATS ? L * N : 1];
    __shared__ float prob[STATS ? kWaves : 1][STATS ? L * N : 1];
    __shared__ double wave_z[kWaves], wave_balance[kWaves];
    __shared__ int wave_tokens[kWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool wide = a.E % C::V == 0;
    const bool sigmoid = a.score == EP_SCORE_SIGMOID, biased = CHOOSE && a.bias;
    float psum[N];
    double z = 0.0;
    int tokens = 0;
    if (STATS || biased) {
        for (int e = threadIdx.x; e < L * N; e += kWaves * 64) {
            if (STATS) count[e] = 0;
            if (biased) bias[e] = e < a.E ? a.bias[e] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) psum[i] = 0.0f;
        __syncthreads();
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWaves * kTokens;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTokens; t0 < a.T; t0 += step) {
        const int l = lane_of_group<L>();
        const bool in = t0 + lane / L < a.T;
        const int64_t t = in ? t0 + lane / L : a.T - 1;
        const bool on = in && (!a.mask || a.mask[t] != 0);
        int pick = -1;
        if (!CHOOSE) pick = a.idx[t * a.K + min(l, a.K - 1)];
        float x[N], e[N];
        uint32_t key[N];
        C::load(x, a.logits, t, a.E, l, wide, on, kept[wave]);
        if (CHOOSE) C::keep(x, kept[wave]);
        Softmax r = {};
        if (STATS || (!sigmoid && (biased || !a.normalise))) r = softmax<L>(x, e);
        // keys, and of e the numerators of the probabilities
        const float *my_bias = bias + l * C::V;
        const uint32_t my_low = kLow - l * C::V;
        auto key_of = [&](float v, int i) { return (ordered_bits(v) & ~kLow) | (my_low - C::at(i)); };
        float all = 0.0f;
        if (sigmoid && (STATS || biased)) {
            const bool low = r.top < 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float rcp;
                const float s = quick_logistic(x[i], &rcp);
                if (STATS) e[i] = low ? e[i] * rcp : s, all += e[i];
                if (CHOOSE) {
                    const float v = x[i] > -INFINITY ? (biased ? s + my_bias[C::at(i)] : x[i] + 0.0f) : -INFINITY;
                    key[i] = v > -INFINITY ? key_of(v, i) : 0;
                }
            }
        } else if (CHOOSE) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float v = x[i] > -INFINITY ? (biased ? __builtin_fmaf(e[i], r.rcp, my_bias[C::at(i)]) : x[i] + 0.0f) : -INFINITY;
                key[i] = v > -INFINITY ? key_of(v, i) : 0;
            }
        }
        if (STATS) {
            const float rcp = !r.live ? 0.0f : sigmoid ? 1.0f / group_sum<L>(all) : r.rcp;
#pragma unroll
            for (int i = 0; i < N; ++i) psum[i] = __builtin_fmaf(e[i], rcp, psum[i]);
            if (l == 0 && r.live) {
                z += static_cast<double>(r.lse) * r.lse;
                ++tokens;
            }
        }
        if (CHOOSE) {
            pick = choose<BF16, L, N>(a, key, r, l, kept[wave]);
            const float w = choice_weight<L>(a, pick, pick >= 0 ? kept[wave][C::place(pick)] : -INFINITY, r);
            if (in && l < a.K) a.idx[t * a.K + l] = pick, a.w[t * a.K + l] = w;
        } else if (!(on && r.live && l < a.K && pick < a.E)) {
            pick = -1;
        }
        if (STATS && pick >= 0) atomicAdd(&count[pick], 1);
    }
    if (!STATS) return;
    // the groups of a wave, then the waves, in a fixed order
    const int l = lane & (L - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float p = across_groups<L>(psum[i]);
        if (lane < L) prob[wave][l * C::V + C::at(i)] = p;
    }
    z = wave_sum(z), tokens = wave_sum(tokens);
    if (lane == 0) wave_z[wave] = z, wave_tokens[wave] = tokens;
    __syncthreads();
    const bool alone = gridDim.x == 1;  // its sums are the call's
    const Partials o = partials(a.workspace, gridDim.x, a.E);
    int32_t *counts = alone ? a.expert_count : o.count + static_cast<int64_t>(blockIdx.x) * a.E;
    float *probs = alone ? a.prob_sum : o.prob + static_cast<int64_t>(blockIdx.x) * a.E;
    double balance = 0.0;
    for (int e = threadIdx.x; e < a.E; e += kWaves * 64) {
        double p = 0.0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) p += prob[w][e];
        counts[e] = count[e];
        probs[e] = static_cast<float>(p);
        balance += p * count[e];
    }
    if (alone) {
        balance = wave_sum(balance);
        if (lane == 0) wave_balance[wave] = balance;
        __syncthreads();
    }
    if (threadIdx.x != 0) return;
    for (int w = 1; w < kWaves; ++w) z += wave_z[w], tokens += wave_tokens[w];
    if (alone) {
        for (int w = 1; w < kWaves; ++w) balance += wave_balance[w];
        write_losses(a, balance, z, tokens);
    } else {
        o.z[blockIdx.x] = z;
        o.tokens[blockIdx.x] = tokens;
        if (blockIdx.x == 0) *o.ticket = 0;
    }
}

// Joins the partial sums: 16 experts a workgroup, its rows the partials in
// turn; the last workgroup to finish adds up the losses.  The workgroups' sums of
// probabilities are fp32, and so is what prob_sum holds and the balance loss is
// made of: a rounding each, of the size of prob_sum's own.  5 us for 256 partials
// of 256 experts: a launch, a read and the ticket, one after the other.
constexpr int kJoinThreads = 1024;
constexpr int kJoinColumns = 16;
__global__ __launch_bounds__(kJoinThreads) void route_join_kernel(RouteArgs a, int G) {
    constexpr int kWaves = kJoinThreads / 64, R = kJoinThreads / kJoinColumns;
    __shared__ int cnt[kWaves][kJoinColumns];
    __shared__ double prob[kWaves][kJoinColumns], zs[kWaves], sums[kWaves];
    __shared__ int toks[kWaves];
    __shared__ bool last;
    const Partials o = partials(a.workspace, G, a.E);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = threadIdx.x % kJoinColumns, e = blockIdx.x * kJoinColumns + c;
    int n = 0;
    double p = 0.0;
    if (e < a.E) {
#pragma unroll 4
        for (int g = threadIdx.x / kJoinColumns; g < G; g += R) {
            n += o.count[static_cast<int64_t>(g) * a.E + e];
            p += o.prob[static_cast<int64_t>(g) * a.E + e];
        }
    }
#pragma unroll
    for (int s = kJoinColumns; s < 64; s <<= 1) n += __shfl_xor(n, s), p += __shfl_xor(p, s);
    if (lane < kJoinColumns) cnt[wave][c] = n, prob[wave][c] = p;
    __syncthreads();
    if (threadIdx.x < kJoinColumns && e < a.E) {
#pragma unroll
        for (int w = 1; w < kWaves; ++w) n += cnt[w][c], p += prob[w][c];
        __hip_atomic_store(a.expert_count + e, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(a.prob_sum + e, static_cast<float>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(o.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    double balance = 0.0, z = 0.0;
    int tokens = 0;
    for (int i = threadIdx.x; i < a.E; i += kJoinThreads) {
        const int ni = __hip_atomic_load(a.expert_count + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        balance += static_cast<double>(ni) * __hip_atomic_load(a.prob_sum + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    for (int g = threadIdx.x; g < G; g += kJoinThreads) z += o.z[g], tokens += o.tokens[g];
    balance = wave_sum(balance), z = wave_sum(z), tokens = wave_sum(tokens);
    if (lane == 0) sums[wave] = balance, zs[wave] = z, toks[wave] = tokens;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < kWaves; ++w) balance += sums[w], z += zs[w], tokens += toks[w];
    write_losses(a, balance, z, tokens);
}

// d logits of the weights and of both losses.  b, the balance loss's gradient
// of p, is taken from the mean count, which the softmax's gradient does not
// see, so that nearly even counts leave their differences and not their sum's rounding.
template <bool BF16, int L, int N>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteArgs a) {
    using C = Columns<BF16, L, N>;
    constexpr int kTokens = 64 / L;
    __shared__ float kept[kRouteWaves][64 * N];
    __shared__ float b[L * N];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool wide = a.E % C::V == 0;
    const bool sigmoid = a.score == EP_SCORE_SIGMOID;
    float *row = kept[wave];
    float zscale = 0.0f;
    if (a.dlosses) {
        const double V = max(*a.token_count, 1);
        const double scale = a.dlosses[0] * static_cast<double>(a.E) / (a.K * V * V), mean = a.K * V / a.E;
        zscale = static_cast<float>(2.0 * a.dlosses[1] / V);
        for (int e = threadIdx.x; e < L * N; e += kRouteThreads)
            b[e] = e < a.E ? static_cast<float>(scale * (a.expert_count[e] - mean)) : 0.0f;
    } else {
        for (int e = threadIdx.x; e < L * N; e += kRouteThreads) b[e] = 0.0f;
    }
    __syncthreads();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWaves * kTokens;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave) * kTokens; t0 < a.T; t0 += step) {
        const int l = lane_of_group<L>();
        const bool in = t0 + lane / L < a.T;
        const int64_t t = in ? t0 + lane / L : a.T - 1;
        const bool on = in && (!a.mask || a.mask[t] != 0);
        int pick = -1;
        float g = 0.0f;
        if (a.dw) {
            const int64_t at = t * a.K + min(l, a.K - 1);
            pick = a.idx[at];
            g = a.scale * a.dw[at];
        }
        float x[N], p[N], d[N];
        C::load(x, a.logits, t, a.E, l, wide, on, row);
        const Softmax r = softmax<L>(x, p);
        // c: what each choice adds to its own logit;  sum: what the softmax of unnormalised weights takes from all
        float c = 0.0f, sum = 0.0f;
        if (a.dw) {
            C::keep(x, row);
            if (!(on && l < a.K && pick >= 0 && pick < a.E)) pick = -1, g = 0.0f;  // whatever dweights hold there
            const float val = pick >= 0 ? row[C::place(pick)] : -INFINITY;
            if (a.normalise) {
                const float top = group_max<L>(val);
                const float e = expf(val - top);
                float u = pick >= 0 ? (sigmoid ? sigmoid_numerator(val, e, top) : e) : 0.0f;
                const float all = group_sum<L>(u);
                u = pick >= 0 ? u / all : 0.0f;
                c = u * (g - group_sum<L>(u * g)) * (sigmoid ? logistic(-val) : 1.0f);
            } else {
                const float s = sigmoid ? logistic(val) : expf(val - r.top) * r.rcp;
                c = pick >= 0 ? g * s : 0.0f;
                if (sigmoid)
                    c *= logistic(-val);
                else
                    sum = group_sum<L>(c);
            }
        }
        const float zt = zscale * r.lse;
        if (!sigmoid) {
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                p[i] *= r.rcp;
                d[i] = b[l * C::V + C::at(i)];
                dot = __builtin_fmaf(p[i], d[i], dot);
            }
            dot = group_sum<L>(dot);
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] = __builtin_fmaf(p[i], d[i] - dot, p[i] * (zt - sum));
        } else {
            // p of the balance loss: the sigmoids over their sum;  the z loss's is the softmax
            float dot = 0.0f, all = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float q = sigmoid_numerator(x[i], p[i], r.top);
                all += q;
                dot = __builtin_fmaf(q, b[l * C::V + C::at(i)], dot);
            }
            all = group_sum<L>(all), dot = group_sum<L>(dot);
            const float rcp = r.live ? 1.0f / all : 0.0f;
            dot *= rcp;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float unused;
                const float q = sigmoid_numerator(x[i], p[i], r.top) * rcp, rest = quick_logistic(-x[i], &unused);  // 1 - s
                d[i] = __builtin_fmaf(q * (b[l * C::V + C::at(i)] - dot), rest, zt * (p[i] * r.rcp));
            }
        }
        if (a.dw) {
            // c to the lanes that hold the logits: through LDS, an expert named twice with the sum of its choices
            float total = 0.0f;
            for (int j = 0; j < a.K; ++j) {
                const int other = __shfl(pick, j, L);
                const float v = __shfl(c, j, L);
                total += other == pick ? v : 0.0f;
            }
            wave_fence();
#pragma unroll
            for (int i = 0; i < N; ++i) row[i * 64 + lane] = 0.0f;
            wave_fence();
            if (pick >= 0) row[C::place(pick)] = total;
            wave_fence();
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] += row[i * 64 + lane];
        }
        if (!r.live) {
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] = 0.0f;
        }
        C::store(d, a.dlogits, t, a.E, l, wide, in, row);
    }
}

// Tokens up to which a token has a whole wave: there are CUs for all of them, and fewer logits a lane make its way shorter,
// the more so where 16 lanes would hold 16 each.  With a choice and statistics, of 256 experts: 4096 tokens 15.9 us by waves
// and 19.1 by 16 lanes, 8192 tokens 20.7 and 19.6; of 64: 1024 tokens 14.7 and 14.2, 256 tokens 14.8 and 20.
constexpr int few_tokens(int32_t E) { return E > 128 ? 4096 : 1024; }
// Choices that 16 lanes hold with candidates to spare (16384 tokens, 12 of 256 experts: 11.3 us, by waves 18).
constexpr int kFewChoices = 12;

// Calls f with the lanes of a token and the logits of a lane.
template <class F>
void with_shape(int32_t T, int32_t E, int32_t K, F f) {
    const bool wave = T <= few_tokens(E) || K > kFewChoices;
    if (E <= 64 && !wave) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
    if (E <= 128 && !wave) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
    if (E <= 256 && !wave) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
    if (E <= 256) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    if (E <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
    if (E <= 1024) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
    f(std::integral_constant<int, 64>{}, std::integral_constant<int, 32>{});
}

int workgroups(int32_t T, int tokens, int most) {
    const int64_t n = (static_cast<int64_t>(T) + tokens - 1) / tokens;
    return static_cast<int>(n < 1 ? 1 : n < most ? n : most);
}

// One workgroup of 16 waves up to as many rounds of a token a wave: it needs no second kernel.  Statistics of 32 tokens
// 10.4 us, with a second kernel 12.9, and with a choice 12 to 13.6 and 14; of 64 tokens 10.4 and 12.9, with a choice 22 and
// 14.  One rule for both: the same statistics come out, bit for bit.
constexpr int kAloneRounds = 2;

template <int L, int N>
int stat_workgroups(int32_t T) {
    constexpr int threads = kThreads<kStats, L, N>, tokens = threads / L;
    if (threads == 1024 && T <= kAloneRounds * tokens) return 1;
    return workgroups(T, tokens, threads == 1024 ? 256 : 512);
}

template <int MODE>
hipError_t launch_stats(const RouteArgs &a, hipStream_t stream) {
    int G = 0;
    with_shape(a.T, a.E, a.K, [&](auto l, auto n) {
        constexpr int L = l(), N = n();
        G = stat_workgroups<L, N>(a.T);
        if (a.bf16)
            route_kernel<true, L, N, MODE><<<G, kThreads<MODE, L, N>, 0, stream>>>(a);
        else
            route_kernel<false, L, N, MODE><<<G, kThreads<MODE, L, N>, 0, stream>>>(a);
    });
    hipError_t rc = hipGetLastError();
    if (rc != hipSuccess || G == 1) return rc;
    route_join_kernel<<<(a.E + kJoinColumns - 1) / kJoinColumns, kJoinThreads, 0, stream>>>(a, G);
    return hipGetLastError();
}

}  // namespace

// An upper bound of what the calls with fewer tokens or choices need too: what is allocated for the longest batch serves
// every shorter one, though a token has more lanes, and the partials are more, up to few_tokens and past kFewChoices.
int64_t route_workspace(int32_t T, int32_t E, int32_t K) {
    int64_t G = 0;
    auto most = [&](int32_t t, int32_t k) {
        with_shape(t, E, k, [&](auto l, auto n) { G = std::max<int64_t>(G, stat_workgroups<l(), n()>(t)); });
    };
    most(T, K);
    most(std::min(T, few_tokens(E)), K);
    return 256 + G * (8 + 4 + static_cast<int64_t>(E) * 8);
}

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
    if (a.losses) return launch_stats<kChooseStats>(a, stream);
    if (a.T == 0) return hipSuccess;
    with_shape(a.T, a.E, a.K, [&](auto l, auto n) {
        const int G = workgroups(a.T, kRouteThreads / l(), 4096);
        if (a.bf16)
            route_kernel<true, l(), n(), kChoose><<<G, kRouteThreads, 0, stream>>>(a);
        else
            route_kernel<false, l(), n(), kChoose><<<G, kRouteThreads, 0, stream>>>(a);
    });
    return hipGetLastError();
}

hipError_t launch_balance(const RouteArgs &a, hipStream_t stream) { return launch_stats<kStats>(a, stream); }

hipError_t launch_route_backward(const RouteArgs &a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    with_shape(a.T, a.E, a.K, [&](auto l, auto n) {
        const int G = workgroups(a.T, kRouteThreads / l(), 4096);
        if (a.bf16)
            route_backward_kernel<true, l(), n()><<<G, kRouteThreads, 0, stream>>>(a);
        else
            route_backward_kernel<false, l(), n()><<<G, kRouteThreads, 0, stream>>>(a);
    });
    return hipGetLastError();
}

}  // namespace epget
