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
#include <limits.h>

#include <type_traits>

#include "../../include/ep_get.h"
#include "device_common.h"
#include "route_internal.h"

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

// Reduction over the group of L lanes; every lane gets the same result, since
// each step joins the same two values on both sides.
template <int L, class V, class Op>
__device__ __forceinline__ V group_reduce(V v, Op op) {
    v = op(v, dpp<0x128>(v));
    v = op(v, dpp<0x124>(v));
    v = op(v, dpp<0x122>(v));
    v = op(v, dpp<0x121>(v));
    if (L >= 32) v = op(v, __shfl_xor(v, 16));
    if (L >= 64) v = op(v, __shfl_xor(v, 32));
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

// The columns of a lane: runs of V neighbours, V values being 16 bytes where
// there are as many.
template <bool BF16, int L, int N>
struct Columns {
    static constexpr int V = BF16 ? (N < 8 ? N : 8) : 4;
    // column of value i of lane 0; that of lane l is l * V further
    static constexpr int at(int i) { return (i / V) * (L * V) + i % V; }

    // Logits of row `row`, -inf past the last column.  wide: E is a multiple
    // of V, so that a run is one aligned load.
    static __device__ __forceinline__ void load(float (&x)[N], const void *logits, int64_t row, int E, int l, bool wide,
                                                bool on) {
        const int64_t base = row * E + l * V;
#pragma unroll
        for (int r = 0; r < N / V; ++r) {
            const int c = l * V + at(r * V);
            if constexpr (BF16) {
                const uint16_t *p = static_cast<const uint16_t *>(logits) + base + at(r * V);
                uint32_t u[V / 2];
#pragma unroll
                for (int i = 0; i < V / 2; ++i) u[i] = 0xFF80FF80u;
                if (wide) {
                    if (on && c < E) {
#pragma unroll
                        for (int i = 0; i < V / 4; ++i) {
                            const u32x2 d = reinterpret_cast<const u32x2 *>(p)[i];
                            u[2 * i] = d[0], u[2 * i + 1] = d[1];
                        }
                    }
                } else if (on) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (c + i < E) u[i / 2] = i & 1 ? (u[i / 2] & 0xFFFFu) | uint32_t{p[i]} << 16 : (u[i / 2] & 0xFFFF0000u) | p[i];
                }
#pragma unroll
                for (int i = 0; i < V; ++i) x[r * V + i] = i & 1 ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]);
            } else {
                const float *p = static_cast<const float *>(logits) + base + at(r * V);
                f32x4 d = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                if (wide) {
                    if (on && c < E) d = *reinterpret_cast<const f32x4 *>(p);
                } else if (on) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (c + i < E) d[i] = p[i];
                }
#pragma unroll
                for (int i = 0; i < V; ++i) x[r * V + i] = d[i];
            }
        }
    }

    static __device__ __forceinline__ void store(const float (&x)[N], void *out, int64_t row, int E, int l, bool wide) {
        const int64_t base = row * E + l * V;
#pragma unroll
        for (int r = 0; r < N / V; ++r) {
            const int c = l * V + at(r * V);
            if constexpr (BF16) {
                uint16_t *p = static_cast<uint16_t *>(out) + base + at(r * V);
                if (wide) {
                    if (c < E) {
#pragma unroll
                        for (int i = 0; i < V / 4; ++i)
                            reinterpret_cast<u32x2 *>(p)[i] = u32x2{pack_bf16x2(x[r * V + 4 * i], x[r * V + 4 * i + 1]),
                                                                    pack_bf16x2(x[r * V + 4 * i + 2], x[r * V + 4 * i + 3])};
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (c + i < E) p[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x[r * V + i]));
                }
            } else {
                float *p = static_cast<float *>(out) + base + at(r * V);
                if (wide) {
                    if (c < E) *reinterpret_cast<f32x4 *>(p) = f32x4{x[r * V], x[r * V + 1], x[r * V + 2], x[r * V + 3]};
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (c + i < E) p[i] = x[r * V + i];
                }
            }
        }
    }
};

// Sums over a token's row that its probabilities need.
struct RowSums {
    float top;      // greatest logit, 0 in a row without any above -inf
    float rcp;      // 1 / sum exp(x - top)
    float lse;
    float sig_rcp;  // 1 / sum of the numerators below (sigmoid scores)
    bool live;      // some logit is not -inf
};

__device__ __forceinline__ float logistic(float x) { return 1.0f / (1.0f + expf(-x)); }

// sigmoid(x) exp(-c) with c = min(top, 0), which no row of small logits takes to 0: e = exp(x - top).
__device__ __forceinline__ float sigmoid_numerator(float x, float e, float top) {
    const float t = expf(-fabsf(x));
    return (top < 0.0f ? e : x >= 0.0f ? 1.0f : x < 0.0f ? t : x) / (1.0f + t);
}

// x becomes p, the probabilities of the balance loss, and soft the softmax.
template <int L, int N>
__device__ __forceinline__ RowSums probabilities(float (&x)[N], float (&soft)[N], bool sigmoid) {
    RowSums r;
    float m = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
    m = group_max<L>(m);
    r.top = m > -INFINITY ? m : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        soft[i] = expf(x[i] - r.top);
        sum += soft[i];
    }
    sum = group_sum<L>(sum);
    r.live = sum != 0.0f;  // NaN counts
    r.rcp = r.live ? 1.0f / sum : 0.0f;
    r.lse = r.live ? r.top + logf(sum) : 0.0f;
    if (sigmoid) {
        float all = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = sigmoid_numerator(x[i], soft[i], r.top);
            all += x[i];
        }
        all = group_sum<L>(all);
        r.sig_rcp = r.live ? 1.0f / all : 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= r.sig_rcp;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        soft[i] *= r.rcp;
        if (!sigmoid) x[i] = soft[i];
    }
    return r;
}

enum RouteMode { kChoose, kChooseStats, kStats };

// Partial sums of a workgroup, by workgroup.
struct Partials {
    int32_t *count;  // [G, E]
    float *prob;     // [G, E]
    double *z;       // [G]
    int32_t *tokens; // [G]
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

// The K choices of a token in keys k (N a lane): lane j % L keeps choice j in
// slot j / L of pick (its expert) and of val (its logit).  Keys are compared exactly;
// of equal ones the lowest expert goes first, and -inf is never chosen.
template <class C, int L, int N, class Key>
__device__ __forceinline__ void choose(Key (&k)[N], const float (&x)[N], int K, int l, int (&pick)[2], float (&val)[2]) {
    const int base = l * C::V;
    for (int j = 0; j < K; ++j) {
        Key best = k[0];
#pragma unroll
        for (int i = 1; i < N; ++i) best = k[i] > best ? k[i] : best;
        best = group_max<L>(best);
        int at = INT_MAX;
#pragma unroll
        for (int i = N - 1; i >= 0; --i) at = k[i] == best ? base + C::at(i) : at;
        at = group_min<L>(at);
        const bool any = best > -static_cast<Key>(INFINITY);
        const int rel = at - base;
        float v = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool hit = rel == C::at(i);
            v = hit ? x[i] : v;
            k[i] = hit ? -static_cast<Key>(INFINITY) : k[i];
        }
        v = group_max<L>(v);
        if (l == j % L) {
            const int e = any ? at : -1;
            if (L >= 32 || j < L)
                pick[0] = e, val[0] = v;
            else
                pick[1] = e, val[1] = v;
        }
    }
}

// The weight of every choice (-1 none) that lane l holds.
template <int L>
__device__ __forceinline__ void choice_weights(const RouteArgs &a, const int (&pick)[2], const float (&val)[2], const RowSums &r,
                                               float (&w)[2]) {
    constexpr int P = L >= 32 ? 1 : 2;
    const bool sigmoid = a.score == EP_SCORE_SIGMOID;
    if (!a.normalise) {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const float s = sigmoid ? logistic(val[q]) : expf(val[q] - r.top) * r.rcp;
            w[q] = pick[q] >= 0 ? a.scale * s : 0.0f;
        }
        return;
    }
    float top = -INFINITY;
#pragma unroll
    for (int q = 0; q < P; ++q) top = fmaxf(top, pick[q] >= 0 ? val[q] : -INFINITY);
    top = group_max<L>(top);
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const float e = expf(val[q] - top);
        w[q] = pick[q] >= 0 ? (sigmoid ? sigmoid_numerator(val[q], e, top) : e) : 0.0f;
        sum += w[q];
    }
    sum = group_sum<L>(sum);
#pragma unroll
    for (int q = 0; q < P; ++q) w[q] = pick[q] >= 0 ? a.scale * (w[q] / sum) : 0.0f;
}

template <bool BF16, int L, int N, int MODE, bool BIASED>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
    using C = Columns<BF16, L, N>;
    constexpr int kTokens = 64 / L;  // of a wave
    constexpr bool STATS = MODE != kChoose;
    __shared__ int count[STATS ? L * N : 1];
    __shared__ float prob[STATS ? L * N : 1];
    __shared__ double wave_z[kRouteWaves];
    __shared__ int wave_tokens[kRouteWaves];
    const int lane = threadIdx.x & 63, l = lane & (L - 1);
    const int wave = threadIdx.x >> 6;
    const bool wide = a.E % C::V == 0;
    const bool sigmoid = a.score == EP_SCORE_SIGMOID;
    float psum[N];
    double z = 0.0;
    int tokens = 0;
    if (STATS) {
        for (int e = threadIdx.x; e < L * N; e += kRouteThreads) count[e] = 0, prob[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) psum[i] = 0.0f;
        __syncthreads();
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWaves * kTokens;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave) * kTokens; t0 < a.T; t0 += step) {
        const int64_t t = t0 + lane / L;
        const bool in = t < a.T;
        const bool on = in && (!a.mask || a.mask[t] != 0);
        float x[N], p[N], soft[N];
        C::load(x, a.logits, t, a.E, l, wide, on);
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = x[i];
        RowSums r = {};
        if (STATS || BIASED || (!sigmoid && !a.normalise)) r = probabilities<L>(p, soft, sigmoid);
        int pick[2] = {-1, -1};
        if (MODE != kStats) {
            float val[2] = {-INFINITY, -INFINITY}, w[2];
            if constexpr (BIASED) {
                // scores in 64 bits: in 32, two experts' sums with the bias may round to one value or change places
                double k[N];
                double sum = 0.0;
                if (!sigmoid) {
#pragma unroll
                    for (int i = 0; i < N; ++i) sum += (k[i] = exp(static_cast<double>(x[i]) - r.top));
                    sum = group_reduce<L>(sum, [](double u, double v) { return u + v; });
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int c = l * C::V + C::at(i);
                    const double s = sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x[i]))) : k[i] / sum;
                    const double b = c < a.E ? a.bias[c] : 0.0;
                    k[i] = x[i] > -INFINITY && s + b > -INFINITY ? s + b : -INFINITY;
                }
                choose<C, L, N>(k, x, a.K, l, pick, val);
            } else {  // scores rise with the logits
                float k[N];
#pragma unroll
                for (int i = 0; i < N; ++i) k[i] = x[i] > -INFINITY ? x[i] : -INFINITY;
                choose<C, L, N>(k, x, a.K, l, pick, val);
            }
            choice_weights<L>(a, pick, val, r, w);
            if (in) {
#pragma unroll
                for (int q = 0; q < (L >= 32 ? 1 : 2); ++q) {
                    const int j = q * L + l;
                    if (j < a.K) a.idx[t * a.K + j] = pick[q], a.w[t * a.K + j] = w[q];
                }
            }
        } else if (on && r.live) {
#pragma unroll
            for (int q = 0; q < (L >= 32 ? 1 : 2); ++q) {
                const int j = q * L + l;
                if (j < a.K) {
                    const int e = a.idx[t * a.K + j];
                    pick[q] = e < a.E ? e : -1;
                }
            }
        }
        if (STATS) {
#pragma unroll
            for (int q = 0; q < (L >= 32 ? 1 : 2); ++q)
                if (pick[q] >= 0) atomicAdd(&count[pick[q]], 1);
#pragma unroll
            for (int i = 0; i < N; ++i) psum[i] += r.live ? p[i] : 0.0f;
            if (l == 0 && r.live) {
                z += static_cast<double>(r.lse) * r.lse;
                ++tokens;
            }
        }
    }
    if (!STATS) return;
    // the groups of a wave, then the waves, in a fixed order
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (L < 32) psum[i] += __shfl_xor(psum[i], 16);
        if (L < 64) psum[i] += __shfl_xor(psum[i], 32);
    }
    for (int s = 32; s >= L; s >>= 1) {
        z += __shfl_xor(z, s);
        tokens += __shfl_xor(tokens, s);
    }
    if (lane == 0) wave_z[wave] = z, wave_tokens[wave] = tokens;
    for (int w = 0; w < kRouteWaves; ++w) {
        if (wave == w && lane < L)
#pragma unroll
            for (int i = 0; i < N; ++i) prob[l * C::V + C::at(i)] += psum[i];
        __syncthreads();
    }
    const Partials o = partials(a.workspace, gridDim.x, a.E);
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
        o.count[static_cast<int64_t>(blockIdx.x) * a.E + e] = count[e];
        o.prob[static_cast<int64_t>(blockIdx.x) * a.E + e] = prob[e];
    }
    if (threadIdx.x == 0) {
        double zz = 0.0;
        int n = 0;
        for (int w = 0; w < kRouteWaves; ++w) zz += wave_z[w], n += wave_tokens[w];
        o.z[blockIdx.x] = zz;
        o.tokens[blockIdx.x] = n;
        if (blockIdx.x == 0) *o.ticket = 0;
    }
}

// Joins the partial sums: 32 experts a workgroup, its rows the partials in
// turn; the last workgroup to finish adds up the losses.
constexpr int kJoinThreads = 1024;
constexpr int kJoinColumns = 32;
__global__ __launch_bounds__(kJoinThreads) void route_join_kernel(RouteArgs a, int G) {
    constexpr int R = kJoinThreads / kJoinColumns;
    __shared__ int cnt[R][kJoinColumns];
    __shared__ double prob[R][kJoinColumns];
    __shared__ double part[kJoinThreads / 64];
    __shared__ int toks[kJoinThreads / 64];
    __shared__ double zs[kJoinThreads / 64];
    __shared__ bool last;
    const Partials o = partials(a.workspace, G, a.E);
    const int c = threadIdx.x % kJoinColumns, r = threadIdx.x / kJoinColumns;
    const int e = blockIdx.x * kJoinColumns + c;
    int n = 0;
    double p = 0.0;
    if (e < a.E) {
        for (int g = r; g < G; g += R) {
            n += o.count[static_cast<int64_t>(g) * a.E + e];
            p += o.prob[static_cast<int64_t>(g) * a.E + e];
        }
    }
    cnt[r][c] = n;
    prob[r][c] = p;
    __syncthreads();
    if (r == 0 && e < a.E) {
        for (int i = 1; i < R; ++i) n += cnt[i][c], p += prob[i][c];
        a.expert_count[e] = n;
        a.prob_sum[e] = static_cast<float>(p);
        __threadfence();
    }
    __syncthreads();
    if (threadIdx.x == 0) last = __hip_atomic_fetch_add(o.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    double sum = 0.0, z = 0.0;
    int tokens = 0;
    for (int i = threadIdx.x; i < a.E; i += kJoinThreads) {
        const int ni = __hip_atomic_load(a.expert_count + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const float pi = __hip_atomic_load(a.prob_sum + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        sum += static_cast<double>(ni) * pi;
    }
    for (int g = threadIdx.x; g < G; g += kJoinThreads) z += o.z[g], tokens += o.tokens[g];
    for (int s = 32; s >= 1; s >>= 1) {
        sum += __shfl_xor(sum, s);
        z += __shfl_xor(z, s);
        tokens += __shfl_xor(tokens, s);
    }
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum, zs[threadIdx.x >> 6] = z, toks[threadIdx.x >> 6] = tokens;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 1; i < kJoinThreads / 64; ++i) sum += part[i], z += zs[i], tokens += toks[i];
    const double V = tokens > 0 ? tokens : 1;
    *a.token_count = tokens;
    a.losses[0] = static_cast<float>(sum * a.E / (a.K * V * V));
    a.losses[1] = static_cast<float>(z / V);
}

// d logits of the weights and of both losses.  b, the balance loss's gradient
// of p, is taken from the mean count, which the softmax's gradient does not
// see, so that nearly even counts leave their differences and not their sum's rounding.
template <bool BF16, int L, int N>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteArgs a) {
    using C = Columns<BF16, L, N>;
    constexpr int kTokens = 64 / L;
    constexpr int P = L >= 32 ? 1 : 2;
    __shared__ float scatter[kRouteWaves][64 * N];
    const int lane = threadIdx.x & 63, l = lane & (L - 1);
    const int wave = threadIdx.x >> 6;
    const bool wide = a.E % C::V == 0;
    const bool sigmoid = a.score == EP_SCORE_SIGMOID;
    float *row = scatter[wave] + (lane / L) * (L * N);
    float b[N], zscale = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = 0.0f;
    if (a.dlosses) {
        const double V = max(*a.token_count, 1);
        const double scale = a.dlosses[0] * static_cast<double>(a.E) / (a.K * V * V), mean = a.K * V / a.E;
        zscale = static_cast<float>(2.0 * a.dlosses[1] / V);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = l * C::V + C::at(i);
            if (c < a.E) b[i] = static_cast<float>(scale * (a.expert_count[c] - mean));
        }
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWaves * kTokens;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouteWaves + wave) * kTokens; t0 < a.T; t0 += step) {
        const int64_t t = t0 + lane / L;
        const bool in = t < a.T;
        const bool on = in && (!a.mask || a.mask[t] != 0);
        float x[N], p[N], soft[N], d[N];
        C::load(x, a.logits, t, a.E, l, wide, on);
        int pick[2] = {-1, -1};
        float val[2] = {-INFINITY, -INFINITY}, g[2] = {0.0f, 0.0f};
        if (a.dw && on) {
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const int j = q * L + l;
                if (j >= a.K) continue;
                const int e = a.idx[t * a.K + j];
                if (e < 0 || e >= a.E) continue;
                pick[q] = e;
                g[q] = a.scale * a.dw[t * a.K + j];
                if constexpr (BF16)
                    val[q] = bf16_lo(static_cast<const uint16_t *>(a.logits)[t * a.E + e]);
                else
                    val[q] = static_cast<const float *>(a.logits)[t * a.E + e];
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = x[i];
        const RowSums r = probabilities<L>(p, soft, sigmoid);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) dot += p[i] * b[i];
        dot = group_sum<L>(dot);
        const float zt = zscale * r.lse;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v = p[i] * (b[i] - dot);
            if (sigmoid) v *= logistic(-x[i]);  // 1 - s
            d[i] = v + zt * soft[i];
        }
        if (a.dw) {
            // c: what each choice adds to its own logit
            float c[2], sum = 0.0f;
            if (a.normalise) {
                float u[2], top = -INFINITY, all = 0.0f;
#pragma unroll
                for (int q = 0; q < P; ++q) top = fmaxf(top, pick[q] >= 0 ? val[q] : -INFINITY);
                top = group_max<L>(top);
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    const float e = expf(val[q] - top);
                    u[q] = pick[q] >= 0 ? (sigmoid ? sigmoid_numerator(val[q], e, top) : e) : 0.0f;
                    all += u[q];
                }
                all = group_sum<L>(all);
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    u[q] = pick[q] >= 0 ? u[q] / all : 0.0f;
                    sum += u[q] * g[q];
                }
                sum = group_sum<L>(sum);
#pragma unroll
                for (int q = 0; q < P; ++q) c[q] = u[q] * (g[q] - sum) * (sigmoid ? logistic(-val[q]) : 1.0f);
            } else {
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    const float s = sigmoid ? logistic(val[q]) : expf(val[q] - r.top) * r.rcp;
                    c[q] = pick[q] >= 0 ? g[q] * s : 0.0f;
                    sum += c[q];
                    if (sigmoid) c[q] *= logistic(-val[q]);
                }
                if (!sigmoid) {
                    sum = group_sum<L>(sum);
#pragma unroll
                    for (int i = 0; i < N; ++i) d[i] -= soft[i] * sum;
                }
            }
            // to the lanes that hold the logits: through LDS, an expert named twice with the sum of its choices
            float total[2] = {0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < P; ++q)
                for (int j = 0; j < min(a.K - q * L, L); ++j) {
                    const int e = __shfl(pick[q], j, L);
                    const float v = __shfl(c[q], j, L);
#pragma unroll
                    for (int s = 0; s < P; ++s) total[s] += e == pick[s] ? v : 0.0f;
                }
#pragma unroll
            for (int i = 0; i < N; ++i) row[l * C::V + C::at(i)] = 0.0f;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int q = 0; q < P; ++q)
                if (pick[q] >= 0) row[pick[q]] = total[q];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] += row[l * C::V + C::at(i)];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        if (!r.live) {
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] = 0.0f;
        }
        if (in) C::store(d, a.dlogits, t, a.E, l, wide);
    }
}

int tokens_of_workgroup(int32_t E) { return kRouteWaves * (E <= 256 ? 4 : E <= 512 ? 2 : 1); }

// Calls f with the lanes of a token and the logits of a lane.
template <class F>
void with_shape(int32_t E, F f) {
    if (E <= 64) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
    if (E <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
    if (E <= 256) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
    if (E <= 512) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
    if (E <= 1024) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
    f(std::integral_constant<int, 64>{}, std::integral_constant<int, 32>{});
}

template <int MODE, bool BIASED>
hipError_t launch_mode(const RouteArgs &a, int G, hipStream_t stream) {
    with_shape(a.E, [&](auto l, auto n) {
        if (a.bf16)
            route_kernel<true, l(), n(), MODE, BIASED><<<G, kRouteThreads, 0, stream>>>(a);
        else
            route_kernel<false, l(), n(), MODE, BIASED><<<G, kRouteThreads, 0, stream>>>(a);
    });
    return hipGetLastError();
}

hipError_t launch_join(const RouteArgs &a, int G, hipStream_t stream) {
    route_join_kernel<<<(a.E + kJoinColumns - 1) / kJoinColumns, kJoinThreads, 0, stream>>>(a, G);
    return hipGetLastError();
}

int workgroups(int32_t T, int32_t E, int most) {
    const int per = tokens_of_workgroup(E);
    const int64_t n = (static_cast<int64_t>(T) + per - 1) / per;
    return static_cast<int>(n < 1 ? 1 : n < most ? n : most);
}

}  // namespace

int32_t route_stat_workgroups(int32_t T, int32_t E) { return workgroups(T, E, 512); }

int64_t route_workspace(int32_t T, int32_t E) {
    const int64_t G = route_stat_workgroups(T, E);
    return 256 + G * (8 + 4 + static_cast<int64_t>(E) * 8);
}

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
    if (!a.losses) {
        if (a.T == 0) return hipSuccess;
        const int G = workgroups(a.T, a.E, 4096);
        return a.bias ? launch_mode<kChoose, true>(a, G, stream) : launch_mode<kChoose, false>(a, G, stream);
    }
    const int G = route_stat_workgroups(a.T, a.E);
    const hipError_t rc = a.bias ? launch_mode<kChooseStats, true>(a, G, stream) : launch_mode<kChooseStats, false>(a, G, stream);
    return rc == hipSuccess ? launch_join(a, G, stream) : rc;
}

hipError_t launch_balance(const RouteArgs &a, hipStream_t stream) {
    const int G = route_stat_workgroups(a.T, a.E);
    const hipError_t rc = launch_mode<kStats, false>(a, G, stream);
    return rc == hipSuccess ? launch_join(a, G, stream) : rc;
}

hipError_t launch_route_backward(const RouteArgs &a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const int G = workgroups(a.T, a.E, 4096);
    with_shape(a.E, [&](auto l, auto n) {
        if (a.bf16)
            route_backward_kernel<true, l(), n()><<<G, kRouteThreads, 0, stream>>>(a);
        else
            route_backward_kernel<false, l(), n()><<<G, kRouteThreads, 0, stream>>>(a);
    });
    return hipGetLastError();
}

}  // namespace epget
