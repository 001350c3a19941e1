// The global norm of many gradients, and clipping, for gfx950.
//
//   square_sum = sum g^2      out = g min(1, max_norm / sqrt(square_sum))
//
// Up to kTableSize gradients share a launch: their addresses and sizes travel
// in the kernel's arguments, so that nothing is copied to the device and a
// captured call holds them itself.  A workgroup takes pieces of kPiece bytes,
// whichever gradient they belong to, so many small gradients and a few
// large ones fill the chip alike.  Squares are summed in 64 bits: an fp32
// square of a large gradient overflows, and the sum of 10^9 small ones loses
// its last digits.
//
// Both calls are bound by memory.  2.8 GB of gradients: the sum 480 us (5.9 TB/s), the clipping 1030 us, a read and a write
// at 5.5 TB/s; together 1515 us with 4096 workgroups, 1538 with 2048.  The clipping's loads and stores are past the caches:
// 1610 us with ordinary ones.  40 small gradients: 5, 3 and 7 us, of which a launch is 2; the rest is 144 workgroups with
// one piece each, which wait for the search of its gradient in the arguments, then for its loads, with nothing behind them.
#include <algorithm>

#include "../../include/ep_get.h"
#include "device_common.h"
#include "grads_internal.h"

namespace epget {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kTableSize = 64;
constexpr int kGradThreads = 256;
constexpr int kVectors = 8;                                 // 16-byte vectors of a thread and piece
constexpr int kPiece = kGradThreads * kVectors * 16;        // bytes
constexpr int kGradWorkgroups = 4096;

struct GradTable {
    const char *grad[kTableSize];
    char *out[kTableSize];
    int64_t count[kTableSize];
    int32_t first[kTableSize + 1];  // pieces of the gradients before each
    int32_t num;
    uint64_t fp32;                  // bit i: gradient i is fp32
};

// The gradient that owns piece `piece`: the last i with first[i] <= piece.
__device__ __forceinline__ int owner(const GradTable &t, int piece) {
    int lo = 0, hi = t.num - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= piece)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float element(const char *p, int64_t i, bool fp32) {
    return fp32 ? reinterpret_cast<const float *>(p)[i] : bf16_lo(reinterpret_cast<const uint16_t *>(p)[i]);
}

// out[i] = p[i] * f, or its very bits without `scale`.  V: float, or double for a factor that fp32 does not hold.
template <class V>
__device__ __forceinline__ void move(char *out, const char *p, int64_t i, bool fp32, bool scale, V f) {
    if (fp32) {
        const uint32_t v = reinterpret_cast<const uint32_t *>(p)[i];
        reinterpret_cast<uint32_t *>(out)[i] = scale ? __float_as_uint(static_cast<float>(__uint_as_float(v) * f)) : v;
    } else {
        const uint16_t v = reinterpret_cast<const uint16_t *>(p)[i];
        reinterpret_cast<uint16_t *>(out)[i] =
            scale ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(static_cast<float>(bf16_lo(v) * f))) : v;
    }
}

__device__ __forceinline__ double square(float v) { return static_cast<double>(v) * v; }

// The values [begin, end) of piece `piece` of a gradient, and the first and
// one past the last that lie in whole 16-byte vectors of its address.
struct Span {
    int64_t begin, end, vec, vec_end;
};
__device__ __forceinline__ Span span_of(const char *grad, int64_t count, int64_t piece, int size) {
    const int per = 16 / size;
    const int64_t head = (-reinterpret_cast<intptr_t>(grad) & 15) / size;  // values before the first aligned one
    Span s;
    // pieces are cut at aligned addresses; the first takes the head as well
    s.begin = piece == 0 ? 0 : head + piece * (kPiece / size);
    s.end = min(count, head + (piece + 1) * (kPiece / size));
    s.vec = min(s.end, piece == 0 ? head : s.begin);
    s.vec_end = s.vec + (s.end - s.vec) / per * per;
    return s;
}

__global__ __launch_bounds__(kGradThreads) void square_sum_kernel(GradTable t, double *partial) {
    __shared__ double wave[kGradThreads / 64];
    double sum = 0.0;
    const int pieces = t.first[t.num];
    for (int piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
        const int g = owner(t, piece);
        const bool fp32 = t.fp32 >> g & 1;
        const char *p = t.grad[g];
        const int size = fp32 ? 4 : 2;
        const Span s = span_of(p, t.count[g], piece - t.first[g], size);
        const u32x4 *v = reinterpret_cast<const u32x4 *>(p + s.vec * size);
        const int n = static_cast<int>((s.vec_end - s.vec) * size / 16);
        u32x4 d[kVectors];
        if (n == kPiece / 16) {
#pragma unroll
            for (int i = 0; i < kVectors; ++i) d[i] = v[threadIdx.x + i * kGradThreads];
        } else {
#pragma unroll
            for (int i = 0; i < kVectors; ++i) {
                const int at = threadIdx.x + i * kGradThreads;
                d[i] = at < n ? v[at] : u32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (fp32)
                    sum += square(__uint_as_float(d[i][q]));
                else
                    sum += square(bf16_lo(d[i][q])) + square(bf16_hi(d[i][q]));
            }
        // fewer than a vector before the first and after the last
        const int64_t head = s.begin + threadIdx.x, tail = s.vec_end + threadIdx.x;
        if (head < s.vec) sum += square(element(p, head, fp32));
        if (tail < s.end) sum += square(element(p, tail, fp32));
    }
    for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
    if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kGradThreads / 64; ++w) sum += wave[w];
        partial[blockIdx.x] = sum;
    }
}

constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void square_join_kernel(const double *partial, int64_t n, double *square_sum) {
    __shared__ double wave[kJoinThreads / 64];
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kJoinThreads) sum += partial[i];
    for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
    if ((threadIdx.x & 63) == 0) wave[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kJoinThreads / 64; ++w) sum += wave[w];
        *square_sum = sum;
    }
}

__device__ __forceinline__ u32x4 scaled(u32x4 d, bool fp32, float f) {
    u32x4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        o[q] = fp32 ? __float_as_uint(__uint_as_float(d[q]) * f) : pack_bf16x2(bf16_lo(d[q]) * f, bf16_hi(d[q]) * f);
    return o;
}

__global__ __launch_bounds__(kGradThreads) void clip_kernel(GradTable t, const double *square_sum, float max_norm,
                                                            float *norm_out) {
    const double norm = sqrt(*square_sum);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
    const bool scale = norm > max_norm && norm < INFINITY;
    const double factor = scale ? max_norm / norm : 1.0;
    const float f = static_cast<float>(factor);
    const int pieces = t.first[t.num];
    if (factor > 0.0 && factor < 0x1p-126) {
        // fp32 holds a factor but for its last rounding down to 2^-126; a smaller one, of a norm of 2^126 times max_norm and
        // more, would lose its digits there or be 0, and multiplies in 64 bits
        for (int piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
            const int g = owner(t, piece);
            const bool fp32 = t.fp32 >> g & 1;
            const Span s = span_of(t.grad[g], t.count[g], piece - t.first[g], fp32 ? 4 : 2);
            for (int64_t i = s.begin + threadIdx.x; i < s.end; i += kGradThreads) move(t.out[g], t.grad[g], i, fp32, true, factor);
        }
        return;
    }
    for (int piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
        const int g = owner(t, piece);
        const bool fp32 = t.fp32 >> g & 1;
        const char *p = t.grad[g];
        char *out = t.out[g];
        if (!scale && out == p) continue;
        const int size = fp32 ? 4 : 2;
        Span s = span_of(p, t.count[g], piece - t.first[g], size);
        if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) {
            // no 16-byte vector is aligned on both sides
            for (int64_t i = s.begin + threadIdx.x; i < s.end; i += kGradThreads) move(out, p, i, fp32, scale, f);
            continue;
        }
        const u32x4 *v = reinterpret_cast<const u32x4 *>(p + s.vec * size);
        u32x4 *o = reinterpret_cast<u32x4 *>(out + s.vec * size);
        const int n = static_cast<int>((s.vec_end - s.vec) * size / 16);
        u32x4 d[kVectors];
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            const int at = threadIdx.x + i * kGradThreads;
            if (at < n) d[i] = __builtin_nontemporal_load(v + at);
        }
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            const int at = threadIdx.x + i * kGradThreads;
            if (at < n) __builtin_nontemporal_store(scale ? scaled(d[i], fp32, f) : d[i], o + at);
        }
        const int64_t head = s.begin + threadIdx.x, tail = s.vec_end + threadIdx.x;
        if (head < s.vec) move(out, p, head, fp32, scale, f);
        if (tail < s.end) move(out, p, tail, fp32, scale, f);
    }
}

int64_t pieces_of(const ep_grad &g) {
    const int64_t size = g.type == EP_GRAD_FP32 ? 4 : 2;
    return (g.count * size + kPiece - 1) / kPiece;
}

// Calls f(table, workgroups) for the gradients in turn, as many in a table as fit it.
template <class F>
hipError_t for_tables(const ep_grad *grads, int32_t num, F f) {
    GradTable t;
    t.num = 0;
    t.fp32 = 0;
    int64_t pieces = 0;
    auto flush = [&] {
        if (t.num == 0) return hipSuccess;
        t.first[t.num] = static_cast<int32_t>(pieces);
        const hipError_t rc = f(t, static_cast<int>(pieces < kGradWorkgroups ? pieces : kGradWorkgroups));
        t.num = 0;
        t.fp32 = 0;
        pieces = 0;
        return rc;
    };
    for (int32_t i = 0; i < num; ++i) {
        const ep_grad &g = grads[i];
        const int64_t n = pieces_of(g);
        if (n == 0) continue;
        if (t.num == kTableSize || pieces + n > INT32_MAX - kGradWorkgroups) {
            const hipError_t rc = flush();
            if (rc != hipSuccess) return rc;
        }
        t.grad[t.num] = static_cast<const char *>(g.grad);
        t.out[t.num] = static_cast<char *>(g.out);
        t.count[t.num] = g.count;
        t.first[t.num] = static_cast<int32_t>(pieces);
        if (g.type == EP_GRAD_FP32) t.fp32 |= uint64_t{1} << t.num;
        ++t.num;
        pieces += n;
    }
    return flush();
}

}  // namespace

// An upper bound of what a part of the list needs too, which is shared among launches in another way: no launch leaves more
// partial sums than kGradWorkgroups, or than it has pieces.
int64_t grad_workspace_bytes(const ep_grad *grads, int32_t num) {
    int64_t pieces = 0, filled = 0;
    for (int32_t i = 0; i < num; ++i) {
        const int64_t n = pieces_of(grads[i]);
        pieces += n;
        filled += n > 0;
    }
    // a launch ends at a full table, or at more pieces than it can number
    const int64_t launches = (filled + kTableSize - 1) / kTableSize + pieces / (INT32_MAX / 2);
    return 256 + std::min(pieces, launches * kGradWorkgroups) * 8;
}

hipError_t launch_square_sum(const ep_grad *grads, int32_t num, double *square_sum, void *workspace, hipStream_t stream) {
    double *partial = static_cast<double *>(workspace);
    int64_t n = 0;
    const hipError_t rc = for_tables(grads, num, [&](const GradTable &t, int G) {
        square_sum_kernel<<<G, kGradThreads, 0, stream>>>(t, partial + n);
        n += G;
        return hipGetLastError();
    });
    if (rc != hipSuccess) return rc;
    square_join_kernel<<<1, kJoinThreads, 0, stream>>>(partial, n, square_sum);
    return hipGetLastError();
}

hipError_t launch_clip(const ep_grad *grads, int32_t num, const double *square_sum, float max_norm, float *norm,
                       hipStream_t stream) {
    bool any = false;
    const hipError_t rc = for_tables(grads, num, [&](const GradTable &t, int G) {
        clip_kernel<<<G, kGradThreads, 0, stream>>>(t, square_sum, max_norm, any ? nullptr : norm);
        any = true;
        return hipGetLastError();
    });
    if (rc != hipSuccess || any || !norm) return rc;
    GradTable none;  // no values: the norm alone
    none.num = 0;
    none.first[0] = 0;
    none.fp32 = 0;
    clip_kernel<<<1, kGradThreads, 0, stream>>>(none, square_sum, max_norm, norm);
    return hipGetLastError();
}

}  // namespace epget
