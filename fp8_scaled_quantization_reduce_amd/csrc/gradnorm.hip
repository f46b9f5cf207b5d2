// gradnorm.hip -- the global norm of many gradients and their clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   coef = min(1, max_norm / (norm + 1e-6)),  out = g coef
// A NaN anywhere gives a NaN norm and a NaN coefficient; an infinite gradient
// gives an infinite norm and the coefficient 0 (1 where max_norm is infinite).
//
// The tensors of a launch are a table in the kernel's arguments, so a call
// copies nothing to the device.  Each tensor is cut into units of kUnit
// elements, the units of all tensors are numbered through, and a fixed grid
// of blocks takes them in turn; a block finds a unit's tensor by bisection in
// the table.  The squares are summed in binary64, which neither overflows (the
// square of the largest binary32 value is 2^256) nor loses small gradients
// next to a long sum; the conversion and the multiply-add run well above the
// memory's rate.  Every block leaves one partial in the stream's slot and
// the clipping kernel's blocks (or, for the norm alone, a one-block kernel)
// add the partials in a fixed order, so equal inputs give equal bits.
#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

namespace {

constexpr int kGnThreads = 256;
constexpr int kUnitVecs = 4;                           // 8-element vectors per lane and unit
constexpr int kUnit = kGnThreads * 8 * kUnitVecs;      // elements of a unit
constexpr int kListMax = 128;                          // tensors of one launch

struct TensorTable {
    const void *g[kListMax];
    void *out[kListMax];
    int64_t n[kListMax];          // elements; bit 62 set: bf16
    uint32_t first[kListMax + 1]; // the tensor's first unit; [count] = all units
    int count;
};
constexpr int64_t kBf16Bit = (int64_t)1 << 62;

__device__ __forceinline__ int find_tensor(const TensorTable &t, uint32_t unit)
{
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= unit) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <typename T> struct Vec8;
template <> struct Vec8<float> {
    typedef float part __attribute__((ext_vector_type(4), aligned(4)));
    static constexpr int kParts = 2;
};
template <> struct Vec8<__bf16> {
    typedef __bf16 part __attribute__((ext_vector_type(8), aligned(2)));
    static constexpr int kParts = 1;
};

// The norm's pass reads with ordinary loads (tensors that fit the last-level
// cache are then found there by the clipping pass); the clipping pass, which
// touches everything for the last time, loads and stores (kLast) with the
// non-temporal hint: 940 MB of fp32 523 -> 510 us, with four times the blocks
// below 480 us.
template <typename T, bool kLast> __device__ __forceinline__ void load8(const T *p, int64_t left, float (&v)[8])
{
    typedef typename Vec8<T>::part P;
    constexpr int kE = 8 / Vec8<T>::kParts;
    if (left >= 8) {
#pragma unroll
        for (int k = 0; k < Vec8<T>::kParts; ++k) {
            const P *q = reinterpret_cast<const P *>(p) + k;
            const P w = kLast ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
            for (int e = 0; e < kE; ++e) v[k * kE + e] = (float)w[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < left ? (float)p[e] : 0.0f;
    }
}

template <typename T> __device__ __forceinline__ void store8(T *p, int64_t left, const float (&v)[8])
{
    typedef typename Vec8<T>::part P;
    constexpr int kE = 8 / Vec8<T>::kParts;
    if (left >= 8) {
#pragma unroll
        for (int k = 0; k < Vec8<T>::kParts; ++k) {
            P w;
#pragma unroll
            for (int e = 0; e < kE; ++e) w[e] = (T)v[k * kE + e];
            __builtin_nontemporal_store(w, reinterpret_cast<P *>(p) + k);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) p[e] = (T)v[e];
    }
}

template <typename T> __device__ __forceinline__ double square_unit(const T *g, int64_t n, int64_t at)
{
    float v[kUnitVecs][8];
#pragma unroll
    for (int u = 0; u < kUnitVecs; ++u) {
        const int64_t i = at + ((int64_t)u * kGnThreads + threadIdx.x) * 8;
        load8<T, false>(g + i, n - i, v[u]);
    }
    double s = 0.0;
#pragma unroll
    for (int u = 0; u < kUnitVecs; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fma((double)v[u][e], (double)v[u][e], s);
    return s;
}

// Sum over the block in a fixed order; every lane gets it.
__device__ __forceinline__ double block_sum(double s)
{
    __shared__ double lds[kGnThreads / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    double r = 0.0;
#pragma unroll
    for (int w = 0; w < kGnThreads / 64; ++w) r += lds[w];
    return r;
}

// Block b's share of the squares -> sq[b] (added to what an earlier launch of
// the same call left there).
__global__ __launch_bounds__(kGnThreads) void square_kernel(TensorTable t, double *sq, bool first)
{
    double s = 0.0;
    for (uint32_t unit = blockIdx.x; unit < t.first[t.count]; unit += gridDim.x) {
        const int k = find_tensor(t, unit);
        const int64_t at = (int64_t)(unit - t.first[k]) * kUnit;
        const int64_t n = t.n[k] & ~kBf16Bit;
        s += t.n[k] & kBf16Bit ? square_unit((const __bf16 *)t.g[k], n, at)
                               : square_unit((const float *)t.g[k], n, at);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) sq[blockIdx.x] = first ? s : sq[blockIdx.x] + s;
}

// norm and coefficient from the partials; every lane gets the coefficient.
__device__ __forceinline__ float clip_coef(const double *sq, int parts, float max_norm, float &norm)
{
    double s = 0.0;
#pragma unroll
    for (int u = 0; u < kParts / kGnThreads; ++u) {
        const int i = u * kGnThreads + threadIdx.x;
        if (i < parts) s += sq[i];
    }
    norm = (float)sqrt(block_sum(s));
    if (max_norm == __builtin_inff()) return norm == norm ? 1.0f : norm; // no bound: inf / inf is not asked
    const float c = max_norm / (norm + 1e-6f);
    return c > 1.0f ? 1.0f : c; // a NaN stays
}

template <typename T>
__device__ __forceinline__ void scale_unit(const T *g, T *out, int64_t n, int64_t at, float coef)
{
    float v[kUnitVecs][8];
#pragma unroll
    for (int u = 0; u < kUnitVecs; ++u) {
        const int64_t i = at + ((int64_t)u * kGnThreads + threadIdx.x) * 8;
        load8<T, true>(g + i, n - i, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnitVecs; ++u) {
        const int64_t i = at + ((int64_t)u * kGnThreads + threadIdx.x) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] *= coef;
        store8<T>(out + i, n - i, v[u]);
    }
}

__global__ __launch_bounds__(kGnThreads) void clip_kernel(TensorTable t, const double *sq, int parts, float max_norm,
                                                          float *norm_out, float *coef_out)
{
    float norm;
    const float coef = clip_coef(sq, parts, max_norm, norm);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) {
        *norm_out = norm;
        *coef_out = coef;
    }
    for (uint32_t unit = blockIdx.x; unit < t.first[t.count]; unit += gridDim.x) {
        const int k = find_tensor(t, unit);
        if (coef == 1.0f && t.out[k] == t.g[k]) continue; // in place: nothing changes
        const int64_t at = (int64_t)(unit - t.first[k]) * kUnit;
        const int64_t n = t.n[k] & ~kBf16Bit;
        if (t.n[k] & kBf16Bit) scale_unit((const __bf16 *)t.g[k], (__bf16 *)t.out[k], n, at, coef);
        else scale_unit((const float *)t.g[k], (float *)t.out[k], n, at, coef);
    }
}

// One partial per block bounds the first grid; the second is larger, so that
// few blocks walk: 2048 blocks 510 us, 16384 480 us, 65536 497 us (940 MB).
constexpr int kSquareGrid = kParts, kClipGrid = 16384;

} // namespace

hipError_t launch_grad_norm_clip(const void *const *g, void *const *out, const int64_t *n, const int32_t *dtype,
                                 int count, float max_norm, bool clip, float *norm, float *coef, double *sq,
                                 hipStream_t s)
{
    // one table per launch; the same walk for the norm and for the clipping
    auto table = [&](int at, TensorTable &t) {
        uint32_t units = 0;
        t.count = 0;
        while (at < count && t.count < kListMax) {
            if (n[at] > 0) {
                const int64_t u = (n[at] + kUnit - 1) / kUnit;
                if (t.count && units + u > 0x7FFFFFFF) break;
                t.g[t.count] = g[at];
                t.out[t.count] = out ? out[at] : const_cast<void *>(g[at]);
                t.n[t.count] = n[at] | (dtype[at] == kBF16 ? kBf16Bit : 0);
                t.first[t.count++] = units;
                units += (uint32_t)u;
            }
            ++at;
        }
        t.first[t.count] = units;
        return at;
    };
    TensorTable t;
    // every launch runs the grid of the largest, so that each slot is written
    int parts = 1;
    for (int at = 0; at < count;) {
        at = table(at, t);
        const int u = (int)(t.first[t.count] < (uint32_t)kSquareGrid ? t.first[t.count] : kSquareGrid);
        parts = u > parts ? u : parts;
    }
    int at = 0;
    do {
        const bool first = at == 0;
        at = table(at, t);
        square_kernel<<<parts, kGnThreads, 0, s>>>(t, sq, first);
    } while (at < count);
    at = 0;
    do {
        const bool first = at == 0;
        at = clip ? table(at, t) : count;
        if (!clip) t.count = 0, t.first[0] = 0;
        const uint32_t u = t.first[t.count];
        const int grid = (int)(u < 1 ? 1 : u < (uint32_t)kClipGrid ? u : (uint32_t)kClipGrid);
        clip_kernel<<<grid, kGnThreads, 0, s>>>(t, sq, parts, max_norm, first ? norm : nullptr, coef);
    } while (at < count);
    return hipGetLastError();
}

} // namespace fp8q
