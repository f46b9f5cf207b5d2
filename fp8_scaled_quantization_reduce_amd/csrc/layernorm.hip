// layernorm.hip -- layer norm over the rows of a matrix and its backward pass,
// the step that produces the activations the FP8 casts read.
//
// Forward, per row of n columns:
//   mean = sum x / n,  var = sum (x - mean)^2 / n,  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd gamma + beta
// Backward, with xh = (x - mean) rstd and h = dy gamma:
//   dx = rstd (h - sum h / n - xh sum(h xh) / n)
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
// All sums and statistics are binary32; the variance is a second pass over
// the row's values in registers (the difference of two large sums would lose
// the variance of rows whose mean is far from zero).  Values are rounded once,
// when y, dx, dgamma and dbeta are stored in their type.
//
// A row is held in registers by R lanes (one wave for short rows, a block of
// 256 or 1024 otherwise), kI vectors of 16 bytes per lane, so x and dy are read
// once.  Rows longer than that are read again for each pass (ln_*_long).
// Rows may start at any element: vectors are loaded with element alignment
// (gfx950 loads and stores 16 bytes at any address) and the row's last,
// partial vector by elements.
#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

namespace {

constexpr int kLnThreads = 256;

template <int DT> struct Elem;
template <> struct Elem<kF32> {
    typedef float type;
    static constexpr int kVec = 4;
};
template <> struct Elem<kBF16> {
    typedef __bf16 type;
    static constexpr int kVec = 8;
};

// kV elements of type DT at p -> floats; elements from `left` on are zero.
template <int DT, int kV>
__device__ __forceinline__ void load_vec(const typename Elem<DT>::type *p, int64_t left, float (&v)[kV])
{
    typedef typename Elem<DT>::type T;
    typedef T vec_t __attribute__((ext_vector_type(kV), aligned(sizeof(T))));
    if (left >= kV) {
        const vec_t w = *reinterpret_cast<const vec_t *>(p);
#pragma unroll
        for (int e = 0; e < kV; ++e) v[e] = (float)w[e];
    } else {
#pragma unroll
        for (int e = 0; e < kV; ++e) v[e] = e < left ? (float)p[e] : 0.0f;
    }
}

template <int DT, int kV>
__device__ __forceinline__ void store_vec(typename Elem<DT>::type *p, int64_t left, const float (&v)[kV])
{
    typedef typename Elem<DT>::type T;
    typedef T vec_t __attribute__((ext_vector_type(kV), aligned(sizeof(T))));
    if (left >= kV) {
        vec_t w;
#pragma unroll
        for (int e = 0; e < kV; ++e) w[e] = (T)v[e];
        *reinterpret_cast<vec_t *>(p) = w;
    } else {
#pragma unroll
        for (int e = 0; e < kV; ++e)
            if (e < left) p[e] = (T)v[e];
    }
}

// Sums over the R lanes that share a row (a wave, or the block through LDS:
// one slot per wave and value, two sets used in turn so that one barrier per
// reduction is enough).
template <int R, int kN>
__device__ __forceinline__ void row_sum(float (&v)[kN], float (*lds)[kN][16], int set)
{
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = wave_sum_f32(v[k]);
    if constexpr (R > 64) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int k = 0; k < kN; ++k)
            if (lane == 0) lds[set][k][wave] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < R / 64; ++w) s += lds[set][k][w];
            v[k] = s;
        }
    }
}

template <int DT, int PT, int R, int kI>
__global__ __launch_bounds__(R > kLnThreads ? R : kLnThreads) void ln_fwd_kernel(
    const typename Elem<DT>::type *__restrict__ x, int64_t rows, int64_t cols,
    const typename Elem<PT>::type *__restrict__ gamma, const typename Elem<PT>::type *__restrict__ beta, float eps,
    typename Elem<DT>::type *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd)
{
    constexpr int kV = Elem<DT>::kVec, kRows = R > kLnThreads ? 1 : kLnThreads / R;
    __shared__ float lds[2][1][16];
    const int t = threadIdx.x % R;
    const float n = (float)cols;
    // a block whose rows are shared by all its lanes walks whole rounds, so
    // that every lane reaches the barriers
    for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / R; row < rows; row += (int64_t)gridDim.x * kRows) {
        const typename Elem<DT>::type *xr = x + row * cols;
        float v[kI][kV];
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const int64_t c = ((int64_t)i * R + t) * kV;
            load_vec<DT, kV>(xr + c, cols - c, v[i]);
#pragma unroll
            for (int e = 0; e < kV; ++e) s[0] += v[i][e];
        }
        row_sum<R, 1>(s, lds, 0);
        const float mu = s[0] / n;
        float q[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const int64_t c = ((int64_t)i * R + t) * kV;
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                v[i][e] -= mu;
                q[0] += c + e < cols ? v[i][e] * v[i][e] : 0.0f;
            }
        }
        row_sum<R, 1>(q, lds, 1);
        const float rs = 1.0f / sqrtf(q[0] / n + eps);
        if (t == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = rs;
        }
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const int64_t c = ((int64_t)i * R + t) * kV;
            float g[kV], b[kV];
            if (gamma) load_vec<PT, kV>(gamma + c, cols - c, g);
            if (beta) load_vec<PT, kV>(beta + c, cols - c, b);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                float o = v[i][e] * rs;
                if (gamma) o *= g[e];
                if (beta) o += b[e];
                v[i][e] = o;
            }
            store_vec<DT, kV>(y + row * cols + c, cols - c, v[i]);
        }
    }
}

// Rows too long for registers: three passes over the row.
constexpr int kLnLong = 1024;

template <int DT, int PT>
__global__ __launch_bounds__(kLnLong) void ln_fwd_long(const typename Elem<DT>::type *__restrict__ x, int64_t rows,
                                                       int64_t cols, const typename Elem<PT>::type *__restrict__ gamma,
                                                       const typename Elem<PT>::type *__restrict__ beta, float eps,
                                                       typename Elem<DT>::type *__restrict__ y,
                                                       float *__restrict__ mean, float *__restrict__ rstd)
{
    constexpr int kV = Elem<DT>::kVec;
    __shared__ float lds[2][1][16];
    const float n = (float)cols;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const typename Elem<DT>::type *xr = x + row * cols;
        float s[1] = {0.0f};
        for (int64_t c = (int64_t)threadIdx.x * kV; c < cols; c += (int64_t)kLnLong * kV) {
            float v[kV];
            load_vec<DT, kV>(xr + c, cols - c, v);
#pragma unroll
            for (int e = 0; e < kV; ++e) s[0] += v[e];
        }
        row_sum<kLnLong, 1>(s, lds, 0);
        const float mu = s[0] / n;
        float q[1] = {0.0f};
        for (int64_t c = (int64_t)threadIdx.x * kV; c < cols; c += (int64_t)kLnLong * kV) {
            float v[kV];
            load_vec<DT, kV>(xr + c, cols - c, v);
#pragma unroll
            for (int e = 0; e < kV; ++e) q[0] += c + e < cols ? (v[e] - mu) * (v[e] - mu) : 0.0f;
        }
        row_sum<kLnLong, 1>(q, lds, 1);
        const float rs = 1.0f / sqrtf(q[0] / n + eps);
        if (threadIdx.x == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = rs;
        }
        for (int64_t c = (int64_t)threadIdx.x * kV; c < cols; c += (int64_t)kLnLong * kV) {
            float v[kV], g[kV], b[kV];
            load_vec<DT, kV>(xr + c, cols - c, v);
            if (gamma) load_vec<PT, kV>(gamma + c, cols - c, g);
            if (beta) load_vec<PT, kV>(beta + c, cols - c, b);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                float o = (v[e] - mu) * rs;
                if (gamma) o *= g[e];
                if (beta) o += b[e];
                v[e] = o;
            }
            store_vec<DT, kV>(y + row * cols + c, cols - c, v);
        }
    }
}

// Backward: each R-lane team walks its share of the rows and keeps its
// columns' sums of dy xh and dy in registers; at the end it writes them to its
// slot of the workspace, [slot][2][cols] (ws null: no parameter gradients).
template <int DT, int PT, int R, int kI>
__global__ __launch_bounds__(R > kLnThreads ? R : kLnThreads) void ln_bwd_kernel(
    const typename Elem<DT>::type *__restrict__ dy, const typename Elem<DT>::type *__restrict__ x, int64_t rows,
    int64_t cols, const typename Elem<PT>::type *__restrict__ gamma, const float *__restrict__ mean,
    const float *__restrict__ rstd, typename Elem<DT>::type *__restrict__ dx, float *__restrict__ ws)
{
    constexpr int kV = Elem<DT>::kVec, kRows = R > kLnThreads ? 1 : kLnThreads / R;
    __shared__ float lds[2][2][16];
    const int t = threadIdx.x % R;
    const int64_t team = (int64_t)blockIdx.x * kRows + threadIdx.x / R;
    const float n = (float)cols;
    float g[kI][kV], dg[kI][kV], db[kI][kV];
#pragma unroll
    for (int i = 0; i < kI; ++i) {
        const int64_t c = ((int64_t)i * R + t) * kV;
        if (gamma) load_vec<PT, kV>(gamma + c, cols - c, g[i]);
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            if (!gamma) g[i][e] = 1.0f;
            dg[i][e] = db[i][e] = 0.0f;
        }
    }
    int set = 0;
    for (int64_t row = team; row < rows; row += (int64_t)gridDim.x * kRows) {
        const float mu = mean[row], rs = rstd[row];
        float xh[kI][kV], h[kI][kV];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const int64_t c = ((int64_t)i * R + t) * kV;
            load_vec<DT, kV>(x + row * cols + c, cols - c, xh[i]);
            load_vec<DT, kV>(dy + row * cols + c, cols - c, h[i]);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                // columns past the row have dy = 0 and add nothing, but their
                // xh must stay finite
                xh[i][e] = c + e < cols ? (xh[i][e] - mu) * rs : 0.0f;
                dg[i][e] += h[i][e] * xh[i][e];
                db[i][e] += h[i][e];
                h[i][e] *= g[i][e];
                s[0] += h[i][e];
                s[1] += h[i][e] * xh[i][e];
            }
        }
        row_sum<R, 2>(s, lds, set);
        set ^= 1;
        const float m1 = s[0] / n, m2 = s[1] / n;
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const int64_t c = ((int64_t)i * R + t) * kV;
#pragma unroll
            for (int e = 0; e < kV; ++e) h[i][e] = (h[i][e] - m1 - xh[i][e] * m2) * rs;
            store_vec<DT, kV>(dx + row * cols + c, cols - c, h[i]);
        }
    }
    if (ws) {
        float *slot = ws + team * 2 * cols;
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const int64_t c = ((int64_t)i * R + t) * kV;
#pragma unroll
            for (int e = 0; e < kV; ++e)
                if (c + e < cols) {
                    slot[c + e] = dg[i][e];
                    slot[cols + c + e] = db[i][e];
                }
        }
    }
}

// dx of rows too long for registers.
template <int DT, int PT>
__global__ __launch_bounds__(kLnLong) void ln_bwd_long(const typename Elem<DT>::type *__restrict__ dy,
                                                       const typename Elem<DT>::type *__restrict__ x, int64_t rows,
                                                       int64_t cols, const typename Elem<PT>::type *__restrict__ gamma,
                                                       const float *__restrict__ mean, const float *__restrict__ rstd,
                                                       typename Elem<DT>::type *__restrict__ dx)
{
    constexpr int kV = Elem<DT>::kVec;
    __shared__ float lds[2][2][16];
    const float n = (float)cols;
    int set = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float mu = mean[row], rs = rstd[row];
        float s[2] = {0.0f, 0.0f};
        for (int64_t c = (int64_t)threadIdx.x * kV; c < cols; c += (int64_t)kLnLong * kV) {
            float v[kV], d[kV], g[kV];
            load_vec<DT, kV>(x + row * cols + c, cols - c, v);
            load_vec<DT, kV>(dy + row * cols + c, cols - c, d);
            if (gamma) load_vec<PT, kV>(gamma + c, cols - c, g);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const float h = gamma ? d[e] * g[e] : d[e];
                s[0] += h;
                s[1] += c + e < cols ? h * ((v[e] - mu) * rs) : 0.0f;
            }
        }
        row_sum<kLnLong, 2>(s, lds, set);
        set ^= 1;
        const float m1 = s[0] / n, m2 = s[1] / n;
        for (int64_t c = (int64_t)threadIdx.x * kV; c < cols; c += (int64_t)kLnLong * kV) {
            float v[kV], d[kV], g[kV];
            load_vec<DT, kV>(x + row * cols + c, cols - c, v);
            load_vec<DT, kV>(dy + row * cols + c, cols - c, d);
            if (gamma) load_vec<PT, kV>(gamma + c, cols - c, g);
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const float h = gamma ? d[e] * g[e] : d[e];
                v[e] = (h - m1 - (v[e] - mu) * rs * m2) * rs;
            }
            store_vec<DT, kV>(dx + row * cols + c, cols - c, v);
        }
    }
}

// Sums of dy xh and dy of 64 columns over a share of the rows (long rows):
// four waves take rows in turn, then fold through LDS into slot blockIdx.y.
template <int DT>
__global__ __launch_bounds__(kLnThreads) void ln_bwd_cols(const typename Elem<DT>::type *__restrict__ dy,
                                                          const typename Elem<DT>::type *__restrict__ x, int64_t rows,
                                                          int64_t cols, const float *__restrict__ mean,
                                                          const float *__restrict__ rstd, float *__restrict__ ws)
{
    __shared__ float lds[2][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float dg = 0.0f, db = 0.0f;
    if (c < cols) {
        for (int64_t row = (int64_t)blockIdx.y * 4 + wave; row < rows; row += (int64_t)gridDim.y * 4) {
            const float d = (float)dy[row * cols + c];
            dg += d * (((float)x[row * cols + c] - mean[row]) * rstd[row]);
            db += d;
        }
    }
    lds[0][wave][lane] = dg;
    lds[1][wave][lane] = db;
    __syncthreads();
    if (wave < 2 && c < cols)
        ws[((int64_t)blockIdx.y * 2 + wave) * cols + c] =
            lds[wave][0][lane] + lds[wave][1][lane] + lds[wave][2][lane] + lds[wave][3][lane];
}

// Fold `slots` partial rows of the workspace: 32 columns per block, eight
// lanes per column taking slots in turn.  blockIdx.y: 0 dgamma, 1 dbeta.
template <int PT>
__global__ __launch_bounds__(kLnThreads) void ln_bwd_fold(const float *__restrict__ ws, int slots, int64_t cols,
                                                          typename Elem<PT>::type *__restrict__ dgamma,
                                                          typename Elem<PT>::type *__restrict__ dbeta)
{
    __shared__ float lds[8][32];
    const int j = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + j;
    typename Elem<PT>::type *out = blockIdx.y ? dbeta : dgamma;
    if (!out) return;
    float s = 0.0f;
    if (c < cols)
        for (int p = k; p < slots; p += 8) s += ws[((int64_t)p * 2 + blockIdx.y) * cols + c];
    lds[k][j] = s;
    __syncthreads();
    if (k == 0 && c < cols) {
#pragma unroll
        for (int p = 1; p < 8; ++p) s += lds[p][j];
        out[c] = (typename Elem<PT>::type)s;
    }
}

// The lanes per row and vectors per lane that hold a row of `cols` elements
// of `vec`-element vectors; lanes 0: the row is too long for registers.
struct LnShape {
    int lanes, vecs;
};
LnShape ln_shape(int64_t cols, int vec)
{
    const int64_t v = (cols + vec - 1) / vec;
    if (v <= 64) return {64, 1};
    if (v <= 128) return {64, 2};
    if (v <= 256) return {256, 1};
    if (v <= 512) return {256, 2};
    if (v <= 1024) return {256, 4};
    if (v <= 2048) return {1024, 2};
    if (v <= 4096) return {1024, 4};
    return {0, 0};
}
int vec_of(int dtype) { return dtype == kF32 ? 4 : 8; }

constexpr int64_t kLnMaxGrid = 1 << 20;
// Blocks of the backward pass: each leaves one partial row per team.
constexpr int kLnBwdBlocks = 512;

int bwd_blocks(int64_t rows, LnShape sh)
{
    const int per = sh.lanes == 64 ? kLnThreads / 64 : 1; // teams per block
    const int64_t want = (rows + per - 1) / per;
    const int cap = kLnBwdBlocks / per;
    return (int)(want < cap ? (want < 1 ? 1 : want) : cap);
}
int bwd_slots(int64_t rows, int64_t cols, int dtype)
{
    const LnShape sh = ln_shape(cols, vec_of(dtype));
    if (sh.lanes == 0) { // ln_bwd_cols: slots of 32 rows or more
        const int64_t s = (rows + 31) / 32;
        return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
    }
    return bwd_blocks(rows, sh) * (sh.lanes == 64 ? kLnThreads / 64 : 1);
}

template <int DT, int PT>
hipError_t fwd(const void *x_, int64_t rows, int64_t cols, const void *gamma_, const void *beta_, float eps, void *y_,
               float *mean, float *rstd, hipStream_t s)
{
    typedef typename Elem<DT>::type T;
    typedef typename Elem<PT>::type P;
    const T *x = (const T *)x_;
    const P *gamma = (const P *)gamma_, *beta = (const P *)beta_;
    T *y = (T *)y_;
    const LnShape sh = ln_shape(cols, Elem<DT>::kVec);
    const int per = sh.lanes == 64 ? kLnThreads / 64 : 1;
    int64_t g = (rows + per - 1) / per;
    const int grid = (int)(g < kLnMaxGrid ? g : kLnMaxGrid);
#define FP8Q_LN(R, I)                                                                                                \
    if (sh.lanes == R && sh.vecs == I)                                                                               \
        ln_fwd_kernel<DT, PT, R, I><<<grid, R > kLnThreads ? R : kLnThreads, 0, s>>>(x, rows, cols, gamma, beta,     \
                                                                                     eps, y, mean, rstd);
    FP8Q_LN(64, 1)
    FP8Q_LN(64, 2)
    FP8Q_LN(256, 1)
    FP8Q_LN(256, 2)
    FP8Q_LN(256, 4)
    FP8Q_LN(1024, 2)
    FP8Q_LN(1024, 4)
#undef FP8Q_LN
    if (sh.lanes == 0) ln_fwd_long<DT, PT><<<grid, kLnLong, 0, s>>>(x, rows, cols, gamma, beta, eps, y, mean, rstd);
    return hipGetLastError();
}

template <int DT, int PT>
hipError_t bwd(const void *dy_, const void *x_, int64_t rows, int64_t cols, const void *gamma_, const float *mean,
               const float *rstd, void *dx_, void *dgamma, void *dbeta, float *ws, hipStream_t s)
{
    typedef typename Elem<DT>::type T;
    typedef typename Elem<PT>::type P;
    const T *dy = (const T *)dy_, *x = (const T *)x_;
    const P *gamma = (const P *)gamma_;
    T *dx = (T *)dx_;
    const bool params = dgamma || dbeta;
    const LnShape sh = ln_shape(cols, Elem<DT>::kVec);
    const int slots = bwd_slots(rows, cols, DT);
    if (rows > 0) {
        const int grid = sh.lanes ? bwd_blocks(rows, sh) : (int)(rows < kLnMaxGrid ? rows : kLnMaxGrid);
        float *w = params ? ws : nullptr;
#define FP8Q_LN(R, I)                                                                                                \
    if (sh.lanes == R && sh.vecs == I)                                                                               \
        ln_bwd_kernel<DT, PT, R, I><<<grid, R > kLnThreads ? R : kLnThreads, 0, s>>>(dy, x, rows, cols, gamma, mean, \
                                                                                     rstd, dx, w);
        FP8Q_LN(64, 1)
        FP8Q_LN(64, 2)
        FP8Q_LN(256, 1)
        FP8Q_LN(256, 2)
        FP8Q_LN(256, 4)
        FP8Q_LN(1024, 2)
        FP8Q_LN(1024, 4)
#undef FP8Q_LN
        if (sh.lanes == 0) {
            ln_bwd_long<DT, PT><<<grid, kLnLong, 0, s>>>(dy, x, rows, cols, gamma, mean, rstd, dx);
            if (params)
                ln_bwd_cols<DT><<<dim3((unsigned)((cols + 63) / 64), (unsigned)slots), kLnThreads, 0, s>>>(
                    dy, x, rows, cols, mean, rstd, w);
        }
    }
    // no rows: the parameter gradients are zero
    if (params)
        ln_bwd_fold<PT><<<dim3((unsigned)((cols + 31) / 32), 2), kLnThreads, 0, s>>>(ws, rows > 0 ? slots : 0, cols,
                                                                                     (P *)dgamma, (P *)dbeta);
    return hipGetLastError();
}

} // namespace

int64_t layernorm_bwd_workspace(int64_t rows, int64_t cols, int dtype)
{
    return (int64_t)bwd_slots(rows, cols, dtype) * 2 * cols * 4;
}

hipError_t launch_layernorm(const void *x, int dtype, int64_t rows, int64_t cols, const void *gamma, const void *beta,
                            int p_dtype, float eps, void *y, float *mean, float *rstd, hipStream_t s)
{
    if (rows == 0) return hipSuccess;
    auto f = dtype == kF32 ? (p_dtype == kF32 ? fwd<kF32, kF32> : fwd<kF32, kBF16>)
                           : (p_dtype == kF32 ? fwd<kBF16, kF32> : fwd<kBF16, kBF16>);
    return f(x, rows, cols, gamma, beta, eps, y, mean, rstd, s);
}

hipError_t launch_layernorm_bwd(const void *dy, const void *x, int dtype, int64_t rows, int64_t cols,
                                const void *gamma, int p_dtype, const float *mean, const float *rstd, void *dx,
                                void *dgamma, void *dbeta, float *ws, hipStream_t s)
{
    auto f = dtype == kF32 ? (p_dtype == kF32 ? bwd<kF32, kF32> : bwd<kF32, kBF16>)
                           : (p_dtype == kF32 ? bwd<kBF16, kF32> : bwd<kBF16, kBF16>);
    return f(dy, x, rows, cols, gamma, mean, rstd, dx, dgamma, dbeta, ws, s);
}

} // namespace fp8q
