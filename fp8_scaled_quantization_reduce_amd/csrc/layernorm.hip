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
// (gfx950 loads and stores 16 bytes at any address).  The last cols % kVec
// columns are one more element of the first lanes.
#include "fp8q_device.h"
#include "fp8q_launch.h"

namespace fp8q {

namespace {

constexpr int kLnThreads = 256;

template <int DT> struct Elem;
template <> struct Elem<kF32> {
    typedef float type;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(4)));
    static constexpr int kVec = 4;
};
template <> struct Elem<kBF16> {
    typedef __bf16 type;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2)));
    static constexpr int kVec = 8;
};

// kV elements of type DT at p -> floats; zeros where there is no vector.
template <int DT, int kV>
__device__ __forceinline__ void load_vec(const typename Elem<DT>::type *p, bool has, float (&v)[kV])
{
    typedef typename Elem<DT>::type T;
    typedef T vec_t __attribute__((ext_vector_type(kV), aligned(sizeof(T))));
    if (has) {
        const vec_t w = *reinterpret_cast<const vec_t *>(p);
#pragma unroll
        for (int e = 0; e < kV; ++e) v[e] = (float)w[e];
    } else {
#pragma unroll
        for (int e = 0; e < kV; ++e) v[e] = 0.0f;
    }
}

// kStream: not read again here (y, dx), so with the non-temporal hint, which
// leaves the caches to the rows being read: 30000x1111 bf16 40.5 -> 35.9 us,
// 2051x5003 fp32 18.2 -> 17.0, the backward pass 16384x4096 76.3 -> 74.3.
template <int DT, int kV, bool kStream>
__device__ __forceinline__ void store_vec(typename Elem<DT>::type *p, bool has, const float (&v)[kV])
{
    typedef typename Elem<DT>::type T;
    typedef T vec_t __attribute__((ext_vector_type(kV), aligned(sizeof(T))));
    if (has) {
        vec_t w;
#pragma unroll
        for (int e = 0; e < kV; ++e) w[e] = (T)v[e];
        if constexpr (kStream) __builtin_nontemporal_store(w, reinterpret_cast<vec_t *>(p));
        else *reinterpret_cast<vec_t *>(p) = w;
    }
}

// kLast: read for the last time, so with the non-temporal hint (the backward
// pass: 16384x4096 bf16 89.4 -> 87.4 us, 8192x4096 fp32 91.2 -> 86.5 us)
template <int DT, bool kLast> __device__ __forceinline__ uint4 load_raw(const typename Elem<DT>::type *p, bool has)
{
    if (!has) return make_uint4(0u, 0u, 0u, 0u);
    const typename Elem<DT>::raw *q = reinterpret_cast<const typename Elem<DT>::raw *>(p);
    const typename Elem<DT>::raw r = kLast ? __builtin_nontemporal_load(q) : *q;
    return make_uint4(r.x, r.y, r.z, r.w);
}

template <int DT, int kV> __device__ __forceinline__ void widen(const uint4 &w, float (&v)[kV])
{
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == kF32) v[k] = __uint_as_float(d[k]);
        else v[2 * k] = bf16_lo(d[k]), v[2 * k + 1] = bf16_hi(d[k]);
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

// Where a lane's columns are: vectors i * R + t of the row's `vecs` whole ones,
// and column tail + t if it is in the row.  kFull: the row is exactly the
// lanes' vectors, and nothing is checked.
template <int R, int kV, bool kFull> struct Cols {
    int t, vecs, tail, cols;
    __device__ __forceinline__ Cols(int t_, int cols_) : t(t_), vecs(cols_ / kV), tail(cols_ / kV * kV), cols(cols_) {}
    __device__ __forceinline__ bool has(int i) const { return kFull || i * R + t < vecs; }
    __device__ __forceinline__ int at(int i) const { return (i * R + t) * kV; }
    __device__ __forceinline__ bool has_tail() const { return !kFull && tail + t < cols; }
    __device__ __forceinline__ int at_tail() const { return tail + t; }
};

// Each R-lane team walks its share of the rows: the next row is fetched before
// the row in hand is reduced, and (kHeld) the gain and bias stay in registers.
// Memory bounds it: 16384x4096 bf16 51.5 us, 5.2 TB/s (63 us without the row
// ahead); 2051x5003 fp32 16.8 us, 4.9 TB/s; one row of 4096 2.7 us, its launch.
template <int DT, int PT, int R, int kI, bool kFull>
__global__ __launch_bounds__(R > kLnThreads ? R : kLnThreads) void ln_fwd_kernel(
    const typename Elem<DT>::type *__restrict__ x, int64_t rows, int64_t cols_,
    const typename Elem<PT>::type *__restrict__ gamma, const typename Elem<PT>::type *__restrict__ beta, float eps,
    typename Elem<DT>::type *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd)
{
    typedef typename Elem<DT>::type T;
    constexpr int kV = Elem<DT>::kVec, kRows = R > kLnThreads ? 1 : kLnThreads / R;
    constexpr bool kHeld = kI * kV <= 16;
    __shared__ float lds[2][1][16];
    const Cols<R, kV, kFull> col(threadIdx.x % R, kFull ? R * kI * kV : (int)cols_);
    const float n = (float)col.cols;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / R;
    uint4 w[kI];
    T wt = (T)0.0f;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < kI; ++i) w[i] = load_raw<DT, false>(x + r * col.cols + col.at(i), col.has(i));
        if (col.has_tail()) wt = x[r * col.cols + col.at_tail()];
    };
    if (kHeld && row < rows) fetch(row);
    float g[kHeld ? kI : 1][kV], b[kHeld ? kI : 1][kV], gt = 1.0f, bt = 0.0f;
    if constexpr (kHeld) {
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            if (gamma) load_vec<PT, kV>(gamma + col.at(i), col.has(i), g[i]);
            if (beta) load_vec<PT, kV>(beta + col.at(i), col.has(i), b[i]);
        }
    }
    if (col.has_tail()) {
        if (gamma) gt = (float)gamma[col.at_tail()];
        if (beta) bt = (float)beta[col.at_tail()];
    }
    // a block whose rows are shared by all its lanes walks whole rounds, so
    // that every lane reaches the barriers
    for (; row < rows; row += step) {
        T *yr = y + row * col.cols;
        if constexpr (!kHeld) fetch(row);
        float v[kI][kV], vt = (float)wt;
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kI; ++i) widen<DT, kV>(w[i], v[i]);
        if (kHeld && row + step < rows) fetch(row + step);
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int e = 0; e < kV; ++e) s[0] += v[i][e];
        if (col.has_tail()) s[0] += vt;
        row_sum<R, 1>(s, lds, 0);
        const float mu = s[0] / n;
        float q[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            float d = 0.0f;
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                v[i][e] -= mu;
                d += v[i][e] * v[i][e];
            }
            q[0] += col.has(i) ? d : 0.0f;
        }
        vt -= mu;
        if (col.has_tail()) q[0] += vt * vt;
        row_sum<R, 1>(q, lds, 1);
        const float rs = 1.0f / sqrtf(q[0] / n + eps);
        if (col.t == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = rs;
        }
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            constexpr int kP = kHeld ? 1 : 0;
            if constexpr (!kHeld) {
                if (gamma) load_vec<PT, kV>(gamma + col.at(i), col.has(i), g[0]);
                if (beta) load_vec<PT, kV>(beta + col.at(i), col.has(i), b[0]);
            }
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                float o = v[i][e] * rs;
                if (gamma) o *= g[kP * i][e];
                if (beta) o += b[kP * i][e];
                v[i][e] = o;
            }
            store_vec<DT, kV, true>(yr + col.at(i), col.has(i), v[i]);
        }
        if (col.has_tail()) yr[col.at_tail()] = (T)(vt * rs * gt + bt);
    }
}

// Rows too long for registers: three passes over the row, in one lane's
// elements of each round (rare, so by elements).  The latency of these short
// loads bounds them: 1000x20000 fp32 66 us, 2.4 TB/s, 300x40001 bf16 40 us, 1.2
// TB/s; the backward pass (ln_bwd_long and ln_bwd_cols) 95 to 103 and 82 us.
constexpr int kLnLong = 1024;
constexpr int kFoldThreads = 1024;

template <int DT, int PT>
__global__ __launch_bounds__(kLnLong) void ln_fwd_long(const typename Elem<DT>::type *__restrict__ x, int64_t rows,
                                                       int64_t cols, const typename Elem<PT>::type *__restrict__ gamma,
                                                       const typename Elem<PT>::type *__restrict__ beta, float eps,
                                                       typename Elem<DT>::type *__restrict__ y,
                                                       float *__restrict__ mean, float *__restrict__ rstd)
{
    __shared__ float lds[2][1][16];
    const float n = (float)cols;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const typename Elem<DT>::type *xr = x + row * cols;
        float s[1] = {0.0f};
#pragma unroll 8
        for (int64_t c = threadIdx.x; c < cols; c += kLnLong) s[0] += (float)xr[c];
        row_sum<kLnLong, 1>(s, lds, 0);
        const float mu = s[0] / n;
        float q[1] = {0.0f};
#pragma unroll 8
        for (int64_t c = threadIdx.x; c < cols; c += kLnLong) {
            const float d = (float)xr[c] - mu;
            q[0] += d * d;
        }
        row_sum<kLnLong, 1>(q, lds, 1);
        const float rs = 1.0f / sqrtf(q[0] / n + eps);
        if (threadIdx.x == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = rs;
        }
#pragma unroll 4
        for (int64_t c = threadIdx.x; c < cols; c += kLnLong) {
            float o = ((float)xr[c] - mu) * rs;
            if (gamma) o *= (float)gamma[c];
            if (beta) o += (float)beta[c];
            y[row * cols + c] = (typename Elem<DT>::type)o;
        }
    }
}

// Backward: each R-lane team walks its share of the rows and keeps its
// columns' sums of dy xh and dy in registers; at the end the block writes them
// to its slot of the workspace, [slot][2][cols] (ws null: no parameter
// gradients).
// The row's x and dy stay as loaded (bf16 pairs) and are widened again after
// the reduction; the next row's are fetched before it, so that a team always
// has a row in flight (kAhead; with eight vectors a lane of fp32 that would
// spill: 2000x16384 122 us, without it 90).  Memory bounds it: 16384x4096 bf16
// 74 us with the fold of the partials, 5.4 TB/s; 16 resident waves a CU.
template <int DT, int PT, int R, int kI, bool kFull>
__global__ __launch_bounds__(R > kLnThreads ? R : kLnThreads, 2) void ln_bwd_kernel(
    const typename Elem<DT>::type *__restrict__ dy, const typename Elem<DT>::type *__restrict__ x, int64_t rows,
    int64_t cols_, const typename Elem<PT>::type *__restrict__ gamma, const float *__restrict__ mean,
    const float *__restrict__ rstd, typename Elem<DT>::type *__restrict__ dx, float *__restrict__ ws)
{
    typedef typename Elem<DT>::type T;
    constexpr int kV = Elem<DT>::kVec, kRows = R > kLnThreads ? 1 : kLnThreads / R;
    constexpr bool kAhead = kI <= 6;
    __shared__ float lds[2][2][16];
    const Cols<R, kV, kFull> col(threadIdx.x % R, kFull ? R * kI * kV : (int)cols_);
    const int64_t team = (int64_t)blockIdx.x * kRows + threadIdx.x / R, step = (int64_t)gridDim.x * kRows;
    const float n = (float)col.cols;
    float g[kI][kV], dg[kI][kV], db[kI][kV], gt = 1.0f, dgt = 0.0f, dbt = 0.0f;
#pragma unroll
    for (int i = 0; i < kI; ++i) {
        if (gamma) load_vec<PT, kV>(gamma + col.at(i), col.has(i), g[i]);
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            if (!gamma) g[i][e] = 1.0f;
            dg[i][e] = db[i][e] = 0.0f;
        }
    }
    if (gamma && col.has_tail()) gt = (float)gamma[col.at_tail()];
    struct Row {
        uint4 x[kI], dy[kI];
        T xt, dyt;
        float mu, rs;
    };
    auto fetch = [&](int64_t row, Row &r) {
        r.mu = mean[row], r.rs = rstd[row];
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            r.x[i] = load_raw<DT, true>(x + row * col.cols + col.at(i), col.has(i));
            r.dy[i] = load_raw<DT, true>(dy + row * col.cols + col.at(i), col.has(i));
        }
        if (col.has_tail()) r.xt = x[row * col.cols + col.at_tail()], r.dyt = dy[row * col.cols + col.at_tail()];
    };
    Row cur;
    if (kAhead && team < rows) fetch(team, cur);
    int set = 0;
    for (int64_t row = team; row < rows; row += step) {
        Row next;
        if constexpr (kAhead) {
            next = cur;
            if (row + step < rows) fetch(row + step, next);
        } else {
            fetch(row, cur);
        }
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            float xv[kV], d[kV];
            widen<DT, kV>(cur.x[i], xv);
            widen<DT, kV>(cur.dy[i], d);
            if (!col.has(i)) continue;
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const float xh = (xv[e] - cur.mu) * cur.rs, h = d[e] * g[i][e];
                dg[i][e] += d[e] * xh;
                db[i][e] += d[e];
                s[0] += h;
                s[1] += h * xh;
            }
        }
        float xht = 0.0f, ht = 0.0f;
        if (col.has_tail()) {
            const float d = (float)cur.dyt;
            xht = ((float)cur.xt - cur.mu) * cur.rs;
            ht = d * gt;
            dgt += d * xht;
            dbt += d;
            s[0] += ht;
            s[1] += ht * xht;
        }
        row_sum<R, 2>(s, lds, set);
        set ^= 1;
        const float m1 = s[0] / n, m2 = s[1] / n;
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            float xv[kV], d[kV];
            widen<DT, kV>(cur.x[i], xv);
            widen<DT, kV>(cur.dy[i], d);
#pragma unroll
            for (int e = 0; e < kV; ++e)
                d[e] = (d[e] * g[i][e] - m1 - (xv[e] - cur.mu) * cur.rs * m2) * cur.rs;
            store_vec<DT, kV, true>(dx + row * col.cols + col.at(i), col.has(i), d);
        }
        if (col.has_tail()) dx[row * col.cols + col.at_tail()] = (T)((ht - m1 - xht * m2) * cur.rs);
        if constexpr (kAhead) cur = next;
    }
    if (ws) {
        if constexpr (kRows > 1) { // the block's waves share a slot
            __shared__ float sums[kRows - 1][2][kI][kV + 1][64];
            const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
            if (wave > 0) {
#pragma unroll
                for (int i = 0; i < kI; ++i)
#pragma unroll
                    for (int e = 0; e < kV; ++e) {
                        sums[wave - 1][0][i][e][lane] = dg[i][e];
                        sums[wave - 1][1][i][e][lane] = db[i][e];
                    }
                sums[wave - 1][0][0][kV][lane] = dgt;
                sums[wave - 1][1][0][kV][lane] = dbt;
            }
            __syncthreads();
            if (wave > 0) return;
#pragma unroll
            for (int w = 0; w < kRows - 1; ++w) {
#pragma unroll
                for (int i = 0; i < kI; ++i)
#pragma unroll
                    for (int e = 0; e < kV; ++e) {
                        dg[i][e] += sums[w][0][i][e][lane];
                        db[i][e] += sums[w][1][i][e][lane];
                    }
                dgt += sums[w][0][0][kV][lane];
                dbt += sums[w][1][0][kV][lane];
            }
        }
        float *slot = ws + (int64_t)blockIdx.x * 2 * col.cols;
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            store_vec<kF32, kV, false>(slot + col.at(i), col.has(i), dg[i]);
            store_vec<kF32, kV, false>(slot + col.cols + col.at(i), col.has(i), db[i]);
        }
        if (col.has_tail()) slot[col.at_tail()] = dgt, slot[col.cols + col.at_tail()] = dbt;
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
    __shared__ float lds[2][2][16];
    const float n = (float)cols;
    int set = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const typename Elem<DT>::type *xr = x + row * cols, *dr = dy + row * cols;
        const float mu = mean[row], rs = rstd[row];
        float s[2] = {0.0f, 0.0f};
#pragma unroll 4
        for (int64_t c = threadIdx.x; c < cols; c += kLnLong) {
            const float h = gamma ? (float)dr[c] * (float)gamma[c] : (float)dr[c];
            s[0] += h;
            s[1] += h * (((float)xr[c] - mu) * rs);
        }
        row_sum<kLnLong, 2>(s, lds, set);
        set ^= 1;
        const float m1 = s[0] / n, m2 = s[1] / n;
#pragma unroll 4
        for (int64_t c = threadIdx.x; c < cols; c += kLnLong) {
            const float h = gamma ? (float)dr[c] * (float)gamma[c] : (float)dr[c];
            dx[row * cols + c] = (typename Elem<DT>::type)((h - m1 - ((float)xr[c] - mu) * rs * m2) * rs);
        }
    }
}

// Sums of dy xh and dy of 64 columns (the launch's from c0 on) over a share of
// the rows (long rows): four waves take rows in turn, then fold through LDS
// into slot blockIdx.y.
template <int DT>
__global__ __launch_bounds__(kLnThreads) void ln_bwd_cols(const typename Elem<DT>::type *__restrict__ dy,
                                                          const typename Elem<DT>::type *__restrict__ x, int64_t rows,
                                                          int64_t cols, const float *__restrict__ mean,
                                                          const float *__restrict__ rstd, float *__restrict__ ws,
                                                          int64_t c0)
{
    __shared__ float lds[2][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = c0 + (int64_t)blockIdx.x * 64 + lane;
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

// Fold `slots` partial rows of the workspace: 32 columns per block (the launch's
// from c0 on), 32 lanes per column taking slots in turn, eight loads in flight
// each.  blockIdx.y: 0 dgamma, 1 dbeta.  The memory's latency bounds it: 799 slots of 147 columns
// 26 us with eight lanes and a load at a time, 4.5 us so.
template <int PT>
__global__ __launch_bounds__(kFoldThreads) void ln_bwd_fold(const float *__restrict__ ws, int slots, int64_t cols,
                                                            typename Elem<PT>::type *__restrict__ dgamma,
                                                            typename Elem<PT>::type *__restrict__ dbeta, int64_t c0)
{
    constexpr int kLanes = kFoldThreads / 32;
    __shared__ float lds[kLanes][32];
    const int j = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = c0 + (int64_t)blockIdx.x * 32 + j;
    typename Elem<PT>::type *out = blockIdx.y ? dbeta : dgamma;
    if (!out) return;
    float s = 0.0f;
    if (c < cols)
        for (int p = k; p < slots; p += 8 * kLanes) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] = p + u * kLanes < slots ? ws[((int64_t)(p + u * kLanes) * 2 + blockIdx.y) * cols + c] : 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
    lds[k][j] = s;
    __syncthreads();
    if (k == 0 && c < cols) {
#pragma unroll
        for (int p = 1; p < kLanes; ++p) s += lds[p][j];
        out[c] = (typename Elem<PT>::type)s;
    }
}

// The lanes per row and vectors per lane that hold a row of `cols` elements
// of `vec`-element vectors; lanes 0: the row is too long for registers.
struct LnShape {
    int lanes, vecs;
};
LnShape fwd_shape(int64_t cols, int vec)
{
    const int64_t v = (cols + vec - 1) / vec;
    if (v <= 64) return {64, 1};
    if (v <= 128) return {64, 2};
    if (v <= 1536) {
        const int i = (int)((v + 255) / 256);
        return {256, i == 5 ? 6 : i};
    }
    if (v <= 2048) return {1024, 2};
    if (v <= 4096) return {1024, 4};
    return {0, 0};
}
#define FP8Q_LN_FWD_SHAPES(X) X(64, 1) X(64, 2) X(256, 1) X(256, 2) X(256, 3) X(256, 4) X(256, 6) X(1024, 2) X(1024, 4)

// The backward pass also holds the lane's gain and its two sums, 12 bytes per
// column beside x and dy: up to 32 columns a lane (24 for fp32 rows at 256
// lanes, more would spill), at 512 lanes 16384 columns.
LnShape bwd_shape(int64_t cols, int vec)
{
    const int64_t v = (cols + vec - 1) / vec;
    if (v <= 64) return {64, 1};
    if (v <= 128) return {64, 2};
    for (int lanes = 256; lanes <= 512; lanes *= 2) {
        const int i = (int)((v + lanes - 1) / lanes);
        if (i * vec > (lanes == 256 ? 24 : 32) && !(vec == 8 && i == 4)) continue;
        return {lanes, i <= 4 ? (lanes == 512 ? 4 : i) : i <= 6 ? 6 : 8};
    }
    return {0, 0};
}
#define FP8Q_LN_BWD_SHAPES(X) X(64, 1) X(64, 2) X(256, 1) X(256, 2) X(256, 3) X(256, 4)
#define FP8Q_LN_BWD_SHAPES_F32(X) X(256, 6) X(512, 4) X(512, 6) X(512, 8)
#define FP8Q_LN_BWD_SHAPES_BF16(X) X(512, 4)
int vec_of(int dtype) { return dtype == kF32 ? 4 : 8; }

// Most blocks of a launch (max_blocks ends below 2^22 of 1024 lanes).  Rows
// beyond are walked, columns (ln_bwd_cols, ln_bwd_fold) get a launch more;
// walking them too cost ln_bwd_cols 2%.
constexpr int64_t kLnMaxGrid = 1 << 20;
// Blocks of the backward pass, each of which leaves one partial row: two per
// CU where a block shares a row, four where its waves have rows of their own
// (short rows, so short partials).
constexpr int kLnBwdBlocks = 512;

int bwd_blocks(int64_t rows, LnShape sh)
{
    const int per = sh.lanes == 64 ? kLnThreads / 64 : 1; // rows a block holds
    const int cap = sh.lanes == 64 ? 2 * kLnBwdBlocks : kLnBwdBlocks;
    const int64_t want = (rows + per - 1) / per;
    return (int)(want < cap ? (want < 1 ? 1 : want) : cap);
}
int bwd_slots(int64_t rows, int64_t cols, int dtype)
{
    const LnShape sh = bwd_shape(cols, vec_of(dtype));
    if (sh.lanes == 0) { // ln_bwd_cols: slots of 32 rows or more
        const int64_t s = (rows + 31) / 32;
        return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
    }
    return bwd_blocks(rows, sh);
}

// Most blocks of the forward pass.  Where the gain and bias are held in
// registers and the next row is fetched early, about what is resident at once
// (16384x4096 bf16: 2048 blocks 51.6 us, one row a block 63.6; 30000x1111:
// 40.4 and 45.0; 3000x16000 fp32: 512 blocks of 1024 lanes 72.7, 94.5); rows
// that leave no registers for it take a block each (8192x8192 bf16 57.1 us,
// 64.4 in 2048 blocks).
int64_t fwd_blocks(LnShape sh, int vec)
{
    if (sh.lanes == 64) return 1024;
    if (sh.lanes == 1024) return 512;
    return sh.lanes && sh.vecs * vec <= 16 ? 2048 : kLnMaxGrid;
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
    const LnShape sh = fwd_shape(cols, Elem<DT>::kVec);
    const int per = sh.lanes == 64 ? kLnThreads / 64 : 1;
    int64_t g = (rows + per - 1) / per;
    const int64_t cap = fwd_blocks(sh, Elem<DT>::kVec), rounds = (g + cap - 1) / cap;
    const int grid = (int)((g + rounds - 1) / rounds);
    const bool full = cols == (int64_t)sh.lanes * sh.vecs * Elem<DT>::kVec;
#define FP8Q_LN(R, I)                                                                                                \
    if (sh.lanes == R && sh.vecs == I) {                                                                             \
        auto k = full ? ln_fwd_kernel<DT, PT, R, I, true> : ln_fwd_kernel<DT, PT, R, I, false>;                      \
        k<<<grid, R > kLnThreads ? R : kLnThreads, 0, s>>>(x, rows, cols, gamma, beta, eps, y, mean, rstd);          \
    }
    FP8Q_LN_FWD_SHAPES(FP8Q_LN)
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
    const LnShape sh = bwd_shape(cols, Elem<DT>::kVec);
    const int slots = bwd_slots(rows, cols, DT);
    // launches of blocks of `width` columns each
    auto by_columns = [&](int width, auto launch) {
        for (int64_t c0 = 0; c0 < cols; c0 += kLnMaxGrid * width) {
            const int64_t blocks = (cols - c0 + width - 1) / width;
            launch((unsigned)(blocks < kLnMaxGrid ? blocks : kLnMaxGrid), c0);
        }
    };
    if (rows > 0) {
        const int grid = sh.lanes ? bwd_blocks(rows, sh) : (int)(rows < kLnMaxGrid ? rows : kLnMaxGrid);
        float *w = params ? ws : nullptr;
        const bool full = cols == (int64_t)sh.lanes * sh.vecs * Elem<DT>::kVec;
#define FP8Q_LN(R, I)                                                                                                \
    if (sh.lanes == R && sh.vecs == I) {                                                                             \
        auto k = full ? ln_bwd_kernel<DT, PT, R, I, true> : ln_bwd_kernel<DT, PT, R, I, false>;                      \
        k<<<grid, R > kLnThreads ? R : kLnThreads, 0, s>>>(dy, x, rows, cols, gamma, mean, rstd, dx, w);             \
    }
        FP8Q_LN_BWD_SHAPES(FP8Q_LN)
        if constexpr (DT == kF32) {
            FP8Q_LN_BWD_SHAPES_F32(FP8Q_LN)
        } else {
            FP8Q_LN_BWD_SHAPES_BF16(FP8Q_LN)
        }
#undef FP8Q_LN
        if (sh.lanes == 0) {
            ln_bwd_long<DT, PT><<<grid, kLnLong, 0, s>>>(dy, x, rows, cols, gamma, mean, rstd, dx);
            if (params)
                by_columns(64, [&](unsigned blocks, int64_t c0) {
                    ln_bwd_cols<DT><<<dim3(blocks, (unsigned)slots), kLnThreads, 0, s>>>(dy, x, rows, cols, mean, rstd,
                                                                                        w, c0);
                });
        }
    }
    // no rows: the parameter gradients are zero
    if (params)
        by_columns(32, [&](unsigned blocks, int64_t c0) {
            ln_bwd_fold<PT><<<dim3(blocks, 2), kFoldThreads, 0, s>>>(ws, rows > 0 ? slots : 0, cols, (P *)dgamma,
                                                                     (P *)dbeta, c0);
        });
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
