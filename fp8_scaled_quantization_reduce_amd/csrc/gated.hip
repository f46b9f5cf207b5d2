// gated.hip -- the gated feed-forward block beside its product: the finishing
// pass of a few-row product, the backward pass from the 8-bit checkpoint, and
// the token-contiguous copy of 8-bit rows.
//
// Codes in 1x128 blocks are the checkpoint: g and u as the forward pass wrote
// them, the block's input as it was quantized.  The backward pass reads them
// once and writes every copy that the products after it read, so neither bf16
// activations nor a columnwise copy are kept between the passes.
#include "gate.h"
#include "gated_tiles.h"
#include "groups.h"

namespace fp8q {

namespace {

// Max over the 16 lanes that share a row's block.
__device__ __forceinline__ uint32_t max_16_lanes(uint32_t m)
{
    m = max(m, FP8Q_DPP(m, 0xB1));  // lane ^ 1
    m = max(m, FP8Q_DPP(m, 0x4E));  // lane ^ 2
    m = max(m, FP8Q_DPP(m, 0x141)); // lane ^ 7
    return max(m, FP8Q_DPP(m, 0x128)); // lane ^ 8
}

// Four codes -> values without their scale.
typedef float v2f __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2v __attribute__((ext_vector_type(2)));
template <int F> __device__ __forceinline__ void decode4(uint32_t c, float *v)
{
    v2f a, b;
    if constexpr (F == kE4M3) {
        a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
        b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    } else {
        a = __builtin_amdgcn_cvt_pk_f32_bf8((int)c, false);
        b = __builtin_amdgcn_cvt_pk_f32_bf8((int)c, true);
    }
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
}

// Eight codes of a row with its block's scale.
template <int F> __device__ __forceinline__ uint2 encode8(const float *v, float scale, bool finite)
{
    return make_uint2(encode_block<F>(v[0], v[1], v[2], v[3], scale, finite),
                      encode_block<F>(v[4], v[5], v[6], v[7], scale, finite));
}

// Eight values of a row into a buffer of bf16 or fp32.
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t to, int dtype, int voff, int soff, const float *v)
{
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    typedef float f32x8 __attribute__((ext_vector_type(8)));
    if (dtype == kBF16) {
        const f32x8 f{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, __builtin_convertvector(f, bf16x8)), to, voff,
                                               soff, kBufferNt);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            __builtin_amdgcn_raw_buffer_store_b128(
                __builtin_bit_cast(u32x4v, v4f{v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]}), to, voff + 16 * k,
                soff, kBufferNt);
    }
}

// The finishing pass of a few-row product: h and its codes, and those of g and
// u, from g and u in binary32.  16 lanes a block, eight columns each.  A launch's
// latency, 3 to 5 us.
constexpr int kFinishThreads = 256;

__global__ __launch_bounds__(kFinishThreads) void gated_finish_kernel(const int32_t *__restrict__ offsets, int groups,
                                                                      int rows, int tiles, int F, GatedOut o)
{
    const int lane = threadIdx.x & 63, blocks = F / 128;
    const int64_t i = (int64_t)blockIdx.x * (kFinishThreads / 16) + (threadIdx.x >> 4);
    const int64_t row = i / blocks, b = i % blocks;
    const int64_t c = b * 128 + 8 * (lane & 15);
    float g[8], u[8], h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = u[e] = 0.0f;
    if (row < rows) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const v4f x = *reinterpret_cast<const v4f *>(o.ws + row * 2 * F + c + 4 * k);
            const v4f y = *reinterpret_cast<const v4f *>(o.ws + row * 2 * F + F + c + 4 * k);
#pragma unroll
            for (int e = 0; e < 4; ++e) g[4 * k + e] = x[e], u[4 * k + e] = y[e];
        }
    }
    // rows that the product's tiles filled, looked up beside the loads of the values
    const bool live = offsets ? row_in_tiles<16>(offsets, groups, rows, tiles, (int)row) : row < rows;
    with_act(o.act, [&](auto a) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = act_f32<decltype(a)::value>(g[e]) * u[e];
    });
    auto codes = [&](const float *v, int fmt, uint8_t *q, float *s, int64_t cols, int64_t col) {
        const uint32_t m = max_16_lanes(absmax_bits<8>(v));
        const Scales sc = block_scales(m, fmt);
        if (!live) return;
        with_fmt(fmt, [&](auto f) {
            st_stream(q + row * cols + col, encode8<decltype(f)::value>(v, sc.scale, m < kInfBits));
        });
        if ((lane & 15) == 0) s[row * (cols / 128) + col / 128] = sc.s;
    };
    if (o.q_gu) {
        codes(g, o.gu_fmt, o.q_gu, o.s_gu, 2 * F, c);
        codes(u, o.gu_fmt, o.q_gu, o.s_gu, 2 * F, F + c);
    }
    if (o.q_h) codes(h, o.h_fmt, o.q_h, o.s_h, F, c);
    if (o.H && live) {
        const int64_t at = row * F + c;
        if (o.h_dtype == kBF16) {
            const v4f lo{h[0], h[1], h[2], h[3]}, hi{h[4], h[5], h[6], h[7]};
            const uint2 a = __builtin_bit_cast(uint2, __builtin_convertvector(lo, bf16x4));
            const uint2 b = __builtin_bit_cast(uint2, __builtin_convertvector(hi, bf16x4));
            st_stream((uint16_t *)o.H + at, make_uint4(a.x, a.y, b.x, b.y));
        } else {
            st_stream((float *)o.H + at, __builtin_bit_cast(uint4, v4f{h[0], h[1], h[2], h[3]}));
            st_stream((float *)o.H + at + 4, __builtin_bit_cast(uint4, v4f{h[4], h[5], h[6], h[7]}));
        }
    }
}

// Block b of a launch -> one of `rows` x `cols` tiles.  A tile's scales are single
// words, 8 tiles' a 32-byte piece of memory in either direction, so the tiles that
// an XCD works on at a time are neighbours: runs of 8 rows of tiles, column by
// column, and a contiguous part of that order for each XCD.  Its L2 then holds the
// pieces until they are whole: without it, 14% more bytes are written
// (8192 x 14336 gradients).
constexpr int kNeighbours = 8;

__device__ __forceinline__ bool neighbours(int b, int rows, int cols, int &row, int &col)
{
    const int per = (rows * cols + kXcds - 1) / kXcds, i = b / kXcds;
    const int at = b % kXcds * per + i;
    if (i >= per || at >= rows * cols) return false;
    const int run = at / (kNeighbours * cols), high = min(kNeighbours, rows - run * kNeighbours);
    const int in = at - run * kNeighbours * cols;
    col = in / high, row = run * kNeighbours + in - col * high;
    return true;
}

// ---------------------------------------------------------------------------
// Backward pass: 128 rows of a group x 128 columns of the gate, of the up
// projection and of h per block of 512 lanes, four rows x eight columns a lane, so
// every input is read once.  Row blocks are 16 lanes, column blocks the whole
// block (four lanes of a wave, then the waves through LDS); column codes are
// transposed through LDS and leave as 128-byte pieces.
//
// Memory bounds it, and close behind the vector ALU (half of the time busy: 34
// instructions an element, two of them transcendental): 8192 x 14336 bf16 with all
// copies 239 us, 4.5 TB/s of the bytes it cannot do without; fp32 GELU, 24594 x
// 1408 over 64 groups 92 us.  Two blocks share a CU, so one's loads run beside the
// other's arithmetic; that takes 128 registers a lane, which three values of 32
// elements fit only as written (see the notes in the kernel).
constexpr int kBwThreads = 512;
constexpr int kTlPitch = 36; // dwords of a column's 128 codes: two columns a lane group apart take other banks

struct GatedBwd {
    const void *dh;
    const uint8_t *q_gu;
    const float *s_gu;
    const int32_t *offsets;
    int groups, rows;
    int64_t F;
    void *D; // [rows][2F] of d_dtype, null: none
    int d_dtype;
    uint8_t *q_d; // row copy, null: none
    float *s_d;
    uint8_t *qc_d; // token-contiguous copy [2F][stride], null: none
    float *sc_d;
    int d_fmt;
    uint8_t *qc_h; // of h [F][stride], null: none
    float *sc_h;
    int h_fmt;
    int64_t stride;
    int t0, tn; // tiles of rows of the launch
};

// Buffers of a tile's rows: rows past the group's last read as zeros and are not
// written, and a row's offset is a scalar of the instruction.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_buffer(const void *p, int64_t first, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc((uint8_t *)p + first, 0, bytes, kRawBufferWord3);
}

// (FG, the checkpoint's format, is a parameter of the template: two versions of the
// values joined by a branch would need 50 registers more than there are)
template <int DT, int ACT, int FG>
__global__ __launch_bounds__(kBwThreads, 4) void gated_backward_kernel(GatedBwd p)
{
    __shared__ __attribute__((aligned(16))) uint32_t tl[3][128 * kTlPitch]; // dg, du, h: [column][row / 4]
    __shared__ __attribute__((aligned(16))) uint32_t colmax[8][3][128];
    __shared__ __attribute__((aligned(16))) float colscale[3][128];
    __shared__ uint32_t colbad; // some column's maximum is NaN or infinite (no scale is zero: amax has a floor)
    GroupTiles<128> tiles(p.offsets, p.groups, p.rows);
    int t, cb;
    if (!neighbours((int)blockIdx.x, min(tiles.total - p.t0, p.tn), (int)(p.F / 128), t, cb)) return;
    t += p.t0;
    const GroupTile gt = tiles.find(t);
    const int ig = threadIdx.x >> 4, jg = threadIdx.x & 15, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t row0 = (int64_t)gt.row0 + 128 * gt.tile, c0 = (int64_t)cb * 128;
    const int F = (int)p.F, last = min(128, gt.size - 128 * gt.tile) - 1; // the tile's last row
    // the caller's columnwise buffers may be too short for these offsets
    const bool columns = (p.qc_d || p.qc_h) && (int64_t)t * 128 + 128 <= p.stride; // block-uniform
    const int v2 = 4 * ig * 2 * F + 8 * jg, vs = 4 * ig * (F / 64) * 4; // the lane's first row of codes, of scales

    float dg[4][8], du[4][8], h[4][8];
    {
        constexpr int kE = DT == kF32 ? 4 : 2;
        const __amdgpu_buffer_rsrc_t rx = tile_buffer(p.dh, (row0 * F + c0) * kE, (last * F + 128) * kE);
        const __amdgpu_buffer_rsrc_t rq = tile_buffer(p.q_gu, row0 * 2 * F + c0, last * 2 * F + F + 128);
        const __amdgpu_buffer_rsrc_t rs = tile_buffer(p.s_gu, (row0 * (F / 64) + cb) * 4, (last * (F / 64) + F / 128 + 1) * 4);
        const int vx = (4 * ig * F + 8 * jg) * kE;
        u32x4v d[4][DT == kF32 ? 2 : 1];
        u32x2v qg[4], qu[4];
        float sg[4], su[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            d[r][0] = __builtin_amdgcn_raw_buffer_load_b128(rx, vx, r * F * kE, 0);
            if constexpr (DT == kF32) d[r][1] = __builtin_amdgcn_raw_buffer_load_b128(rx, vx + 16, r * F * kE, 0);
            qg[r] = __builtin_amdgcn_raw_buffer_load_b64(rq, v2, r * 2 * F, 0);
            qu[r] = __builtin_amdgcn_raw_buffer_load_b64(rq, v2, r * 2 * F + F, 0);
            sg[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, vs, r * (F / 64) * 4, 0));
            su[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, vs, (r * (F / 64) + F / 128) * 4, 0));
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k) { // four columns
                float g[4], u[4], x[4];
                decode4<FG>(qg[r][k], g), decode4<FG>(qu[r][k], u);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = DT == kF32 ? __uint_as_float(d[r][DT == kF32 ? k : 0][e])
                           : e & 1    ? bf16_hi(d[r][0][2 * k + e / 2])
                                      : bf16_lo(d[r][0][2 * k + e / 2]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float gv = g[e] * sg[r], uv = u[e] * su[r];
                    float a, da;
                    act_and_grad<ACT>(gv, a, da);
                    dg[r][4 * k + e] = x[e] * uv * da;
                    du[r][4 * k + e] = x[e] * a;
                    h[r][4 * k + e] = a * uv;
                    // formed here: the compiler would keep both factors up to the columns (145 registers)
                    asm volatile("" : "+v"(h[r][4 * k + e]));
                }
            }
    }
    if (p.D) {
        const int e = p.d_dtype == kBF16 ? 2 : 4;
        const __amdgpu_buffer_rsrc_t rd = tile_buffer(p.D, (row0 * 2 * F + c0) * e, (last * 2 * F + F + 128) * e);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            store8(rd, p.d_dtype, v2 * e, r * 2 * F * e, dg[r]);
            store8(rd, p.d_dtype, v2 * e, (r * 2 * F + F) * e, du[r]);
        }
    }
    if (p.q_d) {
        // maxima of the rows' blocks, one of dg's and du's eight in each pair of the 16 lanes
        uint32_t m[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) m[2 * r] = absmax_bits<8>(dg[r]), m[2 * r + 1] = absmax_bits<8>(du[r]);
        halve_dpp<8, 0x128>(m, lane & 8);
        halve_dpp<4, 0x141>(m, lane & 4);
        halve_dpp<2, 0x4E>(m, lane & 2);
        m[0] = max(m[0], FP8Q_DPP(m[0], 0xB1));
        const Scales sc = block_scales(m[0], p.d_fmt);
        const bool finite = __all(m[0] < kInfBits);
        const __amdgpu_buffer_rsrc_t rq = tile_buffer(p.q_d, row0 * 2 * F + c0, last * 2 * F + F + 128);
        const __amdgpu_buffer_rsrc_t rs = tile_buffer(p.s_d, (row0 * (F / 64) + cb) * 4, (last * (F / 64) + F / 128 + 1) * 4);
        if (!(lane & 1))
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sc.s), rs,
                                                  vs + ((jg >> 2) * (F / 64) + (jg >> 1 & 1) * (F / 128)) * 4, 0, 0);
        // lane 2 i's scale to its 16 lanes
        const uint32_t own = __float_as_uint(sc.scale);
        const float to[8] = {__uint_as_float(FP8Q_DPP(own, 0x150)), __uint_as_float(FP8Q_DPP(own, 0x152)),
                             __uint_as_float(FP8Q_DPP(own, 0x154)), __uint_as_float(FP8Q_DPP(own, 0x156)),
                             __uint_as_float(FP8Q_DPP(own, 0x158)), __uint_as_float(FP8Q_DPP(own, 0x15A)),
                             __uint_as_float(FP8Q_DPP(own, 0x15C)), __uint_as_float(FP8Q_DPP(own, 0x15E))};
        auto rows = [&](auto fc, auto whole) {
            constexpr int FC = decltype(fc)::value;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint2 a = encode8<FC>(dg[r], to[2 * r], decltype(whole)::value);
                const uint2 b = encode8<FC>(du[r], to[2 * r + 1], decltype(whole)::value);
                __builtin_amdgcn_raw_buffer_store_b64(u32x2v{a.x, a.y}, rq, v2, r * 2 * F, kBufferNt);
                __builtin_amdgcn_raw_buffer_store_b64(u32x2v{b.x, b.y}, rq, v2, r * 2 * F + F, kBufferNt);
            }
        };
        with_fmt(p.d_fmt, [&](auto fc) {
            if (__builtin_expect(finite, 1)) rows(fc, PhaseC<1>{});
            else rows(fc, PhaseC<0>{});
        });
    }
    if (!columns) return;
    // a lane's columns over its wave's 16 rows: two of the eight are left to it
    const int c2 = 8 * jg + (lane >> 5) * 4 + (lane >> 4 & 1) * 2;
    auto column_max = [&](const float(&v)[4][8], int k) {
        uint32_t m[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c[4] = {v[0][e], v[1][e], v[2][e], v[3][e]};
            m[e] = absmax_bits<4>(c);
        }
        halve_32<8>(m);
        halve_16<4>(m);
        *reinterpret_cast<uint2 *>(&colmax[wave][k][c2]) = make_uint2(m[0], m[1]);
    };
    if (p.qc_d) column_max(dg, 0), column_max(du, 1);
    if (p.qc_h) column_max(h, 2);
    if (threadIdx.x == 0) colbad = 0;
    __syncthreads();
    if (threadIdx.x < 384) {
        const int k = threadIdx.x >> 7, c = threadIdx.x & 127; // wave-uniform k
        if (k < 2 ? p.qc_d != nullptr : p.qc_h != nullptr) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) m = max(m, colmax[w][k][c]);
            const Scales sc = block_scales(m, k < 2 ? p.d_fmt : p.h_fmt);
            colscale[k][c] = sc.scale;
            if (m >= kInfBits) colbad = 1;
            float *s = k < 2 ? p.sc_d + k * p.F * (p.stride / 128) : p.sc_h;
            s[(c0 + c) * (p.stride / 128) + t] = sc.s;
        }
    }
    __syncthreads();
    const bool finite = __builtin_amdgcn_readfirstlane(colbad) == 0;
    auto transpose = [&](const float(&v)[4][8], int k, int fmt) {
        auto columns_of = [&](auto fc, auto whole) {
            const v4f lo = *reinterpret_cast<const v4f *>(&colscale[k][8 * jg]);
            const v4f hi = *reinterpret_cast<const v4f *>(&colscale[k][8 * jg + 4]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                tl[k][(8 * jg + e) * kTlPitch + (((ig >> 2) ^ (jg >> 1)) << 2 | (ig & 3))] =
                    encode_block<decltype(fc)::value>(v[0][e], v[1][e], v[2][e], v[3][e], e < 4 ? lo[e & 3] : hi[e & 3],
                                                      decltype(whole)::value);
        };
        with_fmt(fmt, [&](auto fc) {
            if (__builtin_expect(finite, 1)) columns_of(fc, PhaseC<1>{});
            else columns_of(fc, PhaseC<0>{});
        });
    };
    if (p.qc_d) transpose(dg, 0, p.d_fmt), transpose(du, 1, p.d_fmt);
    if (p.qc_h) transpose(h, 2, p.h_fmt);
    __syncthreads();
    const int chunk = threadIdx.x & 7, c = threadIdx.x >> 3;
    const int64_t at = (c0 + c) * p.stride + (int64_t)t * 128 + 16 * chunk;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint8_t *q = k < 2 ? p.qc_d : p.qc_h;
        if (!q) continue;
        if (k == 1) q += p.F * p.stride;
#pragma unroll
        for (int n = 0; n < 2; ++n) // columns c and 64 + c
            st_stream(q + at + 64 * n * p.stride,
                      *reinterpret_cast<const uint4 *>(
                          &tl[k][(64 * n + c) * kTlPitch + ((chunk ^ ((64 * n + c) >> 4)) << 2)]));
    }
}

// ---------------------------------------------------------------------------
// Token-contiguous copy of rows in 1x128 blocks: 128 rows of a group x 128
// columns per block of 256 lanes, four rows x 16 columns a lane.
//
// Memory bounds it: 8192 x 4096 12.4 us, 5.6 TB/s; 24594 gathered rows of 2048 over
// 64 groups 24.6 us, where both reads of a row leave the L2 (4.6 TB/s of what
// moves; the same rows without an index or groups 20.3).  Blocks that
// walk several column tiles, with or without the next one fetched ahead, and 512
// lanes of half as many columns were as fast or slower.
constexpr int kRqThreads = 256;

template <int F, int FC>
__global__ __launch_bounds__(kRqThreads) void requantize_kernel(const uint8_t *__restrict__ x,
                                                                const float *__restrict__ s, int64_t x_rows,
                                                                int64_t cols, const int32_t *__restrict__ index,
                                                                int rows, const int32_t *__restrict__ offsets,
                                                                int groups, uint8_t *__restrict__ q_col,
                                                                float *__restrict__ s_col, int64_t stride, int t0,
                                                                int tn)
{
    __shared__ __attribute__((aligned(16))) uint32_t tl[128 * 32]; // column codes, [column][row / 4]
    __shared__ __attribute__((aligned(16))) uint32_t colmax[4][128];
    __shared__ __attribute__((aligned(16))) float colscale[128];
    __shared__ uint32_t colbad;
    const int blocks_c = (int)(cols / 128);
    GroupTiles<128> tiles(offsets, groups, rows);
    int t, cb;
    if (!neighbours((int)blockIdx.x, min(tiles.total - t0, tn), blocks_c, t, cb)) return;
    t += t0;
    if ((int64_t)t * 128 + 128 > stride) return;
    const GroupTile gt = tiles.find(t);
    const int ig = threadIdx.x >> 3, jg = threadIdx.x & 7, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int first = 128 * gt.tile + 4 * ig, live = gt.size - first; // the lane's rows in the group
    uint4 q[4];
    float sc[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t row = (int64_t)gt.row0 + first + r;
        const int64_t src = r < live ? (index ? (int64_t)index[row] : row) : -1;
        q[r] = make_uint4(0u, 0u, 0u, 0u); // a row of zeros
        sc[r] = 1.0f;
        if (src >= 0 && src < x_rows) {
            q[r] = *reinterpret_cast<const uint4 *>(x + src * cols + (int64_t)cb * 128 + 16 * jg);
            sc[r] = s[src * blocks_c + cb];
        }
    }
    float v[4][16]; // x' = fl32(value s)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        decode4<F>(q[r].x, v[r]), decode4<F>(q[r].y, v[r] + 4), decode4<F>(q[r].z, v[r] + 8), decode4<F>(q[r].w, v[r] + 12);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[r][e] *= sc[r];
    }
    // the columns over the wave's 32 rows: two of the 16 are left to a lane
    uint32_t m[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float c[4] = {v[0][e], v[1][e], v[2][e], v[3][e]};
        m[e] = absmax_bits<4>(c);
    }
    halve_32<16>(m);
    halve_16<8>(m);
    halve_dpp<4, 0x128>(m, lane & 8);
    *reinterpret_cast<uint2 *>(&colmax[wave][16 * jg + (lane >> 5) * 8 + (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2]) =
        make_uint2(m[0], m[1]);
    if (threadIdx.x == 0) colbad = 0;
    __syncthreads();
    if (threadIdx.x < 128) {
        const int c = threadIdx.x;
        const uint32_t most = max(max(colmax[0][c], colmax[1][c]), max(colmax[2][c], colmax[3][c]));
        const Scales o = block_scales(most, FC);
        colscale[c] = o.scale;
        if (most >= kInfBits) colbad = 1;
        s_col[((int64_t)cb * 128 + c) * (stride / 128) + t] = o.s;
    }
    __syncthreads();
    float to[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) *reinterpret_cast<v4f *>(to + 4 * k) = *reinterpret_cast<const v4f *>(&colscale[16 * jg + 4 * k]);
    auto put = [&](int e, uint32_t o) { tl[(16 * jg + e) * 32 + ((((ig >> 2) ^ jg) << 2) | (ig & 3))] = o; };
    if (__builtin_expect(__builtin_amdgcn_readfirstlane(colbad) == 0, 1)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) put(e, encode_fit<FC>(v[0][e], v[1][e], v[2][e], v[3][e], to[e]));
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            uint32_t o;
            if (finite_nonzero(to[e])) {
                o = encode_fit<FC>(v[0][e], v[1][e], v[2][e], v[3][e], to[e]);
            } else {
                // a NaN x' (a NaN code, or zero times an infinite scale) has its row code's sign
                o = 0;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t w[4] = {q[r].x, q[r].y, q[r].z, q[r].w};
                    const float x = v[r][e];
                    o |= (x != x ? 0x7Fu | (w[e >> 2] >> (8 * (e & 3)) & 0x80u) : encode_bad(x, to[e])) << (8 * r);
                }
            }
            put(e, o);
        }
    }
    __syncthreads();
    const int chunk = threadIdx.x & 7, c = threadIdx.x >> 3;
    uint8_t *out = q_col + ((int64_t)cb * 128 + c) * stride + (int64_t)t * 128 + 16 * chunk;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        st_stream(out + 32 * k * stride,
                  *reinterpret_cast<const uint4 *>(&tl[(32 * k + c) * 32 + ((chunk ^ ((32 * k + c) >> 4)) << 2)]));
}

template <int DT, int FG> hipError_t launch_backward(GatedBwd p, int act, hipStream_t s)
{
    auto k = act == kActSilu ? gated_backward_kernel<DT, kActSilu, FG>
             : act == kActGelu ? gated_backward_kernel<DT, kActGelu, FG>
                               : gated_backward_kernel<DT, kActRelu, FG>;
    // in launches of as many tiles as one holds
    const int64_t blocks_c = p.F / 128, tiles = max_tiles(p.rows, p.groups, 128);
    const int64_t most = (max_blocks(kBwThreads) - kXcds) / blocks_c;
    for (int64_t t0 = 0; t0 < tiles; t0 += most) {
        p.t0 = (int)t0, p.tn = (int)(tiles - t0 < most ? tiles - t0 : most);
        k<<<(unsigned)(p.tn * blocks_c + kXcds), kBwThreads, 0, s>>>(p);
    }
    return hipGetLastError();
}

template <int F, int FC>
hipError_t launch_columns(const uint8_t *x, const float *s, int64_t x_rows, int64_t cols, const int32_t *index,
                          int64_t rows, const int32_t *offsets, int groups, uint8_t *q_col, float *s_col,
                          int64_t stride, hipStream_t st)
{
    const int64_t tiles = max_tiles(rows, groups, 128), most = (max_blocks(kRqThreads) - kXcds) / (cols / 128);
    for (int64_t t0 = 0; t0 < tiles; t0 += most) {
        const int64_t tn = tiles - t0 < most ? tiles - t0 : most;
        requantize_kernel<F, FC><<<(unsigned)(tn * (cols / 128) + kXcds), kRqThreads, 0, st>>>(
            x, s, x_rows, cols, index, (int)rows, offsets, groups, q_col, s_col, stride, (int)t0, (int)tn);
    }
    return hipGetLastError();
}

} // namespace

#define FP8Q_DECLARE(NAME) hipError_t launch_gated_##NAME(const GatedArgs &a);
FP8Q_DECLARE(e4m3_e4m3)
FP8Q_DECLARE(e5m2_e4m3)
FP8Q_DECLARE(e4m3_e5m2)
FP8Q_DECLARE(e5m2_e5m2)
#undef FP8Q_DECLARE

int64_t gated_gemm_workspace(int64_t rows, int groups, int64_t F, int64_t K)
{
    if (rows == 0 || groups == 0 || F == 0) return 0;
    return gated_tile(rows, groups, F, K, true, compute_units()) == kGated16 ? rows * 2 * F * 4 : 0;
}

bool gated_gemm_fits(int64_t rows, int groups, int64_t F)
{
    return gated_pp_blocks(rows, groups, F, 256) <= max_blocks(kBSThreads);
}

hipError_t launch_gated_gemm(const uint8_t *A, int fa, const float *sA, const uint8_t *B, int fb, const float *sB,
                             const int32_t *offsets, int groups, int64_t rows, int64_t F, int64_t K, int act, void *H,
                             int h_dtype, uint8_t *q_h, float *s_h, int h_fmt, uint8_t *q_gu, float *s_gu, int gu_fmt,
                             float *ws, hipStream_t s)
{
    if (rows == 0 || groups == 0 || F == 0) return hipSuccess;
    const GatedOut out{H, h_dtype, q_h, s_h, h_fmt, q_gu, s_gu, gu_fmt, act, ws};
    const GatedArgs a{A, B, sA, sB, offsets, groups, (int)rows, F, K, out, s, compute_units()};
    const hipError_t e =
        fa == kE4M3 ? (fb == kE4M3 ? launch_gated_e4m3_e4m3(a) : launch_gated_e4m3_e5m2(a))
                    : (fb == kE4M3 ? launch_gated_e5m2_e4m3(a) : launch_gated_e5m2_e5m2(a));
    if (e != hipSuccess || !ws) return e;
    const int64_t units = rows * (F / 128), per = kFinishThreads / 16;
    gated_finish_kernel<<<(unsigned)((units + per - 1) / per), kFinishThreads, 0, s>>>(
        offsets, groups, (int)rows, (int)max_tiles(rows, groups, 16), (int)F, out);
    return hipGetLastError();
}

hipError_t launch_gated_backward(const void *dh, int dh_dtype, const uint8_t *q_gu, const float *s_gu, int gu_fmt,
                                 const int32_t *offsets, int groups, int64_t rows, int64_t F, int act, void *D,
                                 int d_dtype, uint8_t *q_d, float *s_d, uint8_t *qc_d, float *sc_d, int d_fmt,
                                 uint8_t *qc_h, float *sc_h, int h_fmt, int64_t stride, hipStream_t s)
{
    if (rows == 0 || groups == 0 || F == 0) return hipSuccess;
    const GatedBwd p{dh,  q_gu, s_gu, offsets, groups, (int)rows, F,     D,      d_dtype, q_d,
                     s_d, qc_d, sc_d, d_fmt,   qc_h,   sc_h,      h_fmt, stride, 0,       0};
    auto f = dh_dtype == kF32 ? (gu_fmt == kE4M3 ? launch_backward<kF32, kE4M3> : launch_backward<kF32, kE5M2>)
                              : (gu_fmt == kE4M3 ? launch_backward<kBF16, kE4M3> : launch_backward<kBF16, kE5M2>);
    return f(p, act, s);
}

hipError_t launch_requantize_grouped(const uint8_t *x, const float *s, int fmt, int64_t x_rows, int64_t cols,
                                     const int32_t *index, int64_t rows, const int32_t *offsets, int groups,
                                     uint8_t *q_col, float *s_col, int col_fmt, int64_t stride, hipStream_t st)
{
    if (rows == 0 || cols == 0 || groups == 0) return hipSuccess;
    auto f = fmt == kE4M3 ? (col_fmt == kE4M3 ? launch_columns<kE4M3, kE4M3> : launch_columns<kE4M3, kE5M2>)
                          : (col_fmt == kE4M3 ? launch_columns<kE5M2, kE4M3> : launch_columns<kE5M2, kE5M2>);
    return f(x, s, x_rows, cols, index, rows, offsets, groups, q_col, s_col, stride, st);
}

} // namespace fp8q
