// gated_gemm.h -- both projections of a gated feed-forward block, the
// activation and the product in one kernel, over ragged groups of rows or one
// matrix; included by one translation unit per operand-format pair.
//
//   g[t] = sum over slices kb of fma(part_kb, fl32(sA[t, kb] sB[e, n / 128, kb]), .)
//   u[t] likewise with the rows F .. 2F - 1 of B_e,  h[t, n] = act(g) u
//
// in the arithmetic of the grouped product, part_kb on the FP8 matrix instruction,
// whose narrow adder leaves g and u 1.4e-5 to 2e-5 off in the 2-norm.  A binary32 h
// shows that; bf16 (1.7e-3) hides it, and of the codes one in a thousand falls on the
// other side of its rounding, 1.4e-3 in their 2-norm beside the format's 2.6e-2.  That
// is taken for twice the rate of the bf16 instruction on widened codes.  A 1x128 block of h needs 128
// columns of g and of u in one place: the large tiles hold 256, 128 or 64 rows x
// 128 columns of h, so a block's codes leave with the tile.  The tiles for few
// rows hold 16 columns, as many blocks as it takes to read the weights at the
// memory's rate; for codes they leave g and u in binary32 to a finishing pass.
// Between them are tiles of 64 rows x 128 columns.
#ifndef FP8Q_GATED_GEMM_H
#define FP8Q_GATED_GEMM_H

#include "gate.h"
#include "gated_tiles.h"
#include "grouped_gemm.h"

namespace fp8q {

// The results of a kTM x 128 tile of h at row0, n0 (`rows` of its rows are the
// group's): the 1x128 blocks' maxima from the waves' strips through LDS, scales by
// one lane a block, codes staged by all waves and stored as whole lines, values
// staged and stored by each wave.
//
// With codes of h, g and u it takes 5 us more of a 256-row tile than values of h
// alone (11.4 and 6.4 us beside the slices with the chip full): the vector ALU's
// work, 1200 instructions a wave, 390 of them the activation's and 128 of those
// transcendental at a quarter of the rate, while the matrix pipes wait, and 98 KB
// that every CU then writes.
// One pass over a block's maxima with v_maximum3_f32 and halved reductions
// instead of integer maxima, and codes without clamps, took 1.3 us off.
template <int kTM>
__device__ __forceinline__ void gated_finish(uint8_t *st0, uint8_t *st1, float *sx,
                                             v4f (&acc)[4][2 * PPShape<kTM>::kJT], int w, int wm, int wn,
                                             const GatedOut &o, int64_t row0, int n0, int F, int rows)
{
    typedef PPShape<kTM> P;
    constexpr int kQ = P::kQ, kJT = P::kJT, kCS = P::kCS;
    const int tid = threadIdx.x, lane = tid & 63, fr = lane & 15, fg = lane >> 4;
    const int64_t f = F;
    v4f h[4][kJT];
    with_act(o.act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < kJT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) h[i][j][e] = act_f32<decltype(a)::value>(acc[i][j][e]) * acc[i][kJT + j][e];
    });
    uint32_t *most = reinterpret_cast<uint32_t *>(sx);     // [h, g, u][strip][row]
    float *inverse = sx + 3 * kCS * kTM;                   // [h, g, u][row]
    if (o.q_h || o.q_gu) {                                 // uniform
        // a row's maximum over its four lanes: the four rows of 16 i + fr are split between them
        const int row = wm * 64 + 16 * ((lane >> 5) * 2 + (lane >> 4 & 1)) + fr;
        auto maxima = [&](int k, auto v) {
            uint32_t m[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[4 * kJT];
#pragma unroll
                for (int j = 0; j < kJT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[4 * j + e] = v(i, j)[e];
                m[i] = absmax_bits<4 * kJT>(x);
            }
            halve_32<4>(m);
            halve_16<2>(m);
            most[(k * kCS + wn) * kTM + row] = m[0];
        };
        if (o.q_h) maxima(0, [&](int i, int j) { return h[i][j]; });
        if (o.q_gu) {
            maxima(1, [&](int i, int j) { return acc[i][j]; });
            maxima(2, [&](int i, int j) { return acc[i][kJT + j]; });
        }
        __syncthreads();
        for (int b = (o.q_h ? 0 : kTM) + tid; b < (o.q_gu ? 3 : 1) * kTM; b += kBSThreads) {
            const int k = b / kTM, row = b % kTM;
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < kCS; ++c) m = max(m, most[(k * kCS + c) * kTM + row]);
            const Scales sc = block_scales(m, k == 0 ? o.h_fmt : o.gu_fmt);
            inverse[b] = sc.scale;
            if (row < rows) {
                if (k == 0) o.s_h[(row0 + row) * (f / 128) + n0 / 128] = sc.s;
                else o.s_gu[(row0 + row) * (2 * f / 128) + ((k - 1) * f + n0) / 128] = sc.s;
            }
        }
        __syncthreads();
    }
    const int wrow = wm * 64, wcol = n0 + wn * kQ;
    // codes of the wave's columns of part k (h, g, u), v(i, j), into the part's rows of
    // 128 bytes: whole lines leave, which the wave's own half or quarter of one is not
    typedef EpiStage<128, 1, kTM / 8, kTM / 8 * 128> CS;
    auto codes = [&](int k, int fmt, uint8_t *part, auto v) {
        float sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = inverse[k * kTM + wrow + 16 * i + fr];
        auto put = [&](auto fc, auto whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < kJT; ++j) {
                    const v4f x = v(i, j);
                    CS::put(part, wrow + 16 * i + fr, wn * (kQ / 4) + 4 * j + fg,
                            make_uint4(encode_block<decltype(fc)::value>(x[0], x[1], x[2], x[3], sc[i],
                                                                         decltype(whole)::value),
                                       0u, 0u, 0u));
                }
        };
        const bool finite = __all(finite_nonzero(sc[0]) && finite_nonzero(sc[1]) && finite_nonzero(sc[2]) &&
                                  finite_nonzero(sc[3]));
        with_fmt(fmt, [&](auto fc) {
            if (__builtin_expect(finite, 1)) put(fc, PhaseC<1>{});
            else put(fc, PhaseC<0>{});
        });
    };
    uint8_t *const part_g = st0, *const part_u = st0 + kTM * 128, *const part_h = st1;
    static_assert(2 * kTM * 128 <= P::kStage, "codes of g and u share a stage");
    if (o.q_gu) {
        codes(1, o.gu_fmt, part_g, [&](int i, int j) { return acc[i][j]; });
        codes(2, o.gu_fmt, part_u, [&](int i, int j) { return acc[i][kJT + j]; });
    }
    if (o.q_h) codes(0, o.h_fmt, part_h, [&](int i, int j) { return h[i][j]; });
    if (o.q_h || o.q_gu) {
        __syncthreads();
        const int first = w * (kTM / 8), rest = rows - first;
        const int64_t row = row0 + first;
        if (rest > 0) {
            auto store = [&](const uint8_t *part, uint8_t *q, int pitch) {
                store_rows<CS, kTM / 8>(part + first * 128, q, pitch, 128, rest, lane);
            };
            if (o.q_gu) {
                store(part_g, o.q_gu + row * 2 * f + n0, 2 * F);
                store(part_u, o.q_gu + row * 2 * f + F + n0, 2 * F);
            }
            if (o.q_h) store(part_h, o.q_h + row * f + n0, F);
        }
        if (!o.H) return;
        __syncthreads(); // its values take the codes' place
    }
    const int left = rows - wrow;
    if (left <= 0) return;
    row0 += wrow;
    uint8_t *ep = (w < 4 ? st0 : st1) + (w & 3) * (P::kWC * kBK);
    auto values = [&](auto kind) {
        constexpr int kOut = decltype(kind)::value, kB = out_bytes<kOut>();
        typedef EpiStage<kQ, kB, 64, P::kWC * kBK> ES;
        uint32_t m = 0;
        const Epi none{nullptr, kActNone, nullptr};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < kJT; ++j)
                ES::put(ep, 16 * i + fr, 4 * j + fg, pack_out4<kOut, false, false>(0, h[i][j], m, none, 0.0f));
        store_rows<ES, 64>(ep, (uint8_t *)o.H + (row0 * f + wcol) * kB, F * kB, kQ * kB, left, lane);
    };
    if (o.H && o.h_dtype == kBF16) values(PhaseC<kOutBF16>{});
    else if (o.H) values(PhaseC<kOutF32>{});
}

// Tiles of 256 rows x 128 columns of h on the grouped product's ping-pong
// schedule; a group's last tile of at most 128 rows has 128, and what an XCD
// leaves for a last round on at most half of its CUs runs as two of those each.
//
// Long contractions are bound by the card's power, as the grouped product's:
// 8192 rows of 14336 x 4096 with all codes 863 us, 2.2 PFLOP/s (values of h alone
// 2.5 PFLOP/s, the product without a gate, in bf16, 2.5).  Short ones by what a
// tile takes beside its slices: 24594 rows over 64 matrices of 1408 x 2048, 16
// slices, 213 us, 1.3 PFLOP/s (the product without a gate 182).
template <int FA, int FB>
__global__ __launch_bounds__(kBSThreads, 1) void gated_pp_kernel(const uint8_t *__restrict__ A,
                                                                 const float *__restrict__ sA,
                                                                 const uint8_t *__restrict__ B,
                                                                 const float *__restrict__ sB,
                                                                 const int32_t *__restrict__ offsets, int groups,
                                                                 int rows, int F, int K, GatedOut out, int cus)
{
    typedef PPShape<256> P;
    __shared__ __attribute__((aligned(1024))) uint8_t st0[P::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[P::kStage];
    __shared__ __attribute__((aligned(16))) float sx[kScaleGroups * 64 * pp_scale_runs<256, false>()];
    static_assert(sizeof(sx) >= 4 * (3 * 2 * 256 + 3 * 256) && sizeof(sx) >= 4 * (3 * 4 * 128 + 3 * 128), "maxima");
    const int tiles_n = F / 128, nk = K / kBK;
    GroupTiles<256> tiles(offsets, groups, rows);
    const int n = tiles.total * tiles_n, per = (n + kXcds - 1) / kXcds, first = (int)(blockIdx.x % kXcds) * per;
    const int share = min(per, n - first); // this XCD's tiles
    int i = blockIdx.x / kXcds, half = -1;
    const int last = share % cus;
    if (i >= share - last && 2 * last <= cus) {
        half = (i - (share - last)) & 1;
        i = share - last + ((i - (share - last)) >> 1);
    }
    if (i >= share) return;
    const int t = first + i;
    const GroupTile gt = tiles.find(t / tiles_n);
    int tm, tn;
    group_tile(gt.tile * tiles_n + t % tiles_n, (gt.size + 255) / 256, tiles_n, tm, tn);
    const int at = 256 * tm + (half > 0 ? 128 : 0), n0 = 128 * tn;
    const int64_t row0 = gt.row0 + at;
    const int a_rows = min(half < 0 ? 256 : 128, gt.size - at);
    if (a_rows <= 0) return;
    const PPOperand a{A + row0 * K, a_rows * K, K, sA + row0 * nk, a_rows * nk * 4, nk};
    const int s_pitch = F / 128 * nk; // floats from a gate block's scales to its up block's
    const PPOperand b{B + ((int64_t)gt.group * 2 * F + n0) * K, 128 * K, K,
                      sB + ((int64_t)gt.group * 2 * (F / 128) + tn) * nk, (s_pitch + nk) * 4, s_pitch};
    const uint8_t *up = b.base + (int64_t)F * K;
    if (a_rows > 128)
        pp_tile<FA, FB, 256, false, true>(st0, st1, sx, a, b, up, nk, 1, [&](auto &acc, int w, int wm, int wn) {
            gated_finish<256>(st0, st1, sx, acc, w, wm, wn, out, row0, n0, F, a_rows);
        });
    else
        pp_tile<FA, FB, 128, false, true>(st0, st1, sx, a, b, up, nk, 1, [&](auto &acc, int w, int wm, int wn) {
            gated_finish<128>(st0, st1, sx, acc, w, wm, wn, out, row0, n0, F, a_rows);
        });
}

// Tiles of 64 rows x 128 columns of h, for a batch that leaves most of the chip
// without a large tile: eight waves of 64 x (16 + 16), the slices through three
// stages, loaded three ahead, and a slice's fragments read from LDS while the one
// before is multiplied.  All scales of the tile are loaded at the start, which is
// what bounds K (kMidSlices).
//
// What the LDS moves bounds a slice, 96 KB read and 40 KB written, 0.5 us: 301 rows
// of 4096 x 4096 24 us on 160 CUs, 20 of it the 32 slices of a tile, with the weights in
// the last-level cache; from memory 28, and 0.85 us a slice where 32 CUs read all
// of them.  Many weights, their bytes: 32 rows of each of 64 matrices of 1408 x 2048
// 73 to 79 us, 5.1 TB/s.
// Weights straight from memory into registers took 1 us a slice (every load
// touches half a line of 16 rows), four waves of 64 x (32 + 32), which read a third
// less from LDS, 0.7 us (one wave a SIMD waits for its own reads).
template <int FA, int FB>
__global__ __launch_bounds__(kBSThreads, 1) void gated_mid_kernel(const uint8_t *__restrict__ A,
                                                                  const float *__restrict__ sA,
                                                                  const uint8_t *__restrict__ B,
                                                                  const float *__restrict__ sB,
                                                                  const int32_t *__restrict__ offsets, int groups,
                                                                  int rows, int F, int K, GatedOut out)
{
    constexpr int kTM = 64, kRuns = kTM / 16 + 1, kGroup = 64 * kRuns; // runs of 16 rows x 4 slices; B's two scales
    constexpr int kLoads = 5;                                          // of a wave and slice
    typedef PPShape<kTM> P;
    __shared__ __attribute__((aligned(1024))) uint8_t s0[P::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t s1[P::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t s2[P::kStage];
    __shared__ __attribute__((aligned(16))) float sx[kMidSlices / 4 * kGroup];
    static_assert(sizeof(sx) >= 4 * (3 * 8 * kTM + 3 * kTM), "maxima");
    const int tiles_n = F / 128, nk = K / kBK;
    GroupTiles<kTM> tiles(offsets, groups, rows);
    const int n = tiles.total * tiles_n, per = (n + kXcds - 1) / kXcds;
    const int i0 = blockIdx.x / kXcds, t = (int)(blockIdx.x % kXcds) * per + i0;
    if (i0 >= per || t >= n) return;
    const GroupTile gt = tiles.find(t / tiles_n);
    int tm, tn;
    // 16 rows of tiles at a time, so that few rows read the weights once
    group_tile<16>(gt.tile * tiles_n + t % tiles_n, (gt.size + kTM - 1) / kTM, tiles_n, tm, tn);
    const int64_t row0 = gt.row0 + kTM * tm;
    const int n0 = 128 * tn, a_rows = min(kTM, gt.size - kTM * tm);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fg = lane >> 4;
    const uint8_t *gate = B + ((int64_t)gt.group * 2 * F + n0) * K;
    const int s_pitch = F / 128 * nk; // floats from a gate block's scales to its up block's
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc((void *)(A + row0 * K), 0, a_rows * K, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t rg = __builtin_amdgcn_make_buffer_rsrc((void *)gate, 0, 128 * K, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t ru =
        __builtin_amdgcn_make_buffer_rsrc((void *)(gate + (int64_t)F * K), 0, 128 * K, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t rsa =
        __builtin_amdgcn_make_buffer_rsrc((void *)(sA + row0 * nk), 0, a_rows * nk * 4, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t rsb =
        __builtin_amdgcn_make_buffer_rsrc((void *)(sB + ((int64_t)gt.group * 2 * (F / 128) + tn) * nk), 0,
                                          (s_pitch + nk) * 4, kRawBufferWord3);
    // scales: lane -> row lane % 16 of a run, slice lane / 16 of the four (rows of B's run: gate, up, up, ...)
    const int sa_voff = ((lane & 15) * nk + (lane >> 4)) * 4;
    const int sb_voff = (min(lane & 15, 1) * s_pitch + (lane >> 4)) * 4;
    for (int u = w; u < (nk + 3) / 4 * kRuns; u += 8) {
        const int group = u / kRuns, run = u - group * kRuns;
        float *dst = sx + group * kGroup + 64 * run;
        if (run < kTM / 16)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (lds_void *)dst, 4, sa_voff, (16 * run * nk + 4 * group) * 4, 0,
                                                     0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (lds_void *)dst, 4, sb_voff, 4 * group * 4, 0, 0);
    }
    const int voff = (lane >> 3) * K + (((lane & 7) ^ ((4 * w + (lane >> 4)) & 7)) << 4);
    auto load = [&](uint8_t *st, int kb) {
        const int at = kb * kBK;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(st + 8 * w * kBK), 16, voff, 8 * w * K + at, 0, 0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int row = 8 * (w + 8 * u);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rg, (lds_void *)(st + P::oB0 + row * kBK), 16, voff, row * K + at, 0,
                                                     0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ru, (lds_void *)(st + P::oB1 + row * kBK), 16, voff, row * K + at, 0,
                                                     0);
        }
    };
    struct Frags {
        v8i a[4], b[2];
    };
    auto read = [&](const uint8_t *st, Frags &f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f.a[i] = read_frag(st, 16 * i + fr, fg);
        f.b[0] = read_frag(st + P::oB0, 16 * w + fr, fg);
        f.b[1] = read_frag(st + P::oB1, 16 * w + fr, fg);
    };
    v4f acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = v4f{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Frags &f, int kb) {
        const float *s = sx + (kb >> 2) * kGroup + 16 * (kb & 3);
        const float sg = s[64 * (kTM / 16)], su = s[64 * (kTM / 16) + 1];
        v4f p[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) p[i][j] = mfma16x16x128<FB, FA>(f.b[j], f.a[i], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float sa = s[64 * i + fr], wg = sa * sg, wu = sa * su;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[i][0][e] = __builtin_fmaf(p[i][0][e], wg, acc[i][0][e]);
                acc[i][1][e] = __builtin_fmaf(p[i][1][e], wu, acc[i][1][e]);
            }
        }
    };
    // slice kb, its fragments in f: slice kb + 1 has landed in `next` (only kb + 2's loads may
    // be outstanding) and kb's stage is free once all waves are here
    auto slice = [&](int kb, uint8_t *own, const uint8_t *next, const Frags &f, Frags &g) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(kLoads, 0));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        load(own, kb + 3);
        read(next, g);
        multiply(f, kb);
    };
    Frags f, g;
    if (nk > 0) {
        load(s0, 0);
        load(s1, 1);
        load(s2, 2);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(2 * kLoads, 15));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        read(s0, f);
    }
    int kb = 0;
    for (; kb + 6 <= nk; kb += 6) {
        slice(kb, s0, s1, f, g);
        slice(kb + 1, s1, s2, g, f);
        slice(kb + 2, s2, s0, f, g);
        slice(kb + 3, s0, s1, g, f);
        slice(kb + 4, s1, s2, f, g);
        slice(kb + 5, s2, s0, g, f);
    }
    if (kb < nk) slice(kb, s0, s1, f, g);
    if (kb + 1 < nk) slice(kb + 1, s1, s2, g, f);
    if (kb + 2 < nk) slice(kb + 2, s2, s0, f, g);
    if (kb + 3 < nk) slice(kb + 3, s0, s1, g, f);
    if (kb + 4 < nk) slice(kb + 4, s1, s2, f, g);
    // the loads of the slices past the end must land before the stages are reused
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    gated_finish<kTM>(s0, s1, sx, acc, w, 0, w, out, row0, n0, F, a_rows);
}

// Few rows per group, where the weights' bytes are what counts: 16 rows x 16
// columns of h per block, fragments loaded straight from memory into registers,
// kWK waves that take the 128-wide slices in turn and add their sums through LDS.
// The weights' bytes bound it: one row of 14336 x 4096 24.5 us with launch, 4.8
// TB/s; 222 rows over 64 matrices of 1408 x 2048 60 us, 5.9 TB/s, and 5 for the
// finishing pass.
template <int FA, int FB, int kWK>
__global__ __launch_bounds__(64 * kWK) void gated_rows_kernel(const uint8_t *__restrict__ A,
                                                              const float *__restrict__ sA,
                                                              const uint8_t *__restrict__ B,
                                                              const float *__restrict__ sB,
                                                              const int32_t *__restrict__ offsets, int groups,
                                                              int rows, int F, int K, GatedOut out)
{
    __shared__ v4f sums[2][kWK][64]; // of g, of u
    const int tiles_n = F / 16;
    const int t = blockIdx.x / tiles_n, n0 = (int)(blockIdx.x % tiles_n) * 16;
    GroupTiles<16> tiles(offsets, groups, rows);
    if (t >= tiles.total) return;
    const GroupTile gt = tiles.find(t);
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int nk = K / 128;
    const int left = gt.size - 16 * gt.tile; // rows of the tile in the group
    // rows past the group's last repeat it; their results are not stored
    const int64_t row = (int64_t)gt.row0 + 16 * gt.tile + min(r, left - 1);
    const uint8_t *a = A + row * K;
    const float *sa = sA + row * nk;
    const uint8_t *bg = B + ((int64_t)gt.group * 2 * F + n0 + r) * K, *bu = bg + (int64_t)F * K;
    const float *sg = sB + ((int64_t)gt.group * 2 * (F / 128) + n0 / 128) * nk, *su = sg + (int64_t)(F / 128) * nk;
    v4f cg{0.f, 0.f, 0.f, 0.f}, cu{0.f, 0.f, 0.f, 0.f};
    for (int kb = w; kb < nk; kb += kWK) {
        const v8i fg = load_frag(bg + kb * 128, g), fu = load_frag(bu + kb * 128, g), fa = load_frag(a + kb * 128, g);
        const float s = sa[kb], wg = s * sg[kb], wu = s * su[kb];
        const v4f pg = mfma16x16x128<FB, FA>(fg, fa, v4f{0.f, 0.f, 0.f, 0.f});
        const v4f pu = mfma16x16x128<FB, FA>(fu, fa, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            cg[e] = __builtin_fmaf(pg[e], wg, cg[e]);
            cu[e] = __builtin_fmaf(pu[e], wu, cu[e]);
        }
    }
    sums[0][w][lane] = cg, sums[1][w][lane] = cu;
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int k = 1; k < kWK; ++k) cg += sums[0][k][lane], cu += sums[1][k][lane];
    if (r >= left) return;
    const int col = n0 + 4 * g;
    if (out.ws) {
        float *p = out.ws + row * 2 * F + col;
        *reinterpret_cast<v4f *>(p) = cg;
        *reinterpret_cast<v4f *>(p + F) = cu;
        return;
    }
    v4f h;
    with_act(out.act, [&](auto act) {
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = act_f32<decltype(act)::value>(cg[e]) * cu[e];
    });
    if (out.h_dtype == kBF16)
        *reinterpret_cast<uint2 *>((uint16_t *)out.H + row * F + col) =
            __builtin_bit_cast(uint2, __builtin_convertvector(h, bf16x4));
    else
        *reinterpret_cast<v4f *>((float *)out.H + row * F + col) = h;
}

template <int FA, int FB> hipError_t launch_gated(const GatedArgs &a)
{
#define FP8Q_GATED_ROWS(WK)                                                                                          \
    gated_rows_kernel<FA, FB, WK><<<(unsigned)(max_tiles(a.rows, a.groups, 16) * (a.F / 16)), 64 * WK, 0, a.stream>>>( \
        a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows, (int)a.F, (int)a.K, a.out)
    switch (gated_tile(a.rows, a.groups, a.F, a.K, a.out.q_h || a.out.q_gu, a.cus)) {
    case kGated16:
        switch (rows_waves(a.K)) {
        case 4: FP8Q_GATED_ROWS(4); break;
        case 8: FP8Q_GATED_ROWS(8); break;
        default: FP8Q_GATED_ROWS(16);
        }
        break;
    case kGatedMid:
        gated_mid_kernel<FA, FB>
            <<<(unsigned)(max_tiles(a.rows, a.groups, 64) * (a.F / 128) + kXcds), kBSThreads, 0, a.stream>>>(
                a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows, (int)a.F, (int)a.K, a.out);
        break;
    case kGatedPP: {
        const int cus = a.cus / kXcds > 1 ? a.cus / kXcds : 1; // of an XCD
        gated_pp_kernel<FA, FB><<<(unsigned)gated_pp_blocks(a.rows, a.groups, a.F, cus), kBSThreads, 0, a.stream>>>(
            a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows, (int)a.F, (int)a.K, a.out, cus);
    }
    }
#undef FP8Q_GATED_ROWS
    return hipGetLastError();
}

// One operand-format pair's launcher (one translation unit each).
#define FP8Q_GATED_PAIR(NAME, FA, FB)                                                                                \
    hipError_t launch_gated_##NAME(const GatedArgs &a) { return launch_gated<FA, FB>(a); }

} // namespace fp8q

#endif // FP8Q_GATED_GEMM_H
