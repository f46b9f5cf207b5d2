// grouped_gemm.h -- FP8 products of ragged groups of rows with a matrix per
// group (the experts of a layer), included by one translation unit per
// operand-format pair.
//
// fprop / dgrad: rows t of group e, C[t] = sum over 128-wide slices kb of
//   fma(part_kb, fl32(sA[t, kb] sB[e, n / 128, kb]), acc),
//   part_kb the slice's products on the FP8 matrix instruction,
//   B [groups][N][K] codes with 128x128 block scales.
// wgrad: C[e] = A_e B_e^T contracted over the rows (tokens) of group e, from
//   the token-contiguous copies A [M][stride], B [N][stride] with one scale
//   per row and block of 128 tokens; a group's tokens fill whole blocks.
#ifndef FP8Q_GROUPED_GEMM_H
#define FP8Q_GROUPED_GEMM_H

#include "gemm_kernels.h"
#include "groups.h"

namespace fp8q {

// 32 bytes of a 128-byte slice row for lane group g: chunks g and g + 4 (A and
// B use the same ones, so the order inside the slice does not matter)
__device__ __forceinline__ v8i load_frag(const uint8_t *row, int g)
{
    const uint4 lo = *reinterpret_cast<const uint4 *>(row + 16 * g);
    const uint4 hi = *reinterpret_cast<const uint4 *>(row + 64 + 16 * g);
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight codes -> eight bf16 values (exact: bf16 has more exponent and mantissa
// bits than either format).
template <int F> __device__ __forceinline__ bf16x8 widen8(int lo, int hi)
{
    bf16x2 p[4];
    if constexpr (F == kE4M3) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
    }
    return bf16x8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// One slice's 16x16 partial.  kWide: the codes are widened to bf16 and
// multiplied by the bf16 matrix instruction, whose sums are binary32.
// The FP8 instruction adds the products of eight neighbouring bytes on about
// 15 bits under the largest of them (measured on the MI355X with one large
// and one small product at a time), which leaves an fp32 result 1.1e-5 off in
// the 2-norm where the widened one is 1e-8 off: below the rounding of a bf16
// result, but above that of an fp32 one.
template <int FA, int FB, bool kWide> __device__ __forceinline__ v4f slice16(const v8i &b, const v8i &a)
{
    if constexpr (!kWide) {
        return mfma16x16x128<FB, FA>(b, a, v4f{0.f, 0.f, 0.f, 0.f});
    } else {
        v4f c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<FB>(b[2 * s], b[2 * s + 1]),
                                                        widen8<FA>(a[2 * s], a[2 * s + 1]), c, 0, 0, 0);
        return c;
    }
}

struct GroupedArgs {
    const uint8_t *A, *B;
    const float *sA, *sB;
    const int32_t *offsets;
    int groups, rows;
    int64_t M, N, K; // wgrad: M x N per group; K unused
    int64_t stride;  // wgrad: bytes of a row of A and B
    void *C;
    int c_dtype;
    hipStream_t stream;
    int cus;
};

// fprop / dgrad for few rows per group, where the weights' bytes are what
// counts: 16 kMT rows of a group x 16 kNT columns per block, fragments loaded
// straight from memory into registers (a weight byte is used by one wave).
// kWK waves take the 128-wide slices in turn and add their sums through LDS.
template <int FA, int FB, int kMT, int kNT, int kWK>
__global__ __launch_bounds__(64 * kWK) void grouped_rows_kernel(const uint8_t *__restrict__ A,
                                                                const float *__restrict__ sA,
                                                                const uint8_t *__restrict__ B,
                                                                const float *__restrict__ sB,
                                                                const int32_t *__restrict__ offsets, int groups,
                                                                int rows, int N, int K, uint16_t *__restrict__ C)
{
    constexpr int kTM = 16 * kMT, kTN = 16 * kNT, kT = kMT * kNT;
    __shared__ v4f sums[kWK][kT][64];
    const int tiles_n = N / kTN;
    const int t = blockIdx.x / tiles_n, n0 = (int)(blockIdx.x % tiles_n) * kTN;
    GroupTiles<kTM> tiles(offsets, groups, rows);
    if (t >= tiles.total) return;
    const GroupTile gt = tiles.find(t);
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int nk = K / 128;
    const int left = gt.size - kTM * gt.tile; // rows of the tile in the group
    const int64_t row0 = gt.row0 + kTM * gt.tile;
    // rows past the group's last repeat it; their results are not stored
    const uint8_t *Ar[kMT];
    const float *sAr[kMT];
#pragma unroll
    for (int i = 0; i < kMT; ++i) {
        const int64_t row = row0 + min(16 * i + r, left - 1);
        Ar[i] = A + row * K;
        sAr[i] = sA + row * nk;
    }
    const uint8_t *Bg = B + ((int64_t)gt.group * N + n0 + r) * K;
    const float *sBg = sB + ((int64_t)gt.group * (N / 128) + n0 / 128) * nk;
    v4f acc[kMT][kNT];
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int kb = w; kb < nk; kb += kWK) {
        v8i a[kMT], b[kNT];
        float wt[kMT];
        const float sb = sBg[kb];
#pragma unroll
        for (int j = 0; j < kNT; ++j) b[j] = load_frag(Bg + (int64_t)(16 * j) * K + kb * 128, g);
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            a[i] = load_frag(Ar[i] + kb * 128, g);
            wt[i] = sAr[i][kb] * sb;
        }
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
                const v4f p = slice16<FA, FB, false>(b[j], a[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e], wt[i], acc[i][j][e]);
            }
    }
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j) sums[w][i * kNT + j][lane] = acc[i][j];
    __syncthreads();
    for (int q = w; q < kT; q += kWK) {
        const int i = q / kNT, j = q % kNT;
        v4f c = sums[0][q][lane];
#pragma unroll
        for (int k = 1; k < kWK; ++k) c += sums[k][q][lane];
        if (16 * i + r < left)
            *reinterpret_cast<uint2 *>(C + (row0 + 16 * i + r) * N + n0 + 16 * j + 4 * g) =
                __builtin_bit_cast(uint2, __builtin_convertvector(c, bf16x4));
    }
}

// ---------------------------------------------------------------------------
// One kTM x kTN tile of C on eight waves, the ping-pong schedule of
// gemm_bs_pp_kernel for ragged operands: A and B rows past the tile's own are
// loaded as zeros (the buffer records end there) and never stored, and the
// contraction may start anywhere in the operands' rows (wgrad).
//
// Waves: kTM / 64 row strips x kTN / kWC column strips of 64 x kWC, group X
// (waves 0-3) the left half of the columns, Y the right half.  256 x 256 tiles
// have 64 x 128 waves; 128 x 256 and 256 x 128 tiles, for the rows a group
// leaves over and for the widened products, 64 x 64.
//
// kWide (fp32 results): a read phase also widens the fragments it has read to
// bf16, while the other group's matrix instructions run, and a compute phase
// chains four bf16 instructions per 16x16 tile and slice.
struct PPOperand {
    const uint8_t *base; // first row of the tile, first byte of the contraction
    int bytes;           // readable from base
    int pitch;           // bytes of a row
    const float *s;      // scales of the first row (128x128: block row) and slice
    int s_bytes, s_pitch; // readable bytes; floats of a row (of blocks)
};

template <int kTM, int kTN> struct PPShape {
    static constexpr int kRS = kTM / 64;            // row strips
    static constexpr int kCS = 8 / kRS;             // column strips
    static constexpr int kWC = kTN / kCS;           // a wave's columns
    static constexpr int kQ = kWC / 2, kJT = kQ / 16; // a half's columns and 16-wide column tiles
    static constexpr int kA = kTM * kBK, kB2 = kTN / 2 * kBK; // code bytes of A, of B's first / second halves
    static constexpr int oB0 = kA, oB1 = kA + kB2, kStage = kA + 2 * kB2;
};

// Scales of four slices, three groups of them in LDS: a run of 16 rows is 64
// floats, [slice][row].
constexpr int kScaleGroups = 3;
template <int kTM, int kTN, bool kRowB> constexpr int pp_scale_runs() { return kTM / 16 + (kRowB ? kTN / 16 : 1); }

template <int FA, int FB, int kTM, int kTN, bool kRowB, bool kWide, int DC>
__device__ __forceinline__ void pp_tile(uint8_t *st0, uint8_t *st1, float *sx, const PPOperand &A, const PPOperand &B, int kblocks,
                                        int sb_last, void *C, int64_t ldc, int c_rows, int c_cols)
{
    typedef PPShape<kTM, kTN> P;
    constexpr int kQ = P::kQ, kJT = P::kJT;
    constexpr int kAL = kTM / 64, kBL = kTN / 128; // loads per wave of A, of a B half
    constexpr int G1 = kAL + kBL, G2 = kBL + 1; // G2 with the slice's load of scales
    constexpr int kVm = G1 + G2; // younger loads allowed at the end of every phase
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool gx = w < 4;
    const int wm = w % P::kRS, wn = w / P::kRS;
    const int fr = lane & 15, fg = lane >> 4;
    const int ap = A.pitch, bp = B.pitch;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void *)A.base, 0, A.bytes, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void *)B.base, 0, B.bytes, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void *)A.s, 0, A.s_bytes, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t rsb = __builtin_amdgcn_make_buffer_rsrc((void *)B.s, 0, B.s_bytes, kRawBufferWord3);
    const int swz_lane = ((lane & 7) ^ ((4 * w + (lane >> 4)) & 7)) << 4;
    const int avoff = (lane >> 3) * ap + swz_lane, bvoff = (lane >> 3) * bp + swz_lane;
    const int sx_row = lane & 15, sx_slice = lane >> 4;
    const int sa_voff = (sx_row * A.s_pitch + sx_slice) * 4;
    const int sb_voff = ((kRowB ? sx_row : min(sx_row, sb_last)) * B.s_pitch + sx_slice) * 4;

    auto load_b = [&](uint8_t *dst, int h, int kb) {
#pragma unroll
        for (int u = 0; u < kBL; ++u) {
            const int row = 8 * (w + 8 * u);
            const int trow = (row / kQ) * 2 * kQ + kQ * h + row % kQ;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void *)(dst + row * kBK), 16, bvoff, trow * bp + kb * kBK,
                                                     0, 0);
        }
    };
    auto load_g1 = [&](uint8_t *st, int kb) {
#pragma unroll
        for (int u = 0; u < kAL; ++u) {
            const int row = 8 * (w + 8 * u);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(st + row * kBK), 16, avoff, row * ap + kb * kBK,
                                                     0, 0);
        }
        load_b(st + P::oB0, 0, kb);
    };
    // Quarter f % 4 of the scales of slices 4 (f / 4) .. + 3: every wave loads
    // one run of 16 rows, four lanes a row (a load of one slice's scales would
    // touch 64 rows, a line each).  Slice kb issues quarter kb + 6, so a group
    // is whole three slices before it is read and its place has been free for two.
    constexpr int kRuns = pp_scale_runs<kTM, kTN, kRowB>(), kGroup = 64 * kRuns;
    auto load_scales = [&](int f, int place) {
        const int run = min((f & 3) * 8 + w, kRuns - 1);
        float *dst = sx + place * kGroup + 64 * run;
        if (run < kTM / 16)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)dst, 4, sa_voff,
                                                     (16 * run * A.s_pitch + (f & ~3)) * 4, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (lds_void *)dst, 4, sb_voff,
                                                     (16 * (run - kTM / 16) * B.s_pitch + (f & ~3)) * 4, 0, 0);
    };
    auto load_g2 = [&](uint8_t *st, int kb) {
        load_b(st + P::oB1, 1, kb);
    };

    v4f acc[4][2 * kJT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2 * kJT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    v8i a[4], b[kJT];                         // the slice's A fragments, the half's B fragments
    bf16x8 aw[kWide ? 4 : 1][4], bw[kWide ? kJT : 1][4]; // the same widened
    float wi[4];
    v4f sbq[kJT];
    v4f pr[3]; // results awaiting promotion (tile t in pr[t % 3])

    auto promote = [&](auto hc, int t) {
        constexpr int h = decltype(hc)::value;
        const int i = t & 3, jj = t >> 2;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[i][kJT * h + jj][e] =
                __builtin_fmaf(pr[t % 3][e], kRowB ? wi[i] * sbq[jj][e] : wi[i], acc[i][kJT * h + jj][e]);
        asm volatile("" : "+v"(acc[i][kJT * h + jj])); // keeps these FMAs in their phase
    };
    constexpr int kT = 4 * kJT;
    auto compute = [&](auto hc) {
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            if constexpr (kWide) {
                v4f c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bw[t >> 2][s], aw[t & 3][s], c, 0, 0, 0);
                pr[t % 3] = c;
            } else {
                pr[t % 3] = mfma16x16x128<FB, FA>(b[t >> 2], a[t & 3], v4f{0.f, 0.f, 0.f, 0.f});
            }
            if (t >= 2) promote(hc, t - 2);
        }
        if constexpr (!kWide) {
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0); // MFMA
                if (t >= 2) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0); // promotion FMAs
            }
        }
    };
    auto tail = [&](auto hc) {
        promote(hc, kT - 2);
        promote(hc, kT - 1);
    };
    auto read_a = [&](const uint8_t *st) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = read_frag(st, wm * 64 + 16 * i + fr, fg);
    };
    auto read_b = [&](const uint8_t *st) {
#pragma unroll
        for (int jj = 0; jj < kJT; ++jj) b[jj] = read_frag(st, wn * kQ + 16 * jj + fr, fg);
    };
    auto widen_a = [&]() {
        if constexpr (kWide) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int s = 0; s < 4; ++s) aw[i][s] = widen8<FA>(a[i][2 * s], a[i][2 * s + 1]);
        }
    };
    auto widen_b = [&]() {
        if constexpr (kWide) {
#pragma unroll
            for (int jj = 0; jj < kJT; ++jj)
#pragma unroll
                for (int s = 0; s < 4; ++s) bw[jj][s] = widen8<FB>(b[jj][2 * s], b[jj][2 * s + 1]);
        }
    };
    // the scales of the slice whose group and slice start at sg (with the first
    // half, A's and the 128x128 blocks'; B's rows per half)
    auto read_scales = [&](const float *sg, int h) {
        const float *sb = sg + 64 * (kTM / 16);
        if (h == 0) {
            // 128x128 blocks: a wave's columns lie in one column block
            const float blk = kRowB ? 1.0f : sb[kTN == 256 ? wn * P::kWC / 128 : 0];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float sa = sg[64 * (wm * 4 + i) + fr];
                wi[i] = kRowB ? sa : sa * blk;
            }
        }
        if constexpr (kRowB) {
            // half h's column tile jj is tile columns wn * kWC + kQ h + 16 jj ..
#pragma unroll
            for (int jj = 0; jj < kJT; ++jj)
                sbq[jj] = *reinterpret_cast<const v4f *>(sb + 64 * ((wn * P::kWC + kQ * h) / 16 + jj) + 4 * fg);
        }
    };
    auto phase_end = [&](auto wc) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(decltype(wc)::value);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto sync_lds = [&]() { phase_end(PhaseC<waitcnt_imm(kVm, 0)>{}); };
    auto sync = [&]() { phase_end(PhaseC<waitcnt_imm(kVm, 15)>{}); };
    using H0 = PhaseC<0>;
    using H1 = PhaseC<1>;

    int place = 0, place6 = 1; // of slice kb's group of scales, and of slice kb + 6's
    auto slice = [&](int kb, uint8_t *cur, uint8_t *nxt) {
        const float *sg = sx + place * kGroup + 16 * (kb & 3);
        read_a(cur);
        read_b(cur + P::oB0);
        tail(H1{});
        read_scales(sg, 0);
        load_scales(kb + 6, place6);
        load_g2(nxt, kb + 1);
        widen_a();
        widen_b();
        sync_lds();
        compute(H0{});
        sync();
        read_b(cur + P::oB1);
        tail(H0{});
        read_scales(sg, 1);
        load_g1(cur, kb + 2);
        widen_b();
        if ((kb & 3) == 3) place = place == kScaleGroups - 1 ? 0 : place + 1;
        if (((kb + 6) & 3) == 3) place6 = place6 == kScaleGroups - 1 ? 0 : place6 + 1;
        sync_lds();
        compute(H1{});
        sync();
    };

    if (kblocks > 0) {
#pragma unroll
        for (int f = 0; f < 6; ++f) load_scales(f, f >> 2);
        load_g1(st0, 0);
        load_g2(st0, 0);
        load_g1(st1, 1);
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(G2 - 1 + G1, 15));
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int q = 0; q < 3; ++q) pr[q] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) wi[i] = 0.0f;
#pragma unroll
    for (int jj = 0; jj < kJT; ++jj) sbq[jj] = v4f{0.f, 0.f, 0.f, 0.f};
    if (!gx) sync(); // group Y starts one phase later
    int kb = 0;
    for (; kb + 1 < kblocks; kb += 2) {
        slice(kb, st0, st1);
        slice(kb + 1, st1, st0);
    }
    if (kb < kblocks) slice(kb, st0, st1);
    if (gx) sync(); // and ends one phase later
    tail(H1{});
    // the loads of the slices past the end must land before the stages are reused
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    // epilogue: each wave stages its 64 x kWC results and stores whole row pieces
    constexpr int kB = DC == kF32 ? 4 : 2;
    typedef EpiStage<P::kWC, kB, 64, P::kWC * kBK> ES;
    const int wrow = wm * 64, wcol = wn * P::kWC;
    const bool inside = wrow < c_rows && wcol < c_cols;
    uint8_t *ep = (w < 4 ? st0 : st1) + (w & 3) * (P::kWC * kBK);
    uint32_t m = 0;
    const Epi none{nullptr, kActNone, nullptr};
#pragma unroll
    for (int ps = 0; ps < ES::kPasses; ++ps) {
        if (ps > 0) __syncthreads();
        if (inside) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if ((16 * i) / ES::kPassRows != ps) continue;
#pragma unroll
                for (int j = 0; j < 2 * kJT; ++j)
                    ES::put(ep, 16 * i + fr - ps * ES::kPassRows, 4 * j + fg,
                            pack_out4<DC == kF32 ? kOutF32 : kOutBF16, false, false>(0, acc[i][j], m, none, 0.0f));
            }
        }
        __syncthreads();
        if (inside) {
            const int c = lane % ES::kNC, rr = lane / ES::kNC;
            uint8_t *Cb = reinterpret_cast<uint8_t *>(C);
#pragma unroll 4
            for (int s = 0; s < ES::kPassRows / ES::kRowsPerStore; ++s) {
                const int r = s * ES::kRowsPerStore + rr, row = wrow + ps * ES::kPassRows + r;
                const uint4 v = *reinterpret_cast<const uint4 *>(ep + ES::addr(r, c));
                if (row < c_rows) st_stream(Cb + ((int64_t)row * ldc + wcol) * kB + 16 * c, v);
            }
        }
    }
}

// Block b of a grid -> tile of `n` tiles, each XCD a contiguous run; >= n: none.
__device__ __forceinline__ int xcd_tile(int b, int n)
{
    const int per = (n + kXcds - 1) / kXcds, i = b / kXcds;
    return i < per ? (b % kXcds) * per + i : n;
}

// fprop / dgrad in tiles of 256 rows x 256 columns; a group's last tile of at
// most 128 rows runs as a 128 x 256 tile.
template <int FA, int FB>
__global__ __launch_bounds__(kBSThreads, 1) void grouped_pp_kernel(const uint8_t *__restrict__ A,
                                                                   const float *__restrict__ sA,
                                                                   const uint8_t *__restrict__ B,
                                                                   const float *__restrict__ sB,
                                                                   const int32_t *__restrict__ offsets, int groups,
                                                                   int rows, int N, int K, uint16_t *__restrict__ C)
{
    typedef PPShape<256, 256> P;
    __shared__ __attribute__((aligned(1024))) uint8_t st0[P::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[P::kStage];
    __shared__ __attribute__((aligned(16))) float sx[kScaleGroups * 64 * pp_scale_runs<256, 256, false>()];
    const int tiles_n = (N + 255) / 256, nk = K / kBK;
    GroupTiles<256> tiles(offsets, groups, rows);
    const int t = xcd_tile(blockIdx.x, tiles.total * tiles_n);
    if (t >= tiles.total * tiles_n) return;
    const GroupTile gt = tiles.find(t / tiles_n);
    int tm, tn;
    group_tile(gt.tile * tiles_n + t % tiles_n, (gt.size + 255) / 256, tiles_n, tm, tn);
    const int64_t row0 = gt.row0 + 256 * tm, n0 = 256 * tn;
    const int a_rows = min(256, gt.size - 256 * tm), b_rows = min(256, N - (int)n0);
    const PPOperand a{A + row0 * K, a_rows * K, K, sA + row0 * nk, a_rows * nk * 4, nk};
    const int b_blocks = b_rows / 128; // 1 in a last, half-empty tile column
    const PPOperand b{B + ((int64_t)gt.group * N + n0) * K, b_rows * K, K,
                      sB + ((int64_t)gt.group * (N / 128) + n0 / 128) * nk, b_blocks * nk * 4, nk};
    uint16_t *c = C + row0 * N + n0;
    if (a_rows > 128)
        pp_tile<FA, FB, 256, 256, false, false, kBF16>(st0, st1, sx, a, b, nk, b_blocks - 1, c, N, a_rows,
                                                       b_rows);
    else
        pp_tile<FA, FB, 128, 256, false, false, kBF16>(st0, st1, sx, a, b, nk, b_blocks - 1, c, N, a_rows,
                                                       b_rows);
}

// Blocks of 128 tokens before group e and in it (wave-uniform).
__device__ __forceinline__ void group_blocks(const int32_t *offsets, int groups, int rows, int e, int kbs, int &kb0,
                                             int &kbn)
{
    kb0 = kbn = 0;
    for (int g0 = 0; g0 <= e; g0 += 64) {
        int lo, size;
        group_rows(offsets, groups, rows, g0 + (threadIdx.x & 63), lo, size);
        const int count = (int)(((unsigned)size + 127) / 128), sum = wave_scan_i32(count);
        if (e < g0 + 64) {
            kbn = __builtin_amdgcn_readlane(count, e - g0);
            kb0 += __builtin_amdgcn_readlane(sum, e - g0) - kbn;
        } else {
            kb0 += __builtin_amdgcn_readlane(sum, 63);
        }
    }
    // the caller's buffers may be too short for these offsets
    kb0 = min(kb0, kbs);
    kbn = min(kbn, kbs - kb0);
}

// Tile i of an XCD's share of the groups' tiles (`per` each): every group's
// tiles are split over the XCDs, so that they get equal shares of long and of
// short contractions; an XCD's share of a group is a contiguous run of its
// grouped order.  tile >= per: none.
__device__ __forceinline__ void group_share(int xcd, int i, int per, int &e, int &tile)
{
    const int share = (per + kXcds - 1) / kXcds;
    e = i / share;
    const int j = i - e * share;
    tile = xcd * share + j;
}

// wgrad in kTM x kTN tiles of one group's C per block.
template <int FA, int FB, int kTM, int kTN, int DC>
__global__ __launch_bounds__(kBSThreads, 1) void grouped_wgrad_pp_kernel(
    const uint8_t *__restrict__ A, const float *__restrict__ sA, const uint8_t *__restrict__ B,
    const float *__restrict__ sB, const int32_t *__restrict__ offsets, int groups, int rows, int M, int N,
    int64_t stride, void *__restrict__ C)
{
    typedef PPShape<kTM, kTN> P;
    __shared__ __attribute__((aligned(1024))) uint8_t st0[P::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[P::kStage];
    __shared__ __attribute__((aligned(16))) float sx[kScaleGroups * 64 * pp_scale_runs<kTM, kTN, true>()];
    const int tiles_m = (M + kTM - 1) / kTM, tiles_n = (N + kTN - 1) / kTN, per = tiles_m * tiles_n;
    int e, tile, tm, tn, kb0, kbn;
    group_share(blockIdx.x % kXcds, blockIdx.x / kXcds, per, e, tile);
    if (e >= groups || tile >= per) return;
    group_tile(tile, tiles_m, tiles_n, tm, tn);
    const int kbs = (int)(stride / 128);
    group_blocks(offsets, groups, rows, e, kbs, kb0, kbn);
    const int64_t m0 = (int64_t)tm * kTM, n0 = (int64_t)tn * kTN;
    const int a_rows = min(kTM, M - (int)m0), b_rows = min(kTN, N - (int)n0), pitch = (int)stride;
    const PPOperand a{A + m0 * stride + (int64_t)kb0 * 128, a_rows * pitch - kb0 * 128, pitch, sA + m0 * kbs + kb0,
                      (a_rows * kbs - kb0) * 4, kbs};
    const PPOperand b{B + n0 * stride + (int64_t)kb0 * 128, b_rows * pitch - kb0 * 128, pitch, sB + n0 * kbs + kb0,
                      (b_rows * kbs - kb0) * 4, kbs};
    uint8_t *c = reinterpret_cast<uint8_t *>(C) + (((int64_t)e * M + m0) * N + n0) * (DC == kF32 ? 4 : 2);
    pp_tile<FA, FB, kTM, kTN, true, DC == kF32, DC>(st0, st1, sx, a, b, kbn, 0, c, N, a_rows, b_rows);
}

// The tile of an fprop / dgrad launch.  Up to 12 rows a group on average most
// groups fit a 16-row tile, so the weights are read once, and 32 columns a block are
// faster than 16 unless the blocks then do not fill the chip (8 rows over
// eight 14336 x 4096 matrices: 53.6 and 59.1 us; 64 columns 56.8 us).  Above,
// a launch takes about `step` per round of one block per CU, `least` at the
// least: both measured at K = 4096, one 4096-column matrix with 16 to 1024
// rows, in us.  The steps grow slower than the tiles' areas, so the large
// ping-pong tiles win as soon as they fill a part of the chip: 256 rows over
// those eight matrices 109 us against 132 us in 32 x 64 tiles, but 40 rows of
// one 4096 x 4096 matrix 11.7 us in 32 x 32 tiles against 29 us.
enum RowsTile { kRows16x16, kRows16x32, kRows32x32, kRows32x64, kRows64x64, kRowsPP };

inline RowsTile rows_tile(const GroupedArgs &a)
{
    const int64_t cus = a.cus > 0 ? a.cus : 256;
    auto blocks = [&](int tm, int tn) { return max_tiles(a.rows, a.groups, tm) * ((a.N + tn - 1) / tn); };
    const int64_t live = a.rows < a.groups ? a.rows : a.groups;
    if (a.rows <= 12 * live) return blocks(16, 32) >= cus ? kRows16x32 : kRows16x16;
    static const struct {
        int tm, tn;
        double least, step;
    } cost[6] = {{16, 16, 8.7, 5.0},   {16, 32, 8.8, 7.2},   {32, 32, 11.5, 10.5},
                 {32, 64, 15.4, 14.5}, {64, 64, 22.5, 22.0}, {256, 256, 40.0, 40.0}};
    RowsTile best = kRowsPP;
    double least = 0.0;
    for (int i = kRowsPP; i >= kRows16x16; --i) {
        const int64_t rounds = (blocks(cost[i].tm, cost[i].tn) + cus - 1) / cus;
        double us = cost[i].step * (double)rounds;
        if (i == kRowsPP && a.rows <= 128 * live) us *= 29.0 / 40.0; // mostly 128 x 256 tiles
        if (us < cost[i].least) us = cost[i].least;
        if (i == kRowsPP || us < least) best = (RowsTile)i, least = us;
    }
    return best;
}

template <int FA, int FB> hipError_t launch_grouped_rows(const GroupedArgs &a)
{
#define FP8Q_ROWS(MT, NT, WK)                                                                                        \
    grouped_rows_kernel<FA, FB, MT, NT, WK>                                                                          \
        <<<(unsigned)(max_tiles(a.rows, a.groups, 16 * MT) * (a.N / (16 * NT))), 64 * WK, 0, a.stream>>>(            \
            a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows, (int)a.N, (int)a.K, (uint16_t *)a.C)
    switch (rows_tile(a)) {
    case kRows16x16: FP8Q_ROWS(1, 1, 8); break;
    case kRows16x32: FP8Q_ROWS(1, 2, 8); break;
    case kRows32x32: FP8Q_ROWS(2, 2, 8); break;
    case kRows32x64: FP8Q_ROWS(2, 4, 4); break;
    case kRows64x64: FP8Q_ROWS(4, 4, 4); break;
    default: {
        const int64_t tiles = max_tiles(a.rows, a.groups, 256) * ((a.N + 255) / 256);
        grouped_pp_kernel<FA, FB><<<(unsigned)(tiles + kXcds), kBSThreads, 0, a.stream>>>(
            a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows, (int)a.N, (int)a.K, (uint16_t *)a.C);
    }
    }
#undef FP8Q_ROWS
    return hipGetLastError();
}

template <int FA, int FB> hipError_t launch_grouped_wgrad(const GroupedArgs &a)
{
#define FP8Q_WGRAD(TM, TN, DC)                                                                                       \
    grouped_wgrad_pp_kernel<FA, FB, TM, TN, DC>                                                                      \
        <<<(unsigned)(a.groups * kXcds * ((((a.M + TM - 1) / TM) * ((a.N + TN - 1) / TN) + kXcds - 1) / kXcds)),     \
           kBSThreads, 0, a.stream>>>(a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows, (int)a.M, (int)a.N, a.stride, a.C)
    if (a.c_dtype == kBF16) FP8Q_WGRAD(256, 256, kBF16);
    else FP8Q_WGRAD(256, 128, kF32);
#undef FP8Q_WGRAD
    return hipGetLastError();
}

// One operand-format pair's launchers (one translation unit each).
#define FP8Q_GROUPED_PAIR(NAME, FA, FB)                                                                              \
    hipError_t launch_grouped_rows_##NAME(const GroupedArgs &a) { return launch_grouped_rows<FA, FB>(a); }           \
    hipError_t launch_grouped_wgrad_##NAME(const GroupedArgs &a) { return launch_grouped_wgrad<FA, FB>(a); }

} // namespace fp8q

#endif // FP8Q_GROUPED_GEMM_H
