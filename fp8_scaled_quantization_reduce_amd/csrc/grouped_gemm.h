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

constexpr int kBufferNt = 2; // the non-temporal hint of a buffer store

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
// The weights' bytes bound it: 64 rows over eight 14336 x 4096 matrices 86 us,
// 5.5 TB/s; the hint that a weight is read once costs 15%, loads of two or four
// slices at a time change nothing.
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
                const v4f p = mfma16x16x128<FB, FA>(b[j], a[i], v4f{0.f, 0.f, 0.f, 0.f});
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

// A wave's staged results (kRows rows of `bytes` bytes) to C, rows `pitch` bytes
// apart; rows from `left` on lie outside the buffer and are dropped.  The wave
// wrote the stage itself, so it waits for no other.
template <typename ES, int kRows>
__device__ __forceinline__ void store_rows(const uint8_t *ep, void *C, int pitch, int bytes, int left, int lane)
{
    static_assert(ES::kPasses == 1, "a wave's results fit its part of the stages");
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
    asm volatile("" ::: "memory");
    const __amdgpu_buffer_rsrc_t rc =
        __builtin_amdgcn_make_buffer_rsrc(C, 0, (min(kRows, left) - 1) * pitch + bytes, kRawBufferWord3);
    const int c = lane % ES::kNC, rr = lane / ES::kNC, voff = rr * pitch + 16 * c;
#pragma unroll 4
    for (int s = 0; s < kRows / ES::kRowsPerStore; ++s) {
        const uint4 v = *reinterpret_cast<const uint4 *>(ep + ES::addr(s * ES::kRowsPerStore + rr, c));
        __builtin_amdgcn_raw_buffer_store_b128(u32x4v{v.x, v.y, v.z, v.w}, rc, voff, s * ES::kRowsPerStore * pitch,
                                               kBufferNt);
    }
}

// ---------------------------------------------------------------------------
// One kTM x 256 tile of C (bf16) on eight waves, the ping-pong schedule of
// gemm_bs_pp_kernel for ragged operands: A and B rows past the tile's own are
// loaded as zeros (the buffer records end there) and never stored, and the
// contraction may start anywhere in the operands' rows (wgrad).
//
// Waves: kTM / 64 row strips x kTN / kWC column strips of 64 x kWC, group X
// (waves 0-3) the left half of the columns, Y the right half.  256 x 256 tiles
// have 64 x 128 waves; 128 x 256 tiles, for the rows a group leaves over, 64 x 64.
struct PPOperand {
    const uint8_t *base; // first row of the tile, first byte of the contraction
    int bytes;           // readable from base
    int pitch;           // bytes of a row
    const float *s;      // scales of the first row (128x128: block row) and slice
    int s_bytes, s_pitch; // readable bytes; floats of a row (of blocks)
};

template <int kTM> struct PPShape {
    static constexpr int kTN = 256;
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
template <int kTM, bool kRowB> constexpr int pp_scale_runs() { return kTM / 16 + (kRowB ? 16 : 1); }

template <int FA, int FB, int kTM, bool kRowB>
__device__ __forceinline__ void pp_tile(uint8_t *st0, uint8_t *st1, float *sx, const PPOperand &A, const PPOperand &B,
                                        int kblocks, int sb_last, uint16_t *C, int64_t ldc, int c_rows, int c_cols)
{
    constexpr int kTN = 256;
    typedef PPShape<kTM> P;
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
    constexpr int kRuns = pp_scale_runs<kTM, kRowB>(), kGroup = 64 * kRuns;
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
            pr[t % 3] = mfma16x16x128<FB, FA>(b[t >> 2], a[t & 3], v4f{0.f, 0.f, 0.f, 0.f});
            if (t >= 2) promote(hc, t - 2);
        }
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0); // MFMA
            if (t >= 2) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0); // promotion FMAs
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
    // the scales of the slice whose group and slice start at sg (with the first
    // half, A's and the 128x128 blocks'; B's rows per half)
    auto read_scales = [&](const float *sg, int h) {
        const float *sb = sg + 64 * (kTM / 16);
        if (h == 0) {
            // 128x128 blocks: a wave's columns lie in one column block
            const float blk = kRowB ? 1.0f : sb[wn * P::kWC / 128];
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
        sync_lds();
        compute(H0{});
        sync();
        read_b(cur + P::oB1);
        tail(H0{});
        read_scales(sg, 1);
        load_g1(cur, kb + 2);
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

    // epilogue: each wave stages its 64 x kWC results in a part of the stages of
    // its own and stores whole row pieces
    typedef EpiStage<P::kWC, 2, 64, P::kWC * kBK> ES;
    const int wrow = wm * 64, wcol = wn * P::kWC;
    if (wrow >= c_rows || wcol >= c_cols) return;
    uint8_t *ep = (w < 4 ? st0 : st1) + (w & 3) * (P::kWC * kBK);
    uint32_t m = 0;
    const Epi none{nullptr, kActNone, nullptr};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2 * kJT; ++j)
            ES::put(ep, 16 * i + fr, 4 * j + fg, pack_out4<kOutBF16, false, false>(0, acc[i][j], m, none, 0.0f));
    store_rows<ES, 64>(ep, C + (int64_t)wrow * ldc + wcol, (int)ldc * 2, P::kWC * 2, c_rows - wrow, lane);
}

// fprop / dgrad in tiles of 256 rows x 256 columns; a group's last tile of at
// most 128 rows runs as a 128 x 256 tile.  Each XCD has a contiguous run of
// the tiles; what it leaves for a last round on at most half of its CUs runs as
// two 128 x 256 tiles each (9000 rows of three 2048 x 2048 matrices 54.6 -> 49.1 us).
//
// Long contractions are bound by the card's power: 16384 rows over eight
// 14336 x 4096 matrices 0.89 ms, 2.16 PFLOP/s at 1.7 GHz.  A tile also takes 6
// us beside its slices (1.9 us each with the chip full): finding its group,
// the first loads, the stores; 24594 rows over 64 matrices of 2048 x 1408, 11
// slices, 108 us, 1.3 PFLOP/s.
template <int FA, int FB>
__global__ __launch_bounds__(kBSThreads, 1) void grouped_pp_kernel(const uint8_t *__restrict__ A,
                                                                   const float *__restrict__ sA,
                                                                   const uint8_t *__restrict__ B,
                                                                   const float *__restrict__ sB,
                                                                   const int32_t *__restrict__ offsets, int groups,
                                                                   int rows, int N, int K, uint16_t *__restrict__ C, int cus)
{
    typedef PPShape<256> P;
    __shared__ __attribute__((aligned(1024))) uint8_t st0[P::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[P::kStage];
    __shared__ __attribute__((aligned(16))) float sx[kScaleGroups * 64 * pp_scale_runs<256, false>()];
    const int tiles_n = (N + 255) / 256, nk = K / kBK;
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
    const int at = 256 * tm + (half > 0 ? 128 : 0);
    const int64_t row0 = gt.row0 + at, n0 = 256 * tn;
    const int a_rows = min(half < 0 ? 256 : 128, gt.size - at), b_rows = min(256, N - (int)n0);
    if (a_rows <= 0) return;
    const PPOperand a{A + row0 * K, a_rows * K, K, sA + row0 * nk, a_rows * nk * 4, nk};
    const int b_blocks = b_rows / 128; // 1 in a last, half-empty tile column
    const PPOperand b{B + ((int64_t)gt.group * N + n0) * K, b_rows * K, K,
                      sB + ((int64_t)gt.group * (N / 128) + n0 / 128) * nk, b_blocks * nk * 4, nk};
    uint16_t *c = C + row0 * N + n0;
    if (a_rows > 128)
        pp_tile<FA, FB, 256, false>(st0, st1, sx, a, b, nk, b_blocks - 1, c, N, a_rows, b_rows);
    else
        pp_tile<FA, FB, 128, false>(st0, st1, sx, a, b, nk, b_blocks - 1, c, N, a_rows, b_rows);
}

// The groups' blocks of 128 tokens, 64 groups at a time in a wave's lanes.
struct GroupBlocks {
    const int32_t *offsets;
    int groups, rows;
    int count, sum; // blocks of group 64 i + lane and inclusive sums, for the chunk held

    __device__ __forceinline__ void hold(int g0)
    {
        int lo, size;
        group_rows(offsets, groups, rows, g0 + (threadIdx.x & 63), lo, size);
        count = (int)(((unsigned)size + 127) / 128);
        sum = wave_scan_i32(count);
    }
    // chunk 0 is read first: the loads run beside the search for the tile
    __device__ __forceinline__ GroupBlocks(const int32_t *o, int g, int r) : offsets(o), groups(g), rows(r) { hold(0); }

    // The group that comes i-th: those with more than the average first, so
    // that the launch does not end on the longest tiles (up to 64 groups).
    __device__ __forceinline__ int ordered(int i) const
    {
        if (groups > 64) return i;
        const int lane = threadIdx.x & 63, total = __builtin_amdgcn_readlane(sum, 63);
        const bool live = lane < groups, big = live && (int64_t)count * groups > total;
        const uint64_t bigs = __ballot(big), rest = __ballot(live && !big);
        const uint64_t mine = big ? bigs : rest;
        const int before = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mine >> 32),
                                                          __builtin_amdgcn_mbcnt_lo((uint32_t)mine, 0));
        const int rank = live ? before + (big ? 0 : __popcll(bigs)) : 64;
        return __ffsll((unsigned long long)__ballot(rank == i)) - 1;
    }
    // blocks before group e and in it (wave-uniform), clipped to the kbs that the operands hold
    __device__ __forceinline__ void find(int e, int kbs, int &kb0, int &kbn)
    {
        kb0 = 0;
        for (int g0 = 0;; g0 += 64) {
            if (g0 > 0) hold(g0);
            if (e < g0 + 64) break;
            kb0 += __builtin_amdgcn_readlane(sum, 63);
        }
        kbn = __builtin_amdgcn_readlane(count, e & 63);
        kb0 += __builtin_amdgcn_readlane(sum, e & 63) - kbn;
        kb0 = min(kb0, kbs);
        kbn = min(kbn, kbs - kb0);
    }
};

// Tile i of an XCD's share of the groups' tiles (`per` each): every group's
// tiles are split over the XCDs, so that they get equal shares of long and of
// short contractions; an XCD's share of a group is a contiguous run of its
// grouped order.  e: place of the group; tile >= per: none.
__device__ __forceinline__ void group_share(int xcd, int i, int per, int &e, int &tile)
{
    const int share = (per + kXcds - 1) / kXcds;
    e = (int)((unsigned)i / (unsigned)share);
    tile = xcd * share + (i - e * share);
}

// wgrad with bf16 results in 256 x 256 tiles of one group's C.  Every result
// takes a multiply and a multiply-add of scales per slice, which the wave that
// runs its products issues too: 1.9 us a slice against 0.9 of the matrix
// unit, and 7 us a tile for the rest.  24594 tokens, 64 gradients of 1408 x
// 2048: 180 us, 0.79 PFLOP/s (190 us with the groups in their own order); eight of 4096 x 4096 over 32768 tokens 560 us,
// 1.97 PFLOP/s.
template <int FA, int FB>
__global__ __launch_bounds__(kBSThreads, 1) void grouped_wgrad_pp_kernel(
    const uint8_t *__restrict__ A, const float *__restrict__ sA, const uint8_t *__restrict__ B,
    const float *__restrict__ sB, const int32_t *__restrict__ offsets, int groups, int rows, int M, int N,
    int64_t stride, void *__restrict__ C)
{
    constexpr int kTM = 256, kTN = 256;
    typedef PPShape<kTM> P;
    __shared__ __attribute__((aligned(1024))) uint8_t st0[P::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[P::kStage];
    __shared__ __attribute__((aligned(16))) float sx[kScaleGroups * 64 * pp_scale_runs<kTM, true>()];
    const int tiles_m = (M + kTM - 1) / kTM, tiles_n = (N + kTN - 1) / kTN, per = tiles_m * tiles_n;
    int e, tile, tm, tn, kb0, kbn;
    GroupBlocks blocks(offsets, groups, rows);
    group_share(blockIdx.x % kXcds, blockIdx.x / kXcds, per, e, tile);
    if (e >= groups || tile >= per) return;
    group_tile(tile, tiles_m, tiles_n, tm, tn);
    const int kbs = (int)(stride / 128);
    e = blocks.ordered(e);
    blocks.find(e, kbs, kb0, kbn);
    const int64_t m0 = (int64_t)tm * kTM, n0 = (int64_t)tn * kTN;
    const int a_rows = min(kTM, M - (int)m0), b_rows = min(kTN, N - (int)n0), pitch = (int)stride;
    const PPOperand a{A + m0 * stride + (int64_t)kb0 * 128, a_rows * pitch - kb0 * 128, pitch, sA + m0 * kbs + kb0,
                      (a_rows * kbs - kb0) * 4, kbs};
    const PPOperand b{B + n0 * stride + (int64_t)kb0 * 128, b_rows * pitch - kb0 * 128, pitch, sB + n0 * kbs + kb0,
                      (b_rows * kbs - kb0) * 4, kbs};
    uint16_t *c = (uint16_t *)C + ((int64_t)e * M + m0) * N + n0;
    pp_tile<FA, FB, kTM, true>(st0, st1, sx, a, b, kbn, 0, c, N, a_rows, b_rows);
}

// A wave's 64 x 64 tile, its codes read from LDS a slice at a time.  kRowB: B
// has a scale per row (wgrad), else one for all.  fp32 results (kWide): the codes are
// widened to bf16 (exact) and multiplied by the bf16 matrix instruction, whose
// sums are binary32.  The FP8 instruction adds the products of eight
// neighbouring bytes on about 15 bits under the largest of them (measured on
// the MI355X with one large and one small product at a time), which leaves an
// fp32 result 1.1e-5 off in the 2-norm where the widened one is 7e-8 off: below
// the rounding of a bf16 result, above that of an fp32 one.
template <int FA, int FB, bool kRowB, bool kWide> struct Wave64 {
    v16f acc[2][2];
    uint4 a[2][4], b[2][4]; // 32 rows x 128 K bytes each: chunks 4 fg .. 4 fg + 3 of row fr
    bf16x8 aw[kWide ? 2 : 1][8];
    float wi[2];
    int fr, fg;

    __device__ __forceinline__ explicit Wave64(int lane) : fr(lane & 31), fg(lane >> 5)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    }
    // step s of 16 K, widened
    template <int F> __device__ __forceinline__ static bf16x8 step(const uint4 (&v)[4], int s)
    {
        const uint4 c = v[s >> 1];
        return s & 1 ? widen8<F>((int)c.z, (int)c.w) : widen8<F>((int)c.x, (int)c.y);
    }
    __device__ __forceinline__ static v8i half(const uint4 (&v)[4], int s)
    {
        const uint4 lo = v[2 * s], hi = v[2 * s + 1];
        return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    }
    // all codes of a slice from the 64 rows at sa and at sb, so that the stage can be refilled
    __device__ __forceinline__ void read(const uint8_t *sa, const uint8_t *sb)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                a[i][c] = *reinterpret_cast<const uint4 *>(sa + swz(32 * i + fr, 4 * fg + c));
                b[i][c] = *reinterpret_cast<const uint4 *>(sb + swz(32 * i + fr, 4 * fg + c));
            }
        if constexpr (kWide) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int s = 0; s < 8; ++s) aw[i][s] = step<FA>(a[i], s);
        }
    }
    // A's scales: runs of 16 rows' 64 floats apart at ga (with B's one scale at gb)
    __device__ __forceinline__ void weights(const float *ga, const float *gb)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) wi[i] = ga[64 * (2 * i + (fr >> 4)) + (fr & 15)] * (kRowB ? 1.0f : gb[0]);
    }
    // the slice's products, weighted (B's scales per row in runs at gb)
    __device__ __forceinline__ void products(const float *gb)
    {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            v16f p[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) p[i][r] = 0.0f;
            if constexpr (kWide) {
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const bf16x8 bw = step<FB>(b[j], s);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        p[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bw, aw[i][s], p[i], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i) p[i] = mfma32x32x64<FB, FA>(half(b[j], s), half(a[i], s), p[i]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v4f sb{1.0f, 1.0f, 1.0f, 1.0f};
                if constexpr (kRowB)
                    sb = *reinterpret_cast<const v4f *>(gb + 64 * (2 * j + (q >> 1)) + 8 * (q & 1) + 4 * fg);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][j][4 * q + r] = __builtin_fmaf(p[i][4 * q + r], wi[i] * sb[r], acc[i][j][4 * q + r]);
            }
        }
    }
    // columns 8 q + 4 fg .. + 3 of row fr of the 32 x 32 tile (i, j)
    __device__ __forceinline__ v4f quad(int i, int j, int q) const
    {
        return v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    }
};

// What the wgrad kernels below read of a tile: kTile rows of A and of B from
// the first of the group's slices on, and their scales.
struct WgradTile {
    __amdgpu_buffer_rsrc_t a, b, sa, sb;
    int pitch, s_pitch, slices;
    int64_t row0, col0; // of C [groups * M][N]
};

// Block -> tile of kTile x kTile of a group's C; false: none.
template <int kTile>
__device__ __forceinline__ bool wgrad_tile(const uint8_t *A, const float *sA, const uint8_t *B, const float *sB,
                                           const int32_t *offsets, int groups, int rows, int M, int N, int64_t stride,
                                           WgradTile &t)
{
    const int tiles_m = M / kTile, tiles_n = N / kTile, per = tiles_m * tiles_n;
    int e, tile, tm, tn, kb0;
    GroupBlocks blocks(offsets, groups, rows);
    group_share(blockIdx.x % kXcds, blockIdx.x / kXcds, per, e, tile);
    if (e >= groups || tile >= per) return false;
    group_tile(tile, tiles_m, tiles_n, tm, tn);
    const int kbs = (int)(stride / 128), pitch = (int)stride;
    e = blocks.ordered(e);
    blocks.find(e, kbs, kb0, t.slices);
    const int64_t m0 = (int64_t)tm * kTile, n0 = (int64_t)tn * kTile;
    const int bytes = kTile * pitch - kb0 * 128, s_bytes = (kTile * kbs - kb0) * 4;
    t.a = __builtin_amdgcn_make_buffer_rsrc((void *)(A + m0 * stride + (int64_t)kb0 * 128), 0, bytes, kRawBufferWord3);
    t.b = __builtin_amdgcn_make_buffer_rsrc((void *)(B + n0 * stride + (int64_t)kb0 * 128), 0, bytes, kRawBufferWord3);
    t.sa = __builtin_amdgcn_make_buffer_rsrc((void *)(sA + m0 * kbs + kb0), 0, s_bytes, kRawBufferWord3);
    t.sb = __builtin_amdgcn_make_buffer_rsrc((void *)(sB + n0 * kbs + kb0), 0, s_bytes, kRawBufferWord3);
    t.pitch = pitch, t.s_pitch = kbs;
    t.row0 = (int64_t)e * M + m0, t.col0 = n0;
    return true;
}

// wgrad in 128 x 128 tiles, four waves of 64 x 64 per block, two blocks per
// CU: one block's stores and first loads run beside the other's products.  A
// wave reads its share of a slice from LDS into registers at once, so the
// stage is free for the slice after next while the products run.
//
// Eight 14336 x 4096 gradients over 8192 tokens, fp32: 1.15 ms, 0.84 PFLOP/s,
// 1.9 GB written, 2.08 million cycles at the 1.83 GHz that the card's power leaves.
// A library's bf16 product of as many operations, one 14336 x 4096 gradient over
// 8192 tokens, takes 0.75 ms at 1.97 GHz (1.48 million cycles), so power is a
// part of the distance; the rest is work beside the products.  Without the loads
// of the slices the kernel takes 15% less time, without the widening (two waves
// widen every code) 11%, without the scales 9%; a tile also has a fixed cost
// (finding the group, first loads, stores).  256 x 128 ping-pong tiles of one
// block per CU took 3% longer, with 30% more cycles at a higher clock.  Eight
// 4096 x 4096 over 1024 tokens, where the stores count: 113 us against 146.
template <int FA, int FB, int DC>
__global__ __launch_bounds__(256, 2) void grouped_wgrad_kernel(
    const uint8_t *__restrict__ A, const float *__restrict__ sA, const uint8_t *__restrict__ B,
    const float *__restrict__ sB, const int32_t *__restrict__ offsets, int groups, int rows, int M, int N,
    int64_t stride, void *__restrict__ C)
{
    constexpr int kTile = 128, kOp = kTile * kBK, kSx = 16 * 64;
    __shared__ __attribute__((aligned(1024))) uint8_t st0[2 * kOp];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[2 * kOp];
    __shared__ __attribute__((aligned(16))) float sx0[kSx];
    __shared__ __attribute__((aligned(16))) float sx1[kSx];
    WgradTile t;
    if (!wgrad_tile<kTile>(A, sA, B, sB, offsets, groups, rows, M, N, stride, t)) return;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w & 1, wn = w >> 1;
    const int voff = (lane >> 3) * t.pitch + (((lane & 7) ^ ((4 * w + (lane >> 4)) & 7)) << 4);
    const int svoff = ((lane & 15) * t.s_pitch + (lane >> 4)) * 4;
    // past the last slice the offset lies outside the buffer: nothing is read
    auto load = [&](uint8_t *st, int kb) {
        const int at = kb < t.slices ? kb * kBK : 1 << 30;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int row = 8 * (w + 4 * u), off = row * t.pitch + at;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t.a, (lds_void *)(st + row * kBK), 16, voff, off, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t.b, (lds_void *)(st + kOp + row * kBK), 16, voff, off, 0, 0);
        }
    };
    // scales of slices kb .. kb + 3, runs of 16 rows as [slice][row]
    auto load_scales = [&](float *sx, int kb) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int run = w + 4 * u, off = (16 * run * t.s_pitch + kb) * 4;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t.sa, (lds_void *)(sx + 64 * run), 4, svoff, off, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t.sb, (lds_void *)(sx + 64 * (8 + run)), 4, svoff, off, 0, 0);
        }
    };
    auto barrier = [&]() {
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    Wave64<FA, FB, true, DC == kF32> tile(lane);
    load_scales(sx0, 0);
    load(st0, 0);
    load(st1, 1);
    for (int kb = 0;; kb += 8) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (kb + u >= t.slices) goto done;
            uint8_t *st = u & 1 ? st1 : st0;
            const float *sg = (u & 4 ? sx1 : sx0) + 16 * (u & 3);
            // this slice's loads have landed; the next one's (and the scales) may be in flight
            if ((u & 3) == 1) __builtin_amdgcn_s_waitcnt(waitcnt_imm(12, 15));
            else __builtin_amdgcn_s_waitcnt(waitcnt_imm(8, 15));
            barrier();
            tile.read(st + wm * 64 * kBK, st + kOp + wn * 64 * kBK);
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
            barrier(); // every wave has read the stage
            if ((u & 3) == 0) load_scales(u & 4 ? sx0 : sx1, kb + u + 4);
            load(st, kb + u + 2);
            tile.weights(sg + 64 * 4 * wm, sg);
            tile.products(sg + 64 * (8 + 4 * wn));
        }
    }
done:
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    __syncthreads();
    // each wave stages its 64 x 64 results and stores whole row pieces
    typedef EpiStage<64, DC == kF32 ? 4 : 2, 64, 16384> ES;
    uint8_t *ep = (w < 2 ? st0 : st1) + (w & 1) * 16384;
    uint32_t m = 0;
    const Epi none{nullptr, kActNone, nullptr};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                ES::put(ep, 32 * i + tile.fr, 8 * j + 2 * q + tile.fg,
                        pack_out4<DC == kF32 ? kOutF32 : kOutBF16, false, false>(0, tile.quad(i, j, q), m, none, 0.0f));
    constexpr int kB = DC == kF32 ? 4 : 2;
    store_rows<ES, 64>(ep, (uint8_t *)C + ((t.row0 + wm * 64) * N + t.col0 + wn * 64) * kB, N * kB, 64 * kB, 64, lane);
}

// wgrad of few tiles: a 64 x 64 tile of one group's C per block, whose four
// waves take a quarter of the group's slices each, from stages of their own
// (no barrier until the end), and add their sums through LDS in a fixed order.
template <int FA, int FB, int DC>
__global__ __launch_bounds__(256, 1) void grouped_wgrad_split_kernel(
    const uint8_t *__restrict__ A, const float *__restrict__ sA, const uint8_t *__restrict__ B,
    const float *__restrict__ sB, const int32_t *__restrict__ offsets, int groups, int rows, int M, int N,
    int64_t stride, void *__restrict__ C)
{
    constexpr int kTile = 64, kOp = kTile * kBK, kSx = 8 * 64;
    __shared__ __attribute__((aligned(1024))) uint8_t st0s[4][2 * kOp];
    __shared__ __attribute__((aligned(1024))) uint8_t st1s[4][2 * kOp];
    __shared__ __attribute__((aligned(16))) float sx0s[4][kSx];
    __shared__ __attribute__((aligned(16))) float sx1s[4][kSx];
    WgradTile t;
    if (!wgrad_tile<kTile>(A, sA, B, sB, offsets, groups, rows, M, N, stride, t)) return;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int each = (t.slices + 3) / 4, k0 = w * each, kn = min(each, t.slices - k0);
    uint8_t *st0 = st0s[w], *st1 = st1s[w];
    float *sx0 = sx0s[w], *sx1 = sx1s[w];
    int voff[2]; // rows 8 u + lane / 8, u even and odd
#pragma unroll
    for (int u = 0; u < 2; ++u)
        voff[u] = (lane >> 3) * t.pitch + (((lane & 7) ^ ((4 * u + (lane >> 4)) & 7)) << 4);
    const int svoff = ((lane & 15) * t.s_pitch + (lane >> 4)) * 4;
    auto load = [&](uint8_t *st, int k) {
        const int at = k < kn ? (k0 + k) * kBK : 1 << 30;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int row = 8 * u, off = row * t.pitch + at;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t.a, (lds_void *)(st + row * kBK), 16, voff[u & 1], off, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t.b, (lds_void *)(st + kOp + row * kBK), 16, voff[u & 1], off, 0, 0);
        }
    };
    auto load_scales = [&](float *sx, int k) {
#pragma unroll
        for (int run = 0; run < 4; ++run) {
            const int off = (16 * run * t.s_pitch + k0 + k) * 4;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t.sa, (lds_void *)(sx + 64 * run), 4, svoff, off, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t.sb, (lds_void *)(sx + 64 * (4 + run)), 4, svoff, off, 0, 0);
        }
    };
    Wave64<FA, FB, true, DC == kF32> tile(lane);
    load_scales(sx0, 0);
    load(st0, 0);
    load(st1, 1);
    for (int kb = 0;; kb += 8) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (kb + u >= kn) goto done;
            uint8_t *st = u & 1 ? st1 : st0;
            const float *sg = (u & 4 ? sx1 : sx0) + 16 * (u & 3);
            if ((u & 3) == 1) __builtin_amdgcn_s_waitcnt(waitcnt_imm(24, 15));
            else __builtin_amdgcn_s_waitcnt(waitcnt_imm(16, 15));
            asm volatile("" ::: "memory");
            tile.read(st, st + kOp);
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
            asm volatile("" ::: "memory");
            if ((u & 3) == 0) load_scales(u & 4 ? sx0 : sx1, kb + u + 4);
            load(st, kb + u + 2);
            tile.weights(sg, sg);
            tile.products(sg + 64 * 4);
        }
    }
done:
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    // wave w adds and stores the 32 x 32 tile (w / 2, w % 2)
    v4f(*sums)[64] = reinterpret_cast<v4f(*)[64]>(st0);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) sums[(2 * i + j) * 4 + q][lane] = tile.quad(i, j, q);
    __syncthreads();
    typedef EpiStage<32, DC == kF32 ? 4 : 2, 32, 4096> ES;
    uint32_t m = 0;
    const Epi none{nullptr, kActNone, nullptr};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v4f c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 4; ++k) c += reinterpret_cast<const v4f(*)[64]>(st0s[k])[4 * w + q][lane];
        ES::put(st1, tile.fr, 2 * q + tile.fg,
                pack_out4<DC == kF32 ? kOutF32 : kOutBF16, false, false>(0, c, m, none, 0.0f));
    }
    constexpr int kB = DC == kF32 ? 4 : 2;
    store_rows<ES, 32>(st1, (uint8_t *)C + ((t.row0 + 32 * (w >> 1)) * N + t.col0 + 32 * (w & 1)) * kB, N * kB, 32 * kB,
                       32, lane);
}

// fprop / dgrad of few tiles: a 128 x 128 tile per block, whose two sets of four
// waves (64 x 64 each) take half of the slices each, from stages of their own,
// and add their sums through LDS: each set finishes half of the columns.  A
// set's chain of loads, products and scales bounds it, 1.1 us a slice: 320 rows
// over four 4096 x 4096 matrices 22 us.
template <int FA, int FB>
__global__ __launch_bounds__(512, 2) void grouped_halves_kernel(const uint8_t *__restrict__ A,
                                                                const float *__restrict__ sA,
                                                                const uint8_t *__restrict__ B,
                                                                const float *__restrict__ sB,
                                                                const int32_t *__restrict__ offsets, int groups,
                                                                int rows, int N, int K, uint16_t *__restrict__ C)
{
    constexpr int kTile = 128, kOp = kTile * kBK, kSx = 9 * 64; // eight runs of A's scales and B's
    __shared__ __attribute__((aligned(1024))) uint8_t st0s[2][2 * kOp];
    __shared__ __attribute__((aligned(1024))) uint8_t st1s[2][2 * kOp];
    __shared__ __attribute__((aligned(16))) float sx0s[2][kSx];
    __shared__ __attribute__((aligned(16))) float sx1s[2][kSx];
    GroupTiles<kTile> tiles(offsets, groups, rows);
    const int tiles_n = N / kTile, nk = K / kBK;
    const int n = tiles.total * tiles_n, per = (n + kXcds - 1) / kXcds;
    const int i = blockIdx.x / kXcds, t = (int)(blockIdx.x % kXcds) * per + i;
    if (i >= per || t >= n) return;
    const GroupTile gt = tiles.find(t / tiles_n);
    int tm, tn;
    group_tile(gt.tile * tiles_n + t % tiles_n, (gt.size + kTile - 1) / kTile, tiles_n, tm, tn);
    const int64_t row0 = gt.row0 + kTile * tm, n0 = kTile * tn;
    const int a_rows = min(kTile, gt.size - kTile * tm);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);
    const int h = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8), wm = w & 1, wn = w >> 1;
    // both sets run `each` slices; the second one's last may be past the end: zeros
    // for its codes and for its scales
    const int each = (nk + 1) / 2, k0 = h * each, kn = min(each, nk - k0);
    const __amdgpu_buffer_rsrc_t ra =
        __builtin_amdgcn_make_buffer_rsrc((void *)(A + row0 * K), 0, a_rows * K, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(B + ((int64_t)gt.group * N + n0) * K), 0, kTile * K, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t rsa =
        __builtin_amdgcn_make_buffer_rsrc((void *)(sA + row0 * nk), 0, a_rows * nk * 4, kRawBufferWord3);
    const __amdgpu_buffer_rsrc_t rsb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sB + ((int64_t)gt.group * (N / kTile) + tn) * nk), 0, nk * 4, kRawBufferWord3);
    const int voff = (lane >> 3) * K + (((lane & 7) ^ ((4 * w + (lane >> 4)) & 7)) << 4);
    const int svoff = ((lane & 15) * nk + (lane >> 4)) * 4;
    uint8_t *st0 = st0s[h], *st1 = st1s[h];
    float *sx0 = sx0s[h], *sx1 = sx1s[h];
    auto load = [&](uint8_t *st, int k) {
        const int at = k < kn ? (k0 + k) * kBK : 1 << 30;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int row = 8 * (w + 4 * u), off = row * K + at;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(st + row * kBK), 16, voff, off, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void *)(st + kOp + row * kBK), 16, voff, off, 0, 0);
        }
    };
    // Scales of slices k .. k + 3, runs of 16 rows as [slice][row]; every wave loads
    // B's.  A lane whose slice is past a row's last reads a zero: the next row's
    // first scale may be infinite or NaN, which the slice's zeros would not cancel.
    auto load_scales = [&](float *sx, int k) {
        const int at = (k0 + k) * 4;
        const int sav = k0 + k + (lane >> 4) < nk ? svoff : kTile * nk * 4; // the latter outside the buffer
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int run = w + 4 * u;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsa, (lds_void *)(sx + 64 * run), 4, sav, 16 * run * nk * 4 + at, 0,
                                                     0);
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (lds_void *)(sx + 64 * 8), 4, (lane >> 4) * 4, at, 0, 0);
    };
    auto barrier = [&]() {
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    Wave64<FA, FB, false, false> tile(lane);
    float wq[4][2];
    load_scales(sx0, 0);
    load(st0, 0);
    load(st1, 1);
    for (int kb = 0;; kb += 8) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (kb + u >= each) goto done;
            uint8_t *st = u & 1 ? st1 : st0;
            const float *sg = u & 4 ? sx1 : sx0;
            if ((u & 3) == 1) __builtin_amdgcn_s_waitcnt(waitcnt_imm(11, 15));
            else __builtin_amdgcn_s_waitcnt(waitcnt_imm(8, 15));
            barrier();
            tile.read(st + wm * 64 * kBK, st + kOp + wn * 64 * kBK);
            // four slices' scales at once: the compiler waits for every load in
            // flight before it reads them
            if ((u & 3) == 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    tile.weights(sg + 16 * k + 64 * 4 * wm, sg + 16 * k + 64 * 8);
                    wq[k][0] = tile.wi[0], wq[k][1] = tile.wi[1];
                }
            }
            tile.wi[0] = wq[u & 3][0], tile.wi[1] = wq[u & 3][1];
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
            barrier(); // every wave has read the stage
            if ((u & 3) == 0) load_scales(u & 4 ? sx0 : sx1, kb + u + 4);
            load(st, kb + u + 2);
            tile.products(nullptr);
        }
    }
done:
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    __syncthreads();
    // the other set's columns go to it, 32 of the wave's 64
    v4f(*mine)[64] = reinterpret_cast<v4f(*)[64]>(st0 + w * 8192);
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (j != h) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) mine[4 * i + q][lane] = tile.quad(i, j, q);
        }
    __syncthreads();
    const v4f(*other)[64] = reinterpret_cast<const v4f(*)[64]>(st0s[1 - h] + w * 8192);
    typedef EpiStage<32, 2, 64, 4096> ES;
    uint8_t *ep = st1 + w * 4096;
    uint32_t m = 0;
    const Epi none{nullptr, kActNone, nullptr};
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (j == h) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    ES::put(ep, 32 * i + tile.fr, 2 * q + tile.fg,
                            pack_out4<kOutBF16, false, false>(0, tile.quad(i, j, q) + other[4 * i + q][lane], m, none,
                                                              0.0f));
        }
    if (64 * wm < a_rows)
        store_rows<ES, 64>(ep, C + (row0 + 64 * wm) * N + n0 + 64 * wn + 32 * h, N * 2, 64, a_rows - 64 * wm, lane);
}

// The tile of an fprop / dgrad launch.  Up to 12 rows a group on average most
// groups fit a 16-row tile, so the weights are read once, and 32 columns a block are
// faster than 16 unless the blocks then do not fill the chip (8 rows over
// eight 14336 x 4096 matrices: 53.6 and 59.1 us; 64 columns 56.8 us).  Up to 18
// rows the weights still count most and 32 x 64 tiles read them faster than the
// large ones, if they fill the chip (14 rows a group: eight 14336 x 4096 93 and
// 102 us, 20 of 4096 x 2048 36 and 45, 64 of 2048 x 1408 39.6 and 40.6; 20 rows
// 107 and 102, 39 and 45, 43 and 41).  Above,
// a launch takes about `step` per round of one block per CU, `least` at the
// least: both measured at K = 4096, one 4096-column matrix with 16 to 1024
// rows, in us.  The steps grow slower than the tiles' areas, so the large
// ping-pong tiles win as soon as they fill a part of the chip: 256 rows over
// those eight matrices 109 us against 132 us in 32 x 64 tiles, but 40 rows of
// one 4096 x 4096 matrix 11.7 us in 32 x 32 tiles against 29 us, and in between
// 320 rows over four 22 us in 128 x 128 tiles against 30 in the large ones.
//
// Tiles whose launch would pass max_blocks (16 x 32 ones of 65536 groups of one
// row each and 8320 columns) leave the choice to larger ones; the largest fit
// (grouped_gemm_fits).
enum RowsTile { kRows16x16, kRows16x32, kRows32x32, kRows32x64, kRowsHalves, kRowsPP };

// Waves that share a 16 x 32 tile's slices, one to four slices a wave: 64 rows
// over eight 8192-column matrices in us with 4, 8 and 16 waves: K 1024 13.6,
// 15.8, 18.9; 3456 44.5, 43.3, 47.0; 4096 54.4, 53.8, 52.3; 7168 88.1, 87.8, 86.6.
inline int rows_waves(int64_t K) { return K < 2048 ? 4 : K < 4096 ? 8 : 16; }

inline RowsTile rows_tile(const GroupedArgs &a)
{
    const int64_t cus = a.cus > 0 ? a.cus : 256;
    auto blocks = [&](int tm, int tn) { return max_tiles(a.rows, a.groups, tm) * ((a.N + tn - 1) / tn); };
    const int64_t live = a.rows < a.groups ? a.rows : a.groups;
    const struct {
        int tm, tn, lanes;
        double least, step;
    } cost[6] = {{16, 16, 512, 8.7, 5.0},    {16, 32, 64 * rows_waves(a.K), 8.8, 7.2}, {32, 32, 512, 11.5, 10.5},
                 {32, 64, 256, 15.4, 14.5}, {128, 128, 512, 21.0, 21.0},              {256, 256, 512, 40.0, 40.0}};
    auto fits = [&](int i) { return blocks(cost[i].tm, cost[i].tn) + kXcds <= max_blocks(cost[i].lanes); };
    if (a.rows <= 12 * live && fits(kRows16x32)) return blocks(16, 32) >= cus ? kRows16x32 : kRows16x16;
    if (a.rows <= 18 * live && blocks(32, 64) >= cus && fits(kRows32x64)) return kRows32x64;
    RowsTile best = kRowsPP;
    double least = 0.0;
    for (int i = kRowsPP; i >= kRows16x16; --i) {
        if (i != kRowsPP && !fits(i)) continue;
        const int64_t rounds = (blocks(cost[i].tm, cost[i].tn) + cus - 1) / cus;
        double us = cost[i].step * (double)rounds;
        if (i == kRowsPP && a.rows <= 128 * live) us *= 29.0 / 40.0; // mostly 128 x 256 tiles
        if (us < cost[i].least) us = cost[i].least;
        if (i == kRowsPP || us < least) best = (RowsTile)i, least = us;
    }
    return best;
}

// Blocks of a launch of the large tiles on XCDs of `cus` units: with the halves
// of what is left for a last round.
inline int64_t pp_blocks(int64_t rows, int groups, int64_t N, int cus)
{
    return max_tiles(rows, groups, 256) * ((N + 255) / 256) + kXcds * (1 + cus / 2);
}

template <int FA, int FB> hipError_t launch_grouped_rows(const GroupedArgs &a)
{
#define FP8Q_ROWS(MT, NT, WK)                                                                                        \
    grouped_rows_kernel<FA, FB, MT, NT, WK>                                                                          \
        <<<(unsigned)(max_tiles(a.rows, a.groups, 16 * MT) * (a.N / (16 * NT))), 64 * WK, 0, a.stream>>>(            \
            a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows, (int)a.N, (int)a.K, (uint16_t *)a.C)
    switch (rows_tile(a)) {
    case kRows16x16: FP8Q_ROWS(1, 1, 8); break;
    case kRows16x32:
        switch (rows_waves(a.K)) {
        case 4: FP8Q_ROWS(1, 2, 4); break;
        case 8: FP8Q_ROWS(1, 2, 8); break;
        default: FP8Q_ROWS(1, 2, 16);
        }
        break;
    case kRows32x32: FP8Q_ROWS(2, 2, 8); break;
    case kRows32x64: FP8Q_ROWS(2, 4, 4); break;
    case kRowsHalves: {
        const int64_t tiles = max_tiles(a.rows, a.groups, 128) * (a.N / 128);
        grouped_halves_kernel<FA, FB><<<(unsigned)(tiles + kXcds), 512, 0, a.stream>>>(
            a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows, (int)a.N, (int)a.K, (uint16_t *)a.C);
        break;
    }
    default: {
        const int cus = a.cus / kXcds > 1 ? a.cus / kXcds : 1; // of an XCD
        grouped_pp_kernel<FA, FB><<<(unsigned)pp_blocks(a.rows, a.groups, a.N, cus), kBSThreads, 0, a.stream>>>(
            a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows, (int)a.N, (int)a.K, (uint16_t *)a.C, cus);
    }
    }
#undef FP8Q_ROWS
    return hipGetLastError();
}

// The tiles of a wgrad launch, from the time of a round of blocks in us with s
// slices of 128 tokens per group on average.  Measured on one to sixteen
// gradients of 768 x 1152 to 4096 x 4096 with 1 to 128 slices: 256 x 256 (bf16
// only) 7.5 + 1.9 s per tile and CU, 128 x 128 5 + 1.3 s per two tiles and CU
// (0.8 s where there is one; fp32 2.0 and 1.1), split 64 x 64 5 + 0.25 s per
// tile and CU (fp32 0.31).  The large tiles reuse most of what they read, the
// small ones fill the chip where there are few: one 768 x 1152 gradient over
// 16384 tokens 184, 93 and 36 us (bf16), eight 4096 x 4096 over 32768 548 and
// 711 us in the large and the small ones.
enum WgradTiles { kWgradSplit, kWgradSmall, kWgradLarge };

inline WgradTiles wgrad_tiles(const GroupedArgs &a)
{
    const int64_t cus = a.cus > 0 ? a.cus : 256;
    auto tiles = [&](int tile) { return a.groups * ((a.M + tile - 1) / tile) * ((a.N + tile - 1) / tile); };
    auto up = [](int64_t n, int64_t d) { return (double)((n + d - 1) / d); };
    const double s = (double)a.rows / 128.0 / a.groups;
    const bool bf16 = a.c_dtype == kBF16;
    const int64_t small = tiles(128), last = small % (2 * cus);
    const double two = 5.0 + (bf16 ? 1.3 : 2.0) * s, one = 5.0 + (bf16 ? 0.8 : 1.1) * s;
    const double us_small = (double)(small / (2 * cus)) * two + (last == 0 ? 0.0 : last <= cus ? one : two);
    const double us_split = up(tiles(64), cus) * (5.0 + (bf16 ? 0.25 : 0.31) * s);
    const double us_large = up(tiles(256), cus) * (7.5 + 1.9 * s);
    if (us_split < us_small && !(bf16 && us_large < us_split)) return kWgradSplit;
    return bf16 && us_large <= us_small ? kWgradLarge : kWgradSmall;
}

// Blocks of a wgrad launch: the groups' tiles in equal shares of the XCDs.
inline int64_t wgrad_blocks(int groups, int64_t M, int64_t N, int tile)
{
    const int64_t per = ((M + tile - 1) / tile) * ((N + tile - 1) / tile);
    return groups * (int64_t)kXcds * ((per + kXcds - 1) / kXcds);
}

template <int FA, int FB> hipError_t launch_grouped_wgrad(const GroupedArgs &a)
{
    auto grid = [&](int tile) { return (unsigned)wgrad_blocks(a.groups, a.M, a.N, tile); };
    const bool bf16 = a.c_dtype == kBF16;
#define FP8Q_WGRAD(TILE, THREADS, K)                                                                                 \
    K<<<grid(TILE), THREADS, 0, a.stream>>>(a.A, a.sA, a.B, a.sB, a.offsets, a.groups, a.rows, (int)a.M, (int)a.N,  \
                                            a.stride, a.C)
    switch (wgrad_tiles(a)) {
    case kWgradLarge: FP8Q_WGRAD(256, kBSThreads, (grouped_wgrad_pp_kernel<FA, FB>)); break;
    case kWgradSmall:
        if (bf16) FP8Q_WGRAD(128, 256, (grouped_wgrad_kernel<FA, FB, kBF16>));
        else FP8Q_WGRAD(128, 256, (grouped_wgrad_kernel<FA, FB, kF32>));
        break;
    case kWgradSplit:
        if (bf16) FP8Q_WGRAD(64, 256, (grouped_wgrad_split_kernel<FA, FB, kBF16>));
        else FP8Q_WGRAD(64, 256, (grouped_wgrad_split_kernel<FA, FB, kF32>));
        break;
    }
#undef FP8Q_WGRAD
    return hipGetLastError();
}

// One operand-format pair's launchers (one translation unit each).
#define FP8Q_GROUPED_PAIR(NAME, FA, FB)                                                                              \
    hipError_t launch_grouped_rows_##NAME(const GroupedArgs &a) { return launch_grouped_rows<FA, FB>(a); }           \
    hipError_t launch_grouped_wgrad_##NAME(const GroupedArgs &a) { return launch_grouped_wgrad<FA, FB>(a); }

} // namespace fp8q

#endif // FP8Q_GROUPED_GEMM_H
