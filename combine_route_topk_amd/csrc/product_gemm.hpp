// product_gemm.hpp -- the MFMA core of the experts' products and of their
// gradients: one 256 x 256 tile of C = A B^T, summed over K in float32.
//
// Bound. At 256 x 256 x 64 a K-tile moves 64 KiB into LDS for 8.4 MFLOP, so
// the matrix units bound it as long as they are never left waiting: 8 waves,
// two on each SIMD, compute 128 x 64 each in 16 x 16 x 32 MFMAs (128
// accumulator registers).
//
// Schedule. A wave's K-tile is four phases of 16 MFMAs, one for each pair of
// halves of A's rows and B's columns. Waves 0-3 and waves 4-7 run half a
// phase apart, held so by barriers: while one of a SIMD's two waves issues
// MFMAs the other reads the fragments of its next phase from LDS and starts
// the loads of later K-tiles, so the matrix unit always has a wave that is
// ready. Operands go from memory straight to LDS in half tiles of 16 KiB, one
// per phase, into two stages (128 KiB); each half tile is started as soon as
// every wave has read the one it replaces, six phases before it is read, so
// a wait never drains the queue: five half tiles stay in flight across it.
//
// Operands. K-contiguous (rows of x, grad_y and a forward W): LDS holds 128
// rows of 64 k, and a fragment is one 16-byte read per lane. K-strided (W in
// the input gradient; both operands of the weight gradient): LDS holds 64
// k-rows of 128 columns, and a fragment is two transposing reads. In both the
// 16-byte pieces of a row are permuted by the row's number so that the lanes
// of a read fall into different banks. Buffer descriptors end where the
// operand ends, and reads past that end give zeros: rows past an expert's
// last, columns past the width and the tail of K cost no branch.
#pragma once

#include "product_device.hpp"

namespace moe {
namespace {

constexpr int kGemmThreads = 512;
constexpr int kTile = 256, kTileK = 64;
constexpr int kHalfBytes = 128 * kTileK * 2;   // half an operand's tile
constexpr int kStageBytes = 4 * kHalfBytes;    // A half 0, A half 1, B half 0, B half 1
constexpr int kGemmLdsBytes = 2 * kStageBytes;
constexpr int kGemmBufferFlags = 0x00020000;   // raw byte-addressed buffer
constexpr uint32_t kOutside = 0x80000000u;     // an offset past every descriptor's end

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// One operand of a tile: 256 rows (of A) or columns (of B), by K.
template <bool STRIDED>
struct Operand {
    const uint8_t *base;  // first row's (column's) element of K = 0
    int64_t bytes;        // from base to the operand's end (STRIDED)
    int64_t kstep;        // bytes from one K-tile to the next (STRIDED)
    uint32_t records;     // descriptor size (K-contiguous)
    uint32_t off[2][2];   // this lane's byte offset in load i of half h
    uint32_t tail;        // kOutside where this lane's piece lies past K in the last K-tile

    // K-contiguous: `rows` valid rows of K elements from p. half_rows: rows
    // between the halves; row_of: first of the eight rows of load j of a half.
    template <class RowOf>
    __device__ __forceinline__ void init(const uint16_t *p, int64_t rows, int32_t K, int wave, int lane,
                                         int half_rows, RowOf row_of)
    {
        static_assert(!STRIDED, "");
        base = reinterpret_cast<const uint8_t *>(p);
        records = (uint32_t)(max(min(rows, (int64_t)kTile), (int64_t)0) * K * 2);
        const int c = (lane & 7) ^ (lane >> 3);  // piece at LDS position lane % 8 of row lane / 8
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                off[h][i] = (uint32_t)(h * half_rows + row_of(i * 8 + wave) + (lane >> 3)) * (uint32_t)K * 2u + c * 16;
        tail = (K & (kTileK - 1)) && c * 8 >= (K & (kTileK - 1)) ? kOutside : 0u;
    }

    // K-strided: element (k, n) at p[k * ld + n], K rows, n < width.
    __device__ __forceinline__ void init_strided(const uint16_t *p, int64_t K, int32_t ld, int32_t width, int wave,
                                                 int lane)
    {
        base = reinterpret_cast<const uint8_t *>(p);
        // the last row ends at its valid width: rows K and later lie past it
        bytes = K > 0 ? ((K - 1) * ld + width) * 2 : 0;
        kstep = (int64_t)kTileK * ld * 2;
        const int kr = lane >> 4, swz = (kr & 3) | (((wave >> 1) & 1) << 2);
        const int c = (lane & 15) ^ (2 * swz);  // piece at LDS position lane % 16
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = h * 128 + c * 8;  // column of piece c
#pragma unroll
            for (int i = 0; i < 2; ++i)
                off[h][i] = n >= width ? kOutside : (uint32_t)((i * 8 + wave) * 4 + kr) * (uint32_t)ld * 2u + n * 2;
        }
        tail = 0;
    }

    // start the loads of half h of K-tile t (of nk) into LDS at dst
    __device__ __forceinline__ void load(uint8_t *__restrict__ dst, int h, int t, int nk, int wave) const
    {
        if (STRIDED) {
            const int64_t at = (int64_t)t * kstep;
            const int64_t left = t < nk ? bytes - at : 0;
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint8_t *>(base + at), 0, (uint32_t)min(max(left, (int64_t)0), (int64_t)0x7FFFFFFF),
                kGemmBufferFlags);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst + (i * 8 + wave) * 1024, 16, off[h][i], 0, 0, 0);
        } else {
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint8_t *>(base), 0, t < nk ? records : 0u, kGemmBufferFlags);
            const uint32_t cut = t == nk - 1 ? tail : 0u;
            // the descriptor's end is checked less the scalar offset, which must not pass it
            const uint32_t k0 = t < nk ? t * (kTileK * 2) : 0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst + (i * 8 + wave) * 1024, 16, off[h][i] | cut,
                                                         k0, 0, 0);
        }
    }
};

// Fragment reads. They are written as instructions, because the compiler takes
// every LDS read to depend on every load into LDS in flight and would drain
// the queue before each; the schedule orders them with barriers and counted
// waits instead. A block holds a slot's reads, the wait for the loads that the
// next phase reads, the barrier that ends the slot, and the wait for the
// reads themselves, whose latency so passes under the barrier. LDS
// addresses are byte offsets in 32 bits.
__device__ __forceinline__ uint32_t lds_offset(const uint8_t *p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)p;
}

// Lane L's address within a half tile of its part of fragment f (rows or
// columns first + 16 f), for k = kk * 32 + (L / 16) * 8 .. + 7.
__device__ __forceinline__ uint32_t frag_row(int first, int kk, int lane)
{
    const int i = lane & 15, g = lane >> 4;
    return (uint32_t)((first + i) * 128 + (((kk * 4 + g) ^ (i & 7)) << 4));
}
__device__ __forceinline__ uint32_t frag_strided(int first, int f, int lane)
{
    const int i = lane & 15, g = lane >> 4, swz = (i >> 2) | ((g & 1) << 2);
    return (uint32_t)((g * 8 + (i >> 2)) * 256 + (((first / 16 + f) ^ swz) << 5) + (i & 3) * 8);
}

__device__ __forceinline__ bf16x8 join(s16x4 lo, s16x4 hi)
{
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// A: four fragments of 16 rows, B: two of 16 columns, both halves of a K-tile
struct FragA {
    bf16x8 v[2][4];
};
struct FragB {
    bf16x8 v[2][2];
};

// The half tile's offset within its stage is part of the instruction, so that
// one address register serves a stage's four.
#define MOE_READ(d, a, o) "ds_read_b128 %" #d ", %" #a " offset:%[half]+" #o "\n\t"
#define MOE_READ_TR(d, a, o) "ds_read_b64_tr_b16 %" #d ", %" #a " offset:%[half]+" #o "\n\t"
// destination numbers d.., address numbers a..
#define MOE_READ_A(d0, d1, d2, d3, d4, d5, d6, d7, a0, a1)                                              \
    MOE_READ(d0, a0, 0) MOE_READ(d1, a0, 2048) MOE_READ(d2, a0, 4096) MOE_READ(d3, a0, 6144)            \
    MOE_READ(d4, a1, 0) MOE_READ(d5, a1, 2048) MOE_READ(d6, a1, 4096) MOE_READ(d7, a1, 6144)
#define MOE_READ_B(d0, d1, d2, d3, a0, a1) \
    MOE_READ(d0, a0, 0) MOE_READ(d1, a0, 2048) MOE_READ(d2, a1, 0) MOE_READ(d3, a1, 2048)
#define MOE_READ_TR4(d0, d1, d2, d3, a) \
    MOE_READ_TR(d0, a, 0) MOE_READ_TR(d1, a, 1024) MOE_READ_TR(d2, a, 8192) MOE_READ_TR(d3, a, 9216)
#define MOE_SLOT_END "s_waitcnt vmcnt(10)\n\ts_barrier\n\ts_waitcnt lgkmcnt(0)"
#define MOE_OUT_A(r)                                                                                    \
    "=&v"(r.v[0][0]), "=&v"(r.v[0][1]), "=&v"(r.v[0][2]), "=&v"(r.v[0][3]), "=&v"(r.v[1][0]),           \
        "=&v"(r.v[1][1]), "=&v"(r.v[1][2]), "=&v"(r.v[1][3])
#define MOE_OUT_B(r) "=&v"(r.v[0][0]), "=&v"(r.v[0][1]), "=&v"(r.v[1][0]), "=&v"(r.v[1][1])
#define MOE_OUT_TR4(q) "=&v"(q[0]), "=&v"(q[1]), "=&v"(q[2]), "=&v"(q[3])

// the four transposing reads of one fragment: k 0-3, 4-7 of this lane's first
// eight, then of the eight 32 further
typedef s16x4 TrFrag[4];
template <int N, class F>
__device__ __forceinline__ void from_tr(const TrFrag (&q)[N], F &r)
{
#pragma unroll
    for (int f = 0; f < N; ++f) {
        r.v[0][f] = join(q[f][0], q[f][1]);
        r.v[1][f] = join(q[f][2], q[f][3]);
    }
}

template <bool STRIDED, int N>
struct FragAddr {
    uint32_t a[STRIDED ? N : 2];
    __device__ __forceinline__ void init(int first, int lane)
    {
#pragma unroll
        for (int f = 0; f < (STRIDED ? N : 2); ++f)
            a[f] = STRIDED ? frag_strided(first, f, lane) : frag_row(first, f, lane);
    }
};

// The slot that reads a half of B, and the one that reads a half of A.
template <int HALF, bool STRIDED>
__device__ __forceinline__ void slot_b(const FragAddr<STRIDED, 2> &fb, uint32_t stage, FragB &b)
{
    if constexpr (STRIDED) {
        TrFrag q[2];
        asm volatile(MOE_READ_TR4(0, 1, 2, 3, 8) MOE_READ_TR4(4, 5, 6, 7, 9) MOE_SLOT_END
                     : MOE_OUT_TR4(q[0]), MOE_OUT_TR4(q[1])
                     : "v"(stage + fb.a[0]), "v"(stage + fb.a[1]), [half] "n"(HALF * kHalfBytes)
                     : "memory");
        from_tr(q, b);
    } else {
        asm volatile(MOE_READ_B(0, 1, 2, 3, 4, 5) MOE_SLOT_END
                     : MOE_OUT_B(b)
                     : "v"(stage + fb.a[0]), "v"(stage + fb.a[1]), [half] "n"(HALF * kHalfBytes)
                     : "memory");
    }
}
template <int HALF, bool STRIDED>
__device__ __forceinline__ void slot_a(const FragAddr<STRIDED, 4> &fa, uint32_t stage, FragA &a)
{
    if constexpr (STRIDED) {
        TrFrag q[4];
        asm volatile(MOE_READ_TR4(0, 1, 2, 3, 16) MOE_READ_TR4(4, 5, 6, 7, 17) MOE_READ_TR4(8, 9, 10, 11, 18)
                         MOE_READ_TR4(12, 13, 14, 15, 19) MOE_SLOT_END
                     : MOE_OUT_TR4(q[0]), MOE_OUT_TR4(q[1]), MOE_OUT_TR4(q[2]), MOE_OUT_TR4(q[3])
                     : "v"(stage + fa.a[0]), "v"(stage + fa.a[1]), "v"(stage + fa.a[2]), "v"(stage + fa.a[3]),
                       [half] "n"(HALF * kHalfBytes)
                     : "memory");
        from_tr(q, a);
    } else {
        asm volatile(MOE_READ_A(0, 1, 2, 3, 4, 5, 6, 7, 8, 9) MOE_SLOT_END
                     : MOE_OUT_A(a)
                     : "v"(stage + fa.a[0]), "v"(stage + fa.a[1]), [half] "n"(HALF * kHalfBytes)
                     : "memory");
    }
}

// wait until at most N of this wave's vector-memory operations are outstanding
template <int N>
__device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

__device__ __forceinline__ void slot_end()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

// acc[hA][hB][fa][fb]: lane L holds row hA * 128 + wm * 64 + fa * 16 + L % 16
// and four columns, which lie in LDS as rows (K-strided: columns) wn * 32 +
// fb * 16 + (L / 16) * 4 + 0..3 of B's half tile hB. K-contiguous, that half
// holds columns [hB * 32, hB * 32 + 32) of each 64 of the tile (gated: 16 gate
// and 16 up columns [hB * 16, hB * 16 + 16) of each 32), so that a wave's
// columns are consecutive: rows of 128 bytes to write, which took 1.63 ms
// against 1.80 for halves of 128 columns (327680 x 2048 by 2 x 768, gated).
// K-strided, it holds columns [hB * 128, hB * 128 + 128): splitting its
// 256-byte pieces into 64 bytes took 608 against 573 us (32768 x 4096 by
// 2048).
typedef f32x4 Acc[2][2][4][2];

template <bool ASTR, bool BSTR>
struct Gemm {
    Operand<ASTR> A;
    Operand<BSTR> B;
    FragAddr<ASTR, 4> fa;
    FragAddr<BSTR, 2> fb;
    int wave, lane, wm, wn;
    bool low, high;  // whether this wave's rows of A's first and second half are among the tile's

    // A wave whose rows lie past the tile's `rows` takes its part in the loads
    // and barriers only. (A loop of its own for full tiles, without the
    // branches, spilled registers and was no faster.)
    __device__ __forceinline__ void set_rows(int32_t rows)
    {
        low = rows > wm * 64;
        high = rows > 128 + wm * 64;
    }

    __device__ __forceinline__ void init_lane()
    {
        lane = threadIdx.x & (kWave - 1);
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        wm = wave >> 2;
        wn = wave & 3;
        fa.init(wm * 64, lane);
        fb.init(wn * 32, lane);
    }

    // first of the 32 columns that acc[.][hB] holds for this wave
    __device__ __forceinline__ int column(int hB) const { return BSTR ? hB * 128 + wn * 32 : wn * 64 + hB * 32; }

    // the loads that run ahead of the first phase, in the order they are waited for
    __device__ __forceinline__ void start(uint8_t *lds, int nk) const
    {
        uint8_t *s0 = lds, *s1 = lds + kStageBytes;
        B.load(s0 + 2 * kHalfBytes, 0, 0, nk, wave);
        A.load(s0, 0, 0, nk, wave);
        B.load(s0 + 3 * kHalfBytes, 1, 0, nk, wave);
        A.load(s0 + kHalfBytes, 1, 0, nk, wave);
        B.load(s1 + 2 * kHalfBytes, 0, 1, nk, wave);
        A.load(s1, 0, 1, nk, wave);
        B.load(s1 + 3 * kHalfBytes, 1, 1, nk, wave);
    }

    __device__ __forceinline__ static void mfmas(const FragA &a, const FragB &b, f32x4 (&c)[4][2])
    {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    c[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[kk][j], a.v[kk][i], c[i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
    }

    // sum += this wave's quarter of a's rows, fragment wn, summed over k: a
    // product with ones. Lanes L < 16 hold row wm * 64 + wn * 16 + L's.
    __device__ __forceinline__ void add_rows(const FragA &a, f32x4 &sum) const
    {
        const __bf16 one = (__bf16)1.0f;
        const bf16x8 ones = {one, one, one, one, one, one, one, one};
#pragma unroll
        for (int f = 0; f < 4; ++f)
            if (wn == f)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, a.v[kk][f], sum, 0, 0, 0);
    }

    // K-tile t, which lies in stage `cur`; b0 holds its first half of B, and
    // next receives the next K-tile's. A slot between two barriers holds either
    // reads and load starts or MFMAs, and the refill of a half tile starts a
    // barrier or more after every wave's reads of it are complete.
    template <bool SUM>
    __device__ __forceinline__ void ktile(uint8_t *cur, uint8_t *other, int t, int nk, const FragB &b0, FragB &next,
                                          Acc &acc, f32x4 (&sum)[2], bool summed) const
    {
        const uint32_t at = lds_offset(cur), then = lds_offset(other);
        FragA a;
        FragB b1;
        A.load(other + kHalfBytes, 1, t + 1, nk, wave);
        slot_a<0>(fa, at, a);
        if (low)
            mfmas(a, b0, acc[0][0]);
        if (SUM && summed)
            add_rows(a, sum[0]);
        slot_end();
        B.load(cur + 2 * kHalfBytes, 0, t + 2, nk, wave);
        slot_b<3>(fb, at, b1);
        if (low)
            mfmas(a, b1, acc[0][1]);
        slot_end();
        A.load(cur, 0, t + 2, nk, wave);
        if (high) {
            slot_a<1>(fa, at, a);
            mfmas(a, b1, acc[1][1]);
            if (SUM && summed)
                add_rows(a, sum[1]);
        } else {
            wait_loads<10>();
            slot_end();
        }
        slot_end();
        B.load(cur + 3 * kHalfBytes, 1, t + 2, nk, wave);
        slot_b<2>(fb, then, next);
        if (high)
            mfmas(a, b0, acc[1][0]);
        slot_end();
    }

    // The whole K loop; start() has been called. On return every wave has read
    // what it needs of LDS, and the loads still in flight bring only zeros.
    // SUM: where `summed`, sum[h] receives the row sums of A's half h (add_rows).
    template <bool SUM = false>
    __device__ __forceinline__ void run(uint8_t *lds, int nk, Acc &acc, f32x4 (&sum)[2], bool summed) const
    {
        sum[0] = sum[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 16; ++q)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[q >> 3][(q >> 2) & 1][q & 3][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        uint8_t *s0 = lds, *s1 = lds + kStageBytes;
        wait_loads<10>();
        slot_end();
        FragB b0, b1;
        slot_b<2>(fb, lds_offset(s0), b0);
        if (wm)  // the second group of waves starts half a phase later
            slot_end();
        int t = 0;
        for (; t + 1 < nk; t += 2) {
            ktile<SUM>(s0, s1, t, nk, b0, b1, acc, sum, summed);
            ktile<SUM>(s1, s0, t + 1, nk, b1, b0, acc, sum, summed);
        }
        if (t < nk)
            ktile<SUM>(s0, s1, t, nk, b0, b1, acc, sum, summed);
        if (!wm)
            slot_end();
    }
    __device__ __forceinline__ void run(uint8_t *lds, int nk, Acc &acc) const
    {
        f32x4 none[2];
        run<false>(lds, nk, acc, none, false);
    }
};

// Two groups of four bf16 columns, 16 columns apart, of a row that lies across
// lanes L, L + 16, L + 32, L + 48 -> eight consecutive columns in each of
// those lanes, (L / 16) * 8 + 0..7 of 32; and back. One 16-byte access per
// lane then covers 64 consecutive bytes of 16 rows.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b)
{
    const u32x2 r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b)
{
    const u32x2 r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ u32x4 to_rows(u32x2 a, u32x2 b)
{
    uint32_t a0 = a[0], a1 = a[1], b0 = b[0], b1 = b[1];
    swap32(a0, b0);
    swap32(a1, b1);
    swap16(a0, b0);
    swap16(a1, b1);
    return u32x4{a0, a1, b0, b1};
}
__device__ __forceinline__ void from_rows(u32x4 v, u32x2 &a, u32x2 &b)
{
    uint32_t a0 = v[0], a1 = v[1], b0 = v[2], b1 = v[3];
    swap16(a0, b0);
    swap16(a1, b1);
    swap32(a0, b0);
    swap32(a1, b1);
    a = u32x2{a0, a1};
    b = u32x2{b0, b1};
}
__device__ __forceinline__ f32x4 widen(u32x2 v) { return {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)}; }
__device__ __forceinline__ u32x2 narrow(f32x4 v) { return {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}; }

// A tile's rows of a [rows][ld] bf16 tensor, through a descriptor that ends
// with the tile's last row: pairs of column groups as above, this lane's eight
// consecutive columns at byte offset col (kOutside or more past the width) of
// row m + lane % 16, m uniform. The stores carry no
// scalar offset: a 16-byte store with one, followed at once by an instruction
// that writes its last data register, stored the new value in some lanes on
// gfx950, and the compiler keeps the two apart only where there is none.
struct TileRows {
    __amdgpu_buffer_rsrc_t r;
    uint32_t lane_row, ld2;
    __device__ __forceinline__ void init(const uint16_t *p, int64_t row0, int32_t rows, int64_t ld, int lane)
    {
        r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(p + row0 * ld), 0, (uint32_t)(rows * ld * 2),
                                              kGemmBufferFlags);
        ld2 = (uint32_t)ld * 2;
        lane_row = (uint32_t)(lane & 15) * ld2;
    }
    // any m: past the tile's rows it gives zeros
    __device__ __forceinline__ u32x4 fetch(uint32_t m, uint32_t col, uint32_t half = 0) const
    {
        return __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane_row + col + (m * ld2 + half), 0, 0));
    }
    __device__ __forceinline__ static void unpack(u32x4 raw, f32x4 (&v)[2])
    {
        u32x2 a, b;
        from_rows(raw, a, b);
        v[0] = widen(a);
        v[1] = widen(b);
    }
    __device__ __forceinline__ void store(uint32_t m, uint32_t col, const f32x4 (&v)[2], uint32_t half = 0) const
    {
        __builtin_amdgcn_raw_buffer_store_b128(to_rows(narrow(v[0]), narrow(v[1])), r,
                                               lane_row + col + (m * ld2 + half), 0, 0);
    }
};

}  // namespace
}  // namespace moe
