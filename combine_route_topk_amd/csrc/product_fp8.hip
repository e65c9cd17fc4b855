// product_fp8.hip -- the experts' products on FP8 rows, with weights in E4M3
// and a float32 scale for each block of 128 x 128 of them, and the gradient
// with respect to their input (the same product with the transposed weights).
//
// The tiles, the K loop's schedule and the epilogue are the bf16 products'
// (product_gemm.hpp): a K-tile is 128 bytes of a row in both, here 128 values.
// An MFMA takes 16 x 16 x 128 in as many cycles as two of bf16's 16 x 16 x 32,
// so the matrix units' bound is half the bf16 one. The rows' scales, a power
// of two per 32 values, are one of the instruction's scale operands. The
// weights' scale is the same for a wave's columns across a K-tile: its power of
// two is the other scale operand, and what is left of it, between 1 and 2, is
// the unit that the accumulators are kept in. That costs a multiplication of
// each accumulator for each K-tile, as an FMA on sums that start from zero would,
// but no registers for such sums (16384 x 8192 by 8192: 0.99 ms, 1.04 so).
//
// What that rounds. The ratio of two units is a reciprocal's product (1 ulp and
// half of one), and each accumulator's product half an ulp: less than 2^-22 of
// the sum for each K-tile, 2^-16 at K = 8192, where the result's bf16 keeps 2^-9.
// Against float64 it shows as a mean of 8e-8 of the results' size at K = 8192, 5e-7
// at 32768 (the short kernels, which multiply by the scale itself: none), beside an
// rms of 1.5e-5 from the matrix unit's own sums in all three. It aligns the products
// of eight neighbouring k to the largest and drops their bits below 2^-13 of it:
// the price of its rate, which is twice that of the instructions on bf16.
//
// On MI355X a round of 256 tiles takes 1.83 us for each K-tile (2.3 PFLOP/s),
// 16384 x 8192 by 8192 0.98 to 1.05 ms (2.1 to 2.25). Power bounds the K loop: the
// clock falls to 1.9 GHz in it, and operands of zeros run a fifth faster. Short K is
// bound by the stores as well: 327680 rows of 2048 by 2 x 768 in 30 rounds take
// 1.13 ms, 0.91 of them the K loop and 0.22 first loads and bf16 results; with results
// in both types and pre, 1.8 GB, 1.31 to 1.36 ms, 0.40 of them not the K loop
// (from K = 128, 2048 and 4096). Starting the next tile's loads before
// the epilogue, letting its stores run on into that tile's K loop, starting the
// blocks at different times and stores past the caches gained nothing.
#include "product_fp8_some.hpp"

namespace moe {
namespace {

// LDS: both stages of A, then both of B, so that one address register reaches
// each operand's 64 KiB by instruction offsets; then two stages of the rows'
// scales of four K-tiles, 16 bytes for each of the tile's 256 rows.
constexpr int kStage8 = 2 * kHalfBytes, kB8 = 2 * kStage8, kScales8 = 2 * kB8;
constexpr int kScaleStage = kTile * 16;
constexpr uint32_t kBehind = 0x40000000u;  // past the end of every operand of a tile, and no carry with `from`
constexpr int kLds8 = kScales8 + 2 * kScaleStage;
// Fragments of A (four of 16 rows) and B (two of 16 columns): 128 k of a row in
// four lanes, a lane's 32 in two pieces of 16 that lie 64 apart.
struct FragA8 {
    i32x8 v[4];
    uint32_t s[4];  // scale bytes of the lane's row, for its 32 of the K-tile's values
};
struct FragB8 {
    i32x8 v[2];
};
// A block's scale s of the weights as the product of the power of two that the
// MFMA multiplies by, and of a factor of magnitude [1, 2). Accumulators are kept
// in units of the factor: they are multiplied by the old one over the new where
// it changes, which is between 1/2 and 2 whatever the scales are. A scale below
// 2^-126 counts as 2^-127; one that is infinite or NaN gives NaN.
struct Scale8 {
    uint32_t power;  // E8M0
    float factor;
};
__device__ __forceinline__ Scale8 split(float s)
{
    const uint32_t bits = __float_as_uint(s), power = (bits >> 23) & 255;
    return {power, __uint_as_float(power ? (bits & 0x807FFFFFu) | 0x3F800000u : 0x3F800000u)};
}

// An operand of a tile, as Operand<false>, with one offset per lane: the loads of
// other rows lie a uniform distance from it, which is part of the scalar offset.
// The descriptor's end is checked less the scalar offset, which must not pass
// it: where it would, it is the end itself, and every lane gets zeros.
struct Operand8 {
    u32x4 r;
    uint32_t off;
    uint32_t from[2][2];  // of load i of half h

    // `rows` valid rows (one or more), ld bytes apart; `row`: of this wave's load 0 of half 0
    __device__ __forceinline__ void init(const uint8_t *p, int32_t rows, int32_t ld, int lane, int row, int half_rows,
                                         int second_rows)
    {
        // the same in every lane, which the compiler cannot always tell
        r = descriptor(p, __builtin_amdgcn_readfirstlane((uint32_t)(min(rows, kTile) * ld)));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r[i] = __builtin_amdgcn_readfirstlane(r[i]);
        off = (uint32_t)(row + (lane >> 3)) * (uint32_t)ld + ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                from[h][i] = (uint32_t)((h * half_rows + i * second_rows) * ld);
    }
    // Start the two loads of half H of the K-tile at byte k0 of the rows
    // (kBehind for one behind the last: zeros) into LDS at dst + AT and 8 KiB on.
    // One block of instructions, so that the reading slot has few. The first load
    // stands behind five wait states, as its scalar registers need (load_to_lds):
    // 984 us for 16384 x 8192 by 8192, 979 with three.
    template <int H, int AT>
    __device__ __forceinline__ void load(uint32_t dst, uint32_t k0) const
    {
        uint32_t x, y;
        asm volatile("s_add_u32 %[x], %[f0], %[k0]\n\ts_add_u32 m0, %[dst], %[at0]\n\ts_min_u32 %[x], %[x], %[end]\n\ts_nop 1\n\t"
                     "buffer_load_dwordx4 %[v], %[r], %[x] offen lds\n\t"
                     "s_add_u32 %[y], %[f1], %[k0]\n\ts_add_u32 m0, %[dst], %[at1]\n\ts_min_u32 %[y], %[y], %[end]\n\t"
                     "buffer_load_dwordx4 %[v], %[r], %[y] offen lds"
                     : [x] "=&s"(x), [y] "=&s"(y)
                     : [f0] "s"(from[H][0]), [f1] "s"(from[H][1]), [k0] "s"(k0), [dst] "s"(dst), [at0] "n"(AT),
                       [at1] "n"(AT + 8192), [end] "s"(r[2]), [v] "v"(off), [r] "s"(r)
                     : "memory", "scc");
    }
};

// The K loop of one 256 x 256 tile. Schedule as in product_gemm.hpp: phases of
// 8 MFMAs, and waves 0-3 half a phase apart from waves 4-7, so that one of a
// SIMD's two waves reads while the other multiplies. An MFMA holds its SIMD's
// vector issue for 16 of its 32 cycles and its own wave for longer (FMAs
// between a wave's MFMAs delayed each by all of their time), so the
// multiplications that bring accumulators to a K-tile's units are the reading
// wave's: it starts its reads, then multiplies, then waits.
struct Gemm8 {
    Operand8 a8, b8;
    uint32_t lds, lds_wave;   // LDS, and where this wave's loads begin in it
    uint32_t tail;
    uint32_t fa[2], fb[2];    // LDS addresses of this lane's pieces of a fragment: 16 k of the first 64, and of the second
    u32x4 scales;             // descriptor of the tile's row scales
    uint32_t scale_row;       // this lane's row among them when it loads
    uint32_t scale_read;      // and its address in a stage of scales when it reads
    int32_t last_scales;      // scale bytes of the last K-tile, 1 to 4
    const float *ws[2];       // the weights' scales of this wave's columns (gated: gate, up), one for each K-tile
    int wave, lane, wm, wn;
    uint32_t low, high;       // whether this wave's rows of A's first and second half are among the tile's

    __device__ __forceinline__ void init_lane(uint32_t lds_)
    {
        lds = lds_;
        lane = threadIdx.x & (kWave - 1);
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        lds_wave = lds + wave * 1024;
        wm = wave >> 2;
        wn = wave & 3;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            fa[kk] = lds + frag_row(wm * 64, kk, lane);
            fb[kk] = lds + kB8 + frag_row(wn * 32, kk, lane);
        }
    }
    __device__ __forceinline__ void set_rows(int32_t rows)
    {
        low = __builtin_amdgcn_readfirstlane(rows > wm * 64);
        high = __builtin_amdgcn_readfirstlane(rows > 128 + wm * 64);
    }
    // first of the 32 columns that acc[.][hB] holds for this wave
    __device__ __forceinline__ int column(int hB) const { return wn * 64 + hB * 32; }

    __device__ __forceinline__ void init_scales(const uint8_t *p, int32_t rows, int32_t K, int64_t row_bytes)
    {
        tail = K % kTileK8 && ((lane & 7) ^ (lane >> 3)) * 16 >= K % kTileK8 ? kOutside : 0u;
        scales = descriptor(p + K, (uint32_t)(rows * row_bytes - K));
        scale_row = (uint32_t)(wave * kWave + lane) * (uint32_t)row_bytes;
        scale_read = lds + kScales8 + (uint32_t)((wm * 64 + (lane & 15)) * 16 + (lane >> 4));
        last_scales = (K - 1) % kTileK8 / 32 + 1;
    }
    // start the load of the scales of K-tiles 4 q to 4 q + 3: waves 0 to 3, 64 rows each
    __device__ __forceinline__ void load_scales(int q) const
    {
        if (wave < 4)
            load_to_lds(lds + kScales8 + (q & 1) * kScaleStage + wave * (kWave * 16), scales, scale_row, q * 16);
    }
    template <int S, int H>
    __device__ __forceinline__ void load_a(uint32_t k0) const
    {
        a8.load<H, S * kStage8 + H * kHalfBytes>(lds_wave, k0);
    }
    template <int S, int H>
    __device__ __forceinline__ void load_b(uint32_t k0) const
    {
        b8.load<H, kB8 + S * kStage8 + H * kHalfBytes>(lds_wave, k0);
    }
    // from the last K-tile on, pieces past K read as zeros
    __device__ __forceinline__ void cut_tail()
    {
        a8.off |= tail;
        b8.off |= tail;
    }
    __device__ __forceinline__ static uint32_t k_of(int t, int nk) { return t < nk ? (uint32_t)t * kTileK8 : kBehind; }

    // the loads that run ahead of the first phase, in the order they are waited for
    __device__ __forceinline__ void start(int nk)
    {
        load_scales(0);
        if (nk == 1)
            cut_tail();
        load_b<0, 0>(0);
        load_a<0, 0>(0);
        load_b<0, 1>(0);
        load_a<0, 1>(0);
        // K-tile 1's second half of A follows in the loop: its tail is cut there
        const uint32_t k1 = k_of(1, nk);
        if (nk == 2)
            cut_tail();
        load_b<1, 0>(k1);
        load_a<1, 0>(k1);
        load_b<1, 1>(k1);
    }

    // `at`: of the half tile, among its operand's
    __device__ __forceinline__ void read_a(int at, uint32_t scale, FragA8 &a) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a.v[i] = read_frag(fa[0] + (at + i * 2048), fa[1] + (at + i * 2048));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a.s[i] = lds_read<uint8_t>(scale + i * 256);
    }
    __device__ __forceinline__ void read_b(int at, FragB8 &b) const
    {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            b.v[j] = read_frag(fb[0] + (at + j * 2048), fb[1] + (at + j * 2048));
    }

    // c += a b times the weights' powers of two, w[j] for column group j
    __device__ __forceinline__ static void multiply(const FragA8 &a, const FragB8 &b, const Scale8 (&w)[2],
                                                    f32x4 (&c)[4][2])
    {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                c[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v[j], a.v[i], c[i][j], 0, 0, 0, w[j].power, 0,
                                                                           a.s[i]);
        __builtin_amdgcn_s_setprio(0);
    }
    // accumulators from the units of the K-tile before to this one's
    __device__ __forceinline__ static void rescale(const float (&r)[2], f32x4 (&c)[4][2])
    {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    c[i][j][e] *= r[j];
    }

    // The end of a reading slot: the loads that the next phase reads have
    // arrived, for every wave behind the barrier, and so have this wave's reads.
    // (What reads into LDS replaces is so read to its end one barrier before.)
    __device__ __forceinline__ static void reads_end()
    {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(10)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_s_waitcnt((63 & 15) | ((63 >> 4) << 14) | (7 << 4));  // lgkmcnt(0); the compiler counts along
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ static void products_end()
    {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }

    // K-tile t, which lies in stage S; b0 holds its first half of B, and next
    // receives the next K-tile's. w holds its scales and receives the next
    // K-tile's, r takes the accumulators to its units and receives the next's.
    template <int S>
    __device__ __forceinline__ void ktile(int t, int nk, const FragB8 &b0, FragB8 &next, Scale8 (&w)[2], float (&r)[2],
                                          Acc &acc)
    {
        FragA8 a;
        FragB8 b1;
        uint32_t from = scale_read + (((t >> 2) & 1) * kScaleStage + (t & 3) * 4);
        if (t == nk - 1)  // past K zeros meet the last scale that is one, not what lies behind it
            from -= max((lane >> 4) + 1 - last_scales, 0);
        const int tn = min(t + 1, nk - 1);
        const uint32_t k1 = k_of(t + 1, nk), k2 = k_of(t + 2, nk);
        load_a<1 - S, 1>(k1);
        if (t + 3 == nk)
            cut_tail();
        read_a(S * kStage8, from, a);
        rescale(r, acc[0][0]);
        reads_end();
        if (low)
            multiply(a, b0, w, acc[0][0]);
        products_end();
        load_b<S, 0>(k2);
        read_b(S * kStage8 + kHalfBytes, b1);
        rescale(r, acc[0][1]);
        reads_end();
        if (low)
            multiply(a, b1, w, acc[0][1]);
        products_end();
        load_a<S, 0>(k2);
        if ((t & 3) == 0 && t + 4 < nk)  // two slots after every wave's last reads of the stage
            load_scales((t >> 2) + 1);
        read_a(S * kStage8 + kHalfBytes, from + 128 * 16, a);
        rescale(r, acc[1][1]);
        reads_end();
        if (high)
            multiply(a, b1, w, acc[1][1]);
        __builtin_amdgcn_sched_barrier(0);
        // nothing waits for LDS before these are needed, which would wait for them too
        const float s0 = load_uniform(ws[0] + tn), s1 = load_uniform(ws[1] + tn);
        products_end();
        load_b<S, 1>(k2);
        read_b((1 - S) * kStage8, next);
        rescale(r, acc[1][0]);
        reads_end();
        if (high)
            multiply(a, b0, w, acc[1][0]);
        products_end();
        const Scale8 n[2] = {split(s0), split(s1)};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            r[j] = w[j].factor * __builtin_amdgcn_rcpf(n[j].factor);
            w[j] = n[j];
            asm volatile("" : "+v"(w[j].power));  // the MFMA takes it from a vector register
        }
    }

    // The whole K loop; start() has been called. On return every wave has read
    // what it needs of LDS, and the loads still in flight bring only zeros.
    __device__ __forceinline__ void run(int nk, Acc &acc)
    {
#pragma unroll
        for (int q = 0; q < 16; ++q)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[q >> 3][(q >> 2) & 1][q & 3][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        Scale8 w[2] = {split(load_uniform(ws[0])), split(load_uniform(ws[1]))};
        float r[2] = {1.f, 1.f};
        FragB8 b0, b1;
        reads_end();
        read_b(0, b0);
        reads_end();
        if (wm)  // the second group of waves starts half a phase later
            products_end();
        int t = 0;
        for (; t + 1 < nk; t += 2) {
            ktile<0>(t, nk, b0, b1, w, r, acc);
            ktile<1>(t + 1, nk, b1, b0, w, r, acc);
        }
        if (t < nk)
            ktile<0>(t, nk, b0, b1, w, r, acc);
        if (!wm)
            products_end();
        // w holds the last K-tile's scales again
        const float f[2] = {w[0].factor, w[1].factor};
#pragma unroll
        for (int q = 0; q < 4; ++q)
            rescale(f, acc[q >> 1][q & 1]);
    }
};

template <bool GRAD, bool GATED, int ACT>
__global__ __launch_bounds__(kGemmThreads, 2) void product_fp8_kernel(Product8Args p)
{
    constexpr bool PAIR = GATED && !GRAD;
    constexpr int kCols = PAIR ? kTile / 2 : kTile;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds8 > kSomeLds ? kLds8 : kSomeLds];
    __shared__ int32_t first[kMaxLocalExperts + 1];
    const int32_t row_tiles = plan_row_tiles<kGemmThreads, kTile>(p.off, p.El, p.max_rows, first);
    const uint32_t nct = (uint32_t)(p.N + kCols - 1) / kCols;
    const int64_t wide = PAIR ? 2 * (int64_t)p.N : p.N;
    const int nk = (p.K + kTileK8 - 1) / kTileK8;
    const int64_t nbw = (wide + 127) / 128;
    Gemm8 gemm;
    gemm.init_lane(lds_offset(lds));
    // tiles and the slices of a last round as in product.hip
    const uint32_t slot = gridDim.x % 8 ? blockIdx.x : blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
    const uint32_t tiles = row_tiles * nct, rest = tiles % gridDim.x, whole = tiles - rest;
    const uint32_t slices = rest * 4 <= gridDim.x ? 4 : (rest * 2 <= gridDim.x ? 2 : 1);
    // unit u: rows [row0, row0 + rows) of expert l by the columns from n0; none for a slice past the last row
    struct Unit {
        int32_t l, row0, rows, n0;
    };
    auto unit = [&](uint32_t u) {
        const uint32_t tile = u < whole ? u : whole + (u - whole) / slices;
        const int32_t slice = u < whole ? 0 : (int32_t)((u - whole) % slices);
        const int32_t most = u < whole ? kTile : kTile / (int32_t)slices;
        const TileAt which = tile_at(tile, row_tiles, nct);
        const int32_t l = __builtin_amdgcn_readfirstlane(tile_expert(first, p.El, which.row));
        const Rows r = expert_rows(p.off, l, p.max_rows);
        const int64_t at = r.begin + (int64_t)(which.row - first[l]) * kTile + slice * most;
        return Unit{l, __builtin_amdgcn_readfirstlane((int32_t)at),
                    __builtin_amdgcn_readfirstlane((int32_t)max((int64_t)0, min((int64_t)most, r.end - at))),
                    which.col * kCols};
    };
    const uint32_t units = whole + rest * slices;
    uint32_t u = slot;
    for (; u < (slices > 1 ? whole : units); u += gridDim.x) {
        const auto [l, row0, rows, n0] = unit(u);
        if (!rows)
            continue;
        const uint8_t *a = p.a + row0 * p.a_bytes;
        const uint8_t *Wl = p.W + l * wide * p.K;
        gemm.a8.init(a, rows, (int32_t)p.a_bytes, gemm.lane, gemm.wave * 8, 128, 64);
        gemm.init_scales(a, rows, p.K, p.a_bytes);
        const float *ws = p.scale + l * nbw * nk;
        // Rows of B's halves as in product.hip, eight of a wave's load at a time.
        // Columns past the last have no scale of their own: theirs multiplies zeros.
        if constexpr (PAIR) {
            const bool up = (gemm.wave >> 1) & 1;
            gemm.b8.init(Wl + ((up ? (int64_t)p.N : 0) + n0) * p.K, p.N - n0, p.K, gemm.lane,
                         (gemm.wave >> 2) * 32 + (gemm.wave & 1) * 8, 16, 64);
            const int64_t c = min(n0 + gemm.wn * 32, p.N - 32);
            gemm.ws[0] = ws + c / 128 * nk;
            gemm.ws[1] = ws + (p.N + c) / 128 * nk;
        } else {
            gemm.b8.init(Wl + (int64_t)n0 * p.K, p.N - n0, p.K, gemm.lane, (gemm.wave >> 2) * 64 + (gemm.wave & 3) * 8, 32,
                         128);
            gemm.ws[0] = gemm.ws[1] = ws + min((int64_t)(n0 + gemm.wn * 64) / 128, nbw - 1) * nk;
        }
        Acc acc;
        gemm.set_rows(rows);
        gemm.start(nk);
        gemm.run(nk, acc);
        epilogue<GRAD, GATED, ACT, true>(p, gemm, acc, l, row0, rows, n0);
        const int32_t width = GATED && GRAD ? 2 * p.N : p.N;
        if (p.out8 && n0 + kCols >= p.N)
            pad_rows<kGemmThreads>(p.out8 + row0 * p.out8_bytes, rows, width, p.out8_bytes);
        wait_loads<0>();
        slot_end();
    }
    static_assert(kSomeThreads == kGemmThreads && kSomeRows * 2 == kTile && kSomeCols == kTile);
    // A round of slices: product_fp8_some.hpp's loads run further ahead. With 64
    // rows it takes 0.9 us for each 128 k where the loop above takes 1.65 (4 experts
    // of 64 rows, 7168 by 7168, weights partly in the last-level cache: 51 against
    // 91 us).
    if (slices > 1 && u < units) {
        const auto [l, row0, rows, n0] = unit(u);
        if (rows)
            some_tile<GRAD, GATED, ACT>(p, lds_offset(lds), l, row0, rows, n0);
    }
}

template <bool GRAD>
hipError_t launch(const Product8Args &p, int32_t act, bool gated, int cus, hipStream_t stream)
{
    const int kCols = gated && !GRAD ? kTile / 2 : kTile;
    // four blocks a tile, for its slices
    const int64_t units = 4 * ((int64_t)p.max_rows / kTile + p.El) * ((p.N + kCols - 1) / kCols);
    const dim3 grid((unsigned)(units < cus ? units : cus));
#define MOE_PRODUCT_CASE(A)                                                                                        \
    case A:                                                                                                        \
        if (gated)                                                                                                 \
            hipLaunchKernelGGL((product_fp8_kernel<GRAD, true, A>), grid, dim3(kGemmThreads), 0, stream, p);       \
        else                                                                                                       \
            hipLaunchKernelGGL((product_fp8_kernel<GRAD, false, A>), grid, dim3(kGemmThreads), 0, stream, p);      \
        return hipGetLastError();
    switch (act) {
        MOE_PRODUCT_CASE(kActNone)
        MOE_PRODUCT_CASE(kActRelu)
        MOE_PRODUCT_CASE(kActSilu)
        MOE_PRODUCT_CASE(kActGelu)
        MOE_PRODUCT_CASE(kActGeluTanh)
    default:
        return hipErrorInvalidValue;
    }
#undef MOE_PRODUCT_CASE
}

// Which kernel a product runs on. The host knows max_rows, not how the rows lie:
// it takes hit = min(max_rows, E_l) experts with rows; up to three quarters of a
// tile's height each they are taken to have one tile, above that a half-full one
// beside the full ones. On MI355X, in us, weights from HBM, rows drawn at random,
// few rows / some rows / tiles (the last as their 64-row slices where they are few):
//   tiles of 64 rows for less than a quarter of the CUs: 1 expert, 7168 by 2 x
//   2048: 26 / 49 / 50 at 64 and at 128 rows; 8 experts, 2048 by 2 x 768: 10 / 13 / 13
//   at 8 rows each;
//   for less than all: 4 experts, 7168 by 7168: 43 / 51 / 51 at 4 rows each,
//   55 / 54 / 54 at 16, 137 / 62 / 65 at 64;
//   for all: 32 experts, 7168 by 2 x 2048: 163 / 158 / 188 at one row each,
//   275 / 162 / 195 at 32, 438 / 169 / 215 at 64, 784 / 268 / 236 at 128; 64
//   experts, 2048 by 2048: 75 / 54 / 64 at 16, 191 / 64 / 73 at 64, 354 / 96 / 80
//   at 128.
// A round of tiles over the CUs takes about 0.9 us for each 128 k with 64 rows,
// 1.5 with 128 and 1.9 with 256, which decides between the last two.
// Where the estimate errs: rows that lie evenly leave no half-full tiles beside
// full ones. The 32 experts with 100 rows each would take 192 us on some rows
// against 220 (and 240 against 223 where their counts differ by a third); with 128
// each 211 against 228 (268 against 236 at random). And the 8 experts, at 64 rows,
// are taken for 72 tiles of 64 where there are 48: 18.8 us, 17.5 on few rows.
enum class Kernel { kFew, kSome, kTiles };
Kernel choose(const Product8Args &p, bool gated, bool grad, int cus)
{
    const int64_t rows = p.max_rows, hit = rows < p.El ? rows : p.El;
    const int64_t columns = gated && !grad ? kTile / 2 : kTile, across = (p.N + columns - 1) / columns;
    auto tiles = [&](int64_t height) {
        return (4 * rows <= 3 * height * hit ? hit : rows / height + (hit + 1) / 2) * across;
    };
    auto rounds = [&](int64_t n) { return (n + cus - 1) / cus; };
    const int64_t t64 = tiles(64);
    if (!grad && (4 * t64 < cus ? rows <= 128 * (int64_t)p.El : t64 < cus && rows <= 8 * (int64_t)p.El))
        return Kernel::kFew;
    const int64_t some = t64 <= cus ? 9 : 15 * rounds(tiles(kSomeRows));
    return some <= 19 * rounds(tiles(kTile)) ? Kernel::kSome : Kernel::kTiles;
}

}  // namespace

hipError_t launch_product_fp8(const Product8Args &p, int32_t act, bool gated, bool grad, hipStream_t stream)
{
    int cus = 0;
    const hipError_t err = current_cus(&cus);
    if (err != hipSuccess)
        return err;
    switch (choose(p, gated, grad, cus)) {
    case Kernel::kFew:
        return launch_product_fp8_few(p, act, gated, cus, stream);
    case Kernel::kSome:
        return launch_product_fp8_some(p, act, gated, grad, cus, stream);
    default:
        return grad ? launch<true>(p, act, gated, cus, stream) : launch<false>(p, act, gated, cus, stream);
    }
}

}  // namespace moe
