// product_fp8.hip -- the experts' products on FP8 rows, with weights in E4M3
// and a float32 scale for each block of 128 x 128 of them, and the gradient
// with respect to their input (the same product with the transposed weights).
//
// The tiles, the K loop's schedule and the epilogue are the bf16 products'
// (product_gemm.hpp): a K-tile is 128 bytes of a row in both, here 128 values.
// An MFMA takes 16 x 16 x 128 in as many cycles as two of bf16's 16 x 16 x 32,
// so the matrix units' bound is half the bf16 one. The rows' scales, a power
// of two per 32 values, are the instruction's own scale operand. The weights'
// scale is the same for a wave's columns across a K-tile: the MFMA starts from
// zero and its sum is added to the accumulators times the scale, four FMAs of
// 4 cycles beside an MFMA of 32.
#include "product_tile.hpp"

namespace moe {
namespace {

// the rows' scales of four K-tiles: 16 bytes for each of the tile's 256 rows
constexpr int kScaleStage = kTile * 16;
// The scale bytes of a lane's row for a K-tile: of the 32 values numbered
// lane / 16, for each of the eight groups of 16 rows of a wave.
struct RowScales {
    uint32_t v[2][4];
};

// The slot that reads the first half of A, and the K-tile's row scales.
__device__ __forceinline__ void slot_a_scales(const FragAddr<false, 4> &fa, uint32_t stage, uint32_t scale, FragA &a,
                                              RowScales &s)
{
    asm volatile(MOE_READ_A(0, 1, 2, 3, 4, 5, 6, 7, 16, 17)
                 "ds_read_u8 %8, %18\n\tds_read_u8 %9, %18 offset:256\n\t"
                 "ds_read_u8 %10, %18 offset:512\n\tds_read_u8 %11, %18 offset:768\n\t"
                 "ds_read_u8 %12, %18 offset:2048\n\tds_read_u8 %13, %18 offset:2304\n\t"
                 "ds_read_u8 %14, %18 offset:2560\n\tds_read_u8 %15, %18 offset:2816\n\t" MOE_SLOT_END
                 : MOE_OUT_A(a), "=&v"(s.v[0][0]), "=&v"(s.v[0][1]), "=&v"(s.v[0][2]), "=&v"(s.v[0][3]),
                   "=&v"(s.v[1][0]), "=&v"(s.v[1][1]), "=&v"(s.v[1][2]), "=&v"(s.v[1][3])
                 : "v"(stage + fa.a[0]), "v"(stage + fa.a[1]), "v"(scale), [half] "n"(0)
                 : "memory");
}

struct Gemm8 : Gemm<false, false> {
    const uint8_t *scales;    // of the tile's first row
    uint32_t scale_records, scale_row;
    uint32_t scale_read;      // this lane's address in a stage of scales
    int32_t last_scales;      // scale bytes of the last K-tile, 1 to 4
    const float *ws[2];       // the weights' scales of this wave's columns (gated: gate, up), one for each K-tile

    __device__ __forceinline__ void init_scales(const uint8_t *rows_, int32_t rows, int32_t K, int64_t row_bytes)
    {
        scales = rows_ + K;
        scale_records = (uint32_t)(rows * row_bytes - K);
        scale_row = (uint32_t)(wave * kWave + lane) * (uint32_t)row_bytes;
        scale_read = (uint32_t)((wm * 64 + (lane & 15)) * 16 + (lane >> 4));
        last_scales = (K - 1) % kTileK8 / 32 + 1;
    }

    // start the load of the scales of K-tiles 4 q to 4 q + 3: waves 0 to 3, 64 rows each
    __device__ __forceinline__ void load_scales(uint8_t *stages, int q) const
    {
        if (wave < 4)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(scales), 0, scale_records, kGemmBufferFlags),
                stages + (q & 1) * kScaleStage + wave * (kWave * 16), 16, scale_row + q * 16, 0, 0, 0);
    }

    // c += w * (a b), w[j] for column group j
    __device__ __forceinline__ static void mfmas8(const FragA &a, const FragB &b, const uint32_t (&s)[4],
                                                  const float (&w)[2], f32x4 (&c)[4][2])
    {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        f32x4 p[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                p[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    join8(b.v[0][j], b.v[1][j]), join8(a.v[0][i], a.v[1][i]), f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, kOne, 0,
                    s[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    c[i][j][e] = fmaf(w[j], p[i][j][e], c[i][j][e]);
        __builtin_amdgcn_s_setprio(0);
    }

    // As Gemm::ktile. The scales that replace a stage are started two slots
    // after every wave's reads of its last K-tile.
    __device__ __forceinline__ void ktile8(uint8_t *cur, uint8_t *other, uint8_t *stages, int t, int nk, const FragB &b0,
                                           FragB &next, const float (&w)[2], float (&wn_)[2], Acc &acc) const
    {
        const uint32_t at = lds_offset(cur), then = lds_offset(other);
        FragA a;
        FragB b1;
        RowScales s;
        const int tn = min(t + 1, nk - 1);
        wn_[0] = load_uniform(ws[0] + tn);
        wn_[1] = load_uniform(ws[1] + tn);
        A.load(other + kHalfBytes, 1, t + 1, nk, wave);
        uint32_t from = lds_offset(stages) + ((t >> 2) & 1) * kScaleStage + (t & 3) * 4 + scale_read;
        if (t == nk - 1)  // past K zeros meet the last scale that is one, not what lies behind it
            from -= max((lane >> 4) + 1 - last_scales, 0);
        slot_a_scales(fa, at, from, a, s);
        if (low)
            mfmas8(a, b0, s.v[0], w, acc[0][0]);
        slot_end();
        B.load(cur + 2 * kHalfBytes, 0, t + 2, nk, wave);
        slot_b<3>(fb, at, b1);
        if (low)
            mfmas8(a, b1, s.v[0], w, acc[0][1]);
        slot_end();
        A.load(cur, 0, t + 2, nk, wave);
        if ((t & 3) == 0 && t + 4 < nk)
            load_scales(stages, (t >> 2) + 1);
        if (high) {
            slot_a<1>(fa, at, a);
            mfmas8(a, b1, s.v[1], w, acc[1][1]);
        } else {
            wait_loads<10>();
            slot_end();
        }
        slot_end();
        B.load(cur + 3 * kHalfBytes, 1, t + 2, nk, wave);
        slot_b<2>(fb, then, next);
        if (high)
            mfmas8(a, b0, s.v[1], w, acc[1][0]);
        slot_end();
    }

    __device__ __forceinline__ void run8(uint8_t *lds, int nk, Acc &acc) const
    {
#pragma unroll
        for (int q = 0; q < 16; ++q)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[q >> 3][(q >> 2) & 1][q & 3][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        uint8_t *s0 = lds, *s1 = lds + kStageBytes, *stages = lds + kGemmLdsBytes;
        float w0[2] = {load_uniform(ws[0]), load_uniform(ws[1])}, w1[2];
        wait_loads<10>();
        slot_end();
        FragB b0, b1;
        slot_b<2>(fb, lds_offset(s0), b0);
        if (wm)  // the second group of waves starts half a phase later
            slot_end();
        int t = 0;
        for (; t + 1 < nk; t += 2) {
            ktile8(s0, s1, stages, t, nk, b0, b1, w0, w1, acc);
            ktile8(s1, s0, stages, t + 1, nk, b1, b0, w1, w0, acc);
        }
        if (t < nk)
            ktile8(s0, s1, stages, t, nk, b0, b1, w0, w1, acc);
        if (!wm)
            slot_end();
    }
};

template <bool GRAD, bool GATED, int ACT>
__global__ __launch_bounds__(kGemmThreads, 2) void product_fp8_kernel(Product8Args p)
{
    constexpr bool PAIR = GATED && !GRAD;
    constexpr int kCols = PAIR ? kTile / 2 : kTile;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kGemmLdsBytes + 2 * kScaleStage];
    __shared__ int32_t first[kMaxLocalExperts + 1];
    const int32_t row_tiles = plan_row_tiles<kGemmThreads, kTile>(p.off, p.El, p.max_rows, first);
    const uint32_t nct = (uint32_t)(p.N + kCols - 1) / kCols;
    const int64_t wide = PAIR ? 2 * (int64_t)p.N : p.N;
    const int nk = (p.K + kTileK8 - 1) / kTileK8;
    const int64_t nbw = (wide + 127) / 128;
    Gemm8 gemm;
    gemm.init_lane();
    // tiles and the slices of a last round as in product.hip
    const uint32_t slot = gridDim.x % 8 ? blockIdx.x : blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
    const uint32_t tiles = row_tiles * nct, rest = tiles % gridDim.x, whole = tiles - rest;
    const uint32_t slices = rest * 4 <= gridDim.x ? 4 : (rest * 2 <= gridDim.x ? 2 : 1);
    for (uint32_t u = slot; u < whole + rest * slices; u += gridDim.x) {
        const uint32_t tile = u < whole ? u : whole + (u - whole) / slices;
        const int32_t slice = u < whole ? 0 : (int32_t)((u - whole) % slices);
        const int32_t most = u < whole ? kTile : kTile / (int32_t)slices;
        const TileAt which = tile_at(tile, row_tiles, nct);
        const int32_t rt = which.row, n0 = which.col * kCols;
        const int32_t l = __builtin_amdgcn_readfirstlane(tile_expert(first, p.El, rt));
        const Rows r = expert_rows(p.off, l, p.max_rows);
        const int64_t at = r.begin + (int64_t)(rt - first[l]) * kTile + slice * most;
        if (at >= r.end)
            continue;  // a slice past the last row
        const int32_t row0 = __builtin_amdgcn_readfirstlane((int32_t)at);
        const int32_t rows = __builtin_amdgcn_readfirstlane((int32_t)min((int64_t)most, r.end - at));
        const uint8_t *a = p.a + row0 * p.a_bytes;
        const uint16_t *Wl = reinterpret_cast<const uint16_t *>(p.W + l * wide * p.K);  // in pairs of codes, as below
        const int32_t K2 = p.K / 2;
        gemm.A.init(reinterpret_cast<const uint16_t *>(a), rows, K2, (int32_t)(p.a_bytes / 2), gemm.wave, gemm.lane, 128,
                    [](int j) { return j * 8; });
        gemm.init_scales(a, rows, p.K, p.a_bytes);
        const float *ws = p.scale + l * nbw * nk;
        // columns past the last have no scale of their own: theirs multiplies zeros
        if constexpr (PAIR) {
            const bool up = (gemm.wave >> 1) & 1;
            gemm.B.init(Wl + ((up ? (int64_t)p.N : 0) + n0) * K2, p.N - n0, K2, K2, gemm.wave, gemm.lane, 16,
                        [](int j) { return (j >> 2) * 32 + (j & 1) * 8; });
            const int64_t c = min(n0 + gemm.wn * 32, p.N - 32);
            gemm.ws[0] = ws + c / 128 * nk;
            gemm.ws[1] = ws + (p.N + c) / 128 * nk;
        } else {
            gemm.B.init(Wl + (int64_t)n0 * K2, p.N - n0, K2, K2, gemm.wave, gemm.lane, 32,
                        [](int j) { return (j >> 2) * 64 + (j & 3) * 8; });
            gemm.ws[0] = gemm.ws[1] = ws + min((int64_t)(n0 + gemm.wn * 64) / 128, nbw - 1) * nk;
        }
        Acc acc;
        gemm.set_rows(rows);
        gemm.load_scales(lds + kGemmLdsBytes, 0);
        gemm.start(lds, nk);
        gemm.run8(lds, nk, acc);
        epilogue<GRAD, GATED, ACT, true>(p, gemm, acc, l, row0, rows, n0);
        const int32_t width = GATED && GRAD ? 2 * p.N : p.N;
        if (p.out8 && n0 + kCols >= p.N)
            pad_rows<kGemmThreads>(p.out8 + row0 * p.out8_bytes, rows, width, p.out8_bytes);
        wait_loads<0>();
        slot_end();
    }
}

// Whether the kernel for few rows is the faster one, as for bf16.
bool few_rows(int64_t max_rows, int32_t El, int32_t K, int64_t col_tiles)
{
    const int64_t tiles = (max_rows < El ? max_rows : El) * col_tiles;
    if (tiles < 256)
        return max_rows <= 20 * (int64_t)El;
    return K < 4096 && max_rows <= 16 * (int64_t)El;
}

template <bool GRAD>
hipError_t launch(const Product8Args &p, int32_t act, bool gated, hipStream_t stream)
{
    int cus = 0;
    const hipError_t err = current_cus(&cus);
    if (err != hipSuccess)
        return err;
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

}  // namespace

hipError_t launch_product_fp8(const Product8Args &p, int32_t act, bool gated, bool grad, hipStream_t stream)
{
    if (!grad && few_rows(p.max_rows, p.El, p.K, (p.N + (gated ? kTile / 2 : kTile) - 1) / (gated ? kTile / 2 : kTile)))
        return launch_product_fp8_few(p, act, gated, stream);
    return grad ? launch<true>(p, act, gated, stream) : launch<false>(p, act, gated, stream);
}

}  // namespace moe
