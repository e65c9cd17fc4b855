// product.hip -- the experts' products on expert-major rows and the gradient
// with respect to their input, with bias, activation, gate and residual (or
// the activation's gradient) applied to the float32 sums before the one
// rounding to bf16.
//
// A persistent block per CU takes tiles of 256 rows of one expert by 256
// columns (gated: 128 gate columns and the 128 columns they gate, laid out
// so that a lane holds both); product_gemm.hpp has the K loop.
#include "product_epilogue.hpp"
#include "product_gemm.hpp"

namespace moe {
namespace {

// Bias, activation, gate, residual (or the activation's gradient) on the
// sums, and their one rounding. A group of 16 rows past the tile's last is
// skipped; the rest is without branches: the descriptors drop rows and
// columns outside.
template <bool GRAD, bool GATED, int ACT, class G>
__device__ __forceinline__ void epilogue(const ProductArgs &p, const G &gemm, const Acc &acc, int32_t l,
                                         int32_t row0, int32_t rows, int32_t n0)
{
    constexpr bool PAIR = GATED && !GRAD;
    constexpr int NP = PAIR ? 1 : 2;  // pairs of a lane's groups of four columns
    const int64_t N = p.N, wide = GATED ? 2 * N : N;
    const uint32_t N2 = (uint32_t)N * 2;
    uint32_t col[NP];
    f32x4 b[NP][2], bu[NP][2];
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        const int32_t c0 = n0 + (PAIR ? gemm.wn * 32 : gemm.column(q));
        const int32_t c8 = c0 + (gemm.lane >> 4) * 8;
        col[q] = c8 < N ? (uint32_t)c8 * 2 : kOutside;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int32_t c4 = c0 + j * 16 + (gemm.lane >> 4) * 4;
            b[q][j] = bu[q][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (!GRAD && p.bias && c4 < N) {
                b[q][j] = widen(*reinterpret_cast<const u32x2 *>(p.bias + l * wide + c4));
                if (PAIR)
                    bu[q][j] = widen(*reinterpret_cast<const u32x2 *>(p.bias + l * wide + N + c4));
            }
        }
    }
    TileRows out, aux;
    out.init(p.out, row0, rows, GRAD ? wide : N, gemm.lane);
    if (GRAD) {
        if (p.pre_in)
            aux.init(p.pre_in, row0, rows, wide, gemm.lane);
    } else if (p.residual) {
        aux.init(p.residual, row0, rows, N, gemm.lane);
    }
    TileRows pre;
    if (!GRAD && p.pre_out)
        pre.init(p.pre_out, row0, rows, wide, gemm.lane);
    // What a group of 16 rows reads (pre, or the residual) is fetched while the
    // group before it is computed: a wave has only one other on its SIMD to
    // hide that latency.
    constexpr int NF = GRAD && GATED ? 2 : 1;
    const bool reads = GRAD ? (GATED || p.pre_in) : p.residual != nullptr;
    u32x4 ahead[2][NP][NF];
    auto row_of = [&](int s) { return (s >> 2) * 128 + gemm.wm * 64 + (s & 3) * 16; };
    auto fetch = [&](int s) {
#pragma unroll
        for (int q = 0; q < NP; ++q)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                ahead[s & 1][q][f] = aux.fetch(row_of(s), col[q], f * N2);
    };
    if (reads)
        fetch(0);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
        const int h = s >> 2, i = s & 3;
        if (reads && s < 7)
            fetch(s + 1);
        const int32_t m = row_of(s);
        if (m >= rows)
            continue;
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            f32x4 v[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                v[j] = PAIR ? acc[h][j][i][0] : acc[h][q][i][j];
            if (GRAD && GATED) {
                f32x4 z[2], u[2], dz[2], du[2];
                TileRows::unpack(ahead[s & 1][q][0], z);
                TileRows::unpack(ahead[s & 1][q][NF - 1], u);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float f, df;
                        act_and_grad<ACT>(z[j][e], f, df);
                        dz[j][e] = v[j][e] * u[j][e] * df;
                        du[j][e] = v[j][e] * f;
                    }
                out.store(m, col[q], dz);
                out.store(m, col[q], du, N2);
            } else if (GRAD) {
                if (p.pre_in) {
                    f32x4 z[2];
                    TileRows::unpack(ahead[s & 1][q][0], z);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float f, df;
                            act_and_grad<ACT>(z[j][e], f, df);
                            v[j][e] *= df;
                        }
                }
                out.store(m, col[q], v);
            } else {
                f32x4 g[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    v[j] += b[q][j];
                    g[j] = PAIR ? acc[h][j][i][1] + bu[q][j] : f32x4{};
                }
                if (p.pre_out) {
                    pre.store(m, col[q], v);
                    if (PAIR)
                        pre.store(m, col[q], g, N2);
                }
                f32x4 r[2] = {};
                if (p.residual)
                    TileRows::unpack(ahead[s & 1][q][0], r);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[j][e] = (PAIR ? act<ACT>(v[j][e]) * g[j][e] : act<ACT>(v[j][e])) + r[j][e];
                out.store(m, col[q], v);
            }
        }
    }
}

template <bool GRAD, bool GATED, int ACT>
__global__ __launch_bounds__(kGemmThreads, 2) void product_kernel(ProductArgs p)
{
    constexpr bool PAIR = GATED && !GRAD;
    constexpr int kCols = PAIR ? kTile / 2 : kTile;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kGemmLdsBytes];
    __shared__ int32_t first[kMaxLocalExperts + 1];
    const int32_t row_tiles = plan_row_tiles<kGemmThreads, kTile>(p.off, p.El, p.max_rows, first);
    const uint32_t nct = (uint32_t)(p.N + kCols - 1) / kCols;
    const int64_t wide = PAIR ? 2 * (int64_t)p.N : p.N;
    const int nk = (p.K + kTileK - 1) / kTileK;
    Gemm<false, GRAD> gemm;
    gemm.init_lane();
    // each XCD (blockIdx % 8) takes runs of consecutive tiles
    const uint32_t slot = gridDim.x % 8 ? blockIdx.x : blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
    // A last round that would leave half the blocks or more idle takes its
    // tiles in two or four slices of rows, one for each block.
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
        gemm.A.init(p.a + (int64_t)row0 * p.K, rows, p.K, gemm.wave, gemm.lane, 128, [](int j) { return j * 8; });
        const uint16_t *Wl = p.W + (int64_t)l * wide * p.K;
        if constexpr (GRAD) {
            gemm.B.init_strided(Wl + n0, p.K, p.N, p.N - n0, gemm.wave, gemm.lane);
        } else if constexpr (GATED) {
            // rows of a half: for each wave's 32 columns, 16 gate then 16 up
            const bool up = (gemm.wave >> 1) & 1;
            gemm.B.init(Wl + ((up ? (int64_t)p.N : 0) + n0) * p.K, p.N - n0, p.K, gemm.wave, gemm.lane, 16,
                        [](int j) { return (j >> 2) * 32 + (j & 1) * 8; });
        } else {
            gemm.B.init(Wl + (int64_t)n0 * p.K, p.N - n0, p.K, gemm.wave, gemm.lane, 32,
                        [](int j) { return (j >> 2) * 64 + (j & 3) * 8; });
        }
        Acc acc;
        gemm.set_rows(rows);
        gemm.start(lds, nk);
        gemm.run(lds, nk, acc);
        epilogue<GRAD, GATED, ACT>(p, gemm, acc, l, row0, rows, n0);
        // (Starting the next tile's loads ahead of the epilogue spilled registers
        // and took 1.87 against 1.71 ms: 327680 x 2048 by 2 x 768, gated.)
        wait_loads<0>();
        slot_end();
    }
}


// Whether the kernel for few rows is the faster one, by the average rows of an
// expert. The host knows max_rows, not the rows there are: a buffer sized for
// the worst case takes the tiles however few of its rows are used, at the cost
// that the figures show for few rows. On MI355X, in us, few against tiles:
//   too few tiles for the CUs: 8 experts, 2048 by 2 x 768: 12 against 27 at 1
//   row, 16 / 28 at 32, 25 / 28 at 48; 4 experts, 7168 by 7168: 79 / 105 at
//   1 row, 97 / 107 at 16, 112 / 108 at 24;
//   enough tiles, short K: 64 experts, 2048 by 2048: 103 / 128 at 1 row,
//   124 / 127 at 16, 138 / 127 at 24;
//   enough tiles, long K: 32 experts, 7168 by 2 x 2048: 319 / 307 at 4 rows,
//   355 / 308 at 16 (one row each: 321 / 311).
bool few_rows(int64_t max_rows, int32_t El, int32_t K, int64_t col_tiles)
{
    const int64_t tiles = (max_rows < El ? max_rows : El) * col_tiles;
    if (tiles < 256)
        return max_rows <= 20 * (int64_t)El;
    return K < 4096 && max_rows <= 16 * (int64_t)El;
}

template <bool GRAD>
hipError_t launch(const ProductArgs &p, int32_t act, bool gated, hipStream_t stream)
{
    int cus = 0;
    const hipError_t err = current_cus(&cus);
    if (err != hipSuccess)
        return err;
    const int kCols = gated && !GRAD ? kTile / 2 : kTile;
    // four blocks a tile, for its slices
    const int64_t units = 4 * ((int64_t)p.max_rows / kTile + p.El) * ((p.N + kCols - 1) / kCols);
    const dim3 grid((unsigned)(units < cus ? units : cus));
#define MOE_PRODUCT_LAUNCH(G, A)                                                                 \
    hipLaunchKernelGGL((product_kernel<GRAD, G, A>), grid, dim3(kGemmThreads), 0, stream, p);    \
    return hipGetLastError()
#define MOE_PRODUCT_ACT(A)                \
    case A:                               \
        if (gated) {                      \
            MOE_PRODUCT_LAUNCH(true, A);  \
        } else {                          \
            MOE_PRODUCT_LAUNCH(false, A); \
        }
    switch (act) {
        MOE_PRODUCT_ACT(kActNone)
        MOE_PRODUCT_ACT(kActRelu)
        MOE_PRODUCT_ACT(kActSilu)
        MOE_PRODUCT_ACT(kActGelu)
        MOE_PRODUCT_ACT(kActGeluTanh)
    default:
        return hipErrorInvalidValue;
    }
#undef MOE_PRODUCT_ACT
#undef MOE_PRODUCT_LAUNCH
}

}  // namespace

hipError_t launch_expert_product(const uint16_t *x, const int32_t *off, int32_t El,
                                 int64_t max_rows, int32_t H, int32_t O, const uint16_t *W,
                                 const uint16_t *bias, const uint16_t *residual, int32_t act,
                                 bool gated, uint16_t *pre, uint16_t *y, hipStream_t stream)
{
    const ProductArgs p = {x, off, W, bias, residual, nullptr, pre, y, El, (int32_t)max_rows, H, O};
    if (few_rows(max_rows, El, H, (O + (gated ? kTile / 2 : kTile) - 1) / (gated ? kTile / 2 : kTile)))
        return launch_product_few(p, act, gated, stream);
    return launch<false>(p, act, gated, stream);
}

hipError_t launch_expert_dgrad(const uint16_t *grad_y, const int32_t *off, int32_t El,
                               int64_t max_rows, int32_t O, int32_t H, const uint16_t *W,
                               const uint16_t *pre, int32_t act, bool gated, uint16_t *grad_x,
                               hipStream_t stream)
{
    const ProductArgs p = {grad_y, off, W, nullptr, nullptr, pre, nullptr, grad_x, El, (int32_t)max_rows, O, H};
    return launch<true>(p, act, gated, stream);
}

}  // namespace moe
