// product_wgrad.hip -- the gradients of the experts' weights and biases:
// grad_W[l] = grad_y[rows of l]^T x[rows of l], summed over the rows in
// float32. Both operands are K-strided (K is the rows); product_gemm.hpp has
// the K loop.
//
// Split. A tile is 256 x 256 of one expert's grad_W. With few tiles for the
// CUs, or a last round that would leave many idle, each expert's rows are cut
// into S pieces, whose float32 sums go to the workspace and are added in
// ascending order by a second kernel: the result does not depend on which
// block computed what. S comes from the sizes the host knows (plan()). Blocks
// take the pieces of the experts with the most rows first, in alternating
// direction from round to round, which evens out ragged experts: with 8
// experts of 25,000 to 60,000 rows and three rounds, blocks' shares differ by
// a few percent.
#include "product_epilogue.hpp"
#include "product_gemm.hpp"

namespace moe {
namespace {

constexpr int kPlanCUs = 256;  // MI355X; the plan, hence the result, is the same on any device
constexpr int kMaxSplit = 16;
constexpr int64_t kMaxPieces = 4096;  // of a split: 1 GiB of partial sums
constexpr int64_t kTileFloats = kTile * kTile;

struct WgradPlan {
    int64_t no, nh, tiles;  // tiles of O, of H, and of all experts
    int32_t S;              // pieces of an expert's rows
};

// S minimises an estimate of the time in K-tiles (1.5 us each on MI355X): the
// rounds of blocks, with 6 K-tiles for a tile's start and end, and for S > 1
// the partial sums' way to memory and back, 512 KiB a tile (0.07), and the
// second launch.
WgradPlan plan(int32_t El, int64_t max_rows, int32_t O, int32_t H)
{
    WgradPlan p;
    p.no = (O + kTile - 1) / kTile;
    p.nh = (H + kTile - 1) / kTile;
    p.tiles = El * p.no * p.nh;
    const double nk = (double)max_rows / kTileK / El;
    double best = 0;
    p.S = 1;
    for (int32_t s = 1; s <= kMaxSplit && (s == 1 || (nk >= 4 * s && p.tiles * s <= kMaxPieces)); ++s) {
        const int64_t rounds = (p.tiles * s + kPlanCUs - 1) / kPlanCUs;
        const double t = rounds * (nk / s + 6) + (s > 1 ? 0.07 * p.tiles * s + 4 : 0);
        if (s == 1 || t < best) {
            best = t;
            p.S = s;
        }
    }
    return p;
}

size_t partial_bytes(const WgradPlan &p) { return p.S > 1 ? (size_t)(p.tiles * p.S * kTileFloats * 4) : 0; }

struct WgradArgs {
    const uint16_t *gy, *x;
    const int32_t *off;
    void *gW;
    float *gb;       // NULL: no bias gradient
    float *partial;  // [El][S][tile][kTileFloats] in accumulator order
    float *partial_gb;  // [El][S][O]
    int32_t El, max_rows, O, H, S;
};

// Two groups of four float columns, 16 columns apart, of rows r = L % 16: a
// becomes rows 0-7 (lanes with r < 8 the first group of row r, the others the
// second of row r - 8), b rows 8-15 in the same way.
__device__ __forceinline__ void to_lines(f32x4 &a, f32x4 &b)
{
    constexpr int kRowRor8 = 0x128;  // lane i of 16 <- lane i ^ 8
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t x = __float_as_uint(a[e]), y = __float_as_uint(b[e]);
        // lanes 8-15 of a take b of the lane eight below, lanes 0-7 of b take a of the lane eight above
        const uint32_t p = (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)y, kRowRor8, 0xF, 0xC, false);
        const uint32_t q = (uint32_t)__builtin_amdgcn_update_dpp((int)y, (int)x, kRowRor8, 0xF, 0x3, false);
        a[e] = __uint_as_float(p);
        b[e] = __uint_as_float(q);
    }
}

// One tile to grad_W. Rows of 16 columns of O lie across the lanes.
template <bool FP32, bool ACCUMULATE, class G>
__device__ __forceinline__ void write_tile(const WgradArgs &p, const G &gemm, const Acc &acc, int32_t l, int32_t o0,
                                           int32_t h0)
{
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t o = o0 + ha * 128 + gemm.wm * 64 + i * 16 + (gemm.lane & 15);
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
                const int64_t at = ((int64_t)l * p.O + o) * p.H + h0 + gemm.column(hb);
                const int32_t left = p.H - h0 - gemm.column(hb), c4 = (gemm.lane >> 4) * 4;
                if (FP32) {
                    // Whole 128-byte lines, rows 0-7 of the 16 in one access and 8-15 in
                    // the other, written past the caches: 131 us against 138 for the
                    // lanes' own pieces of 64 bytes (6 x 1536 x 7168, 4093 rows), and
                    // 148 for those written past the caches.
                    f32x4 v[2] = {acc[ha][hb][i][0], acc[ha][hb][i][1]};
                    to_lines(v[0], v[1]);
                    const int32_t r8 = gemm.lane & 7, c = (gemm.lane & 8) * 2 + c4;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int32_t row = o - (gemm.lane & 15) + j * 8 + r8;
                        if (row >= p.O || c >= left)
                            continue;
                        f32x4 *q = reinterpret_cast<f32x4 *>(
                            static_cast<float *>(p.gW) + ((int64_t)l * p.O + row) * p.H + h0 + gemm.column(hb) + c);
                        if (ACCUMULATE)
                            v[j] += *q;
                        __builtin_nontemporal_store(v[j], q);
                    }
                } else {
                    const u32x4 v = to_rows(narrow(acc[ha][hb][i][0]), narrow(acc[ha][hb][i][1]));
                    if (o < p.O && c4 * 2 < left)
                        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.gW) + at + c4 * 2) = v;
                }
            }
        }
}

// The bias gradients of a tile's 256 columns, from the sums of grad_y that the
// blocks of the first column of tiles make: grad_y's K-tile is in their
// registers anyway, so 2 MFMAs in 18 cost them 6% and the other tiles nothing
// (a kernel of its own, at the least, reads grad_y again).
template <class G>
__device__ __forceinline__ void write_bias(const G &gemm, const f32x4 (&sum)[2], float *q, int32_t o0, int32_t O,
                                           bool accumulate)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int32_t o = o0 + h * 128 + gemm.wm * 64 + gemm.wn * 16 + gemm.lane;
        if (gemm.lane < 16 && o < O)
            q[o] = accumulate ? q[o] + sum[h][0] : sum[h][0];
    }
}

// accumulator fragment n of this lane within a partial tile
__device__ __forceinline__ int64_t frag_at(int n, int wave, int lane) { return ((int64_t)(wave * 32 + n) * kWave + lane) * 4; }

template <bool FP32, bool ACCUMULATE, bool SPLIT, bool BIAS>
__global__ __launch_bounds__(kGemmThreads, 2) void wgrad_kernel(WgradArgs p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kGemmLdsBytes];
    __shared__ uint16_t by_rows[kMaxLocalExperts];  // experts, most rows first
    const uint32_t nh = (uint32_t)(p.H + kTile - 1) / kTile, no = (uint32_t)(p.O + kTile - 1) / kTile, tp = no * nh;
    const uint32_t units = p.El * (SPLIT ? p.S : 1) * tp;
    const bool sorted = units > gridDim.x;
    if (sorted) {
        // rank by counting, from row counts staged where the tiles will lie
        int32_t *n = reinterpret_cast<int32_t *>(lds);
        for (int32_t l = threadIdx.x; l < p.El; l += kGemmThreads) {
            const Rows r = expert_rows(p.off, l, p.max_rows);
            n[l] = r.end - r.begin;
        }
        __syncthreads();
        for (int32_t l = threadIdx.x; l < p.El; l += kGemmThreads) {
            const int32_t mine = n[l];
            int32_t rank = 0;
            for (int32_t q = 0; q < p.El; ++q)
                rank += n[q] > mine || (n[q] == mine && q < l);
            by_rows[rank] = (uint16_t)l;
        }
        __syncthreads();
    }
    Gemm<true, true> gemm;
    gemm.init_lane();
    const uint32_t slot = gridDim.x % 8 ? blockIdx.x : blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
    // One unit: a tile's piece s of expert l's rows.
    struct Unit {
        uint32_t tile;
        int32_t l, s, o0, h0, nk;
    } next = {0, 0, 0, 0, 0, 0};
    uint32_t round = 0;
    // Finds this block's next unit, points the operands at it and starts its
    // first loads; false when there is none.
    auto begin = [&]() -> bool {
        for (; round * gridDim.x < units; ++round) {
            const uint32_t u = round * gridDim.x + (round & 1 ? gridDim.x - 1 - slot : slot);
            if (u >= units)
                continue;
            const uint32_t piece = u / tp;
            next.tile = u - piece * tp;
            const TileAt which = tile_at(next.tile, no, nh);
            next.o0 = which.row * kTile;
            next.h0 = which.col * kTile;
            const int32_t e = (int32_t)(SPLIT ? piece / p.S : piece);
            next.s = SPLIT ? __builtin_amdgcn_readfirstlane((int32_t)(piece % p.S)) : 0;
            next.l = __builtin_amdgcn_readfirstlane(sorted ? by_rows[e] : e);
            const Rows r = expert_rows(p.off, next.l, p.max_rows);
            const int32_t rows = __builtin_amdgcn_readfirstlane(r.end - r.begin);
            const int64_t all = (rows + (int64_t)kTileK - 1) / kTileK;
            const int64_t t0 = SPLIT ? all * next.s / p.S : 0, t1 = SPLIT ? all * (next.s + 1) / p.S : all;
            next.nk = (int)(t1 - t0);
            if (SPLIT && next.nk == 0)
                continue;
            const int64_t first = __builtin_amdgcn_readfirstlane(r.begin) + t0 * kTileK;
            const int64_t n = min(rows - t0 * kTileK, next.nk * (int64_t)kTileK);
            gemm.A.init_strided(p.gy + first * p.O + next.o0, n, p.O, p.O - next.o0, gemm.wave, gemm.lane);
            gemm.B.init_strided(p.x + first * p.H + next.h0, n, p.H, p.H - next.h0, gemm.wave, gemm.lane);
            gemm.set_rows(p.O - next.o0);
            gemm.start(lds, next.nk);
            ++round;
            return true;
        }
        return false;
    };
    bool more = begin();
    while (more) {
        const Unit u = next;
        Acc acc;
        f32x4 sum[2];
        gemm.template run<BIAS>(lds, u.nk, acc, sum, u.h0 == 0);
        // the next unit's first loads run under this one's stores
        more = begin();
        if (BIAS && u.h0 == 0)
            write_bias(gemm, sum, SPLIT ? p.partial_gb + ((int64_t)u.l * p.S + u.s) * p.O : p.gb + (int64_t)u.l * p.O,
                       u.o0, p.O, !SPLIT && ACCUMULATE);
        if (SPLIT) {
            float *q = p.partial + (((int64_t)u.l * p.S + u.s) * tp + u.tile) * kTileFloats;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                *reinterpret_cast<f32x4 *>(q + frag_at(i, gemm.wave, gemm.lane)) =
                    acc[i >> 4][(i >> 3) & 1][(i >> 1) & 3][i & 1];
        } else {
            write_tile<FP32, ACCUMULATE>(p, gemm, acc, u.l, u.o0, u.h0);
        }
    }
    // loads past the last K-tile may still be on their way into LDS
    wait_loads<0>();
}

// The pieces of one tile, added in ascending order.
template <bool FP32, bool ACCUMULATE>
__global__ __launch_bounds__(kGemmThreads, 2) void join_kernel(WgradArgs p)
{
    const uint32_t nh = (uint32_t)(p.H + kTile - 1) / kTile, no = (uint32_t)(p.O + kTile - 1) / kTile, tp = no * nh;
    Gemm<true, true> gemm;
    gemm.init_lane();
    const int32_t l = (int32_t)(blockIdx.x / tp);
    const uint32_t tile = blockIdx.x % tp;
    const Rows r = expert_rows(p.off, l, p.max_rows);
    const int64_t all = ((int64_t)r.end - r.begin + kTileK - 1) / kTileK;
    Acc acc;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        acc[i >> 4][(i >> 3) & 1][(i >> 1) & 3][i & 1] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int32_t s = 0; s < p.S; ++s) {
        if (all * s / p.S == all * (s + 1) / p.S)
            continue;
        const float *q = p.partial + (((int64_t)l * p.S + s) * tp + tile) * kTileFloats;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            acc[i >> 4][(i >> 3) & 1][(i >> 1) & 3][i & 1] +=
                __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(q + frag_at(i, gemm.wave, gemm.lane)));
    }
    const TileAt which = tile_at(tile, no, nh);
    const int32_t o0 = which.row * kTile;
    write_tile<FP32, ACCUMULATE>(p, gemm, acc, l, o0, which.col * kTile);
    if (!p.gb || which.col != 0 || threadIdx.x >= kTile || o0 + (int32_t)threadIdx.x >= p.O)
        return;
    const int32_t o = o0 + threadIdx.x;
    float b = 0.f;
    for (int32_t s = 0; s < p.S; ++s)
        if (all * s / p.S != all * (s + 1) / p.S)
            b += p.partial_gb[((int64_t)l * p.S + s) * p.O + o];
    float *q = p.gb + (int64_t)l * p.O + o;
    *q = ACCUMULATE ? *q + b : b;
}

}  // namespace

size_t wgrad_workspace_bytes(int32_t El, int64_t max_rows, int32_t O, int32_t H)
{
    const WgradPlan p = plan(El, max_rows, O, H);
    return p.S > 1 ? partial_bytes(p) + (size_t)El * p.S * O * sizeof(float) : 0;
}

hipError_t launch_expert_wgrad(const uint16_t *grad_y, const uint16_t *x, const int32_t *off,
                               int32_t El, int64_t max_rows, int32_t O, int32_t H, bool fp32,
                               bool accumulate, void *grad_W, float *grad_bias, void *workspace,
                               hipStream_t stream)
{
    int cus = 0;
    hipError_t err = current_cus(&cus);
    if (err != hipSuccess)
        return err;
    const WgradPlan plan_ = plan(El, max_rows, O, H);
    const int64_t units = plan_.tiles * plan_.S;
    const dim3 grid((unsigned)(units < cus ? units : cus)), block(kGemmThreads);
    const WgradArgs p = {grad_y, x, off, grad_W, grad_bias, static_cast<float *>(workspace),
                         reinterpret_cast<float *>(static_cast<char *>(workspace) + partial_bytes(plan_)),
                         El, (int32_t)max_rows, O, H, plan_.S};
#define MOE_WGRAD_LAUNCH(F, A, S)                                                              \
    do {                                                                                       \
        if (grad_bias)                                                                         \
            hipLaunchKernelGGL((wgrad_kernel<F, A, S, true>), grid, block, 0, stream, p);      \
        else                                                                                   \
            hipLaunchKernelGGL((wgrad_kernel<F, A, S, false>), grid, block, 0, stream, p);     \
    } while (0)
    if (plan_.S > 1) {
        MOE_WGRAD_LAUNCH(true, false, true);
        if ((err = hipGetLastError()) != hipSuccess)
            return err;
        const dim3 joins((unsigned)plan_.tiles);
        if (accumulate)
            hipLaunchKernelGGL((join_kernel<true, true>), joins, block, 0, stream, p);
        else if (fp32)
            hipLaunchKernelGGL((join_kernel<true, false>), joins, block, 0, stream, p);
        else
            hipLaunchKernelGGL((join_kernel<false, false>), joins, block, 0, stream, p);
    } else if (accumulate) {
        MOE_WGRAD_LAUNCH(true, true, false);
    } else if (fp32) {
        MOE_WGRAD_LAUNCH(true, false, false);
    } else {
        MOE_WGRAD_LAUNCH(false, false, false);
    }
#undef MOE_WGRAD_LAUNCH
    return hipGetLastError();
}

}  // namespace moe
