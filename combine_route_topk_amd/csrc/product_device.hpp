// product_device.hpp -- what the experts' products and their gradients share:
// the row tiles of an expert-major buffer, and the activations.
#pragma once

#include "device.hpp"
#include "launch.hpp"

namespace moe {
namespace {

// Expert l's rows, kept inside [0, max_rows] whatever the offsets hold.
struct Rows {
    int32_t begin, end;
};
__device__ __forceinline__ Rows expert_rows(const int32_t *__restrict__ off, int32_t l, int32_t max_rows)
{
    Rows r;
    r.begin = min(max(off[l], 0), max_rows);
    r.end = min(max(off[l + 1], r.begin), max_rows);
    return r;
}

// first[l] = row tiles of BM rows before expert l, for l <= El (El <= 1024);
// returns their total, or 0 where the offsets decrease (otherwise the experts'
// rows are disjoint, and the total at most max_rows / BM + El). Every thread of the block takes part; `first` is in
// LDS and ready after the call. One pass over at most 1025 offsets by the
// block itself costs a launch less than a table written by another kernel.
template <int THREADS, int BM>
__device__ int32_t plan_row_tiles(const int32_t *__restrict__ off, int32_t El, int32_t max_rows,
                                  int32_t *first)
{
    constexpr int PER = (kMaxLocalExperts + THREADS - 1) / THREADS;
    constexpr int WAVES = THREADS / kWave;
    __shared__ int32_t wave_total[WAVES];
    __shared__ bool wave_bad[WAVES];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave;
    int32_t n[PER], part = 0;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int l = tid * PER + u;
        n[u] = 0;
        if (l < El) {
            const Rows r = expert_rows(off, l, max_rows);
            n[u] = (int32_t)(((int64_t)r.end - r.begin + BM - 1) / BM);
            bad |= off[l + 1] < off[l];
        }
        part += n[u];
    }
    const int32_t inc = wave_inclusive_sum(part);
    const uint64_t any_bad = ballot64(bad);
    if (lane == kWave - 1) {
        wave_total[w] = inc;
        wave_bad[w] = any_bad != 0;
    }
    __syncthreads();
    int32_t run = inc - part, all = 0;
#pragma unroll
    for (int u = 0; u < WAVES; ++u) {
        run += u < w ? wave_total[u] : 0;
        all += wave_total[u];
    }
    bad = false;
#pragma unroll
    for (int u = 0; u < WAVES; ++u)
        bad |= wave_bad[u];
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int l = tid * PER + u;
        if (l < El)
            first[l] = run;
        run += n[u];
    }
    if (tid == 0)
        first[El] = all;
    __syncthreads();
    return bad ? 0 : all;
}

// the expert whose tiles hold tile t: the largest l with first[l] <= t
__device__ __forceinline__ int32_t tile_expert(const int32_t *first, int32_t El, int32_t t)
{
    int32_t lo = 0, hi = El - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (first[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Row and column of tile t in a rows x cols grid of tiles. Wide grids are
// walked four rows at a time, so that the 32 consecutive tiles of an XCD are
// about four by eight and share their operands in its L2: 114 against 118 us
// for 16 x 28 tiles (4093 x 2048 by 7168, bias and residual), 733 against 783 us
// for 32 x 32 (8192 cubed).
struct TileAt {
    int32_t row, col;
};
// Tile numbers fit 32 bits with room: no memory holds the rows or weights of
// 2^31 tiles of 256 by 128. (64-bit quotients took 1.3 us a tile.)
__device__ __forceinline__ TileAt tile_at(uint32_t t, uint32_t rows, uint32_t cols)
{
    uint32_t r = t / cols, c = t - r * cols;
    if (cols > 8) {
        const uint32_t r0 = t / (4 * cols) * 4, in = t - r0 * cols, n = min(4u, rows - r0);
        c = in / n;
        r = r0 + in - c * n;
    }
    // the same in every lane; saying so keeps what follows, buffer descriptors
    // above all, in scalar registers (the quotient's vector arithmetic would
    // put a loop around every load)
    return {__builtin_amdgcn_readfirstlane((int32_t)r), __builtin_amdgcn_readfirstlane((int32_t)c)};
}

// act(z) in float32, ACT a moe_act value. Arguments of the
// exponentials are bounded where a product with an overflowed factor would
// give NaN: beyond |z| = 30 both GELUs' cdf and derivative are 0 or 1 in
// float32, and SiLU's are once |z| > 104.
enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// 2^x and 1 / x by the hardware's instructions, each within a step or two of
// float32: an activation's value is rounded to bf16 next, 2^16 times coarser.
// Where exp(-z) overflows the quotient is 0, which misses at most 2^-126.
__device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kSqrt2OverPi = 0.79788456080286536f;
constexpr float kGeluCubic = 0.044715f;

// z within [-30, 30]; NaN stays NaN (a minimum and maximum alone would drop it)
__device__ __forceinline__ float within_30(float z) { return z != z ? z : fminf(fmaxf(z, -30.f), 30.f); }

// with u = sqrt(2 / pi) (z + c z^3), (1 + tanh u) / 2 = sigmoid(2 u)
__device__ __forceinline__ float gelu_tanh_cdf(float z)
{
    const float b = fminf(fmaxf(z, -30.f), 30.f);
    return sigmoid(2.f * kSqrt2OverPi * (b + kGeluCubic * b * b * b));
}

template <int ACT>
__device__ __forceinline__ float act(float z)
{
    switch (ACT) {
    case kActRelu: return z > 0.f ? z : (z != z ? z : 0.f);
    case kActSilu: return z * sigmoid(z);
    case kActGelu: return 0.5f * z * erfcf(-z * kSqrtHalf);
    case kActGeluTanh: return z * gelu_tanh_cdf(z);
    default: return z;
    }
}

// act(z) and act'(z) together: they share their exponential.
template <int ACT>
__device__ __forceinline__ void act_and_grad(float z, float &f, float &df)
{
    switch (ACT) {
    case kActRelu:
        f = act<ACT>(z);
        df = z > 0.f ? 1.f : (z != z ? z : 0.f);
        return;
    case kActSilu: {
        const float p = sigmoid(z);
        f = z * p;
        df = p * (1.f + fminf(fmaxf(z, -104.f), 104.f) * (1.f - p));
        return;
    }
    case kActGelu: {
        const float b = within_30(z), cdf = 0.5f * erfcf(-b * kSqrtHalf);
        f = z * cdf;
        df = cdf + b * __builtin_amdgcn_exp2f(-0.72134752044448170f * b * b) * kInvSqrt2Pi;
        return;
    }
    case kActGeluTanh: {
        const float b = within_30(z), p = gelu_tanh_cdf(b);
        f = z * p;
        df = p + 2.f * b * p * (1.f - p) * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * b * b);
        return;
    }
    default:
        f = z;
        df = 1.f;
    }
}

}  // namespace
}  // namespace moe
