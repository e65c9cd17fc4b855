// norm.hip -- the RMS norm in front of a layer, with the residual's addition,
// and its gradient.
//
//   t = round(x + residual);  y = t * rsqrt(mean(t^2) + eps) * weight
//   dt = r (g - t r^2 mean(g t)) + grad_total,  g = grad_y * weight
//   grad_weight = sum over tokens of grad_y t r,  r = rsqrt(mean(t^2) + eps)
//
// Bound by HBM: a row is read once, held in registers across its sum, and
// written once in every form that is asked for (bf16, FP8 rows, the sum).
// The norm is of t as it is stored, so that the gradient, which reads t,
// differentiates the very function that ran; r is recomputed there from the
// row that is in registers anyway.
#include "fp8_device.hpp"
#include "launch.hpp"

namespace moe {
namespace {

// lane 63 ends with the wave's sum; the order is fixed
__device__ __forceinline__ float wave_sum(float v)
{
    auto add = [](float a, uint32_t b) { return a + __uint_as_float(b); };
    v = add(v, dpp::mov<dpp::kQuadSwap1>(__float_as_uint(v), 0u));
    v = add(v, dpp::mov<dpp::kQuadSwap2>(__float_as_uint(v), 0u));
    v = add(v, dpp::mov<dpp::kRowHalfMirror>(__float_as_uint(v), 0u));
    v = add(v, dpp::mov<dpp::kRowMirror>(__float_as_uint(v), 0u));
    v = add(v, dpp::mov<dpp::kRowBcast15, 0xA>(__float_as_uint(v), 0u));
    v = add(v, dpp::mov<dpp::kRowBcast31, 0xC>(__float_as_uint(v), 0u));
    return __uint_as_float(readlane_u32(__float_as_uint(v), kWave - 1));
}

// A lane's eight columns of 512 that a wave takes: neighbours, or (SPLIT) two
// fours 256 apart, so that float32 rows too are read and written as consecutive
// bytes of a wave (8192 x 7168: forward 135 against 154 us, gradient 141 against
// 154).
template <bool SPLIT>
struct Columns {
    static constexpr int kParts = SPLIT ? 2 : 1;
    int32_t first;  // the same in every lane
    uint32_t mine;  // the lane's first, from there
    __device__ __forceinline__ Columns(int32_t first_, int lane) : first(first_), mine(lane * (SPLIT ? 4 : 8)) {}
    __device__ __forceinline__ int32_t start(int k) const { return first + k * 256; }
    __device__ __forceinline__ int32_t at(int k) const { return start(k) + (int32_t)mine; }
    __device__ __forceinline__ bool in(int k, int32_t H) const { return (int32_t)mine < H - start(k); }
};

// Their values as they lie in memory, bf16 or float32; zeros where there is no
// column or row.
template <bool FP32, bool SPLIT>
struct Raw8 {
    static constexpr int kWords = FP32 ? 8 : 4, kPart = kWords / Columns<SPLIT>::kParts;
    typedef uint32_t piece __attribute__((ext_vector_type(kPart < 4 ? kPart : 4)));  // of one load
    static constexpr int kPiece = kPart < 4 ? kPart : 4;
    static constexpr int kSize = FP32 ? 4 : 2;
    uint32_t q[kWords];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            q[i] = 0;
    }
    // part k of columns c of the row that begins at element `row`, the same in every lane
    template <bool STREAM>
    __device__ __forceinline__ void load_as(const void *p, int64_t row, const Columns<SPLIT> &c, int k)
    {
        const piece *s = reinterpret_cast<const piece *>(static_cast<const uint8_t *>(p) + (row + c.start(k)) * kSize +
                                                         c.mine * (uint32_t)kSize);
#pragma unroll
        for (int u = 0; u < kPart / kPiece; ++u) {
            const piece v = STREAM ? __builtin_nontemporal_load(s + u) : s[u];
#pragma unroll
            for (int i = 0; i < kPiece; ++i)
                q[k * kPart + u * kPiece + i] = v[i];
        }
    }
    // rows, each once: past the caches (105 against 113 us, 32768 x 2048 forward)
    __device__ __forceinline__ void load(const void *p, int64_t row, const Columns<SPLIT> &c, int k)
    {
        load_as<true>(p, row, c, k);
    }
    // the weight, for every row
    __device__ __forceinline__ void load_cached(const void *p, const Columns<SPLIT> &c, int k) { load_as<false>(p, 0, c, k); }
    __device__ __forceinline__ void store(void *p, int64_t row, const Columns<SPLIT> &c, int k) const
    {
        piece *s = reinterpret_cast<piece *>(static_cast<uint8_t *>(p) + (row + c.start(k)) * kSize + c.mine * (uint32_t)kSize);
#pragma unroll
        for (int u = 0; u < kPart / kPiece; ++u) {
            piece v;
#pragma unroll
            for (int i = 0; i < kPiece; ++i)
                v[i] = q[k * kPart + u * kPiece + i];
            __builtin_nontemporal_store(v, s + u);
        }
    }
    __device__ __forceinline__ float get(int i) const
    {
        if (FP32)
            return __uint_as_float(q[i % kWords]);
        return i & 1 ? bf16_hi(q[i >> 1]) : bf16_lo(q[i >> 1]);
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            q[i] = FP32 ? __float_as_uint(v[i]) : pack_bf16x2(v[2 * i & 7], v[(2 * i + 1) & 7]);
    }
};

// WPR waves take a row, each lane CH chunks of eight columns; a block of at
// least four waves.
constexpr int norm_threads(int wpr) { return wpr < 4 ? 256 : wpr * kWave; }
constexpr int kScaleLine = 128;  // scale bytes of 4096 values

template <bool FP32, bool WFP32, int WPR, int CH>
__global__ __launch_bounds__(norm_threads(WPR)) void rms_norm_kernel(NormArgs p)
{
    constexpr int kRows = norm_threads(WPR) / kWave / WPR;
    constexpr int kLines = (WPR * CH * 512 + 4095) / 4096;
    // wider rows need the registers: the weight is read when it is used, the
    // residual by a few chunks (float32, 1024 x 40960: 104 us, 213 with many
    // registers spilled; bf16 rows past 32768 columns still spill three)
    constexpr bool kEarly = WPR < 16 || CH <= 2;
    constexpr int kBatch = kEarly ? CH : (FP32 ? 2 : 4);
    __shared__ float part[2][kRows][WPR];
    __shared__ __attribute__((aligned(16))) uint8_t scales[kRows][kLines * kScaleLine];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int slot = wave / WPR, wr = wave % WPR;  // the wave's row of the block, and its place in it
    const int32_t pad = (p.H + 4095) / 4096 * kScaleLine;  // scale bytes of a row
    if (p.y8) {  // padding stays zero: no wave writes it below
        for (int i = threadIdx.x; i < kRows * kLines * kScaleLine / 4; i += norm_threads(WPR))
            reinterpret_cast<uint32_t *>(scales)[i] = 0;
        __syncthreads();
    }
    int parity = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < p.T; t0 += (int64_t)gridDim.x * kRows) {
        const int64_t t = t0 + slot;
        const int32_t H = t < p.T ? p.H : 0;  // no columns in a row past the last
        Raw8<FP32, FP32> h[CH];
        Raw8<WFP32, FP32> w[CH];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Columns<FP32> c((i * WPR + wr) * 512, lane);
            h[i].clear();
            w[i].clear();
#pragma unroll
            for (int k = 0; k < c.kParts; ++k)
                if (c.in(k, H)) {
                    h[i].load(p.x, t * p.H, c, k);
                    if (kEarly)
                        w[i].load_cached(p.weight, c, k);
                }
        }
        if (p.residual) {
#pragma unroll
            for (int first = 0; first < CH; first += kBatch) {
                Raw8<FP32, FP32> r[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const Columns<FP32> c(((first + b) * WPR + wr) * 512, lane);
                    r[b].clear();
#pragma unroll
                    for (int k = 0; k < c.kParts; ++k)
                        if (c.in(k, H))
                            r[b].load(p.residual, t * p.H, c, k);
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int i = first + b;
                    const Columns<FP32> c((i * WPR + wr) * 512, lane);
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = h[i].get(e) + r[b].get(e);
                    h[i].set(v);
#pragma unroll
                    for (int k = 0; k < c.kParts; ++k)
                        if (c.in(k, H))
                            h[i].store(p.total, t * p.H, c, k);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = fmaf(h[i].get(e), h[i].get(e), sum);
        sum = wave_sum(sum);
        if (WPR > 1) {
            if (lane == 0)
                part[parity][slot][wr] = sum;
            __syncthreads();
            sum = part[parity][slot][0];
#pragma unroll
            for (int u = 1; u < WPR; ++u)
                sum += part[parity][slot][u];
            parity ^= 1;
        }
        const float r = rsqrtf(sum / (float)p.H + p.eps);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Columns<FP32> c((i * WPR + wr) * 512, lane);
            if (!kEarly)
#pragma unroll
                for (int k = 0; k < c.kParts; ++k)
                    if (c.in(k, H))
                        w[i].load_cached(p.weight, c, k);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = h[i].get(e) * r * w[i].get(e);
            Raw8<false, FP32> o;
            o.set(v);
#pragma unroll
            for (int k = 0; k < c.kParts; ++k) {
                if (!c.in(k, H))
                    continue;
                if (p.y)
                    o.store(p.y, t * p.H, c, k);
                if (p.y8) {
                    // H is a multiple of 32: the lanes of a block, four or eight, are all here
                    constexpr int kValues = 8 / Columns<FP32>::kParts;
                    float m = 0.f;
#pragma unroll
                    for (int e = 0; e < kValues; ++e)
                        m = max_abs(m, v[k * kValues + e]);
                    m = fmaxf(m, __uint_as_float(dpp::mov<dpp::kQuadSwap1>(__float_as_uint(m), 0u)));
                    m = fmaxf(m, __uint_as_float(dpp::mov<dpp::kQuadSwap2>(__float_as_uint(m), 0u)));
                    if (FP32)
                        m = fmaxf(m, __uint_as_float(dpp::mov<dpp::kRowHalfMirror>(__float_as_uint(m), 0u)));
                    const int32_t e = fp8_exponent(m);
                    const float mul = fp8_multiplier(e);
                    uint32_t codes[kValues / 4];
#pragma unroll
                    for (int u = 0; u < kValues / 4; ++u) {
                        const int f = k * kValues + u * 4;
                        codes[u] = fp8_encode4(v[f], v[f + 1], v[f + 2], v[f + 3], mul);
                    }
                    uint8_t *at = p.y8 + (t * p.y8_bytes + c.start(k)) + c.mine;
                    if constexpr (kValues == 8)
                        __builtin_nontemporal_store(u32x2{codes[0], codes[1]}, reinterpret_cast<u32x2 *>(at));
                    else
                        __builtin_nontemporal_store(codes[0], reinterpret_cast<uint32_t *>(at));
                    if ((lane & (32 / kValues - 1)) == 0)
                        scales[slot][c.at(k) >> 5] = (uint8_t)(e + 127);
                }
            }
        }
        if (p.y8) {
            if (WPR > 1)
                __syncthreads();
            else
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const int i = wr * kWave + lane;  // the row's scale bytes in whole lines
            if (H && i < pad / 16)
                store_stream(reinterpret_cast<u32x4 *>(p.y8 + t * p.y8_bytes + p.H) + i,
                             reinterpret_cast<const u32x4 *>(scales[slot])[i]);
            if (WPR > 1)
                __syncthreads();
            else
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
}

// r and mean(g t) r^2 of one row in every lane of its waves
struct RowStats {
    float r, c;
};

// The gradient of rows blockIdx.x * kRows + slot, and further ones, in columns
// from blockIdx.y * (the columns that the waves cover). GIVEN: the row's
// statistics are read from p.stats, since a block covers only a part of the row.
template <bool FP32, bool WFP32, int WPR, int CH, bool GIVEN>
__global__ __launch_bounds__(norm_threads(WPR)) void rms_norm_backward_kernel(NormGradArgs p)
{
    constexpr int kRows = norm_threads(WPR) / kWave / WPR;
    __shared__ float part[2][2][kRows][WPR];
    __shared__ float sums[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? WPR * CH * 512 : 1];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int slot = wave / WPR, wr = wave % WPR;
    const int32_t c0 = GIVEN ? blockIdx.y * (WPR * CH * 512) : 0;
    float acc[CH][8];
    Raw8<WFP32, FP32> w[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc[i][e] = 0.f;
        const Columns<FP32> c(c0 + (i * WPR + wr) * 512, lane);
        w[i].clear();
#pragma unroll
        for (int k = 0; k < c.kParts; ++k)
            if (c.in(k, p.H))
                w[i].load_cached(p.weight, c, k);
    }
    int parity = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < p.T; t0 += (int64_t)gridDim.x * kRows) {
        const int64_t t = t0 + slot;
        const int32_t H = t < p.T ? p.H : 0;  // no columns in a row past the last
        Raw8<FP32, FP32> h[CH], d[CH];
        Raw8<false, FP32> g[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Columns<FP32> c(c0 + (i * WPR + wr) * 512, lane);
            h[i].clear();
            g[i].clear();
            d[i].clear();
#pragma unroll
            for (int k = 0; k < c.kParts; ++k)
                if (c.in(k, H)) {
                    h[i].load(p.t, t * p.H, c, k);
                    g[i].load(p.grad_y, t * p.H, c, k);
                    if (p.grad_x && p.grad_total)
                        d[i].load(p.grad_total, t * p.H, c, k);
                }
        }
        if (!WFP32)  // kept as it lies in memory: widened ahead of the loop it would take twice the registers
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    asm volatile("" : "+v"(w[i].q[u]));
        RowStats s = {0.f, 0.f};
        if (GIVEN) {
            if (H)
                s = RowStats{p.stats[2 * t], p.stats[2 * t + 1]};
        } else {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s0 = fmaf(h[i].get(e), h[i].get(e), s0);
                    s1 = fmaf(g[i].get(e) * w[i].get(e), h[i].get(e), s1);
                }
            s0 = wave_sum(s0);
            s1 = wave_sum(s1);
            if (WPR > 1) {
                if (lane == 0) {
                    part[parity][0][slot][wr] = s0;
                    part[parity][1][slot][wr] = s1;
                }
                __syncthreads();
                s0 = part[parity][0][slot][0];
                s1 = part[parity][1][slot][0];
#pragma unroll
                for (int u = 1; u < WPR; ++u) {
                    s0 += part[parity][0][slot][u];
                    s1 += part[parity][1][slot][u];
                }
                parity ^= 1;
            }
            s.r = rsqrtf(s0 / (float)p.H + p.eps);
            s.c = s1 / (float)p.H * s.r * s.r;
        }
        // their products are made again: kept across the sums they would take twice the registers
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                asm volatile("" : "+v"(g[i].q[u]));
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Columns<FP32> c(c0 + (i * WPR + wr) * 512, lane);
            if (!c.in(0, H))
                continue;  // the second part lies further right
            if (p.grad_x) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = s.r * (g[i].get(e) * w[i].get(e) - h[i].get(e) * s.c);
                if (p.grad_total)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] += d[i].get(e);
                Raw8<FP32, FP32> o;
                o.set(v);
#pragma unroll
                for (int k = 0; k < c.kParts; ++k)
                    if (c.in(k, H))
                        o.store(p.grad_x, t * p.H, c, k);
            }
            if (p.partial)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[i][e] = fmaf(g[i].get(e), h[i].get(e) * s.r, acc[i][e]);
        }
    }
    if (!p.partial)
        return;
    // the block's rows together, in the order of its waves
    if (kRows > 1) {
        if (slot > 0)
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sums[slot - 1][((i * WPR + wr) * 8 + e) * kWave + lane] = acc[i][e];
        __syncthreads();
        if (slot > 0)
            return;
#pragma unroll
        for (int u = 0; u < kRows - 1; ++u)
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[i][e] += sums[u][((i * WPR + wr) * 8 + e) * kWave + lane];
    }
    float *out = p.partial + (int64_t)blockIdx.x * p.H;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const Columns<FP32> c(c0 + (i * WPR + wr) * 512, lane);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int32_t at = FP32 ? c.at(k) : c.at(0) + k * 4;
            if (at < p.H)
                *reinterpret_cast<u32x4 *>(out + at) =
                    u32x4{__float_as_uint(acc[i][k * 4]), __float_as_uint(acc[i][k * 4 + 1]),
                          __float_as_uint(acc[i][k * 4 + 2]), __float_as_uint(acc[i][k * 4 + 3])};
        }
    }
}

// Statistics of rows too wide for one block's registers: a block per row.
constexpr int kStatThreads = 512;
template <bool FP32, bool WFP32>
__global__ __launch_bounds__(kStatThreads) void rms_norm_stats_kernel(NormGradArgs p)
{
    __shared__ float part[2][kStatThreads / kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        float s0 = 0.f, s1 = 0.f;
        for (int32_t first = wave * 512; first < p.H; first += kStatThreads * 8) {
            const Columns<FP32> c(first, lane);
            Raw8<FP32, FP32> h;
            Raw8<false, FP32> g;
            Raw8<WFP32, FP32> w;
            h.clear();
            g.clear();
            w.clear();
#pragma unroll
            for (int k = 0; k < c.kParts; ++k)
                if (c.in(k, p.H)) {
                    h.load(p.t, t * p.H, c, k);
                    g.load(p.grad_y, t * p.H, c, k);
                    w.load_cached(p.weight, c, k);
                }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s0 = fmaf(h.get(e), h.get(e), s0);
                s1 = fmaf(g.get(e) * w.get(e), h.get(e), s1);
            }
        }
        s0 = wave_sum(s0);
        s1 = wave_sum(s1);
        __syncthreads();  // the row before has been read
        if (lane == 0) {
            part[0][wave] = s0;
            part[1][wave] = s1;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            s0 = s1 = 0.f;
            for (int u = 0; u < kStatThreads / kWave; ++u) {
                s0 += part[0][u];
                s1 += part[1][u];
            }
            const float r = rsqrtf(s0 / (float)p.H + p.eps);
            p.stats[2 * t] = r;
            p.stats[2 * t + 1] = s1 / (float)p.H * r * r;
        }
    }
}

// grad_weight[h] (+)= sum of the blocks' partial sums, in the blocks' order
// within each wave and then the waves': 64 columns a block.
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(kJoinWaves *kWave) void rms_norm_join_kernel(const float *__restrict__ partial,
                                                                          int32_t blocks, int32_t H, bool accumulate,
                                                                          float *__restrict__ grad_weight)
{
    __shared__ float part[kJoinWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int32_t h = blockIdx.x * kWave + lane;
    const int32_t each = (blocks + kJoinWaves - 1) / kJoinWaves;
    const int32_t end = min(blocks, (wave + 1) * each);
    float s = 0.f;
    if (h < H)
#pragma unroll 8
        for (int32_t b = wave * each; b < end; ++b)
            s += partial[(int64_t)b * H + h];
    part[wave][lane] = s;
    __syncthreads();
    if (wave || h >= H)
        return;
#pragma unroll
    for (int u = 1; u < kJoinWaves; ++u)
        s += part[u][lane];
    grad_weight[h] = accumulate ? grad_weight[h] + s : s;
}

constexpr int32_t kNormWide = 16384;  // wider rows' gradients take their statistics first

// Blocks of the gradient's kernel: about as many as the GPU holds at once, each
// with a partial sum of the weight's gradient. Four rows a block up to 2048
// columns, else one. In us, with 3/4 of these numbers / these / 3/2 / twice them:
// 4099 x 7168 float32 81.1 / 76.3 / 77.2 / 79.6, bf16 47.8 / 48.5 / 51.3 / 52.8;
// 32768 x 7168 float32 616 / 592 / 590 / 593; 32768 x 2048 bf16 100 / 94 / 95.5 / 97;
// 8192 x 4096 bf16 55.1 / 57.2 / 56.4 / 58.5; 2000 x 40000 float32 298 / 301 / 308 / 313.
int32_t grad_blocks(int64_t T, int32_t H)
{
    const int64_t n = H <= 2048 ? (T + 3) / 4 : T, most = H <= 4096 ? 1024 : 512;
    return (int32_t)(n < most ? n : most);
}

template <bool FP32, bool WFP32, int WPR, int CH>
hipError_t launch_norm(const NormArgs &p, hipStream_t stream)
{
    constexpr int kRows = norm_threads(WPR) / kWave / WPR;
    // a launch takes fewer than 2^32 threads; kMaxRowBlocks of 1024 would be as many
    constexpr int64_t kMost = kMaxRowBlocks * 256 / norm_threads(WPR);
    static_assert(kMost * norm_threads(WPR) < (int64_t)1 << 32);
    const int64_t blocks = (p.T + kRows - 1) / kRows;
    hipLaunchKernelGGL((rms_norm_kernel<FP32, WFP32, WPR, CH>), dim3((unsigned)(blocks < kMost ? blocks : kMost)),
                       dim3(norm_threads(WPR)), 0, stream, p);
    return hipGetLastError();
}

// One wave per row and no barrier up to 2048 columns; wider rows take a wave
// per 512 columns, which shortens a single row's way: 128 x 7168 took 4.4 us with
// 16 waves and 5.8 with four.
template <bool FP32, bool WFP32>
hipError_t norm_by_width(const NormArgs &p, hipStream_t stream)
{
    if (p.H <= 512)
        return launch_norm<FP32, WFP32, 1, 1>(p, stream);
    if (p.H <= 1024)
        return launch_norm<FP32, WFP32, 1, 2>(p, stream);
    if (p.H <= 2048)
        return launch_norm<FP32, WFP32, 1, 4>(p, stream);
    if (p.H <= 4096)
        return launch_norm<FP32, WFP32, 8, 1>(p, stream);
    if (p.H <= 8192)
        return launch_norm<FP32, WFP32, 16, 1>(p, stream);
    if (p.H <= 16384)
        return launch_norm<FP32, WFP32, 16, 2>(p, stream);
    if (p.H <= 32768)
        return launch_norm<FP32, WFP32, 16, 4>(p, stream);
    return launch_norm<FP32, WFP32, 16, 8>(p, stream);
}

template <bool FP32, bool WFP32, int WPR, int CH, bool GIVEN = false>
hipError_t launch_norm_grad(const NormGradArgs &p, int32_t blocks, hipStream_t stream)
{
    const dim3 grid((unsigned)blocks, GIVEN ? (unsigned)((p.H + WPR * CH * 512 - 1) / (WPR * CH * 512)) : 1);
    hipLaunchKernelGGL((rms_norm_backward_kernel<FP32, WFP32, WPR, CH, GIVEN>), grid, dim3(norm_threads(WPR)), 0, stream,
                       p);
    return hipGetLastError();
}

template <bool FP32, bool WFP32>
hipError_t norm_grad_by_width(const NormGradArgs &p, hipStream_t stream)
{
    const int32_t blocks = grad_blocks(p.T, p.H);
    if (p.H <= 512)
        return launch_norm_grad<FP32, WFP32, 1, 1>(p, blocks, stream);
    if (p.H <= 1024)
        return launch_norm_grad<FP32, WFP32, 1, 2>(p, blocks, stream);
    if (p.H <= 2048)
        return launch_norm_grad<FP32, WFP32, 1, 4>(p, blocks, stream);
    if (p.H <= 4096)
        return launch_norm_grad<FP32, WFP32, 8, 1>(p, blocks, stream);
    if (p.H <= 8192)
        return launch_norm_grad<FP32, WFP32, 8, 2>(p, blocks, stream);
    if (p.H <= kNormWide)
        return launch_norm_grad<FP32, WFP32, 16, 2>(p, blocks, stream);
    static_assert(kMaxRowBlocks * kStatThreads < (int64_t)1 << 32);
    hipLaunchKernelGGL((rms_norm_stats_kernel<FP32, WFP32>), dim3((unsigned)(p.T < kMaxRowBlocks ? p.T : kMaxRowBlocks)),
                       dim3(kStatThreads), 0, stream, p);
    const hipError_t err = hipGetLastError();
    return err == hipSuccess ? launch_norm_grad<FP32, WFP32, 8, 2, true>(p, blocks, stream) : err;
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &p, bool fp32, hipStream_t stream)
{
    if (p.weight_fp32)
        return fp32 ? norm_by_width<true, true>(p, stream) : norm_by_width<false, true>(p, stream);
    return fp32 ? norm_by_width<true, false>(p, stream) : norm_by_width<false, false>(p, stream);
}

// partial sums of the weight's gradient where it is wanted, then the statistics of wide rows
size_t rms_norm_backward_workspace_bytes(int64_t T, int32_t H, bool weight)
{
    return (weight ? (size_t)grad_blocks(T, H) * H * 4 : 0) + (H > kNormWide ? (size_t)T * 8 : 0);
}

hipError_t launch_rms_norm_backward(NormGradArgs p, bool fp32, bool accumulate, float *grad_weight, void *workspace,
                                    hipStream_t stream)
{
    const int32_t blocks = grad_blocks(p.T, p.H);
    p.partial = grad_weight ? static_cast<float *>(workspace) : nullptr;
    p.stats = static_cast<float *>(workspace) + (grad_weight ? (size_t)blocks * p.H : 0);
    if (p.T > 0) {
        const hipError_t err =
            p.weight_fp32 ? (fp32 ? norm_grad_by_width<true, true>(p, stream) : norm_grad_by_width<false, true>(p, stream))
                          : (fp32 ? norm_grad_by_width<true, false>(p, stream) : norm_grad_by_width<false, false>(p, stream));
        if (err != hipSuccess || !grad_weight)
            return err;
    }
    hipLaunchKernelGGL(rms_norm_join_kernel, dim3((unsigned)((p.H + kWave - 1) / kWave)), dim3(kJoinWaves * kWave), 0,
                       stream, p.partial, blocks, p.H, accumulate, grad_weight);
    return hipGetLastError();
}

}  // namespace moe
