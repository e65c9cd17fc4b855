// combine_backward.hip -- the gradients of the gate-weighted combine: each
// kept replica's row of grad_y is its weight times the token's grad_out, and
// its weight's gradient the inner product of grad_out with its expert row.
//
// Bound by HBM: per kept replica one row read and one written, in one pass.
// One, two or four waves take a token by its width, each lane 8 columns at a
// time. Up to four replicas' 16-byte loads are issued before the first is
// used; y is read and grad_y written past the caches, each row once. The
// inner products stay in registers over the row, then are reduced over the
// wave by DPP in a fixed order and over the token's waves through LDS.
#include "device.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int kBatch = 4, kMaxReplicas = 32;

__device__ __forceinline__ void widen8(const u32x4 &a, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(a[i]);
        v[2 * i + 1] = bf16_hi(a[i]);
    }
}

template <bool FP32>
__device__ __forceinline__ void load8(const void *p, int64_t chunk, float (&v)[8])
{
    if (FP32) {
        const u32x4 *q = static_cast<const u32x4 *>(p) + 2 * chunk;
        const u32x4 a = q[0], b = q[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(a[i]);
            v[4 + i] = __uint_as_float(b[i]);
        }
    } else {
        widen8(static_cast<const u32x4 *>(p)[chunk], v);
    }
}

// lane 63 ends with the wave's sum
__device__ __forceinline__ float wave_sum(float v)
{
    auto add = [](float a, uint32_t b) { return a + __uint_as_float(b); };
    v = add(v, dpp::mov<dpp::kQuadSwap1>(__float_as_uint(v), 0u));
    v = add(v, dpp::mov<dpp::kQuadSwap2>(__float_as_uint(v), 0u));
    v = add(v, dpp::mov<dpp::kRowHalfMirror>(__float_as_uint(v), 0u));
    v = add(v, dpp::mov<dpp::kRowMirror>(__float_as_uint(v), 0u));
    v = add(v, dpp::mov<dpp::kRowBcast15, 0xA>(__float_as_uint(v), 0u));
    return add(v, dpp::mov<dpp::kRowBcast31, 0xC>(__float_as_uint(v), 0u));
}

// WPT waves per token.
template <bool FP32, int WPT>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(
    const void *__restrict__ grad_out, const u32x4 *__restrict__ y, int64_t y_rows,
    const int32_t *__restrict__ pos, const float *__restrict__ topk_w, int64_t T, int32_t C16, int32_t k,
    u32x4 *__restrict__ grad_y, float *__restrict__ grad_w)
{
    constexpr int kTokens = kRowThreads / kWave / WPT;
    __shared__ float part[kTokens][WPT][kMaxReplicas];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t t = (int64_t)blockIdx.x * kTokens + wave / WPT;
    const bool valid = t < T;  // the same for a token's waves
    // lane j < k holds replica j's position and weight
    int32_t pl = -1;
    float wl = 0.f;
    if (valid && lane < k) {
        pl = pos[t * k + lane];
        if (grad_y)
            wl = topk_w[t * k + lane];
    }
    const bool dots = grad_w != nullptr, rows = grad_y != nullptr;
    for (int j0 = 0; valid && j0 < k; j0 += kBatch) {
        int32_t p[kBatch];
        float w[kBatch], dot[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int32_t q = (int32_t)readlane_u32((uint32_t)pl, (j0 + j) & (kWave - 1));
            p[j] = j0 + j < k && q >= 0 && q < y_rows ? q : -1;
            w[j] = __uint_as_float(readlane_u32(__float_as_uint(wl), (j0 + j) & (kWave - 1)));
            dot[j] = 0.f;
        }
        for (int32_t c = (wave % WPT) * kWave + lane; c < C16; c += WPT * kWave) {
            float g[8];
            u32x4 v[kBatch];
            load8<FP32>(grad_out, t * C16 + c, g);
            if (dots) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (p[j] >= 0)
                        v[j] = load_stream(y + (int64_t)p[j] * C16 + c);
            }
            if (rows) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (p[j] >= 0) {
                        u32x4 o;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[i] = pack_bf16x2(w[j] * g[2 * i], w[j] * g[2 * i + 1]);
                        store_stream(grad_y + (int64_t)p[j] * C16 + c, o);
                    }
            }
            if (dots) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (p[j] >= 0) {
                        float r[8];
                        widen8(v[j], r);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            dot[j] = fmaf(g[i], r[i], dot[j]);
                    }
            }
        }
        if (dots) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const float s = wave_sum(dot[j]);
                if (lane == kWave - 1 && j0 + j < kMaxReplicas)
                    part[wave / WPT][wave % WPT][j0 + j] = s;
            }
        }
    }
    if (!dots)
        return;
    __syncthreads();
    if (valid && wave % WPT == 0 && lane < k) {
        float s = part[wave / WPT][0][lane];
#pragma unroll
        for (int u = 1; u < WPT; ++u)
            s += part[wave / WPT][u][lane];
        grad_w[t * k + lane] = s;
    }
}

template <bool FP32, int WPT>
hipError_t launch(const void *grad_out, const uint16_t *y, int64_t y_rows, const int32_t *pos,
                  const float *topk_w, int64_t T, int32_t H, int32_t k, uint16_t *grad_y, float *grad_w,
                  hipStream_t stream)
{
    constexpr int64_t kTokens = kRowThreads / kWave / WPT;
    const int64_t chunk = kMaxRowBlocks * kTokens;
    for (int64_t t0 = 0; t0 < T; t0 += chunk) {
        const int64_t n = T - t0 < chunk ? T - t0 : chunk;
        hipLaunchKernelGGL((combine_backward_kernel<FP32, WPT>), dim3((unsigned)((n + kTokens - 1) / kTokens)),
                           dim3(kRowThreads), 0, stream,
                           static_cast<const char *>(grad_out) + t0 * H * (FP32 ? 4 : 2),
                           reinterpret_cast<const u32x4 *>(y), y_rows, pos + t0 * k, topk_w ? topk_w + t0 * k : nullptr,
                           n, H / 8, k, reinterpret_cast<u32x4 *>(grad_y), grad_w ? grad_w + t0 * k : nullptr);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_combine_backward(const void *grad_out, bool fp32, const uint16_t *y,
                                   int64_t y_rows, const int32_t *pos, const float *topk_w,
                                   int64_t T, int32_t H, int32_t k, uint16_t *grad_y,
                                   float *grad_w, hipStream_t stream)
{
    // as many waves as have columns: one per 512, at most four
    const int waves = H <= 512 ? 1 : (H <= 1024 ? 2 : 4);
#define MOE_COMBINE_GRAD(F)                                                                                    \
    (waves == 1   ? launch<F, 1>(grad_out, y, y_rows, pos, topk_w, T, H, k, grad_y, grad_w, stream)            \
     : waves == 2 ? launch<F, 2>(grad_out, y, y_rows, pos, topk_w, T, H, k, grad_y, grad_w, stream)            \
                  : launch<F, 4>(grad_out, y, y_rows, pos, topk_w, T, H, k, grad_y, grad_w, stream))
    return fp32 ? MOE_COMBINE_GRAD(true) : MOE_COMBINE_GRAD(false);
#undef MOE_COMBINE_GRAD
}

}  // namespace moe
