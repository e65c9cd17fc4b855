// combine_backward.hip -- the gradients of the gate-weighted combine: each
// kept replica's row of grad_y is its weight times the token's grad_out, and
// its weight's gradient the inner product of grad_out with its expert row.
//
// Plain form: a block per token, its replicas one after the other.
#include "device.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kRowThreads = 256;

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
        const u32x4 a = static_cast<const u32x4 *>(p)[chunk];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(a[i]);
            v[2 * i + 1] = bf16_hi(a[i]);
        }
    }
}

template <bool FP32>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(
    const void *__restrict__ grad_out, const u32x4 *__restrict__ y, int64_t y_rows,
    const int32_t *__restrict__ pos, const float *__restrict__ topk_w, int32_t C16, int32_t k,
    u32x4 *__restrict__ grad_y, float *__restrict__ grad_w)
{
    __shared__ float part[kRowThreads];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    for (int j = 0; j < k; ++j) {
        const int32_t q = pos[t * k + j];
        const bool kept = q >= 0 && q < y_rows;
        float dot = 0.f;
        if (kept) {
            const float w = grad_y ? topk_w[t * k + j] : 0.f;
            for (int32_t c = tid; c < C16; c += kRowThreads) {
                float g[8];
                load8<FP32>(grad_out, t * C16 + c, g);
                if (grad_w) {
                    float r[8];
                    load8<false>(y, (int64_t)q * C16 + c, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dot = fmaf(g[i], r[i], dot);
                }
                if (grad_y) {
                    u32x4 o;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = pack_bf16x2(w * g[2 * i], w * g[2 * i + 1]);
                    grad_y[(int64_t)q * C16 + c] = o;
                }
            }
        }
        if (grad_w) {
            part[tid] = dot;
            __syncthreads();
            for (int s = kRowThreads / 2; s > 0; s >>= 1) {
                if (tid < s)
                    part[tid] += part[tid + s];
                __syncthreads();
            }
            if (tid == 0)
                grad_w[t * k + j] = part[0];
            __syncthreads();
        }
    }
}

}  // namespace

hipError_t launch_combine_backward(const void *grad_out, bool fp32, const uint16_t *y,
                                   int64_t y_rows, const int32_t *pos, const float *topk_w,
                                   int64_t T, int32_t H, int32_t k, uint16_t *grad_y,
                                   float *grad_w, hipStream_t stream)
{
    const int32_t C16 = H / 8;
    for (int64_t t0 = 0; t0 < T; t0 += kMaxRowBlocks) {
        const int64_t n = T - t0 < kMaxRowBlocks ? T - t0 : kMaxRowBlocks;
        const void *go = static_cast<const char *>(grad_out) + t0 * H * (fp32 ? 4 : 2);
        const float *tw = topk_w ? topk_w + t0 * k : nullptr;
        float *gw = grad_w ? grad_w + t0 * k : nullptr;
        const u32x4 *yv = reinterpret_cast<const u32x4 *>(y);
        u32x4 *gy = reinterpret_cast<u32x4 *>(grad_y);
        if (fp32)
            hipLaunchKernelGGL((combine_backward_kernel<true>), dim3((unsigned)n), dim3(kRowThreads), 0,
                               stream, go, yv, y_rows, pos + t0 * k, tw, C16, k, gy, gw);
        else
            hipLaunchKernelGGL((combine_backward_kernel<false>), dim3((unsigned)n), dim3(kRowThreads), 0,
                               stream, go, yv, y_rows, pos + t0 * k, tw, C16, k, gy, gw);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace moe
