// product_wgrad.hip -- the gradients of the experts' weights and biases:
// grad_W[l] = grad_y[rows of l]^T x[rows of l], summed over the rows in
// float32.
//
// Plain form: a block computes 64 x 64 of one expert's grad_W, 4 x 4 sums
// per thread, with operands staged through LDS in float32.
#include "product_device.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256, kBM = 64, kBN = 64, kBK = 16;
constexpr int kMaxBlocks = 2048;

template <bool FP32, bool ACCUMULATE>
__global__ __launch_bounds__(kThreads) void wgrad_kernel(
    const uint16_t *__restrict__ gy, const uint16_t *__restrict__ x, const int32_t *__restrict__ off,
    int32_t El, int32_t max_rows, int32_t O, int32_t H, void *__restrict__ gW, float *__restrict__ gb)
{
    __shared__ float As[kBK][kBM + 1], Bs[kBK][kBN + 1];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int64_t nh = (H + kBN - 1) / kBN, no = (O + kBM - 1) / kBM;
    for (int64_t u = blockIdx.x; u < El * no * nh; u += gridDim.x) {
        const int32_t h0 = (int32_t)(u % nh) * kBN, o0 = (int32_t)(u / nh % no) * kBM;
        const int32_t l = (int32_t)(u / (nh * no));
        const Rows r = expert_rows(off, l, max_rows);
        float acc[4][4] = {}, bsum = 0.f;
        for (int64_t k0 = r.begin; k0 < r.end; k0 += kBK) {
            for (int i = tid; i < kBM * kBK; i += kThreads) {
                const int k = i / kBM, m = i % kBM;
                const bool in = k0 + k < r.end;
                As[k][m] = in && o0 + m < O ? bf16_to_f32(gy[(k0 + k) * O + o0 + m]) : 0.f;
                Bs[k][m] = in && h0 + m < H ? bf16_to_f32(x[(k0 + k) * H + h0 + m]) : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kBK; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx * 4 + j], acc[i][j]);
                if (tid < kBM)
                    bsum += As[k][tid];
            }
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int32_t o = o0 + ty * 4 + i, h = h0 + tx * 4 + j;
                if (o >= O || h >= H)
                    continue;
                const int64_t at = ((int64_t)l * O + o) * H + h;
                if (FP32) {
                    float *p = static_cast<float *>(gW) + at;
                    *p = ACCUMULATE ? *p + acc[i][j] : acc[i][j];
                } else {
                    static_cast<uint16_t *>(gW)[at] = f32_to_bf16(acc[i][j]);
                }
            }
        if (gb && h0 == 0 && tid < kBM && o0 + tid < O) {
            float *p = gb + (int64_t)l * O + o0 + tid;
            *p = ACCUMULATE ? *p + bsum : bsum;
        }
    }
}

}  // namespace

size_t wgrad_workspace_bytes(int32_t, int64_t, int32_t, int32_t) { return 0; }

hipError_t launch_expert_wgrad(const uint16_t *grad_y, const uint16_t *x, const int32_t *off,
                               int32_t El, int64_t max_rows, int32_t O, int32_t H, bool fp32,
                               bool accumulate, void *grad_W, float *grad_bias, void *,
                               hipStream_t stream)
{
    const int64_t tiles = (int64_t)El * ((O + kBM - 1) / kBM) * ((H + kBN - 1) / kBN);
    const dim3 grid((unsigned)(tiles < kMaxBlocks ? tiles : kMaxBlocks));
#define MOE_WGRAD_LAUNCH(F, A)                                                                     \
    hipLaunchKernelGGL((wgrad_kernel<F, A>), grid, dim3(kThreads), 0, stream, grad_y, x, off, El, \
                       (int32_t)max_rows, O, H, grad_W, grad_bias)
    if (accumulate)
        MOE_WGRAD_LAUNCH(true, true);
    else if (fp32)
        MOE_WGRAD_LAUNCH(true, false);
    else
        MOE_WGRAD_LAUNCH(false, false);
#undef MOE_WGRAD_LAUNCH
    return hipGetLastError();
}

}  // namespace moe
