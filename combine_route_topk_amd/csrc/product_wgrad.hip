// product_wgrad.hip -- the gradients of the experts' weights and biases:
// grad_W[l] = grad_y[rows of l]^T x[rows of l], summed over the rows in
// float32. Both operands are K-strided (K is the rows); product_gemm.hpp has
// the K loop. grad_bias is summed by a kernel of its own.
#include "product_gemm.hpp"

namespace moe {
namespace {

struct WgradArgs {
    const uint16_t *gy, *x;
    const int32_t *off;
    void *gW;
    int32_t El, max_rows, O, H;
};

template <bool FP32, bool ACCUMULATE>
__global__ __launch_bounds__(kGemmThreads, 2) void wgrad_kernel(WgradArgs p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kGemmLdsBytes];
    const int64_t no = (p.O + kTile - 1) / kTile, nh = (p.H + kTile - 1) / kTile;
    Gemm<true, true> gemm;
    gemm.init_lane();
    const int32_t per_xcd = gridDim.x / 8;
    const int64_t slot = gridDim.x % 8 ? blockIdx.x : (int64_t)(blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
    for (int64_t u = slot; u < p.El * no * nh; u += gridDim.x) {
        const int32_t h0 = (int32_t)(u % nh) * kTile, o0 = (int32_t)(u / nh % no) * kTile;
        const int32_t l = (int32_t)(u / (nh * no));
        const Rows r = expert_rows(p.off, l, p.max_rows);
        const int32_t begin = __builtin_amdgcn_readfirstlane(r.begin);
        const int32_t n = __builtin_amdgcn_readfirstlane(r.end - r.begin);
        const int nk = (n + kTileK - 1) / kTileK;
        gemm.A.init_strided(p.gy + (int64_t)begin * p.O + o0, n, p.O, p.O - o0, gemm.wave, gemm.lane);
        gemm.B.init_strided(p.x + (int64_t)begin * p.H + h0, n, p.H, p.H - h0, gemm.wave, gemm.lane);
        Acc acc;
        gemm.start(lds, nk);
        gemm.run(lds, nk, acc);
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
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (o >= p.O || j * 16 + c4 >= left)
                                continue;
                            f32x4 v = acc[ha][hb][i][j];
                            f32x4 *q = reinterpret_cast<f32x4 *>(static_cast<float *>(p.gW) + at + j * 16 + c4);
                            if (ACCUMULATE)
                                v += *q;
                            *q = v;
                        }
                    } else {
                        const u32x4 v = to_rows(narrow(acc[ha][hb][i][0]), narrow(acc[ha][hb][i][1]));
                        if (o < p.O && c4 * 2 < left)
                            *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.gW) + at + c4 * 2) = v;
                    }
                }
            }
        wait_loads<0>();
        slot_end();
    }
}

// A block sums 256 columns of one expert's rows.
__global__ __launch_bounds__(256) void bias_grad_kernel(const uint16_t *__restrict__ gy,
                                                        const int32_t *__restrict__ off, int32_t max_rows,
                                                        int32_t O, bool accumulate, float *__restrict__ gb)
{
    const int32_t o = blockIdx.x * 256 + threadIdx.x, l = blockIdx.y;
    const Rows r = expert_rows(off, l, max_rows);
    if (o >= O)
        return;
    float s = 0.f;
    for (int64_t i = r.begin; i < r.end; ++i)
        s += bf16_to_f32(gy[i * O + o]);
    float *q = gb + (int64_t)l * O + o;
    *q = accumulate ? *q + s : s;
}

}  // namespace

size_t wgrad_workspace_bytes(int32_t, int64_t, int32_t, int32_t) { return 0; }

hipError_t launch_expert_wgrad(const uint16_t *grad_y, const uint16_t *x, const int32_t *off,
                               int32_t El, int64_t max_rows, int32_t O, int32_t H, bool fp32,
                               bool accumulate, void *grad_W, float *grad_bias, void *,
                               hipStream_t stream)
{
    int device = 0, cus = 0;
    hipError_t err = hipGetDevice(&device);
    if (err == hipSuccess)
        err = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device);
    if (err != hipSuccess)
        return err;
    const int64_t tiles = (int64_t)El * ((O + kTile - 1) / kTile) * ((H + kTile - 1) / kTile);
    const dim3 grid((unsigned)(tiles < cus ? tiles : cus));
    const WgradArgs p = {grad_y, x, off, grad_W, El, (int32_t)max_rows, O, H};
    if (accumulate)
        hipLaunchKernelGGL((wgrad_kernel<true, true>), grid, dim3(kGemmThreads), 0, stream, p);
    else if (fp32)
        hipLaunchKernelGGL((wgrad_kernel<true, false>), grid, dim3(kGemmThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((wgrad_kernel<false, false>), grid, dim3(kGemmThreads), 0, stream, p);
    err = hipGetLastError();
    if (err != hipSuccess || !grad_bias)
        return err;
    hipLaunchKernelGGL(bias_grad_kernel, dim3((unsigned)((O + 255) / 256), (unsigned)El), dim3(256), 0, stream,
                       grad_y, off, (int32_t)max_rows, O, accumulate, grad_bias);
    return hipGetLastError();
}

}  // namespace moe
