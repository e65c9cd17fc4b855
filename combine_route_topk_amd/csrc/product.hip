// product.hip -- the experts' products on expert-major rows and the gradient
// with respect to their input, with bias, activation, gate and residual (or
// the activation's gradient) applied to the float32 sums before the one
// rounding to bf16.
//
// Plain form: a block computes 64 rows of one expert by 64 columns (gated:
// 32 gate columns and the 32 columns they gate), 4 x 4 sums per thread, with
// operands staged through LDS in float32.
#include "product_device.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256, kBM = 64, kBN = 64, kBK = 16;
constexpr int kMaxBlocks = 2048;

// GRAD: B(n, k) = W[l][k][n], K = O; otherwise B(n, k) = W[l][n][k], K = H.
// N: columns of the product's own output (O, or H for GRAD); PAIR: tile
// column n < 32 is output n0 + n and column 32 + n the one it gates.
template <bool GRAD, bool GATED, int ACT>
__global__ __launch_bounds__(kThreads) void product_kernel(
    const uint16_t *__restrict__ a, const int32_t *__restrict__ off, int32_t El, int32_t max_rows,
    int32_t K, int32_t N, const uint16_t *__restrict__ W, const uint16_t *__restrict__ bias,
    const uint16_t *residual, const uint16_t *pre_in, uint16_t *pre_out, uint16_t *out)
{
    constexpr bool PAIR = GATED && !GRAD;
    constexpr int kCols = PAIR ? kBN / 2 : kBN;
    __shared__ int32_t first[kMaxLocalExperts + 1];
    __shared__ float As[kBK][kBM + 1], Bs[kBK][kBN + 1];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int32_t row_tiles = plan_row_tiles<kThreads, kBM>(off, El, max_rows, first);
    const int64_t nct = (N + kCols - 1) / kCols;
    const int64_t wide = PAIR ? 2 * (int64_t)N : N;
    for (int64_t u = blockIdx.x; u < row_tiles * nct; u += gridDim.x) {
        const int32_t rt = (int32_t)(u / nct), n0 = (int32_t)(u % nct) * kCols;
        const int32_t l = tile_expert(first, El, rt);
        const Rows r = expert_rows(off, l, max_rows);
        const int64_t row0 = r.begin + (int64_t)(rt - first[l]) * kBM;
        const int rows = (int)min((int64_t)kBM, r.end - row0);
        const uint16_t *Wl = W + (int64_t)l * wide * K;
        float acc[4][4] = {};
        for (int32_t k0 = 0; k0 < K; k0 += kBK) {
            for (int i = tid; i < kBM * kBK; i += kThreads) {
                const int m = i / kBK, k = i % kBK;
                As[k][m] = m < rows && k0 + k < K ? bf16_to_f32(a[(row0 + m) * K + k0 + k]) : 0.f;
                const int n = m;
                const int32_t col = PAIR ? n0 + n % 32 : n0 + n;
                const int64_t wrow = PAIR && n >= 32 ? (int64_t)N + col : col;
                float b = 0.f;
                if (col < N && k0 + k < K)
                    b = bf16_to_f32(GRAD ? Wl[(int64_t)(k0 + k) * N + col] : Wl[wrow * K + k0 + k]);
                Bs[k][n] = b;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kBK; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][(j / 2) * 32 + tx * 2 + j % 2], acc[i][j]);
            }
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i) {
            const int m = ty * 4 + i;
            if (m >= rows)
                continue;
            const int64_t row = row0 + m;
            for (int j = 0; j < (PAIR ? 2 : 4); ++j) {
                const int32_t c = n0 + (j / 2) * 32 + tx * 2 + j % 2;
                if (c >= N)
                    continue;
                float v = acc[i][j];
                if (GRAD) {
                    if (GATED) {
                        const float g = bf16_to_f32(pre_in[row * 2 * N + c]);
                        const float up = bf16_to_f32(pre_in[row * 2 * N + N + c]);
                        out[row * 2 * N + c] = f32_to_bf16(v * up * act_grad<ACT>(g));
                        out[row * 2 * N + N + c] = f32_to_bf16(v * act<ACT>(g));
                    } else {
                        if (pre_in)
                            v *= act_grad<ACT>(bf16_to_f32(pre_in[row * N + c]));
                        out[row * N + c] = f32_to_bf16(v);
                    }
                    continue;
                }
                if (bias)
                    v += bf16_to_f32(bias[l * wide + c]);
                if (pre_out)
                    pre_out[row * wide + c] = f32_to_bf16(v);
                v = act<ACT>(v);
                if (PAIR) {
                    float g = acc[i][j + 2];
                    if (bias)
                        g += bf16_to_f32(bias[l * wide + N + c]);
                    if (pre_out)
                        pre_out[row * wide + N + c] = f32_to_bf16(g);
                    v *= g;
                }
                if (residual)
                    v += bf16_to_f32(residual[row * N + c]);
                out[row * N + c] = f32_to_bf16(v);
            }
        }
    }
}

template <bool GRAD>
hipError_t launch(const uint16_t *a, const int32_t *off, int32_t El, int64_t max_rows, int32_t K,
                  int32_t N, const uint16_t *W, const uint16_t *bias, const uint16_t *residual,
                  const uint16_t *pre_in, int32_t act, bool gated, uint16_t *pre_out, uint16_t *out,
                  hipStream_t stream)
{
    const int64_t tiles = (max_rows / kBM + El) * ((N + 31) / 32);
    const dim3 grid((unsigned)(tiles < kMaxBlocks ? tiles : kMaxBlocks));
#define MOE_PRODUCT_LAUNCH(G, A)                                                                    \
    hipLaunchKernelGGL((product_kernel<GRAD, G, A>), grid, dim3(kThreads), 0, stream, a, off, El,   \
                       (int32_t)max_rows, K, N, W, bias, residual, pre_in, pre_out, out);           \
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
    return launch<false>(x, off, El, max_rows, H, O, W, bias, residual, nullptr, act, gated, pre, y,
                         stream);
}

hipError_t launch_expert_dgrad(const uint16_t *grad_y, const int32_t *off, int32_t El,
                               int64_t max_rows, int32_t O, int32_t H, const uint16_t *W,
                               const uint16_t *pre, int32_t act, bool gated, uint16_t *grad_x,
                               hipStream_t stream)
{
    return launch<true>(grad_y, off, El, max_rows, O, H, W, nullptr, nullptr, pre, act, gated,
                        nullptr, grad_x, stream);
}

}  // namespace moe
