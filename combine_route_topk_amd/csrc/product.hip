// product.hip -- the experts' products on expert-major rows and the gradient
// with respect to their input, with bias, activation, gate and residual (or
// the activation's gradient) applied to the float32 sums before the one
// rounding to bf16.
//
// A persistent block per CU takes tiles of 256 rows of one expert by 256
// columns (gated: 128 gate columns and the 128 columns they gate, laid out
// so that a lane holds both); product_gemm.hpp has the K loop.
#include "product_gemm.hpp"

namespace moe {
namespace {

__device__ __forceinline__ f32x4 load_bf16x4(const uint16_t *p)
{
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
}
__device__ __forceinline__ void store_bf16x4(uint16_t *p, f32x4 v)
{
    uint2 o;
    o.x = pack_bf16x2(v[0], v[1]);
    o.y = pack_bf16x2(v[2], v[3]);
    *reinterpret_cast<uint2 *>(p) = o;
}

struct ProductArgs {
    const uint16_t *a;         // x, or grad_y (GRAD)
    const int32_t *off;
    const uint16_t *W, *bias, *residual, *pre_in;
    uint16_t *pre_out, *out;
    int32_t El, max_rows, K, N;  // N: columns before a gate doubles them
};

// four columns of one row, c a multiple of 4
template <bool GRAD, bool GATED, int ACT>
__device__ __forceinline__ void finish(const ProductArgs &p, int32_t l, int64_t row, int32_t c, f32x4 v, f32x4 g)
{
    const int64_t N = p.N;
    if (GRAD) {
        if (GATED) {
            const f32x4 z = load_bf16x4(p.pre_in + row * 2 * N + c), u = load_bf16x4(p.pre_in + row * 2 * N + N + c);
            f32x4 dz, du;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dz[i] = v[i] * u[i] * act_grad<ACT>(z[i]);
                du[i] = v[i] * act<ACT>(z[i]);
            }
            store_bf16x4(p.out + row * 2 * N + c, dz);
            store_bf16x4(p.out + row * 2 * N + N + c, du);
            return;
        }
        if (p.pre_in) {
            const f32x4 z = load_bf16x4(p.pre_in + row * N + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] *= act_grad<ACT>(z[i]);
        }
        store_bf16x4(p.out + row * N + c, v);
        return;
    }
    const int64_t wide = GATED ? 2 * N : N;
    if (p.bias) {
        v += load_bf16x4(p.bias + l * wide + c);
        if (GATED)
            g += load_bf16x4(p.bias + l * wide + N + c);
    }
    if (p.pre_out) {
        store_bf16x4(p.pre_out + row * wide + c, v);
        if (GATED)
            store_bf16x4(p.pre_out + row * wide + N + c, g);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = GATED ? act<ACT>(v[i]) * g[i] : act<ACT>(v[i]);
    if (p.residual)
        v += load_bf16x4(p.residual + row * N + c);
    store_bf16x4(p.out + row * N + c, v);
}

template <bool GRAD, bool GATED, int ACT>
__global__ __launch_bounds__(kGemmThreads, 2) void product_kernel(ProductArgs p)
{
    constexpr bool PAIR = GATED && !GRAD;
    constexpr int kCols = PAIR ? kTile / 2 : kTile;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kGemmLdsBytes];
    __shared__ int32_t first[kMaxLocalExperts + 1];
    const int32_t row_tiles = plan_row_tiles<kGemmThreads, kTile>(p.off, p.El, p.max_rows, first);
    const int64_t nct = (p.N + kCols - 1) / kCols;
    const int64_t wide = PAIR ? 2 * (int64_t)p.N : p.N;
    const int nk = (p.K + kTileK - 1) / kTileK;
    Gemm<false, GRAD> gemm;
    gemm.init_lane();
    // each XCD (blockIdx % 8) takes runs of consecutive tiles
    const int32_t per_xcd = gridDim.x / 8;
    const int64_t slot = gridDim.x % 8 ? blockIdx.x : (int64_t)(blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
    for (int64_t u = slot; u < row_tiles * nct; u += gridDim.x) {
        const int32_t rt = (int32_t)(u / nct), n0 = (int32_t)(u % nct) * kCols;
        const int32_t l = __builtin_amdgcn_readfirstlane(tile_expert(first, p.El, rt));
        const Rows r = expert_rows(p.off, l, p.max_rows);
        const int32_t row0 = __builtin_amdgcn_readfirstlane(r.begin + (rt - first[l]) * kTile);
        const int32_t rows = __builtin_amdgcn_readfirstlane(min(kTile, r.end - row0));
        if (rows <= 0)
            continue;
        gemm.A.init(p.a + (int64_t)row0 * p.K, rows, p.K, gemm.wave, gemm.lane, 128, [](int j) { return j * 8; });
        const uint16_t *Wl = p.W + (int64_t)l * wide * p.K;
        if constexpr (GRAD) {
            gemm.B.init_strided(Wl + n0, p.K, p.N, p.N - n0, gemm.wave, gemm.lane);
        } else if constexpr (GATED) {
            // rows of a half: for each wave's 32 columns, 16 gate then 16 up
            const bool up = (gemm.wave >> 1) & 1;
            gemm.B.init(Wl + ((up ? (int64_t)p.N : 0) + n0) * p.K, p.N - n0, p.K, gemm.wave, gemm.lane, 64,
                        [](int j) { return (j >> 2) * 16 + (j & 1) * 8; });
        } else {
            gemm.B.init(Wl + (int64_t)n0 * p.K, p.N - n0, p.K, gemm.wave, gemm.lane, 128, [](int j) { return j * 8; });
        }
        Acc acc;
        gemm.start(lds, nk);
        gemm.run(lds, nk, acc);
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t m = ha * 128 + gemm.wm * 64 + i * 16 + (gemm.lane & 15);
                if (m >= rows)
                    continue;
#pragma unroll
                for (int hb = 0; hb < 2; ++hb) {
                    if (PAIR) {
                        const int32_t c = n0 + hb * 64 + gemm.wn * 16 + (gemm.lane >> 4) * 4;
                        if (c < p.N)
                            finish<GRAD, GATED, ACT>(p, l, (int64_t)row0 + m, c, acc[ha][hb][i][0], acc[ha][hb][i][1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int32_t c = n0 + hb * 128 + gemm.wn * 32 + j * 16 + (gemm.lane >> 4) * 4;
                            if (c < p.N)
                                finish<GRAD, GATED, ACT>(p, l, (int64_t)row0 + m, c, acc[ha][hb][i][j], f32x4{});
                        }
                    }
                }
            }
        wait_loads<0>();
        slot_end();
    }
}

template <bool GRAD>
hipError_t launch(const ProductArgs &p, int32_t act, bool gated, hipStream_t stream)
{
    int device = 0, cus = 0;
    hipError_t err = hipGetDevice(&device);
    if (err == hipSuccess)
        err = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device);
    if (err != hipSuccess)
        return err;
    const int kCols = gated && !GRAD ? kTile / 2 : kTile;
    const int64_t tiles = ((int64_t)p.max_rows / kTile + p.El) * ((p.N + kCols - 1) / kCols);
    const dim3 grid((unsigned)(tiles < cus ? tiles : cus));
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
