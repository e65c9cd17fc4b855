// product_fp8_few.hip -- the experts' product on FP8 rows for few rows per
// expert (decoding): the weights' way from memory bounds it, as in bf16
// (product_few.hip), at half the bytes.
//
// A block of eight waves takes up to 32 rows of one expert by 32 output columns
// (gated: 32 gate columns and the 32 they gate). Its waves share K, 128 values
// at a time in turn, so that a block reads 1024 consecutive bytes of each W
// row, and add their sums through LDS, in the waves' order. A lane's two
// 16-byte pieces of 128 values lie 64 bytes apart: that is where the scaled
// MFMA's lanes hold them, and its scales, one per 32 values, follow from it.
#include "product_fp8_device.hpp"

namespace moe {
namespace {

constexpr int kFewThreads = 512, kFewWaves = kFewThreads / kWave;
constexpr int kFewRows = 32, kFewCols = 32;
constexpr int kFewStep = kFewWaves * kTileK8;  // k of one round of the block's waves

// A wave's operands: MT groups of 16 rows of x, NG of 16 rows of W (gated: two
// of gate columns, then the two that they gate).
template <int MT, int NG>
struct FewOperands {
    __amdgpu_buffer_rsrc_t w[NG], x;
    uint32_t woff, xoff[MT], soff[MT];  // this lane's bytes of k = 0, and its scale byte
    const float *ws[NG == 4 ? 2 : 1];   // the weights' scales along K
    uint32_t K, k_lane, s_lane;         // first k of this lane's pieces and of its 32 values
};

// 128 k from k0. TAIL: pieces past K read as zeros, in x and W alike.
template <int MT, int NG, bool TAIL>
__device__ __forceinline__ void few_step(const FewOperands<MT, NG> &o, uint32_t k0, f32x4 (&c)[NG][MT])
{
    i32x4 a[NG][2], b[MT][2];
    uint32_t s[MT];
    float w[NG == 4 ? 2 : 1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t cut = TAIL && k0 + h * 64 + o.k_lane >= o.K ? kOutside : 0u;
#pragma unroll
        for (int g = 0; g < NG; ++g)
            a[g][h] = __builtin_bit_cast(
                i32x4, __builtin_amdgcn_raw_buffer_load_b128(o.w[g], (o.woff + k0 + h * 64) | cut, 0, 0));
#pragma unroll
        for (int m = 0; m < MT; ++m)
            b[m][h] = __builtin_bit_cast(
                i32x4, __builtin_amdgcn_raw_buffer_load_b128(o.x, (o.xoff[m] + k0 + h * 64) | cut, 0, 0));
    }
    const uint32_t cut = TAIL && k0 + o.s_lane >= o.K ? kOutside : 0u;
#pragma unroll
    for (int m = 0; m < MT; ++m)
        s[m] = __builtin_amdgcn_raw_buffer_load_b8(o.x, (o.soff[m] + k0 / 32) | cut, 0, 0);
#pragma unroll
    for (int q = 0; q < NG / 2; ++q)
        w[q] = TAIL && k0 >= o.K ? 0.f : load_uniform(o.ws[q] + k0 / kTileK8);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                __builtin_shufflevector(a[g][0], a[g][1], 0, 1, 2, 3, 4, 5, 6, 7),
                __builtin_shufflevector(b[m][0], b[m][1], 0, 1, 2, 3, 4, 5, 6, 7), f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                kOne, 0, s[m]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c[g][m][e] = fmaf(w[g >> 1], p[e], c[g][m][e]);
        }
}

template <int MT, int NG, bool GATED, int ACT>
__device__ void few_tile(const Product8Args &p, int32_t l, int32_t row0, int32_t rows, int32_t n0,
                         f32x4 (*part)[2 * NG][kWave])
{
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t wide = GATED ? 2 * (int64_t)p.N : p.N;
    const int64_t nbk = (p.K + 127) / 128, nbw = (wide + 127) / 128;
    const uint8_t *Wl = p.W + (l * wide + n0) * p.K;
    FewOperands<MT, NG> o;
    o.K = (uint32_t)p.K;
#pragma unroll
    for (int g = 0; g < NG; ++g)  // N is a multiple of 32: both groups of 16 are whole
        o.w[g] = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t *>(Wl + ((int64_t)(g >> 1) * p.N + (g & 1) * 16) * p.K), 0, 16 * o.K, kGemmBufferFlags);
    o.x = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p.a + row0 * p.a_bytes), 0,
                                            (uint32_t)(rows * p.a_bytes), kGemmBufferFlags);
    o.k_lane = (uint32_t)(lane >> 4) * 16;
    o.s_lane = (uint32_t)(lane >> 4) * 32;
    o.woff = (uint32_t)(lane & 15) * o.K + o.k_lane;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const uint32_t row = (uint32_t)(m * 16 + (lane & 15)) * (uint32_t)p.a_bytes;
        o.xoff[m] = row + o.k_lane;
        o.soff[m] = row + o.K + (uint32_t)(lane >> 4);
    }
#pragma unroll
    for (int q = 0; q < NG / 2; ++q)
        o.ws[q] = p.scale + (l * nbw + (q * (int64_t)p.N + n0) / 128) * nbk;
    f32x4 c[NG][MT];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            c[g][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int32_t full = p.K / kFewStep;  // rounds that need no check of k
    for (int32_t i = 0; i < full; ++i)
        few_step<MT, NG, false>(o, (uint32_t)(i * kFewStep + wave * kTileK8), c);
    if (full * kFewStep < p.K)
        few_step<MT, NG, true>(o, (uint32_t)(full * kFewStep + wave * kTileK8), c);
    // the waves' sums in their order; wave m finishes 16 rows
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            part[wave][g * MT + m][lane] = c[g][m];
    __syncthreads();
    if (wave < MT) {
        f32x4 v[4] = {};
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            v[g] = part[0][g * MT + wave][lane];
#pragma unroll
            for (int q = 1; q < kFewWaves; ++q)
                v[g] += part[q][g * MT + wave][lane];
        }
        const int32_t i = wave * 16 + (lane & 15);
        f32x4 z[2] = {v[0], v[1]}, u[2] = {v[2], v[3]};
        finish32<GATED, ACT>(p, l, (int64_t)row0 + i, i < rows, n0, lane, z, u);
    }
    if (p.out8 && n0 + kFewCols == p.N)
        pad_rows<kFewThreads>(p.out8 + row0 * p.out8_bytes, rows, p.N, p.out8_bytes);
    __syncthreads();
}

template <bool GATED, int ACT>
__global__ __launch_bounds__(kFewThreads, 4) void product_fp8_few_kernel(Product8Args p)
{
    constexpr int NG = GATED ? 4 : 2;
    __shared__ int32_t first[kMaxLocalExperts + 1];
    __shared__ f32x4 part[kFewWaves][2 * NG][kWave];
    const int32_t row_tiles = plan_row_tiles<kFewThreads, kFewRows>(p.off, p.El, p.max_rows, first);
    const uint32_t nct = (uint32_t)p.N / kFewCols;
    for (uint32_t u = blockIdx.x; u < row_tiles * nct; u += gridDim.x) {
        const int32_t rt = __builtin_amdgcn_readfirstlane((int32_t)(u / nct));
        const int32_t n0 = __builtin_amdgcn_readfirstlane((int32_t)(u % nct)) * kFewCols;
        const int32_t l = __builtin_amdgcn_readfirstlane(tile_expert(first, p.El, rt));
        const Rows r = expert_rows(p.off, l, p.max_rows);
        const int32_t row0 = __builtin_amdgcn_readfirstlane((int32_t)(r.begin + (int64_t)(rt - first[l]) * kFewRows));
        const int32_t rows = __builtin_amdgcn_readfirstlane(min(kFewRows, r.end - row0));
        if (rows <= 16)
            few_tile<1, NG, GATED, ACT>(p, l, row0, rows, n0, part);
        else
            few_tile<2, NG, GATED, ACT>(p, l, row0, rows, n0, part);
    }
}

}  // namespace

hipError_t launch_product_fp8_few(const Product8Args &p, int32_t act, bool gated, int cus, hipStream_t stream)
{
    const int64_t tiles = ((int64_t)p.max_rows / kFewRows + p.El) * (p.N / kFewCols);
    const dim3 grid((unsigned)(tiles < 2 * cus ? tiles : 2 * cus));
#define MOE_FEW_CASE(A)                                                                                        \
    case A:                                                                                                    \
        if (gated)                                                                                             \
            hipLaunchKernelGGL((product_fp8_few_kernel<true, A>), grid, dim3(kFewThreads), 0, stream, p);      \
        else                                                                                                   \
            hipLaunchKernelGGL((product_fp8_few_kernel<false, A>), grid, dim3(kFewThreads), 0, stream, p);     \
        return hipGetLastError();
    switch (act) {
        MOE_FEW_CASE(kActNone)
        MOE_FEW_CASE(kActRelu)
        MOE_FEW_CASE(kActSilu)
        MOE_FEW_CASE(kActGelu)
        MOE_FEW_CASE(kActGeluTanh)
    default:
        return hipErrorInvalidValue;
    }
#undef MOE_FEW_CASE
}

}  // namespace moe
