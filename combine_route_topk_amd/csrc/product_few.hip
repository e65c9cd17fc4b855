// product_few.hip -- the experts' product for few rows per expert (decoding):
// the weights' way from memory bounds it, so W is read once, straight into
// MFMA fragments, with as many bytes in flight as registers allow.
//
// A block of eight waves takes up to 32 rows of one expert by 32 output columns
// (gated: 32 gate columns and the 32 they gate). Its waves share K, 64 at a
// time in turn, so that a block reads 1024 consecutive bytes of each W row,
// and add their sums through LDS, in the waves' order. A lane loads 32
// consecutive bytes of W and of x for every 64 k: the k of an MFMA's lane are
// permuted, alike for both operands, so that four lanes read a row's whole
// 128-byte line. 32 columns make two blocks per CU where a single token leaves
// eight experts with a row each and 2048 columns.
#include "product_gemm.hpp"
#include "product_epilogue.hpp"

namespace moe {
namespace {

constexpr int kFewThreads = 512, kFewWaves = kFewThreads / kWave;
constexpr int kFewRows = 32, kFewCols = 32;
constexpr int kFewStep = kFewWaves * kTileK;  // k of one round of the block's waves

// One wave's share of the sums: MT groups of 16 rows, NG of 16 W rows (gated:
// two of gate columns, then the two that they gate).
template <int MT, int NG>
struct FewSums {
    f32x4 c[NG][MT];
};

// 64 k from k0: this lane's two fragments of W rows and of x rows
template <int MT, int NG>
__device__ __forceinline__ void few_step(const __amdgpu_buffer_rsrc_t (&w)[NG], __amdgpu_buffer_rsrc_t x,
                                         uint32_t woff, const uint32_t (&xoff)[MT], uint32_t kb, FewSums<MT, NG> &s)
{
    bf16x8 a[NG][2], b[MT][2];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            a[g][h] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(w[g], woff + kb + h * 16, 0, 0));
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            b[m][h] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(x, xoff[m] + kb + h * 16, 0, 0));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                s.c[g][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[g][h], b[m][h], s.c[g][m], 0, 0, 0);
}

template <int MT, int NG, bool GATED, int ACT>
__device__ void few_tile(const ProductArgs &p, int32_t l, int32_t row0, int32_t rows, int32_t n0,
                         f32x4 (*part)[2 * NG][kWave])
{
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t K2 = (uint32_t)p.K * 2;
    const uint16_t *Wl = p.W + ((int64_t)l * (GATED ? 2 * (int64_t)p.N : p.N) + n0) * p.K;
    __amdgpu_buffer_rsrc_t w[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int32_t cols = min(16, p.N - n0 - (g & 1) * 16);
        w[g] = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t *>(Wl + ((int64_t)(g >> 1) * p.N + (g & 1) * 16) * p.K), 0, cols > 0 ? cols * K2 : 0u,
            kGemmBufferFlags);
    }
    const __amdgpu_buffer_rsrc_t x = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t *>(p.a + (int64_t)row0 * p.K), 0, rows * K2, kGemmBufferFlags);
    const uint32_t at = (uint32_t)(wave * kTileK + (lane >> 4) * 16) * 2;  // of this lane's k
    const uint32_t woff = (uint32_t)(lane & 15) * K2 + at;
    uint32_t xoff[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        xoff[m] = (uint32_t)(m * 16 + (lane & 15)) * K2 + at;
    FewSums<MT, NG> s;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            s.c[g][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int32_t full = p.K / kFewStep;  // rounds that need no check of k
    for (int32_t i = 0; i < full; ++i)
        few_step<MT, NG>(w, x, woff, xoff, (uint32_t)i * (kFewStep * 2), s);
    if (full * kFewStep < p.K) {
        // the last round: pieces past K read as zeros, in x and W alike
        const uint32_t kb = (uint32_t)full * (kFewStep * 2);
        bf16x8 a[NG][2], b[MT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t cut = kb + at + h * 16 >= K2 ? kOutside : 0u;
#pragma unroll
            for (int g = 0; g < NG; ++g)
                a[g][h] = __builtin_bit_cast(
                    bf16x8, __builtin_amdgcn_raw_buffer_load_b128(w[g], (woff + kb + h * 16) | cut, 0, 0));
#pragma unroll
            for (int m = 0; m < MT; ++m)
                b[m][h] = __builtin_bit_cast(
                    bf16x8, __builtin_amdgcn_raw_buffer_load_b128(x, (xoff[m] + kb + h * 16) | cut, 0, 0));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    s.c[g][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[g][h], b[m][h], s.c[g][m], 0, 0, 0);
    }
    // the waves' sums in their order; wave q finishes one group of rows and columns
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            part[wave][g * MT + m][lane] = s.c[g][m];
    __syncthreads();
    if (wave < 2 * MT) {
        const int m = wave >> 1, cg = wave & 1;
        f32x4 v[2] = {};
#pragma unroll
        for (int g = 0; g < NG / 2; ++g) {
            v[g] = part[0][(g * 2 + cg) * MT + m][lane];
#pragma unroll
            for (int q = 1; q < kFewWaves; ++q)
                v[g] += part[q][(g * 2 + cg) * MT + m][lane];
        }
        const int32_t i = m * 16 + (lane & 15), c = n0 + cg * 16 + (lane >> 4) * 4;
        if (i < rows && c < p.N)
            finish4<GATED, ACT>(p, l, (int64_t)row0 + i, c, v[0], v[1]);
    }
    __syncthreads();
}

template <bool GATED, int ACT>
__global__ __launch_bounds__(kFewThreads, 4) void product_few_kernel(ProductArgs p)
{
    constexpr int NG = GATED ? 4 : 2;
    __shared__ int32_t first[kMaxLocalExperts + 1];
    __shared__ f32x4 part[kFewWaves][2 * NG][kWave];
    const int32_t row_tiles = plan_row_tiles<kFewThreads, kFewRows>(p.off, p.El, p.max_rows, first);
    const uint32_t nct = (uint32_t)(p.N + kFewCols - 1) / kFewCols;
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

hipError_t launch_product_few(const ProductArgs &p, int32_t act, bool gated, hipStream_t stream)
{
    int cus = 0;
    const hipError_t err = current_cus(&cus);
    if (err != hipSuccess)
        return err;
    const int64_t tiles = ((int64_t)p.max_rows / kFewRows + p.El) * ((p.N + kFewCols - 1) / kFewCols);
    const dim3 grid((unsigned)(tiles < 2 * cus ? tiles : 2 * cus));
#define MOE_FEW_CASE(A)                                                                                        \
    case A:                                                                                                    \
        if (gated)                                                                                             \
            hipLaunchKernelGGL((product_few_kernel<true, A>), grid, dim3(kFewThreads), 0, stream, p);          \
        else                                                                                                   \
            hipLaunchKernelGGL((product_few_kernel<false, A>), grid, dim3(kFewThreads), 0, stream, p);         \
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
