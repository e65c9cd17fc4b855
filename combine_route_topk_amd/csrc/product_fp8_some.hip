// product_fp8_some.hip -- the kernel for some tens of rows per expert, and its
// launch; product_fp8_some.hpp has the tile.
#include "product_fp8_some.hpp"

namespace moe {
namespace {

template <bool GRAD, bool GATED, int ACT>
__global__ __launch_bounds__(kSomeThreads, 2) void product_fp8_some_kernel(Product8Args p)
{
    constexpr int kCols = GATED && !GRAD ? kSomeCols / 2 : kSomeCols;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kSomeLds];
    __shared__ int32_t first[kMaxLocalExperts + 1];
    const uint32_t nct = (uint32_t)(p.N + kCols - 1) / kCols;
    // 64 rows a tile where all tiles are computed at once: more blocks, and fewer rows for each (4 experts of
    // 128 rows, 7168 by 7168: 65 us, 75 with 128).
    int32_t height = kSomeRows / 2;
    int32_t row_tiles =
        __builtin_amdgcn_readfirstlane(plan_row_tiles<kSomeThreads, kSomeRows / 2>(p.off, p.El, p.max_rows, first));
    if (row_tiles * nct > gridDim.x) {
        height = kSomeRows;
        row_tiles = __builtin_amdgcn_readfirstlane(plan_row_tiles<kSomeThreads, kSomeRows>(p.off, p.El, p.max_rows, first));
    }
    // An XCD's blocks take neighbouring tiles, which share rows (64 experts of 64 rows, 2048 by 2048: 53 against
    // 58 us), where there are tiles for all (4 of 64, 7168 by 7168: 59 against 50).
    const bool all = gridDim.x % 8 == 0 && row_tiles * nct >= gridDim.x;
    const uint32_t slot = all ? blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8 : blockIdx.x;
    for (uint32_t u = slot; u < row_tiles * nct; u += gridDim.x) {
        const int32_t rt = __builtin_amdgcn_readfirstlane((int32_t)(u / nct));
        const int32_t n0 = __builtin_amdgcn_readfirstlane((int32_t)(u % nct)) * kCols;
        const int32_t l = __builtin_amdgcn_readfirstlane(tile_expert(first, p.El, rt));
        const Rows r = expert_rows(p.off, l, p.max_rows);
        const int32_t row0 = __builtin_amdgcn_readfirstlane((int32_t)(r.begin + (int64_t)(rt - first[l]) * height));
        const int32_t rows = __builtin_amdgcn_readfirstlane(min(height, r.end - row0));
        some_tile<GRAD, GATED, ACT>(p, lds_offset(lds), l, row0, rows, n0);
    }
}

template <bool GRAD>
hipError_t launch_some(const Product8Args &p, int32_t act, bool gated, int cus, hipStream_t stream)
{
    const int kCols = gated && !GRAD ? kSomeCols / 2 : kSomeCols;
    const int64_t tiles = (2 * (int64_t)p.max_rows / kSomeRows + p.El) * ((p.N + kCols - 1) / kCols);
    const dim3 grid((unsigned)(tiles < cus ? tiles : cus));
#define MOE_SOME_CASE(A)                                                                                              \
    case A:                                                                                                           \
        if (gated)                                                                                                    \
            hipLaunchKernelGGL((product_fp8_some_kernel<GRAD, true, A>), grid, dim3(kSomeThreads), 0, stream, p);     \
        else                                                                                                          \
            hipLaunchKernelGGL((product_fp8_some_kernel<GRAD, false, A>), grid, dim3(kSomeThreads), 0, stream, p);    \
        return hipGetLastError();
    switch (act) {
        MOE_SOME_CASE(kActNone)
        MOE_SOME_CASE(kActRelu)
        MOE_SOME_CASE(kActSilu)
        MOE_SOME_CASE(kActGelu)
        MOE_SOME_CASE(kActGeluTanh)
    default:
        return hipErrorInvalidValue;
    }
#undef MOE_SOME_CASE
}

}  // namespace

hipError_t launch_product_fp8_some(const Product8Args &p, int32_t act, bool gated, bool grad, int cus, hipStream_t stream)
{
    return grad ? launch_some<true>(p, act, gated, cus, stream) : launch_some<false>(p, act, gated, cus, stream);
}

}  // namespace moe
