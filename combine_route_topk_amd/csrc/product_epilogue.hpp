// product_epilogue.hpp -- the arguments of the experts' product kernels, and
// what the kernel for few rows does to each sum.
#pragma once

#include "product_device.hpp"

namespace moe {

struct ProductArgs {
    const uint16_t *a;         // x, or grad_y of the input gradient
    const int32_t *off;
    const uint16_t *W, *bias, *residual, *pre_in;
    uint16_t *pre_out, *out;
    int32_t El, max_rows, K, N;  // N: columns before a gate doubles them
};

hipError_t launch_product_few(const ProductArgs &p, int32_t act, bool gated, hipStream_t stream);

// compute units of the current device
inline hipError_t current_cus(int *cus)
{
    int device = 0;
    const hipError_t err = hipGetDevice(&device);
    return err == hipSuccess ? hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, device) : err;
}

namespace {

__device__ __forceinline__ void load4(const uint16_t *p, float (&v)[4])
{
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    v[0] = bf16_lo(w.x);
    v[1] = bf16_hi(w.x);
    v[2] = bf16_lo(w.y);
    v[3] = bf16_hi(w.y);
}
__device__ __forceinline__ void store4(uint16_t *p, const float (&v)[4])
{
    *reinterpret_cast<uint2 *>(p) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// Four columns of one row from their sums z (gated: and those they gate, g):
// bias, activation, gate and residual, then the one rounding.
template <bool GATED, int ACT, class V>
__device__ __forceinline__ void finish4(const ProductArgs &p, int32_t l, int64_t row, int32_t c, const V &zs,
                                        const V &gs)
{
    const int64_t wide = GATED ? 2 * (int64_t)p.N : p.N;
    float z[4], g[4], b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        z[e] = zs[e];
        g[e] = gs[e];
    }
    if (p.bias) {
        load4(p.bias + l * wide + c, b);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            z[e] += b[e];
        if (GATED) {
            load4(p.bias + l * wide + p.N + c, b);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                g[e] += b[e];
        }
    }
    if (p.pre_out) {
        store4(p.pre_out + row * wide + c, z);
        if (GATED)
            store4(p.pre_out + row * wide + p.N + c, g);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        z[e] = GATED ? act<ACT>(z[e]) * g[e] : act<ACT>(z[e]);
    if (p.residual) {
        load4(p.residual + row * p.N + c, b);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            z[e] += b[e];
    }
    store4(p.out + row * p.N + c, z);
}

}  // namespace
}  // namespace moe
