// product_fp8_device.hpp -- what the products' kernels on FP8 rows share.
#pragma once

#include "product_tile.hpp"

namespace moe {
namespace {

// A load of 16 bytes per lane into LDS, at `dst` and 16 bytes on for each lane.
// It is written as an instruction (it has no register result) so that the
// compiler does not know of it: it would wait for all such loads in flight
// before every LDS read. The schedule below orders them with barriers and
// counted waits instead. (M0 cannot be named as overwritten; nothing else in
// these kernels uses it.) Nor does it look here for hazards: a scalar register
// that a vector instruction wrote, such as one read back from where it was
// spilled, may be read by a load five wait states later, which the block holds
// itself.
__device__ __forceinline__ void load_to_lds(uint32_t dst, u32x4 r, uint32_t off, uint32_t soff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(dst), "v"(off), "s"(r), "s"(soff)
                 : "memory");
}

__device__ __forceinline__ u32x4 descriptor(const uint8_t *p, uint32_t records)
{
    const uint64_t at = (uint64_t)(uintptr_t)p;
    return u32x4{(uint32_t)at, (uint32_t)(at >> 32), records, (uint32_t)kGemmBufferFlags};
}

template <class T>
__device__ __forceinline__ T lds_read(uint32_t at)
{
    return *(__attribute__((address_space(3))) const T *)(uintptr_t)at;
}

__device__ __forceinline__ i32x8 read_frag(uint32_t at0, uint32_t at1)
{
    const i32x4 lo = lds_read<i32x4>(at0), hi = lds_read<i32x4>(at1);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 32 finished columns from c0 of the output's rows, which hold `width` values:
// to bf16, to FP8 or to both.
__device__ __forceinline__ void put32(const Product8Args &p, int64_t row, bool in, int32_t width, int32_t c0, int lane,
                                      const f32x4 (&v)[2])
{
    if (p.out && in)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<u32x2 *>(p.out + row * width + c0 + j * 16 + (lane >> 4) * 4) = narrow(v[j]);
    if (p.out8) {
        uint32_t codes[2];
        const uint32_t scale = encode32(v, codes);
        uint8_t *at = p.out8 + row * p.out8_bytes;
        if (in) {
            *reinterpret_cast<u32x2 *>(at + c0 + (lane >> 4) * 8) = u32x2{codes[0], codes[1]};
            if (lane < 16)
                at[width + c0 / 32] = (uint8_t)scale;
        }
    }
}

// 32 columns from n0 of 16 rows, a row in lanes i, i + 16, i + 32 and i + 48:
// columns j * 16 + (lane / 16) * 4 + 0..3 of sums z[j] (gated: and those that
// they gate, u[j]). Bias, activation, gate and residual, then the one rounding
// of each output. Lanes with `in` false take part in the row's maximum only.
template <bool GATED, int ACT>
__device__ __forceinline__ void finish32(const Product8Args &p, int32_t l, int64_t row, bool in, int32_t n0, int lane,
                                         f32x4 (&z)[2], f32x4 (&u)[2])
{
    const int64_t wide = GATED ? 2 * (int64_t)p.N : p.N;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int32_t c = n0 + j * 16 + (lane >> 4) * 4;
        auto read = [](const uint16_t *q) { return widen(*reinterpret_cast<const u32x2 *>(q)); };
        auto write = [](uint16_t *q, f32x4 v) { *reinterpret_cast<u32x2 *>(q) = narrow(v); };
        if (p.bias) {
            z[j] += read(p.bias + l * wide + c);
            if (GATED)
                u[j] += read(p.bias + l * wide + p.N + c);
        }
        if (p.pre_out && in) {
            write(p.pre_out + row * wide + c, z[j]);
            if (GATED)
                write(p.pre_out + row * wide + p.N + c, u[j]);
        }
        f32x4 r = {0.f, 0.f, 0.f, 0.f};
        if (p.residual && in)
            r = read(p.residual + row * p.N + c);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            z[j][e] = (GATED ? act<ACT>(z[j][e]) * u[j][e] : act<ACT>(z[j][e])) + r[e];
    }
    put32(p, row, in, p.N, n0, lane, z);
}

// As finish32 for the input gradient: d through the activation's gradient at pre.
template <bool GATED, int ACT>
__device__ __forceinline__ void finish32_grad(const Product8Args &p, int64_t row, bool in, int32_t n0, int lane,
                                              f32x4 (&d)[2])
{
    const int64_t wide = GATED ? 2 * (int64_t)p.N : p.N;
    f32x4 du[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int32_t c = n0 + j * 16 + (lane >> 4) * 4;
        f32x4 z = {0.f, 0.f, 0.f, 0.f}, u = z;
        if (p.pre_in && in) {
            z = widen(*reinterpret_cast<const u32x2 *>(p.pre_in + row * wide + c));
            if (GATED)
                u = widen(*reinterpret_cast<const u32x2 *>(p.pre_in + row * wide + p.N + c));
        }
        if (p.pre_in)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float f, df;
                act_and_grad<ACT>(z[e], f, df);
                du[j][e] = d[j][e] * f;
                d[j][e] *= GATED ? u[e] * df : df;
            }
    }
    put32(p, row, in, (int32_t)wide, n0, lane, d);
    if (GATED)
        put32(p, row, in, (int32_t)wide, p.N + n0, lane, du);
}

}  // namespace
}  // namespace moe
