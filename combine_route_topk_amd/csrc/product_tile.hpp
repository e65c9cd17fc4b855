// product_tile.hpp -- what the products' kernels do to a tile's sums.
#pragma once

#include "fp8_device.hpp"
#include "product_epilogue.hpp"
#include "product_gemm.hpp"

namespace moe {
namespace {

constexpr int kTileK8 = 128;  // values of a K-tile in 8 bits: 128 bytes, as kTileK in bf16
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kOne = 127;  // the scale byte of 1

// a scalar load: `p` is the same in every lane and not written by this kernel
typedef __attribute__((address_space(4))) const float *uniform_floats;
__device__ __forceinline__ float load_uniform(const float *p) { return *(uniform_floats)(uintptr_t)p; }

// Zeros behind the scale bytes of FP8 rows, up to their last whole line.
template <int THREADS>
__device__ __forceinline__ void pad_rows(uint8_t *rows_, int32_t rows, int32_t width, int64_t row_bytes)
{
    const int32_t used = width / 32, words = (int32_t)(row_bytes - width) / 4, first = used / 4;
    for (int32_t i = threadIdx.x; i < rows * (words - first); i += THREADS) {
        const int32_t row = i / (words - first), word = first + i % (words - first);
        uint8_t *at = rows_ + row * row_bytes + width + word * 4;
        if (word * 4 >= used) {
            *reinterpret_cast<uint32_t *>(at) = 0;
        } else {
            for (int32_t b = used - word * 4; b < 4; ++b)
                at[b] = 0;
        }
    }
}

// the larger of this lane's value and those of the lanes 16 and 32 away
__device__ __forceinline__ float max_of_row(float m)
{
    u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    m = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// 32 columns of 16 rows, a row in lanes i, i + 16, i + 32 and i + 48 by two
// groups of four columns, 16 apart: the codes of this lane's eight consecutive
// columns, (lane / 16) * 8 + 0..7, and the scale byte that the row's 32 share.
__device__ __forceinline__ uint32_t encode32(const f32x4 (&v)[2], uint32_t (&codes)[2])
{
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        top = max_abs(max_abs(top, v[0][e]), v[1][e]);
    const int32_t exp = fp8_exponent(max_of_row(top));
    const float mul = fp8_multiplier(exp);
#pragma unroll
    for (int j = 0; j < 2; ++j)
        codes[j] = fp8_encode4(v[j][0], v[j][1], v[j][2], v[j][3], mul);
    swap32(codes[0], codes[1]);
    swap16(codes[0], codes[1]);
    return (uint32_t)(exp + 127);
}

// A tile's rows of an FP8 tensor of `width` values, through a descriptor that
// ends with the tile's last row, as TileRows for bf16.
struct TileRows8 {
    __amdgpu_buffer_rsrc_t r;
    uint32_t lane_row, rb, width;
    __device__ __forceinline__ void init(uint8_t *p, int64_t row0, int32_t rows, int64_t row_bytes, int32_t values,
                                         int lane)
    {
        r = __builtin_amdgcn_make_buffer_rsrc(p + row0 * row_bytes, 0, (uint32_t)(rows * row_bytes), kGemmBufferFlags);
        rb = (uint32_t)row_bytes;
        width = (uint32_t)values;
        lane_row = (uint32_t)(lane & 15) * rb;
    }
    // columns c0 to c0 + 31 of row m + lane % 16
    __device__ __forceinline__ void store(uint32_t m, int32_t c0, const f32x4 (&v)[2], int lane) const
    {
        uint32_t codes[2];
        const uint32_t scale = encode32(v, codes);
        const uint32_t at = lane_row + m * rb;
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{codes[0], codes[1]}, r, at + c0 + (lane >> 4) * 8, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b8((uint8_t)scale, r,
                                             lane < 16 ? at + width + ((uint32_t)c0 >> 5) : kOutside, 0, 0);
    }
};

// Bias, activation, gate, residual (or the activation's gradient) on the
// sums, and their one rounding. A group of 16 rows past the tile's last is
// skipped; the rest is without branches: the descriptors drop rows and
// columns outside. F8: the result goes to bf16 rows, to FP8 rows or to both.
template <bool GRAD, bool GATED, int ACT, bool F8, class Args, class G>
__device__ __forceinline__ void epilogue(const Args &p, const G &gemm, const Acc &acc, int32_t l,
                                         int32_t row0, int32_t rows, int32_t n0)
{
    constexpr bool PAIR = GATED && !GRAD;
    constexpr int NP = PAIR ? 1 : 2;  // pairs of a lane's groups of four columns
    const int64_t N = p.N, wide = GATED ? 2 * N : N;
    const uint32_t N2 = (uint32_t)N * 2;
    uint32_t col[NP];
    f32x4 b[NP][2], bu[NP][2];
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        const int32_t c0 = n0 + (PAIR ? gemm.wn * 32 : gemm.column(q));
        const int32_t c8 = c0 + (gemm.lane >> 4) * 8;
        col[q] = c8 < N ? (uint32_t)c8 * 2 : kOutside;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int32_t c4 = c0 + j * 16 + (gemm.lane >> 4) * 4;
            b[q][j] = bu[q][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (!GRAD && p.bias && c4 < N) {
                b[q][j] = widen(*reinterpret_cast<const u32x2 *>(p.bias + l * wide + c4));
                if (PAIR)
                    bu[q][j] = widen(*reinterpret_cast<const u32x2 *>(p.bias + l * wide + N + c4));
            }
        }
    }
    TileRows out, aux;
    if (!F8 || p.out)
        out.init(p.out, row0, rows, GRAD ? wide : N, gemm.lane);
    TileRows8 out8;
    if constexpr (F8) {
        if (p.out8)
            out8.init(p.out8, row0, rows, p.out8_bytes, (int32_t)(GRAD ? wide : N), gemm.lane);
    }
    // pair q of this lane's groups, 32 columns with the three other lanes of its row
    auto put = [&](int32_t m, int q, const f32x4 (&v)[2], bool second) {
        if (!F8 || p.out)
            out.store(m, col[q], v, second ? N2 : 0u);
        if constexpr (F8) {
            const int32_t c0 = n0 + (PAIR ? gemm.wn * 32 : gemm.column(q));
            if (p.out8 && c0 < N)
                out8.store(m, second ? (int32_t)N + c0 : c0, v, gemm.lane);
        }
    };
    if (GRAD) {
        if (p.pre_in)
            aux.init(p.pre_in, row0, rows, wide, gemm.lane);
    } else if (p.residual) {
        aux.init(p.residual, row0, rows, N, gemm.lane);
    }
    TileRows pre;
    if (!GRAD && p.pre_out)
        pre.init(p.pre_out, row0, rows, wide, gemm.lane);
    // What a group of 16 rows reads (pre, or the residual) is fetched while the
    // group before it is computed: a wave has only one other on its SIMD to
    // hide that latency.
    constexpr int NF = GRAD && GATED ? 2 : 1;
    const bool reads = GRAD ? (GATED || p.pre_in) : p.residual != nullptr;
    u32x4 ahead[2][NP][NF];
    auto row_of = [&](int s) { return (s >> 2) * 128 + gemm.wm * 64 + (s & 3) * 16; };
    auto fetch = [&](int s) {
#pragma unroll
        for (int q = 0; q < NP; ++q)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                ahead[s & 1][q][f] = aux.fetch(row_of(s), col[q], f * N2);
    };
    if (reads)
        fetch(0);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
        const int h = s >> 2, i = s & 3;
        if (reads && s < 7)
            fetch(s + 1);
        const int32_t m = row_of(s);
        if (m >= rows)
            continue;
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            f32x4 v[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                v[j] = PAIR ? acc[h][j][i][0] : acc[h][q][i][j];
            if (GRAD && GATED) {
                f32x4 z[2], u[2], dz[2], du[2];
                TileRows::unpack(ahead[s & 1][q][0], z);
                TileRows::unpack(ahead[s & 1][q][NF - 1], u);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float f, df;
                        act_and_grad<ACT>(z[j][e], f, df);
                        dz[j][e] = v[j][e] * u[j][e] * df;
                        du[j][e] = v[j][e] * f;
                    }
                put(m, q, dz, false);
                put(m, q, du, true);
            } else if (GRAD) {
                if (p.pre_in) {
                    f32x4 z[2];
                    TileRows::unpack(ahead[s & 1][q][0], z);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float f, df;
                            act_and_grad<ACT>(z[j][e], f, df);
                            v[j][e] *= df;
                        }
                }
                put(m, q, v, false);
            } else {
                f32x4 g[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    v[j] += b[q][j];
                    g[j] = PAIR ? acc[h][j][i][1] + bu[q][j] : f32x4{};
                }
                if (p.pre_out) {
                    pre.store(m, col[q], v);
                    if (PAIR)
                        pre.store(m, col[q], g, N2);
                }
                f32x4 r[2] = {};
                if (p.residual)
                    TileRows::unpack(ahead[s & 1][q][0], r);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[j][e] = (PAIR ? act<ACT>(v[j][e]) * g[j][e] : act<ACT>(v[j][e])) + r[j][e];
                put(m, q, v, false);
            }
        }
    }
}

}  // namespace
}  // namespace moe
