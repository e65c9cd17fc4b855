// product_fp8_some.hpp -- the experts' product on FP8 rows for some tens of rows
// per expert (a decoding batch): the weights' way from memory bounds it, but
// the rows are too many to be read again for every 32 columns
// (product_fp8_few.hip), and too few to fill the 256 rows of product_fp8.hip,
// whose LDS then holds mostly zeros and whose loads in flight are half A's.
//
// A block of eight waves takes up to 64 or 128 rows of one expert by 256 rows of
// W (gated: 128 gate rows and the 128 they gate), 128 k at a time: 48 KiB, in
// three stages. Loads go from memory straight to LDS; while a stage is
// multiplied the next two are in flight, 64 KiB of W for each CU, and one
// barrier a stage orders both the stage's arrival and its reuse. Waves 0 to 3
// take 16 of each 32 rows, waves 4 to 7 the others, 64 rows of W each.
// On MI355X, 32 experts, 7168 by 2 x 2048, rows spread evenly: 158 us for 32 rows
// (6.0 TB/s of weights), 162 for 1024, 167 for 2048, 211 for 4096; few 163, 215, 372
// and 715, tiles of 256 rows 188, 192, 211 and 237.
#pragma once

#include "product_fp8_device.hpp"

namespace moe {
namespace {

constexpr int kSomeThreads = 512;
constexpr int kSomeRows = 128, kSomeCols = 256, kStages = 3;
constexpr int kSomeA = kSomeCols * kTileK8;                       // of A in a stage, behind W
constexpr int kSomeStage = kSomeA + kSomeRows * kTileK8;
constexpr int kSomeScales = kStages * kSomeStage, kSomeGroup = kSomeRows * 16;  // scales of four K-tiles, two groups
constexpr int kSomeLds = kSomeScales + 2 * kSomeGroup;
constexpr int kSomeLoads = 5;                                     // of a wave for a stage, one more past 64 rows

struct SomeOperands {
    u32x4 w[2], x, s;            // descriptors: 128 rows of W each, the rows, their scales
    uint32_t woff, xoff, soff;   // this lane's bytes in a wave's load
    uint32_t second;             // from one load of W's rows to the next, 64 rows on
    uint32_t xsecond;            // and of x's; zero where the tile has no more than 64
};

// Starts a stage's loads, of the 128 k at byte k0 of the rows (kNothing: zeros).
constexpr uint32_t kNothing = 0x40000000u;  // past every descriptor's end here, and no carry
__device__ __forceinline__ void some_load(const SomeOperands &o, uint32_t dst, uint32_t k0)
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            // the descriptor's end is checked less the scalar offset, which must not pass it
            load_to_lds(dst + (h * 2 + i) * 8192, o.w[h], o.woff, min(k0 + i * o.second, o.w[h][2]));
    load_to_lds(dst + kSomeA, o.x, o.xoff, min(k0, o.x[2]));
    if (o.xsecond)
        load_to_lds(dst + kSomeA + 8192, o.x, o.xoff, min(k0 + o.xsecond, o.x[2]));
}

// One tile: `rows` rows of expert l from row0 by kCols columns from n0. Every
// thread of the block takes part. LDS may be overwritten until the call, and
// again on return.
template <bool GRAD, bool GATED, int ACT>
__device__ void some_tile(const Product8Args &p, uint32_t lds, int32_t l, int32_t row0, int32_t rows, int32_t n0)
{
    constexpr bool PAIR = GATED && !GRAD;
    constexpr int kCols = PAIR ? kSomeCols / 2 : kSomeCols;
    const int64_t wide = PAIR ? 2 * (int64_t)p.N : p.N;
    const int nk = (p.K + kTileK8 - 1) / kTileK8;
    const int64_t nbw = (wide + 127) / 128;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wr = wave >> 2, wc = wave & 3;
    // a wave's load covers eight rows; pieces are permuted by the row's number, as in product_gemm.hpp
    const int load_row = wave * 8 + (lane >> 3), piece = ((lane & 7) ^ (lane >> 3)) * 16;
    const uint32_t tail = p.K % kTileK8 && piece >= p.K % kTileK8 ? kOutside : 0u;
    const int last_scales = (p.K - 1) % kTileK8 / 32 + 1;
    uint32_t fx[2], fw[2];  // this lane's pieces of a fragment: 16 k of the first 64, and of the second
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
        fx[kk] = lds + kSomeA + frag_row(wr * 16, kk, lane);
        // gated: 32 gate rows, then the 32 up rows 128 further
        fw[kk] = lds + frag_row(PAIR ? wc * 32 : wc * 64, kk, lane);
    }
    constexpr int kUp = (PAIR ? 128 : 32) * kTileK8;  // from fragments 0, 1 to 2, 3
    const uint32_t scale_at = lds + kSomeScales + (uint32_t)((wr * 16 + (lane & 15)) * 16 + (lane >> 4));
    SomeOperands o;
    const uint8_t *Wl = p.W + (l * wide + n0) * p.K;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int32_t left = PAIR ? p.N - n0 : p.N - n0 - h * 128;
        o.w[h] = descriptor(Wl + (PAIR ? h * (int64_t)p.N : h * 128) * p.K,
                            __builtin_amdgcn_readfirstlane((uint32_t)(min(max(left, 0), 128) * p.K)));
    }
    const uint8_t *x = p.a + row0 * p.a_bytes;
    o.x = descriptor(x, __builtin_amdgcn_readfirstlane((uint32_t)(rows * p.a_bytes)));
    o.s = descriptor(x + p.K, __builtin_amdgcn_readfirstlane((uint32_t)(rows * p.a_bytes - p.K)));
    o.woff = (uint32_t)load_row * (uint32_t)p.K + piece;
    o.xoff = (uint32_t)load_row * (uint32_t)p.a_bytes + piece;
    o.soff = (uint32_t)(wave * kWave + lane) * (uint32_t)p.a_bytes;
    o.second = 64u * (uint32_t)p.K;
    const bool tall = rows > 64;
    o.xsecond = tall ? 64u * (uint32_t)p.a_bytes : 0u;
    // the weights' scales along K: of this wave's first 32 rows of W and of its last 32
    const float *ws[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t c = PAIR ? j * (int64_t)p.N + min(n0 + wc * 32, p.N - 32) : min(n0 + wc * 64 + j * 32, p.N - 32);
        ws[j] = p.scale + (l * nbw + c / 128) * nk;
    }
    // rows m * 32 + wr * 16 and on of group m, so that few rows too are shared by all waves
    constexpr int kGroups = kSomeRows / 32;
    f32x4 c[4][kGroups];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int m = 0; m < kGroups; ++m)
            c[g][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t mine = lds + wave * 1024;  // where this wave's loads begin
    auto load_stage = [&](int t) {
        if (t == nk - 1) {  // its pieces past K read as zeros, in x and W alike
            o.woff |= tail;
            o.xoff |= tail;
        }
        some_load(o, mine + t % kStages * kSomeStage, t < nk ? (uint32_t)t * kTileK8 : kNothing);
    };
    auto load_scales = [&](int q) {  // of K-tiles 4 q to 4 q + 3
        if (wave < kSomeRows / kWave)
            load_to_lds(lds + kSomeScales + (q & 1) * kSomeGroup + wave * (kWave * 16), o.s, o.soff, q * 16);
    };
    load_scales(0);
    load_stage(0);
    load_stage(1);
    for (int t = 0; t < nk; ++t) {
        // this stage has arrived, and every wave has read the one before it to its end
        if (tall)
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kSomeLoads + 1) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kSomeLoads) : "memory");
        const float w[2] = {load_uniform(ws[0] + t), load_uniform(ws[1] + t)};
        if ((t & 3) == 0 && t + 4 < nk)
            load_scales((t >> 2) + 1);
        load_stage(t + 2);
        const uint32_t at = t % kStages * kSomeStage;
        uint32_t from = scale_at + (t >> 2 & 1) * kSomeGroup + (t & 3) * 4;
        if (t == nk - 1)  // past K zeros meet the last scale that is one, not what lies behind it
            from -= max((lane >> 4) + 1 - last_scales, 0);
        if (rows <= wr * 16)
            continue;
        i32x8 a[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
            a[g] = read_frag(fw[0] + (at + (g >> 1) * kUp + (g & 1) * 2048), fw[1] + (at + (g >> 1) * kUp + (g & 1) * 2048));
#pragma unroll
        for (int m = 0; m < kGroups; ++m) {
            if (rows <= m * 32 + wr * 16)
                break;
            const i32x8 b = read_frag(fx[0] + (at + m * 4096), fx[1] + (at + m * 4096));
            const uint32_t s = lds_read<uint8_t>(from + m * 512);
            f32x4 q[4];
#pragma unroll
            for (int g = 0; g < 4; ++g)
                q[g] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[g], b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, kOne, 0, s);
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    c[g][m][e] = fmaf(w[g >> 1], q[g][e], c[g][m][e]);
        }
    }
    // the last stage's reads are done before the next tile's loads; those still in flight bring zeros
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int m = 0; m < kGroups; ++m) {
        const int32_t i = m * 32 + wr * 16 + (lane & 15);
        if (rows <= m * 32 + wr * 16)
            continue;
        const bool in = i < rows;
        if (PAIR) {
            if (n0 + wc * 32 < p.N) {
                f32x4 z[2] = {c[0][m], c[1][m]}, g[2] = {c[2][m], c[3][m]};
                finish32<true, ACT>(p, l, (int64_t)row0 + i, in, n0 + wc * 32, lane, z, g);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (n0 + wc * 64 + j * 32 < p.N) {
                    f32x4 z[2] = {c[2 * j][m], c[2 * j + 1][m]}, g[2] = {};
                    if constexpr (GRAD)
                        finish32_grad<GATED, ACT>(p, (int64_t)row0 + i, in, n0 + wc * 64 + j * 32, lane, z);
                    else
                        finish32<false, ACT>(p, l, (int64_t)row0 + i, in, n0 + wc * 64 + j * 32, lane, z, g);
                }
        }
    }
    if (p.out8 && n0 + kCols >= p.N)
        pad_rows<kSomeThreads>(p.out8 + row0 * p.out8_bytes, rows, GATED && GRAD ? 2 * p.N : p.N, p.out8_bytes);
}

}  // namespace
}  // namespace moe
