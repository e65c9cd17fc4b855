// quantize_weights.hip -- the experts' weights as E4M3 codes with a float32
// scale for each block of 128 x 128, and transposed for the input gradient.
//
//   scale = max|W| of the block / 448 (1 for a block of zeros);
//   code  = E4M3 nearest to W * (1 / scale)
//
// The reciprocal and the product are each rounded to float32 first: a quotient
// within 2^-23 of itself of the middle between two codes may get the other one
// than a division would give it. The definition is this one, bit for bit.
//
// Bound by HBM: W is read once and each form written once. A block of 256
// threads takes one 128 x 128 block and holds it in registers between the
// maximum and the codes, eight rows of eight columns per thread: rows as
// 256-byte (float32: 512-byte) reads, codes as whole 128-byte lines. The
// transposed codes pass through LDS, where a thread's eight codes of a column
// are one 8-byte write, and leave as whole lines too. Codes are written past the
// caches (492 against 514 us, 32 x 4096 x 7168). Weights that the last-level
// cache can hold are read through it, since what updated them may have left them
// there (8 x 1536 x 2048, read again: 16.2 against 19.6 us); larger ones past it
// (492 against 512 us).
#include "fp8_device.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kQThreads = 256;
constexpr int64_t kCached = (int64_t)128 << 20;  // half of the last-level cache
constexpr int kQStride = 144;  // bytes of an LDS row of 128: 16-byte reads stay aligned
// An LDS row's 16-byte pieces are permuted by the row's eight, since the 16
// threads that write together lie eight rows apart, a multiple of the banks: two
// share a bank, where eight would (8 x 1536 x 2048, both layouts: 16.2 against 17.0 us).
__device__ __forceinline__ int32_t lds_at(int32_t row, int32_t byte) { return row * kQStride + (byte ^ ((row >> 3 & 7) << 4)); }

template <bool FP32, bool STREAM>
__global__ __launch_bounds__(kQThreads) void quantize_weights_kernel(QuantizeArgs p)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[128 * kQStride];
    __shared__ float part[kQThreads / kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int32_t nbO = (p.O + 127) / 128, nbH = (p.H + 127) / 128;
    const int64_t bh = blockIdx.x % nbH, bo = blockIdx.x / nbH % nbO, n = blockIdx.x / nbH / nbO + p.first;
    const int32_t r0 = threadIdx.x / 16 * 8, c = threadIdx.x % 16 * 8;  // this thread's rows and columns
    const int32_t o0 = (int32_t)bo * 128, h = (int32_t)bh * 128 + c;
    const int32_t rows = min(8, p.O - o0 - r0);  // a multiple of 8, as are O and H
    const bool in = rows > 0 && h < p.H;
    float v[8][8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u32x4 q0 = {0u, 0u, 0u, 0u}, q1 = q0;
        if (in) {
            const int64_t at = (n * p.O + o0 + r0 + i) * p.H + h;
            const u32x4 *W = static_cast<const u32x4 *>(p.W) + at / (FP32 ? 4 : 8);
            q0 = STREAM ? load_stream(W) : W[0];
            if (FP32)
                q1 = STREAM ? load_stream(W + 1) : W[1];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[i][e] = FP32 ? __uint_as_float(e < 4 ? q0[e & 3] : q1[e & 3])
                           : (e & 1 ? bf16_hi(q0[e >> 1]) : bf16_lo(q0[e >> 1]));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            m = max_abs(m, v[i][e]);
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1)
        m = fmaxf(m, __shfl_xor(m, d, kWave));
    if (lane == 0)
        part[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    // no smaller than float32's least normal, so that its reciprocal is finite
    const float scale = m > 0.f ? fmaxf(m / 448.f, 1.17549435e-38f) : 1.f;
    const float mul = 1.f / scale;
    u32x2 code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        code[i] = u32x2{fp8_encode4(v[i][0], v[i][1], v[i][2], v[i][3], mul),
                        fp8_encode4(v[i][4], v[i][5], v[i][6], v[i][7], mul)};
    if (in)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            __builtin_nontemporal_store(code[i], reinterpret_cast<u32x2 *>(p.codes + (n * p.O + o0 + r0 + i) * p.H + h));
    if (threadIdx.x == 0) {
        p.scale[(n * nbO + bo) * nbH + bh] = scale;
        if (p.codes_t)
            p.scale_t[(n * nbH + bh) * nbO + bo] = scale;
    }
    if (!p.codes_t)
        return;
    // column e of the thread's eight rows: byte e of each row's codes
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        u32x2 col;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t a = code[4 * q][e >> 2], b = code[4 * q + 1][e >> 2], d = code[4 * q + 2][e >> 2],
                           f = code[4 * q + 3][e >> 2];
            const uint32_t s = (uint32_t)(e & 3);
            const uint32_t lo = __builtin_amdgcn_perm(b, a, s | (s + 4) << 8 | 0x0C0C0000u);
            const uint32_t hi = __builtin_amdgcn_perm(f, d, s | (s + 4) << 8 | 0x0C0C0000u);
            col[q] = lo | hi << 16;
        }
        *reinterpret_cast<u32x2 *>(lds + lds_at(c + e, r0)) = col;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = i * 32 + threadIdx.x / 8, piece = threadIdx.x % 8 * 16;  // a column of W, 16 of its codes
        const int32_t hr = (int32_t)bh * 128 + row;
        if (hr < p.H && o0 + piece < p.O)  // O is a multiple of 32: a piece is whole
            store_stream(reinterpret_cast<u32x4 *>(p.codes_t + (n * p.H + hr) * p.O + o0 + piece),
                         *reinterpret_cast<const u32x4 *>(lds + lds_at(row, piece)));
    }
}

}  // namespace

hipError_t launch_quantize_weights(QuantizeArgs p, int64_t n, bool fp32, hipStream_t stream)
{
    const int64_t each = (int64_t)((p.O + 127) / 128) * ((p.H + 127) / 128);  // at most 2^19
    const int64_t most = kMaxRowBlocks / each;
    const bool stream_in = n * p.O * p.H * (fp32 ? 4 : 2) > kCached;
    for (p.first = 0; p.first < n; p.first += most) {
        const dim3 grid((unsigned)((n - p.first < most ? n - p.first : most) * each));
#define MOE_QUANTIZE(F, S) hipLaunchKernelGGL((quantize_weights_kernel<F, S>), grid, dim3(kQThreads), 0, stream, p)
        if (fp32) {
            if (stream_in)
                MOE_QUANTIZE(true, true);
            else
                MOE_QUANTIZE(true, false);
        } else {
            if (stream_in)
                MOE_QUANTIZE(false, true);
            else
                MOE_QUANTIZE(false, false);
        }
#undef MOE_QUANTIZE
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace moe
