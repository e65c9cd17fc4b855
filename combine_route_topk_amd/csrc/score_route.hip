// score_route.hip -- top-k routing on softmax or sigmoid scores with a
// selection bias on the scores, and the gradient of its weights.
//
// Plain form: one wavefront per token, everything in 64-bit floating point.
#include "device.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kMaxE = 1024, kSlots = kMaxE / kWave;

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *p, int64_t i)
{
    if (BF16)
        return __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
    return static_cast<const float *>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store_logit(void *p, int64_t i, float v)
{
    if (BF16)
        static_cast<uint16_t *>(p)[i] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
    else
        static_cast<float *>(p)[i] = v;
}

__device__ __forceinline__ double wave_sum(double v)
{
    for (int d = 1; d < kWave; d <<= 1)
        v += __shfl_xor(v, d, kWave);
    return v;
}
__device__ __forceinline__ double wave_max(double v)
{
    for (int d = 1; d < kWave; d <<= 1)
        v = fmax(v, __shfl_xor(v, d, kWave));
    return v;
}

// score of one logit: sigmoid, or softmax given the row's maximum and sum
template <bool SIGMOID>
__device__ __forceinline__ double score(double l, double m, double z)
{
    if (l == -INFINITY)
        return 0.;
    return SIGMOID ? 1. / (1. + exp(-l)) : exp(l - m) / z;
}

template <bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void route_scored_kernel(
    const void *__restrict__ logits, const float *__restrict__ bias, int64_t T, int32_t E, int32_t k,
    int32_t n_groups, int32_t topk_groups, bool top2, bool normalize, float scale,
    int32_t *__restrict__ topk_idx, float *__restrict__ topk_w)
{
    __shared__ double sel_lds[kWaves][kMaxE];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= T)
        return;
    double *sel = sel_lds[wave];
    double m = -INFINITY, z = 0.;
    if (!SIGMOID) {
        for (int e = lane; e < E; e += kWave)
            m = fmax(m, (double)load_logit<BF16>(logits, t * E + e));
        m = wave_max(m);
        for (int e = lane; e < E; e += kWave)
            z += m == -INFINITY ? 0. : exp((double)load_logit<BF16>(logits, t * E + e) - m);
        z = wave_sum(z);
    }
    // order: groups out of the selection, then NaN, then -inf, then numbers
    constexpr double kNaNRank = -1.7e308;  // below every finite score; -inf is moved above it
    for (int e = lane; e < E; e += kWave) {
        const double l = load_logit<BF16>(logits, t * E + e);
        double s = l == -INFINITY ? -INFINITY : score<SIGMOID>(l, m, z) + (bias ? (double)bias[e] : 0.);
        s = s != s ? kNaNRank : (s == -INFINITY ? -1.6e308 : s);
        sel[e] = s;
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    uint64_t chosen = ~0ull;
    const int gsize = n_groups > 0 ? E / n_groups : E;
    if (n_groups > 0) {
        double b1 = -INFINITY, b2 = -INFINITY;
        if (lane < n_groups)
            for (int i = 0; i < gsize; ++i) {
                const double s = sel[lane * gsize + i];
                if (s > b1) {
                    b2 = b1;
                    b1 = s;
                } else if (s > b2) {
                    b2 = s;
                }
            }
        double g = -INFINITY;
        if (lane < n_groups) {
            g = b1;
            if (top2 && gsize > 1)
                g = b2 <= -1.6e308 ? (b2 < -1.65e308 || b1 < -1.65e308 ? kNaNRank : -1.6e308) : b1 + b2;
        }
        bool used = lane >= n_groups;
        chosen = 0;
        for (int q = 0; q < topk_groups; ++q) {
            const double best = wave_max(used ? -INFINITY : g);
            const uint64_t who = ballot64(!used && g == best);
            const int w = __ffsll((unsigned long long)who) - 1;
            chosen |= 1ull << w;
            used |= lane == w;
        }
    }
    uint32_t taken = 0;  // of this lane's slots
    int my_e = 0;
    for (int j = 0; j < k; ++j) {
        double best = -INFINITY;
        int slot = 0;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int e = i * kWave + lane;
            if (e < E && !((taken >> i) & 1u) && (n_groups == 0 || ((chosen >> (e / gsize)) & 1ull)) &&
                sel[e] > best) {
                best = sel[e];
                slot = i;
            }
        }
        const double top = wave_max(best);
        int id = best == top ? slot * kWave + lane : 0x7FFFFFFF;
        for (int d = 1; d < kWave; d <<= 1)
            id = min(id, __shfl_xor(id, d, kWave));
        if (id % kWave == lane)
            taken |= 1u << (id / kWave);
        if (lane == j)
            my_e = id;
    }
    double p = 0.;
    if (lane < k)
        p = score<SIGMOID>(load_logit<BF16>(logits, t * E + my_e), m, z);
    const double sum = normalize ? wave_sum(p) : 1.;
    if (lane < k) {
        topk_idx[t * k + lane] = my_e;
        topk_w[t * k + lane] = sum == 0. ? 0.f : (float)(scale * (p / sum));
    }
}

template <bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void route_scored_backward_kernel(
    const void *__restrict__ logits, const int32_t *__restrict__ topk_idx,
    const float *__restrict__ grad_w, int64_t T, int32_t E, int32_t k, bool normalize, float scale,
    void *__restrict__ grad_logits)
{
    __shared__ float row_lds[kWaves][kMaxE];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= T)
        return;
    float *row = row_lds[wave];
    for (int e = lane; e < E; e += kWave)
        row[e] = 0.f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    int e = -1;
    double l = -INFINITY, g = 0.;
    if (lane < k) {
        e = topk_idx[t * k + lane];
        if (e >= 0 && e < E) {
            l = load_logit<BF16>(logits, t * E + e);
            g = grad_w[t * k + lane];
        } else {
            e = -1;
        }
    }
    double m = -INFINITY, z = 0.;
    if (!SIGMOID) {
        for (int i = lane; i < E; i += kWave)
            m = fmax(m, (double)load_logit<BF16>(logits, t * E + i));
        m = wave_max(m);
        for (int i = lane; i < E; i += kWave)
            z += m == -INFINITY ? 0. : exp((double)load_logit<BF16>(logits, t * E + i) - m);
        z = wave_sum(z);
    }
    const double p = e >= 0 ? score<SIGMOID>(l, m, z) : 0.;
    const double sum = wave_sum(p);
    const double w = normalize ? (sum == 0. ? 0. : p / sum) : p;
    const double gw = wave_sum(g * w);
    double d;
    if (SIGMOID)
        d = normalize ? w * (1. - p) * (g - gw) : g * p * (1. - p);
    else
        d = normalize ? w * (g - gw) : p * (g - gw);
    if (!SIGMOID && !normalize)
        for (int i = lane; i < E; i += kWave)
            row[i] = (float)(-scale * score<false>(load_logit<BF16>(logits, t * E + i), m, z) * gw);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (e >= 0)
        row[e] = (float)(scale * d);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int i = lane; i < E; i += kWave)
        store_logit<BF16>(grad_logits, t * E + i, row[i]);
}

}  // namespace

hipError_t launch_route_scored(const void *logits, const float *bias, int64_t T, int32_t E,
                               int32_t k, int32_t n_groups, int32_t topk_groups,
                               const ScoreOpts &o, int32_t *topk_idx, float *topk_w,
                               hipStream_t stream)
{
    const int64_t chunk = kMaxRowBlocks * kWaves;
    for (int64_t t0 = 0; t0 < T; t0 += chunk) {
        const int64_t n = T - t0 < chunk ? T - t0 : chunk;
        const dim3 grid((unsigned)((n + kWaves - 1) / kWaves));
        const void *lg = static_cast<const char *>(logits) + t0 * E * (o.bf16 ? 2 : 4);
#define MOE_SCORED_LAUNCH(B, S)                                                                       \
    hipLaunchKernelGGL((route_scored_kernel<B, S>), grid, dim3(kThreads), 0, stream, lg, bias, n, E, \
                       k, n_groups, topk_groups, o.top2, o.normalize, o.scale, topk_idx + t0 * k,     \
                       topk_w + t0 * k)
        if (o.bf16 && o.sigmoid)
            MOE_SCORED_LAUNCH(true, true);
        else if (o.bf16)
            MOE_SCORED_LAUNCH(true, false);
        else if (o.sigmoid)
            MOE_SCORED_LAUNCH(false, true);
        else
            MOE_SCORED_LAUNCH(false, false);
#undef MOE_SCORED_LAUNCH
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

hipError_t launch_route_scored_backward(const void *logits, const int32_t *topk_idx,
                                        const float *grad_w, int64_t T, int32_t E, int32_t k,
                                        const ScoreOpts &o, void *grad_logits, hipStream_t stream)
{
    const int64_t chunk = kMaxRowBlocks * kWaves;
    for (int64_t t0 = 0; t0 < T; t0 += chunk) {
        const int64_t n = T - t0 < chunk ? T - t0 : chunk;
        const dim3 grid((unsigned)((n + kWaves - 1) / kWaves));
        const int64_t at = t0 * E * (o.bf16 ? 2 : 4);
        const void *lg = static_cast<const char *>(logits) + at;
        void *gl = static_cast<char *>(grad_logits) + at;
#define MOE_SCORED_LAUNCH(B, S)                                                                  \
    hipLaunchKernelGGL((route_scored_backward_kernel<B, S>), grid, dim3(kThreads), 0, stream, lg, \
                       topk_idx + t0 * k, grad_w + t0 * k, n, E, k, o.normalize, o.scale, gl)
        if (o.bf16 && o.sigmoid)
            MOE_SCORED_LAUNCH(true, true);
        else if (o.bf16)
            MOE_SCORED_LAUNCH(true, false);
        else if (o.sigmoid)
            MOE_SCORED_LAUNCH(false, true);
        else
            MOE_SCORED_LAUNCH(false, false);
#undef MOE_SCORED_LAUNCH
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace moe
