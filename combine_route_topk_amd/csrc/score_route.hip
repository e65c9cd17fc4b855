// score_route.hip -- top-k routing on softmax or sigmoid scores with a
// selection bias on the scores, and the gradient of its weights.
//
// Forward. One wavefront routes one token (2 to 16 tokens for short rows), as
// in route_topk.hip, whose selection it shares: lanes hold the scores as
// order-preserving 32-bit keys. Without a bias the scores of both kinds rise
// with the logit, so the logit itself is the key and the order is exact. With
// one, keys are float32 scores, each within a derived bound of the exact
// value; when two neighbours among the k best are closer than their bounds, or
// the last of them and the best one left (the last group taken and the best
// one left) closer than a bound for every one left, the whole wave ranks that
// token again in 64-bit arithmetic. Random scores need that for under 1% of
// tokens, so the float32 pass sets the time. Rows of more than 512 experts are
// ranked in 64 bits from the start.
//
// Backward. Scores are recomputed from the logits. The k gradients of a token
// are scattered into a row of LDS, so that every lane then reads what belongs
// to its experts and writes whole 16-byte pieces of the gradient's row.
#include "launch.hpp"
#include "route_device.hpp"

namespace moe {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kU = 5.9604644775390625e-8f;  // 2^-24, half a step of float32

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *row, int32_t e)
{
    if (BF16)
        return __uint_as_float((uint32_t)static_cast<const uint16_t *>(row)[e] << 16);
    return static_cast<const float *>(row)[e];
}

// The row's logits (or the biases) in this lane's slots (slot_id's order),
// -inf past E.
template <bool BF16, int NSLOT, int VEC, int HW>
__device__ __forceinline__ void load_row(const void *row, int32_t E, int gl, bool valid, float (&l)[NSLOT])
{
    if (VEC == 4) {
#pragma unroll
        for (int q = 0; q < NSLOT / 4; ++q) {
            f32x4 v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (valid && q * 4 * HW + 4 * gl < E) {
                if (BF16) {
                    const u32x2 w = __builtin_nontemporal_load(static_cast<const u32x2 *>(row) + q * HW + gl);
                    v = {bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
                } else {
                    v = __builtin_nontemporal_load(static_cast<const f32x4 *>(row) + q * HW + gl);
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                l[4 * q + c] = v[c];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NSLOT; ++i) {
            const int32_t e = i * HW + gl;
            l[i] = valid && e < E ? load_logit<BF16>(row, e) : -INFINITY;
        }
    }
}

// 2^(x log2 e) by the hardware's instruction; exact 0 for -inf
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// A softmax's maximum (0 where the row has no finite logit, so that no
// difference is NaN), and the reciprocal of its sum (0 for a sum of 0).
struct Norm {
    float m, inv;
    // numerator of a softmax's score, 1 for the maximum whatever its magnitude:
    // l log2 e - m log2 e by fma would leave the rounding of m's product in the
    // exponent, hundreds of steps for |m| >= 1e10, and infinity near the type's
    // lowest value
    __device__ __forceinline__ float term(float l) const { return fast_exp(l - m); }
};
template <int TPW, int NSLOT>
__device__ __forceinline__ Norm softmax_norm(const float (&l)[NSLOT])
{
    using G = Group<TPW>;
    float m = l[0];
#pragma unroll
    for (int i = 1; i < NSLOT; ++i)
        m = fmaxf(m, l[i]);
    m = G::max_f32(m);
    m = m == -INFINITY ? 0.f : m;
    Norm n = {m, 0.f};
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < NSLOT; ++i)
        z += n.term(l[i]);
    z = G::sum_f32(z);
    n.inv = z == 0.f ? 0.f : 1.f / z;
    return n;
}

// Score of a logit, plus b. -inf gives a score of 0.
template <bool SIGMOID>
__device__ __forceinline__ float score(float l, const Norm &n, float b)
{
    if (SIGMOID)
        return __builtin_amdgcn_rcpf(1.f + fast_exp(-l)) + b;
    return fmaf(n.term(l), n.inv, b);
}

// How far score() is from the exact sum. The exponent x is rounded twice
// and scaled by a rounded constant (2.5 |x| kU in all), the exponential,
// sum and reciprocal each by one or two steps; a sigmoid takes (1 - p) of its
// exponential's share, a softmax's sum at most 43 kU more (its terms' shares
// weighted by the terms, and up to 23 additions). The last addition rounds s.
// |x| is bounded where p has long vanished (exp(-104) is below float32's
// smallest), so that a finite logit in place of a mask gives 0 and not 0 times
// infinity, which would pass every comparison as certain.
template <bool SIGMOID>
__device__ __forceinline__ float score_error(float l, float p, float s, const Norm &n)
{
    const float x = fminf(fabsf(SIGMOID ? l : l - n.m), 1e4f);
    const float share = SIGMOID ? (1.f - p) * (2.5f * x + 2.f) + 4.f : 2.5f * x + 50.f;
    return (p * share + fabsf(s)) * kU + 2.3509887e-38f;
}
// The same for any expert whose score is at most s, as one bound: experts
// behind the best one left may have far larger errors than that one, where a
// large p cancels against its bias. p share is at most 4.3 for a sigmoid, and
// for a softmax largest at the row's maximum, whose p is n.inv.
template <bool SIGMOID>
__device__ __forceinline__ float rest_error(float s, const Norm &n)
{
    return ((SIGMOID ? 5.f : 51.f * n.inv) + fabsf(s)) * kU + 2.3509887e-38f;
}
// The same for a group's score, of experts whose scores are at most `most` in
// magnitude: p share is at most 5.1 for a sigmoid and 51 for a softmax, twice
// that for the sum of two, whose terms and whose sum round once each (the two
// terms may cancel, so their size counts and not the sum's).
template <bool SIGMOID>
__device__ __forceinline__ float group_error(float most)
{
    return (SIGMOID ? 12.f : 104.f) * kU + 6.f * most * kU;
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    // inverse of score_key: 1 stands for NaN
    return k == 1u ? NAN : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// best and second of two ordered pairs
__device__ __forceinline__ void merge_top2(uint32_t &a1, uint32_t &a2, uint32_t b1, uint32_t b2)
{
    const uint32_t lo = min(a1, b1);
    a1 = max(a1, b1);
    a2 = max(lo, max(a2, b2));
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ void merge_lanes(uint32_t &a1, uint32_t &a2)
{
    const uint32_t b1 = dpp::mov<CTRL, ROW_MASK>(a1, 0u), b2 = dpp::mov<CTRL, ROW_MASK>(a2, 0u);
    merge_top2(a1, a2, b1, b2);
}
// over a token's lanes; every lane gets its own token's pair
template <int TPW>
__device__ __forceinline__ void reduce_top2(uint32_t &a1, uint32_t &a2)
{
    constexpr int HW = kWave / TPW;
    merge_lanes<dpp::kQuadSwap1>(a1, a2);
    merge_lanes<dpp::kQuadSwap2>(a1, a2);
    if (HW >= 8)
        merge_lanes<dpp::kRowHalfMirror>(a1, a2);
    if (HW >= 16)
        merge_lanes<dpp::kRowMirror>(a1, a2);
    if (HW <= 16)
        return;
    merge_lanes<dpp::kRowBcast15, 0xA>(a1, a2);
    if (TPW == 1) {
        merge_lanes<dpp::kRowBcast31, 0xC>(a1, a2);
        a1 = readlane_u32(a1, kWave - 1);
        a2 = readlane_u32(a2, kWave - 1);
        return;
    }
    const bool low = (threadIdx.x & (kWave - 1)) < 32;
    const uint32_t l1 = readlane_u32(a1, 31), h1 = readlane_u32(a1, 63);
    const uint32_t l2 = readlane_u32(a2, 31), h2 = readlane_u32(a2, 63);
    a1 = low ? l1 : h1;
    a2 = low ? l2 : h2;
}

__device__ __forceinline__ uint32_t group_key(uint32_t k1, uint32_t k2, bool top2)
{
    return top2 && k2 != 0u ? score_key(key_value(k1) + key_value(k2) + 0.0f) : k1;
}

// Zeroes the keys of experts outside the token's best topk_groups groups.
// Returns, the same in all the token's lanes, how far the last group taken
// lies above the best one left (infinite where that does not matter).
template <int NSLOT, int VEC, int TPW>
__device__ __forceinline__ float keep_groups(uint32_t (&key)[NSLOT], int32_t E, int32_t n_groups, int32_t topk_groups,
                                             bool top2)
{
    using G = Group<TPW>;
    constexpr int HW = G::HW;
    const int lane = threadIdx.x & (kWave - 1), gl = lane & (HW - 1);
    const int32_t gsize = E / n_groups;
    int gid[NSLOT];
    uint32_t mine = 0u;  // key of group gl
    if (VEC == 4 && TPW == 1 && (gsize == 16 || gsize == 32 || gsize == 64)) {
        // a slot quad's group is a segment of gsize / 4 lanes (route_device.hpp)
        const int shift = gsize == 16 ? 2 : (gsize == 32 ? 3 : 4), per_quad = kWave >> shift;
#pragma unroll
        for (int q = 0; q < NSLOT / 4; ++q) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                gid[4 * q + c] = q * per_quad + (gl >> shift);
            uint32_t k1 = max(key[4 * q], key[4 * q + 1]), k2 = min(key[4 * q], key[4 * q + 1]);
            merge_top2(k1, k2, max(key[4 * q + 2], key[4 * q + 3]), min(key[4 * q + 2], key[4 * q + 3]));
            merge_lanes<dpp::kQuadSwap1>(k1, k2);
            merge_lanes<dpp::kQuadSwap2>(k1, k2);
            if (shift >= 3)
                merge_lanes<dpp::kRowHalfMirror>(k1, k2);
            if (shift >= 4)
                merge_lanes<dpp::kRowMirror>(k1, k2);
            const uint32_t g = group_key(k1, k2, top2);
            const int gq = lane - q * per_quad;
            const bool here = gq >= 0 && gq < per_quad;
            const uint32_t got = (uint32_t)__builtin_amdgcn_ds_bpermute((here ? gq << shift : 0) << 2, (int)g);
            mine = here ? got : mine;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NSLOT; ++i)
            gid[i] = (int)(slot_id<VEC, HW>(i, gl) / (uint32_t)gsize);
        for (int g = 0; g < n_groups; ++g) {
            uint32_t k1 = 0u, k2 = 0u;
#pragma unroll
            for (int i = 0; i < NSLOT; ++i)
                merge_top2(k1, k2, gid[i] == g ? key[i] : 0u, 0u);
            reduce_top2<TPW>(k1, k2);
            const uint32_t v = group_key(k1, k2, top2);
            mine = gl == g ? v : mine;
        }
    }
    if (gl >= n_groups)
        mine = 0u;
    uint64_t chosen = 0;
    uint32_t last = 0u;
    for (int m = 0; m < topk_groups; ++m) {
        last = G::max_u32(mine);
        const int g = (int)G::min_u32(mine == last && gl < n_groups ? (uint32_t)gl : 0xFFFFFFFFu);
        chosen |= 1ull << (g & 63);
        mine = gl == g ? 0u : mine;
    }
    const uint32_t rest = G::max_u32(mine);
#pragma unroll
    for (int i = 0; i < NSLOT; ++i)
        key[i] = ((chosen >> (gid[i] & 63)) & 1ull) ? key[i] : 0u;
    return rest <= 1u ? INFINITY : key_value(last) - key_value(rest);
}

// The k + 1 largest of a wave's keys, ties to the smaller id, for one token per
// wave: lane j of the result holds round j's id, lane k the best one left.
// A key that at least k + 1 lanes' largest reach, found by bisection (a compare
// and a count of lanes each time), lets k + 1 experts and few more through;
// those are gathered, one for each lane, and placed by counting the ones ahead
// of them: 33.3 us where select_topk's k rounds of a maximum over the wave took
// 36.2 (32768 tokens, 512 experts, k = 10, with a bias). False where fewer
// than k + 1 lanes have an expert, or ties let more than 64 through.
template <int NSLOT, int VEC>
__device__ __forceinline__ bool pick_topk(const uint32_t (&key)[NSLOT], int32_t k, uint64_t *__restrict__ buf,
                                          Selected &r)
{
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t top = key[0];
#pragma unroll
    for (int i = 1; i < NSLOT; ++i)
        top = max(top, key[i]);
    uint32_t lo = 1u, hi = 0xFF800001u;  // +inf's key and one
    int n = __popcll(ballot64(top >= lo));
    if (n <= k)
        return false;
    while (n > k + 6 && hi - lo > 1u) {
        const uint32_t mid = lo + (hi - lo) / 2u;
        const int c = __popcll(ballot64(top >= mid));
        if (c > k) {
            lo = mid;
            n = c;
        } else {
            hi = mid;
        }
    }
    int C = 0;
#pragma unroll
    for (int i = 0; i < NSLOT; ++i) {
        const bool in = key[i] >= lo;
        const uint64_t who = ballot64(in);
        if (who) {
            const int at = C + (int)count_below(who);
            if (in && at < kWave)
                buf[at] = ((uint64_t)key[i] << 32) | (0xFFFFFFFFu - slot_id<VEC, kWave>(i, lane));
            C += __popcll(who);
        }
    }
    if (C > kWave)
        return false;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const uint64_t mine = lane < C ? buf[lane] : 0u;
    const uint32_t hi32 = (uint32_t)(mine >> 32), lo32 = (uint32_t)mine;
    int ahead = 0;
    for (int q = 0; q < C; ++q) {
        const uint64_t o = ((uint64_t)readlane_u32(hi32, q) << 32) | readlane_u32(lo32, q);
        ahead += o > mine;
    }
    const int to = lane < C ? ahead : lane;  // a permutation of the lanes
    r.e = (uint32_t)__builtin_amdgcn_ds_permute(to << 2, (int)(0xFFFFFFFFu - lo32));
    r.next_e = r.e;
    r.next_key = 1u;
    return true;
}

// ---- the same ranking of one token in 64 bits, by the whole wave ----

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
__device__ __forceinline__ int wave_min(int v)
{
    for (int d = 1; d < kWave; d <<= 1)
        v = min(v, __shfl_xor(v, d, kWave));
    return v;
}

// Ranks below every score, in order: an expert that may not be taken (or is
// not there), NaN, -inf. Scores are finite or +inf.
constexpr double kOut = -INFINITY, kNaNRank = -1.7e308, kMasked = -1.6e308;

// Lane j returns the id of round j. NS slots of 64 experts. Without groups, no
// expert whose score is below `least` is among the k best; the few others are
// gathered, one for each lane, and placed by counting those ahead of them.
// Rounds of a maximum over the wave, 64 bits at a time, took three times as
// long, and are left for groups and for more than 64 candidates.
struct Candidates {
    double s[kWave];
    int32_t e[kWave];
};
// !FEW: every expert takes part in the rounds, and without a bias the logits
// are ranked (their scores only where groups go by the sum of two).
template <int NS, bool BF16, bool SIGMOID, bool FEW>
__device__ int rank_exactly(const void *row, const float *__restrict__ bias, int32_t E, int32_t k, int32_t n_groups,
                            int32_t topk_groups, bool top2, float least, Candidates *__restrict__ cand)
{
    const int lane = threadIdx.x & (kWave - 1);
    const bool by_logit = !FEW && !bias && !(n_groups > 0 && top2);
    double s[NS], m = -INFINITY, z = 0.;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int32_t e = i * kWave + lane;
        s[i] = e < E ? (double)load_logit<BF16>(row, e) : -INFINITY;
        m = fmax(m, s[i]);
    }
    if (!SIGMOID) {
        m = wave_max(m);
        m = m == -INFINITY ? 0. : m;
    }
#pragma unroll
    for (int i = 0; i < NS && !by_logit; ++i) {
        const double l = s[i];
        const double u = l == -INFINITY ? 0. : exp(SIGMOID ? -l : l - m);
        if (SIGMOID)
            s[i] = l == -INFINITY ? -INFINITY : 1. / (1. + u);
        else
            s[i] = l == -INFINITY ? -INFINITY : u;
        z += SIGMOID ? 0. : u;
    }
    if (!SIGMOID)
        z = wave_sum(z);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int32_t e = i * kWave + lane;
        if (e >= E) {
            s[i] = kOut;
            continue;
        }
        double v = s[i];
        if (v != -INFINITY && !by_logit)
            v = (SIGMOID ? v : v / z) + (bias ? (double)bias[e] : 0.);
        s[i] = v != v ? kNaNRank : (v == -INFINITY ? kMasked : v);
    }
    if (FEW && n_groups == 0) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const bool is = s[i] >= (double)least;
            const uint64_t who = ballot64(is);
            const int at = n + (int)count_below(who);
            if (is && at < kWave) {
                cand->s[at] = s[i];
                cand->e[at] = i * kWave + lane;
            }
            n += __popcll(who);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (n >= k && n <= kWave) {
            const double mine = lane < n ? cand->s[lane] : kOut;
            const int32_t e = lane < n ? cand->e[lane] : 0x7FFFFFFF;
            int ahead = 0;
            for (int q = 0; q < n; ++q) {
                const double o = cand->s[q];
                ahead += o > mine || (o == mine && cand->e[q] < e);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (lane < n)
                cand->e[ahead] = e;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            return cand->e[lane];
        }
    }
    if (n_groups > 0) {
        const int32_t gsize = E / n_groups;
        double mine = kOut;
        for (int g = 0; g < n_groups; ++g) {
            double b1 = kOut, b2 = kOut;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const double v = (i * kWave + lane) / gsize == g ? s[i] : kOut;
                const double lo = fmin(b1, v);
                b1 = fmax(b1, v);
                b2 = fmax(b2, lo);
            }
            for (int d = 1; d < kWave; d <<= 1) {
                const double o1 = __shfl_xor(b1, d, kWave), o2 = __shfl_xor(b2, d, kWave);
                const double lo = fmin(b1, o1);
                b1 = fmax(b1, o1);
                b2 = fmax(lo, fmax(b2, o2));
            }
            double v = b1;
            if (top2 && b2 != kOut)
                v = b2 > kMasked ? b1 + b2 : (b2 == kNaNRank || b1 == kNaNRank ? kNaNRank : kMasked);
            mine = lane == g ? v : mine;
        }
        uint64_t chosen = 0;
        for (int q = 0; q < topk_groups; ++q) {
            const double best = wave_max(mine);
            const int g = wave_min(mine == best && lane < n_groups ? lane : kWave - 1);
            chosen |= 1ull << g;
            mine = lane == g ? kOut : mine;
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int32_t e = i * kWave + lane;
            if (e >= E)
                continue;
            if (!((chosen >> (e / gsize)) & 1ull)) {
                s[i] = kOut;
            } else if (!bias) {  // the logits' order, also where their scores are the same in 64 bits
                const double l = load_logit<BF16>(row, e);
                s[i] = l != l ? kNaNRank : (l == -INFINITY ? kMasked : l);
            }
        }
    }
    int id = 0;
    for (int j = 0; j < k; ++j) {
        double best = s[0];
#pragma unroll
        for (int i = 1; i < NS; ++i)
            best = fmax(best, s[i]);
        best = wave_max(best);
        int e = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < NS; ++i)
            e = s[i] == best ? min(e, i * kWave + lane) : e;
        e = wave_min(e);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            s[i] = i * kWave + lane == e ? kOut : s[i];
        id = lane == j ? e : id;
    }
    return id;
}

struct ScoredArgs {
    const void *logits;
    const float *bias;
    int64_t T;
    int32_t E, k, n_groups, topk_groups;
    bool top2, normalize;
    float scale;
    int32_t *topk_idx;
    float *topk_w;
};

// The weight of a token's selected expert, before the scale: my_l is its logit
// in the lanes of `mine`, -inf in the others; n is needed for a softmax that is
// not normalised.
template <class G, bool SIGMOID>
__device__ __forceinline__ float selected_weight(float my_l, bool mine, bool normalize, const Norm &n)
{
    if (normalize) {
        // softmax over the selected; a sigmoid's e^m scales every term alike,
        // so that scores far below float32's range keep their ratios
        const float m = G::max_f32(my_l);
        float u = 0.f;
        if (SIGMOID)
            u = my_l > 0.f ? 1.f / (1.f + expf(-my_l)) : expf(my_l - fminf(m, 0.f)) / (1.f + expf(my_l));
        else
            u = expf(my_l - m);
        u = mine && my_l != -INFINITY ? u : 0.f;
        const float z = G::sum_f32(u);
        return z == 0.f ? 0.f : u / z;
    }
    if (my_l == -INFINITY)
        return 0.f;
    return SIGMOID ? 1.f / (1.f + expf(-my_l)) : n.term(my_l) * n.inv;
}

template <int NSLOT, int VEC, int TPW, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kRouteThreads, 8) void route_scored_kernel(ScoredArgs a)
{
    // eight waves a SIMD: the 64-bit ranking of eight slots, a function of its
    // own, saves registers to scratch for it; the kernels spill none
    __shared__ Candidates cand[kWavesPerBlock];
    using G = Group<TPW>;
    constexpr int HW = G::HW;
    constexpr int NC = NSLOT >= 8 ? 3 : 2;
    const int64_t t0 = ((int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave) * TPW;
    if (t0 >= a.T)
        return;  // whole waves
    const int lane = threadIdx.x & (kWave - 1), gl = lane & (HW - 1), gbase = lane - gl;
    const int64_t t = t0 + lane / HW;
    const bool valid = t < a.T;
    const int64_t row_bytes = (int64_t)a.E * (BF16 ? 2 : 4);
    const char *row = static_cast<const char *>(a.logits) + (valid ? t : t0) * row_bytes;

    float l[NSLOT];
    load_row<BF16, NSLOT, VEC, HW>(row, a.E, gl, valid, l);
    Norm n = {0.f, 0.f};
    const bool grouped = a.n_groups > 0, by_score = a.bias || (grouped && a.top2 && a.E > a.n_groups);
    if (!SIGMOID && (by_score || !a.normalize))
        n = softmax_norm<TPW>(l);

    uint32_t key[NSLOT];
    if (by_score) {
        float b[NSLOT];
#pragma unroll
        for (int i = 0; i < NSLOT; ++i)
            b[i] = 0.f;
        if (a.bias)
            load_row<false, NSLOT, VEC, HW>(a.bias, a.E, gl, true, b);
        float low = l[0];
#pragma unroll
        for (int i = 1; i < NSLOT; ++i)
            low = fminf(low, l[i]);
        if (ballot64(low == -INFINITY)) {  // masked experts, or slots past E
#pragma unroll
            for (int i = 0; i < NSLOT; ++i)
                l[i] = l[i] == -INFINITY ? -INFINITY : score<SIGMOID>(l[i], n, b[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NSLOT; ++i)
                l[i] = score<SIGMOID>(l[i], n, b[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < NSLOT; ++i)
        key[i] = valid && (int32_t)slot_id<VEC, HW>(i, gl) < a.E ? score_key(l[i] + 0.0f) : 0u;
    bool near = false;  // the float32 order is not certain
    if (grouped) {
        float most = 0.f;  // the largest score's magnitude; masked ones do not count
#pragma unroll
        for (int i = 0; i < NSLOT; ++i)
            most = fmaxf(most, key[i] && l[i] != -INFINITY ? fabsf(l[i]) : 0.f);
        const float gap = keep_groups<NSLOT, VEC, TPW>(key, a.E, a.n_groups, a.topk_groups, a.top2);
        near = by_score && gap <= 2.f * group_error<SIGMOID>(G::max_f32(most));
        if (by_score && !a.bias) {
            // groups by their scores, experts within them by their logits
            load_row<BF16, NSLOT, VEC, HW>(row, a.E, gl, valid, l);
#pragma unroll
            for (int i = 0; i < NSLOT; ++i)
                key[i] = key[i] ? score_key(l[i] + 0.0f) : 0u;
        }
    }
    Selected sel;
    bool picked = false;
    if constexpr (TPW == 1)
        picked = pick_topk<NSLOT, VEC>(key, a.k, reinterpret_cast<uint64_t *>(cand[threadIdx.x / kWave].s), sel);
    if (!picked)
        sel = select_topk<NSLOT, VEC, TPW, NC, true>(key, a.k);
    uint32_t my_e = sel.e;
    const bool mine = valid && gl < a.k;
    float my_l = -INFINITY, least = -INFINITY;
    if (a.bias) {
        // lane j: the expert of round j, lane k: the best one left
        const bool is = mine || (valid && gl == a.k && sel.next_key != 0u);
        const uint32_t e = gl == a.k ? sel.next_e : my_e;
        float b = 0.f;
        if (is) {
            my_l = load_logit<BF16>(row, (int32_t)e);
            b = a.bias[e];
        }
        const float p = score<SIGMOID>(my_l, n, 0.f);
        const float s = my_l == -INFINITY ? -INFINITY : score<SIGMOID>(my_l, n, b);
        const float err = my_l == -INFINITY ? 0.f : score_error<SIGMOID>(my_l, p, s, n);
        // the next lane's, across the wave
        constexpr int kShl1 = 0x130;
        const float l2 = __uint_as_float(dpp::mov<kShl1>(__float_as_uint(my_l), 0u));
        const float b2 = __uint_as_float(dpp::mov<kShl1>(__float_as_uint(b), 0u));
        const float s2 = __uint_as_float(dpp::mov<kShl1>(__float_as_uint(s), __float_as_uint(-INFINITY)));
        float err2 = __uint_as_float(dpp::mov<kShl1>(__float_as_uint(err), 0u));
        if (gl == a.k - 1)  // the next lane's stands for all that are left (-inf: masked, or none)
            err2 = s2 == -INFINITY ? 0.f : rest_error<SIGMOID>(s2, n);
        // An equal pair is ranked by its ids, but where it straddles the last
        // place it may hide a third expert next to it. Masked ones (-inf) give
        // NaN here: their order is known.
        near |= mine && (s - s2 <= err + err2) && (gl == a.k - 1 || !(my_l == l2 && b == b2));
        my_l = mine ? my_l : -INFINITY;
        // The k best score at least the smallest of these, exactly. Twice the
        // bound, which holds half a step of s, covers the difference's rounding.
        least = my_l == -INFINITY ? -INFINITY : s - 2.f * err;
    } else if (mine) {
        my_l = load_logit<BF16>(row, (int32_t)my_e);
    }
    uint64_t again = ballot64(near && valid);
    if (again)
        least = -G::max_f32(mine ? -least : -INFINITY);
    while (again) {  // tokens of this wave, one after the other
        const int first = __ffsll((unsigned long long)again) - 1;
        const int base = first & ~(HW - 1);
        const uint64_t lanes = HW == 64 ? ~0ull : ((1ull << HW) - 1) << base;
        again &= ~lanes;
        const char *r = static_cast<const char *>(a.logits) + (t0 + base / HW) * row_bytes;
        constexpr int NS = (NSLOT * HW + kWave - 1) / kWave;
        const float from = __shfl(least, base, kWave);
        Candidates *const c = &cand[threadIdx.x / kWave];
        int id;
        [[clang::noinline]] id = rank_exactly<NS, BF16, SIGMOID, true>(r, a.bias, a.E, a.k, a.n_groups, a.topk_groups,
                                                                       a.top2, from, c);
        const int got = __shfl(id, gl, kWave);
        if (gbase == base) {
            my_e = (uint32_t)got;
            my_l = mine ? load_logit<BF16>(row, (int32_t)my_e) : -INFINITY;
        }
    }

    const float w = selected_weight<G, SIGMOID>(my_l, mine, a.normalize, n);
    if (mine) {
        a.topk_idx[t * a.k + gl] = (int32_t)my_e;
        a.topk_w[t * a.k + gl] = a.scale * w;
    }
}

// More than 512 experts: one wave ranks a token in 64 bits from the start, 16
// experts a lane, every value in registers at four waves a SIMD: 183 us for
// 32768 tokens, 1024 experts, k = 8, softmax with a bias; bound by the rounds'
// reductions over the wave. Float32 keys, 16 a lane at eight waves, took 111 us
// and spilled up to 47 registers, the row's address among them, to scratch. One
// such launch ended in a memory fault that the kernel's own accesses do not
// explain (followed lane by lane, every address is in bounds), so that kernel
// is not used.
template <bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kRouteThreads, 4) void route_scored_wide_kernel(ScoredArgs a)
{
    constexpr int kSlots = 16;
    const int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave;
    if (t >= a.T)
        return;  // whole waves
    const int lane = threadIdx.x & (kWave - 1);
    const char *row = static_cast<const char *>(a.logits) + t * a.E * (BF16 ? 2 : 4);
    int32_t e;
    [[clang::always_inline]] e = rank_exactly<kSlots, BF16, SIGMOID, false>(
        row, a.bias, a.E, a.k, a.n_groups, a.topk_groups, a.top2 && a.E > a.n_groups, -INFINITY, nullptr);
    Norm n = {0.f, 0.f};
    if (!SIGMOID && !a.normalize) {
        float l[kSlots];
        load_row<BF16, kSlots, 1, kWave>(row, a.E, lane, true, l);
        n = softmax_norm<1>(l);
    }
    const bool mine = lane < a.k;
    const float my_l = mine ? load_logit<BF16>(row, e) : -INFINITY;
    const float w = selected_weight<Group<1>, SIGMOID>(my_l, mine, a.normalize, n);
    if (mine) {
        a.topk_idx[t * a.k + lane] = e;
        a.topk_w[t * a.k + lane] = a.scale * w;
    }
}

struct ScoredGradArgs {
    const void *logits;
    const int32_t *topk_idx;
    const float *grad_w;
    int64_t T;
    int32_t E, k;
    bool normalize;
    float scale;
    void *grad_logits;
};

template <int NSLOT, int VEC, int TPW, bool BF16, bool SIGMOID>
__global__ __launch_bounds__(kRouteThreads) void route_scored_backward_kernel(ScoredGradArgs a)
{
    using G = Group<TPW>;
    constexpr int HW = G::HW;
    __shared__ __attribute__((aligned(16))) float rows[kWavesPerBlock][TPW][NSLOT * HW];
    const int lane = threadIdx.x & (kWave - 1), gl = lane & (HW - 1), wave = threadIdx.x / kWave;
    const int64_t t0 = ((int64_t)blockIdx.x * kWavesPerBlock + wave) * TPW;
    if (t0 >= a.T)
        return;
    const int64_t t = t0 + lane / HW;
    const bool valid = t < a.T, dense = !SIGMOID && !a.normalize;
    const int64_t row_bytes = (int64_t)a.E * (BF16 ? 2 : 4);
    const char *row = static_cast<const char *>(a.logits) + (valid ? t : t0) * row_bytes;
    float *grads = rows[wave][lane / HW];

    // gl < k: the selected expert's logit and gradient, -inf and 0 where its id is none
    int32_t e = -1;
    float le = -INFINITY, g = 0.f;
    if (valid && gl < a.k) {
        e = a.topk_idx[t * a.k + gl];
        g = a.grad_w[t * a.k + gl];
        if (e < 0 || e >= a.E) {
            e = -1;
            g = 0.f;
        } else {
            le = load_logit<BF16>(row, e);
        }
    }
    float l[NSLOT];
    Norm n = {0.f, 0.f};
    if (dense) {
        load_row<BF16, NSLOT, VEC, HW>(row, a.E, gl, valid, l);
        n = softmax_norm<TPW>(l);
    }
    if (VEC == 4) {
#pragma unroll
        for (int q = 0; q < NSLOT / 4; ++q)
            *reinterpret_cast<f32x4 *>(grads + 4 * (q * HW + gl)) = f32x4{0.f, 0.f, 0.f, 0.f};
    } else {
#pragma unroll
        for (int i = 0; i < NSLOT; ++i)
            grads[i * HW + gl] = 0.f;
    }
    float gw;  // sum of gradient times weight
    float d;
    if (dense) {
        const float p = n.term(le) * n.inv;
        gw = G::sum_f32(g * p);
        d = g;
    } else {
        const float p = SIGMOID ? (le == -INFINITY ? 0.f : 1.f / (1.f + expf(-le))) : 0.f;
        float w = p;
        if (a.normalize) {
            const float m = G::max_f32(le);
            float u = 0.f;
            if (SIGMOID)
                u = le > 0.f ? p : expf(le - fminf(m, 0.f)) / (1.f + expf(le));
            else
                u = expf(le - m);
            u = le == -INFINITY ? 0.f : u;
            const float z = G::sum_f32(u);
            w = z == 0.f ? 0.f : u / z;
        }
        gw = G::sum_f32(g * w);
        // 1 - p = 1 / (1 + e^l), without its cancellation
        const float q = SIGMOID ? (le == -INFINITY ? 0.f : 1.f / (1.f + expf(le))) : 1.f;
        d = a.scale * w * q * (a.normalize ? g - gw : g);
    }
    // the wave's own row of LDS: its stores and reads are in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (e >= 0)
        grads[e] = d;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    char *out = static_cast<char *>(a.grad_logits) + (valid ? t : t0) * row_bytes;
    const float c = a.scale * n.inv;
    if (VEC == 4) {
#pragma unroll
        for (int q = 0; q < NSLOT / 4; ++q) {
            f32x4 v = *reinterpret_cast<const f32x4 *>(grads + 4 * (q * HW + gl));
            if (dense)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = n.term(l[4 * q + i]) * c * (v[i] - gw);
            if (valid && q * 4 * HW + 4 * gl < a.E) {
                if (BF16)
                    __builtin_nontemporal_store(u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])},
                                                reinterpret_cast<u32x2 *>(out) + q * HW + gl);
                else
                    __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(out) + q * HW + gl);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NSLOT; ++i) {
            const int32_t x = i * HW + gl;
            float v = grads[x];
            if (dense)
                v = n.term(l[i]) * c * (v - gw);
            if (valid && x < a.E) {
                if (BF16)
                    reinterpret_cast<uint16_t *>(out)[x] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
                else
                    reinterpret_cast<float *>(out)[x] = v;
            }
        }
    }
}

// one launch per kMaxRowBlocks blocks of tokens
template <class Args, class Launch>
hipError_t in_chunks(Args a, int64_t per_block, Launch launch)
{
    const int64_t T = a.T, chunk = kMaxRowBlocks * per_block;
    for (int64_t t0 = 0; t0 < T; t0 += chunk) {
        a.T = T - t0 < chunk ? T - t0 : chunk;
        launch(a, t0, dim3((unsigned)((a.T + per_block - 1) / per_block)));
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

template <int NSLOT, int VEC, int TPW, bool BF16, bool SIGMOID>
hipError_t launch(const ScoredArgs &args, hipStream_t stream)
{
    return in_chunks(args, (int64_t)kWavesPerBlock * TPW, [&](ScoredArgs a, int64_t t0, dim3 grid) {
        a.logits = static_cast<const char *>(a.logits) + t0 * a.E * (BF16 ? 2 : 4);
        a.topk_idx += t0 * a.k;
        a.topk_w += t0 * a.k;
        if constexpr (NSLOT <= 8)
            hipLaunchKernelGGL((route_scored_kernel<NSLOT, VEC, TPW, BF16, SIGMOID>), grid, dim3(kRouteThreads), 0,
                               stream, a);
        else
            hipLaunchKernelGGL((route_scored_wide_kernel<BF16, SIGMOID>), grid, dim3(kRouteThreads), 0, stream, a);
    });
}
template <int NSLOT, int VEC, int TPW, bool BF16, bool SIGMOID>
hipError_t launch(const ScoredGradArgs &args, hipStream_t stream)
{
    return in_chunks(args, (int64_t)kWavesPerBlock * TPW, [&](ScoredGradArgs a, int64_t t0, dim3 grid) {
        const int64_t at = t0 * a.E * (BF16 ? 2 : 4);
        a.logits = static_cast<const char *>(a.logits) + at;
        a.grad_logits = static_cast<char *>(a.grad_logits) + at;
        a.topk_idx += t0 * a.k;
        a.grad_w += t0 * a.k;
        hipLaunchKernelGGL((route_scored_backward_kernel<NSLOT, VEC, TPW, BF16, SIGMOID>), grid, dim3(kRouteThreads),
                           0, stream, a);
    });
}

// The widths a wave is built for. Four logits per access where rows allow it
// (E % 4 == 0 and aligned rows), so 4 per lane and slot quad; a short row
// takes a part of the wave that holds its experts, k + 1 ids and its groups.
template <bool BF16, bool SIGMOID, class Args>
hipError_t launch_width(const Args &a, bool vec4, int32_t groups, hipStream_t stream)
{
    int seg = 4;
    while (seg < (a.E + 3) / 4 || seg <= a.k || seg < groups)
        seg *= 2;
    if (vec4) {
        switch (seg) {
        case 4: return launch<4, 4, 16, BF16, SIGMOID>(a, stream);
        case 8: return launch<4, 4, 8, BF16, SIGMOID>(a, stream);
        case 16: return launch<4, 4, 4, BF16, SIGMOID>(a, stream);
        case 32: return launch<4, 4, 2, BF16, SIGMOID>(a, stream);
        case 64: return launch<4, 4, 1, BF16, SIGMOID>(a, stream);
        case 128: return launch<8, 4, 1, BF16, SIGMOID>(a, stream);
        default: return launch<16, 4, 1, BF16, SIGMOID>(a, stream);
        }
    }
    if (a.E <= 4 * kWave)
        return launch<4, 1, 1, BF16, SIGMOID>(a, stream);
    if (a.E <= 8 * kWave)
        return launch<8, 1, 1, BF16, SIGMOID>(a, stream);
    return launch<16, 1, 1, BF16, SIGMOID>(a, stream);
}
template <class Args>
hipError_t launch_type(const Args &a, bool vec4, int32_t groups, const ScoreOpts &o, hipStream_t stream)
{
    if (o.bf16)
        return o.sigmoid ? launch_width<true, true>(a, vec4, groups, stream)
                         : launch_width<true, false>(a, vec4, groups, stream);
    return o.sigmoid ? launch_width<false, true>(a, vec4, groups, stream)
                     : launch_width<false, false>(a, vec4, groups, stream);
}

}  // namespace

hipError_t launch_route_scored(const void *logits, const float *bias, int64_t T, int32_t E,
                               int32_t k, int32_t n_groups, int32_t topk_groups,
                               const ScoreOpts &o, int32_t *topk_idx, float *topk_w,
                               hipStream_t stream)
{
    const ScoredArgs a = {logits, bias,    T,           E,       k,        n_groups, topk_groups,
                          o.top2, o.normalize, o.scale, topk_idx, topk_w};
    const bool vec4 = E % 4 == 0 && (uintptr_t)logits % (o.bf16 ? 8 : 16) == 0 && (uintptr_t)bias % 16 == 0;
    return launch_type(a, vec4, n_groups, o, stream);
}

hipError_t launch_route_scored_backward(const void *logits, const int32_t *topk_idx,
                                        const float *grad_w, int64_t T, int32_t E, int32_t k,
                                        const ScoreOpts &o, void *grad_logits, hipStream_t stream)
{
    const ScoredGradArgs a = {logits, topk_idx, grad_w, T, E, k, o.normalize, o.scale, grad_logits};
    const uintptr_t align = o.bf16 ? 8 : 16;
    const bool vec4 = E % 4 == 0 && (uintptr_t)logits % align == 0 && (uintptr_t)grad_logits % align == 0;
    return launch_type(a, vec4, 0, o, stream);
}

}  // namespace moe
