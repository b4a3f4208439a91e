// route_scored.cu -- scored routing: softmax or sigmoid scores, a bias that
// takes part in the choice but not in the weight, expert groups, top-k and
// (re)normalised weights.  One warp per token.
//
//   s_e = 1 / (1 + exp(-l_e))            or   exp(l_e - m) / sum exp(l - m)
//   c_e = s_e + b_e                       (the choice; masked experts: none)
//   group score = sum of the group_top best choices of the group
//   the topk_group best groups stay; the k best choices of their experts win
//   w_j = s_j [ / sum s ] * scale
//
// Which expert wins is decided on scores of 64 bits: c is a sum of a score and
// a bias, and over a prefill chunk's millions of scores a few pairs at the k-th
// place are closer than fp32 rounding, where an id would depend on the order of
// operations.  The order of two choices is that of a 64-bit key (the double's
// bits made monotone, 0 for a masked expert), ties to the lower id.
#include <math.h>

#include "ops.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 4;  // tokens per CTA

// Above the type's lowest value: false for NaN, -inf and the lowest itself, the
// values that a mask writes.
__device__ __forceinline__ bool is_live(float v) { return v > -3.402823466e+38f; }

__device__ __forceinline__ uint64_t choice_key(double c) {
    const long long b = __double_as_longlong(c);
    return (uint64_t)(b < 0 ? ~b : (b | (long long)0x8000000000000000ull));
}
__device__ __forceinline__ double key_choice(uint64_t key) {
    const long long b = (long long)key;
    return __longlong_as_double(b < 0 ? (b & 0x7fffffffffffffffll) : ~b);
}

// Largest key of the warp (64 bits: the high words first, then the low words of
// the lanes that hold the largest high word).
__device__ __forceinline__ uint64_t warp_max_key(uint64_t key) {
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(key >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}

// Score of a live logit (m, z: the token's largest live logit and the softmax
// denominator; l == m also covers a logit of +inf).
__device__ __forceinline__ double score_of(float l, bool sigmoid, float m, double z) {
    if (sigmoid) return 1.0 / (1.0 + exp(-(double)l));
    return (l == m ? 1.0 : exp((double)l - (double)m)) / z;
}

// Lane l holds experts l, l+32, ...; with groups the keys also go to shared
// memory, where each group is read by a set of 32 / (groups, rounded up to a
// power of two) lanes.
template <int VPL>
__global__ void __launch_bounds__(32 * kWarps) k_route_scored(const ScoredArgs a) {
    extern __shared__ uint64_t s_keys[];  // [kWarps][E] with groups
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= a.T) return;
    const float *row = a.logits + (size_t)t * a.E;
    float l[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = lane + 32 * i < a.E ? __ldg(row + lane + 32 * i) : -INFINITY;

    float m = 0.0f;
    double z = 1.0;
    if (!a.sigmoid) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = is_live(l[i]) ? fmaxf(m, l[i]) : m;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
        z = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (is_live(l[i])) z += score_of(l[i], false, m, 1.0);
        z = warp_sum(z);
    }
    uint64_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        key[i] = 0;
        if (e < a.E && is_live(l[i])) {
            const float b = a.bias ? __ldg(a.bias + e) : 0.0f;
            if (is_live(b)) key[i] = choice_key(score_of(l[i], a.sigmoid, m, z) + (double)b);
        }
    }

    if (a.n_group > 1) {
        uint64_t *sk = s_keys + (size_t)warp * a.E;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane + 32 * i < a.E) sk[lane + 32 * i] = key[i];
        __syncwarp();
        const int p2 = 1 << (32 - __clz(a.n_group - 1));  // groups, rounded up to a power of two
        const int per = 32 / p2, g = lane / per, sub = lane % per;
        uint64_t k1 = 0, k2 = 0;  // the two best of the group
        if (g < a.n_group)
            for (int j = sub; j < a.group_size; j += per) {
                const uint64_t v = sk[g * a.group_size + j];
                k2 = max(k2, min(k1, v));
                k1 = max(k1, v);
            }
        for (int off = per >> 1; off > 0; off >>= 1) {
            const uint64_t o1 = __shfl_xor_sync(kAll, k1, off), o2 = __shfl_xor_sync(kAll, k2, off);
            k2 = max(min(k1, o1), max(k2, o2));
            k1 = max(k1, o1);
        }
        uint64_t gk = 0;  // the group's key, on its first lane
        if (sub == 0 && k1 != 0)
            gk = choice_key(key_choice(k1) + (a.group_top > 1 && k2 != 0 ? key_choice(k2) : 0.0));
        uint32_t kept = 0;
        for (int r = 0; r < a.topk_group; ++r) {
            const uint64_t best = warp_max_key(gk);
            if (best == 0) break;  // only groups without a live expert are left
            const int win = __reduce_min_sync(kAll, gk == best ? g : 32);
            if (g == win) gk = 0;
            kept |= 1u << win;
        }
        // group of expert e by a multiplication: exact for e < 1024
        const uint32_t mul = ((1u << 22) + a.group_size - 1) / a.group_size;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (!((kept >> (((uint32_t)(lane + 32 * i) * mul) >> 22)) & 1u)) key[i] = 0;
    }

    int mine = -1;  // lane j: the expert of place j
    for (int j = 0; j < a.k; ++j) {
        uint64_t bk = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < VPL; ++i)
            if (key[i] > bk) {
                bk = key[i];
                bi = i;
            }
        const uint64_t best = warp_max_key(bk);
        if (best == 0) break;  // every live expert of the kept groups is taken
        const int win = __reduce_min_sync(kAll, bk == best ? lane + 32 * bi : 0x7fffffff);
        if (lane == (win & 31)) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i == (win >> 5)) key[i] = 0;
        }
        if (lane == j) mine = win;
    }
    double s = mine >= 0 ? score_of(__ldg(row + mine), a.sigmoid, m, z) : 0.0;
    if (a.renorm) {
        const double sum = warp_sum(s);
        s = sum > 0.0 ? s / sum : 0.0;
    }
    if (lane < a.k) {
        a.ids[(size_t)t * a.k + lane] = mine;
        a.w[(size_t)t * a.k + lane] = (float)(s * (double)a.scale);
    }
}

}  // namespace

cudaError_t launch_route_scored(const ScoredArgs &a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    const int vpl = (a.E + 31) / 32;
    const dim3 block(32 * kWarps), grid((unsigned)((a.T + kWarps - 1) / kWarps));
    const size_t smem = a.n_group > 1 ? (size_t)kWarps * a.E * sizeof(uint64_t) : 0;  // <= 32 KiB (E <= 1024)
    if (vpl <= 1) return launch_pdl(k_route_scored<1>, grid, block, smem, s, a);
    if (vpl <= 2) return launch_pdl(k_route_scored<2>, grid, block, smem, s, a);
    if (vpl <= 4) return launch_pdl(k_route_scored<4>, grid, block, smem, s, a);
    if (vpl <= 8) return launch_pdl(k_route_scored<8>, grid, block, smem, s, a);
    if (vpl <= 16) return launch_pdl(k_route_scored<16>, grid, block, smem, s, a);
    return launch_pdl(k_route_scored<32>, grid, block, smem, s, a);
}

}  // namespace moe
