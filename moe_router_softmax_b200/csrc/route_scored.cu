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
// operations.  Nearly every token is decided in fp32 all the same: its choices and
// group scores are formed in fp32 with a bound on their error, and where every
// gap that the result rests on (between consecutive winners, between the last one
// and the next, between the last kept group and the next) exceeds the two errors,
// 64 bits would decide alike.  The other tokens, a few in a thousand and all with ties,
// are done over in 64 bits.  The winners' weights are always formed in 64 bits.
//
// Bound by instruction issue: 8192 tokens of 256 experts in 8 groups read 8.4 MB
// (1.3 us of HBM), and a warp's k rounds of reductions take a few hundred instructions.
// 64 bits throughout took 23.9 us there.
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

// Two best keys of the lane's group: `mine1` and `mine2` are those among the lane's
// own, the group's lanes are `per` consecutive ones.
template <class Key>
__device__ __forceinline__ void merge_best(Key &k1, Key &k2, int per) {
    for (int off = per >> 1; off > 0; off >>= 1) {
        const Key o1 = __shfl_xor_sync(kAll, k1, off), o2 = __shfl_xor_sync(kAll, k2, off);
        k2 = max(min(k1, o1), max(k2, o2));
        k1 = max(k1, o1);
    }
}
// Same for any group size: the keys (lane l: experts l V .. l V + V-1) go through
// shared memory, where each group is read by 32 / (groups, rounded up to a power of two)
// lanes.  Returns the group of this lane's set (>= n_group: none) and its size.
template <int VPL, class Key>
__device__ __forceinline__ int group_best(const ScoredArgs &a, const Key key[VPL], Key *sk, Key *k1, Key *k2, int *per) {
    const int lane = threadIdx.x & 31, V = (a.E + 31) / 32;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (i < V && lane * V + i < a.E) sk[lane * V + i] = key[i];
    __syncwarp();
    *per = 32 >> (32 - __clz(a.n_group - 1));
    const int g = lane / *per;
    *k1 = *k2 = 0;
    if (g < a.n_group)
        for (int j = lane % *per; j < a.group_size; j += *per) {
            const Key v = sk[g * a.group_size + j];
            *k2 = max(*k2, min(*k1, v));
            *k1 = max(*k1, v);
        }
    merge_best(*k1, *k2, *per);
    return g;
}
// Group of expert e by a multiplication: exact for e < 1024.
__device__ __forceinline__ uint32_t group_mul(int size) { return ((1u << 22) + size - 1) / size; }

// One token in 64 bits; returns the expert of place `lane`, or -1.
template <int VPL>
__device__ __noinline__ int route_exact(const ScoredArgs &a, const float *row, float m, uint64_t *sk) {
    const int lane = threadIdx.x & 31, V = (a.E + 31) / 32;
    double z = 1.0;
    if (!a.sigmoid) {
        z = 0.0;
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            const float l = e < a.E ? __ldg(row + e) : -INFINITY;
            if (is_live(l)) z += score_of(l, false, m, 1.0);
        }
        z = warp_sum(z);
    }
    uint64_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane * V + i;
        key[i] = 0;
        if (i >= V || e >= a.E) continue;
        const float l = __ldg(row + e), b = a.bias ? __ldg(a.bias + e) : 0.0f;
        if (is_live(l) && is_live(b)) key[i] = choice_key(score_of(l, a.sigmoid, m, z) + (double)b);
    }
    if (a.n_group > 1) {
        uint64_t k1, k2;
        int per;
        const int g = group_best<VPL>(a, key, sk, &k1, &k2, &per);
        uint64_t gk = 0;  // the group's key, on its first lane
        if (lane % per == 0 && k1 != 0)
            gk = choice_key(key_choice(k1) + (a.group_top > 1 && k2 != 0 ? key_choice(k2) : 0.0));
        uint32_t kept = 0;
        for (int r = 0; r < a.topk_group; ++r) {
            const uint64_t best = warp_max_key(gk);
            if (best == 0) break;  // only groups without a live expert are left
            const int win = __reduce_min_sync(kAll, gk == best ? g : 32);
            if (g == win) gk = 0;
            kept |= 1u << win;
        }
        const uint32_t mul = group_mul(a.group_size);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (!((kept >> (((uint32_t)(lane * V + i) * mul) >> 22)) & 1u)) key[i] = 0;
    }
    int mine = -1;
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
        const int id = lane * V + bi, win = __reduce_min_sync(kAll, bk == best ? id : 0x7fffffff);
        if (id == win) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i == bi) key[i] = 0;
        }
        if (lane == j) mine = win;
    }
    return mine;
}

// fp32 choices.  A score s in [0, 1] formed with the fast exponential and division is
// off by less than 2^-19: sigmoid, s (1 - s) times the exponential's 2 + 1.2 |l| steps,
// and 2 steps of the division; softmax, s times the steps of its exponential (weighed by
// it), of the sum (their mean, and VPL + 5 roundings) and of the division, below 60 half
// steps together.  Adding the bias rounds by half a step of c.  So two choices whose gap
// exceeds 2^-17 + 2^-21 (|c| + |c'|), four times those bounds, stand in the same
// order in 64 bits; for group scores, sums of two, twice that.
__device__ __forceinline__ bool far_apart(float c, float d, float times) {
    return c - d > times * (0x1p-17f + 0x1p-21f * (fabsf(c) + fabsf(d)));  // false for a NaN (inf - inf)
}
__device__ __forceinline__ uint32_t key32(float c) {  // of a number that is not NaN; never 0
    const uint32_t b = __float_as_uint(c + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float choice32(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// Lane l holds experts l V .. l V + V-1, V = ceil(E / 32) <= VPL.
template <int VPL>
__global__ void __launch_bounds__(32 * kWarps) k_route_scored(const ScoredArgs a) {
    extern __shared__ uint64_t s_keys[];  // [kWarps][E] with groups
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= a.T) return;
    const int V = (a.E + 31) / 32, e0 = lane * V;
    const float *row = a.logits + (size_t)t * a.E;
    uint64_t *sk = s_keys + (size_t)warp * a.E;
    float c[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = i < V && e0 + i < a.E ? __ldg(row + e0 + i) : -INFINITY;
    float m = 0.0f, rz = 1.0f;
    uint32_t live = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) live |= (uint32_t)is_live(c[i]) << i;
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = __fdividef(1.0f, 1.0f + __expf(-c[i]));
    } else {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = (live >> i) & 1u ? fmaxf(m, c[i]) : m;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            c[i] = (live >> i) & 1u ? (c[i] == m ? 1.0f : __expf(c[i] - m)) : 0.0f;
            z += c[i];
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(kAll, z, off);
        rz = __fdividef(1.0f, z);
    }
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const float b = a.bias && i < V && e0 + i < a.E ? __ldg(a.bias + e0 + i) : 0.0f;
        key[i] = ((live >> i) & 1u) && is_live(b) ? key32(c[i] * rz + b) : 0u;
    }
    bool sure = true;
    if (a.n_group > 1) {
        uint32_t k1 = 0, k2 = 0;
        int g, per;
        if (a.E == 32 * V && (a.n_group & (a.n_group - 1)) == 0) {
            // a group is a power of two of whole lanes
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                k2 = max(k2, min(k1, key[i]));
                k1 = max(k1, key[i]);
            }
            per = 32 / a.n_group;
            g = lane / per;
            merge_best(k1, k2, per);
        } else {
            g = group_best<VPL>(a, key, reinterpret_cast<uint32_t *>(sk), &k1, &k2, &per);
        }
        uint32_t gk = 0;
        if (lane % per == 0 && k1 != 0) gk = key32(choice32(k1) + (a.group_top > 1 && k2 != 0 ? choice32(k2) : 0.0f));
        uint32_t kept = 0;
        float last = 0.0f;
        for (int r = 0; r <= a.topk_group; ++r) {
            const uint32_t best = __reduce_max_sync(kAll, gk);
            if (best == 0) break;
            if (r == a.topk_group) {
                sure = far_apart(last, choice32(best), 2.0f);
                break;
            }
            const int win = __reduce_min_sync(kAll, gk == best ? g : 32);
            if (g == win) gk = 0;
            kept |= 1u << win;
            last = choice32(best);
        }
        const uint32_t mul = group_mul(a.group_size);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (!((kept >> (((uint32_t)(e0 + i) * mul) >> 22)) & 1u)) key[i] = 0;
    }

    int mine = -1;  // lane j: the expert of place j
    float prev = 0.0f;
    for (int j = 0; j <= a.k && sure; ++j) {
        uint32_t bk = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < VPL; ++i)
            if (key[i] > bk) {
                bk = key[i];
                bi = i;
            }
        const uint32_t best = __reduce_max_sync(kAll, bk);
        if (best == 0) break;  // every live expert of the kept groups is taken
        const float now = choice32(best);
        if (j > 0) sure = far_apart(prev, now, 1.0f);
        if (j == a.k) break;
        prev = now;
        const int id = e0 + bi, win = __reduce_min_sync(kAll, bk == best ? id : 0x7fffffff);
        if (bk == best && id == win) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i == bi) key[i] = 0;
        }
        if (lane == j) mine = win;
    }
    if (!sure) mine = route_exact<VPL>(a, row, m, sk);

    // weights.  The softmax denominator cancels where they are renormalised
    double z = 1.0;
    if (!a.sigmoid && !a.renorm) {
        z = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if ((live >> i) & 1u) z += score_of(__ldg(row + e0 + i), false, m, 1.0);
        z = warp_sum(z);
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
