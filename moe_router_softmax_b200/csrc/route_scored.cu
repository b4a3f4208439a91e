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
// operations.  Choices and group scores are formed in fp32 first, with a bound on their
// error, and where every gap that the result rests on (between consecutive winners,
// between the last one and the next, between the last kept group and the next) exceeds the
// two errors, 64 bits would decide alike.  Elsewhere the candidates
// are put in order in 64 bits: the experts that no gap separates from the k-th, one
// to a lane, or the groups; where more than 32 are that close, the whole token.  The
// winners' weights are always formed in 64 bits.
//
// How many tokens leave the fp32 decision depends on how far apart the k best choices lie
// (counted over normal logits, without groups): 1 to 3 in a hundred at k = 8, up to
// 512 experts and logits of spread 1.5 to 2, softmax or sigmoid; but 71 (10 of them as a whole)
// at 1024 experts and k = 32, whose softmax scores are small beside a bound that does not shrink with
// them, and 64 to 97 where sigmoid scores saturate (spread 5, 128 to 256 experts, no bias).
//
// Bound by latency: 8192 tokens of 256 experts in 8 groups read 8.4 MB (1.3 us of HBM) and
// take some 1100 warp instructions each, issued in 53% of the cycles (integer pipe 44%) from the 28
// warps that 68 registers leave room for, each a chain of reductions and votes and then the
// winners' exponentials and divisions in 64 bits; a small batch is one such chain.  Measured on
// B200, 64 bits throughout -> this: one token 5.5 -> 3.4 us, 61 tokens of 165 experts 7.9 ->
// 6.5, 8192 tokens 23.7 -> 15.3.  Without groups: 8192 tokens of 256 experts 10.4 us (sigmoid
// scores of spread 5, in 64 bits: 12.9), of 1024 experts with k = 8 44 us, with k = 32 182 us.
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

// Softmax denominator of a token in 64 bits.
__device__ __forceinline__ double denominator(const ScoredArgs &a, const float *row, float m) {
    double z = 0.0;
#pragma unroll 8
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
        const float l = __ldg(row + e);
        const double v = score_of(l, false, m, 1.0);
        z += is_live(l) ? v : 0.0;
    }
    return warp_sum(z);
}

// 64-bit keys of the lane's experts.  (Scores of masked experts are formed like the
// others, so that the lane's exponentials run side by side.)
template <int VPL>
__device__ __forceinline__ void exact_keys(const ScoredArgs &a, const float *row, float m, uint64_t key[VPL]) {
    const int lane = threadIdx.x & 31, V = (a.E + 31) / 32;
    const double z = a.sigmoid ? 1.0 : denominator(a, row, m);
    float l[VPL], b[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const bool in = i < V && lane * V + i < a.E;
        l[i] = in ? __ldg(row + lane * V + i) : -INFINITY;
        b[i] = in && a.bias ? __ldg(a.bias + lane * V + i) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const uint64_t k = choice_key(score_of(l[i], a.sigmoid, m, z) + (double)b[i]);
        key[i] = is_live(l[i]) && is_live(b[i]) ? k : 0;
    }
}

// The kept groups (a bit each), decided in 64 bits.
template <int VPL>
__device__ __forceinline__ uint32_t exact_groups(const ScoredArgs &a, const uint64_t key[VPL], uint64_t *sk) {
    uint64_t k1, k2;
    int per;
    const int g = group_best<VPL>(a, key, sk, &k1, &k2, &per);
    uint64_t gk = 0;  // the group's key, on its first lane
    if ((threadIdx.x & 31) % per == 0 && k1 != 0)
        gk = choice_key(key_choice(k1) + (a.group_top > 1 && k2 != 0 ? key_choice(k2) : 0.0));
    uint32_t kept = 0;
    for (int r = 0; r < a.topk_group; ++r) {
        const uint64_t best = warp_max_key(gk);
        if (best == 0) break;  // only groups without a live expert are left
        const int win = __reduce_min_sync(kAll, gk == best ? g : 32);
        if (g == win) gk = 0;
        kept |= 1u << win;
    }
    return kept;
}
template <int VPL>
__device__ __noinline__ uint32_t groups_exact(const ScoredArgs &a, const float *row, float m, uint64_t *sk) {
    uint64_t key[VPL];
    exact_keys<VPL>(a, row, m, key);
    return exact_groups<VPL>(a, key, sk);
}

// One token in 64 bits; returns the expert of place `lane`, or -1.
template <int VPL>
__device__ __noinline__ int route_exact(const ScoredArgs &a, const float *row, float m, uint64_t *sk) {
    const int lane = threadIdx.x & 31, V = (a.E + 31) / 32;
    uint64_t key[VPL];
    exact_keys<VPL>(a, row, m, key);
    if (a.n_group > 1) {
        const uint32_t kept = exact_groups<VPL>(a, key, sk), mul = group_mul(a.group_size);
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

// fp32 choices.  What the fast exponential and division (2 + 1.2 |x| and 2 units in
// the last place, 2^-23 relative) and the roundings leave in a score s:
//   sigmoid  s (1 - s) (2 + 1.2 |l|) + 0.5 s + 2 s units, below 2^-21
//   softmax  s times its exponential's error, weighed by it (2 units), the sum's (a
//            mean of such errors, 4, and up to 37 roundings) and the division's: below
//            28 units of s; taken at s = 1 for every score, 2^-18.2, so that small scores
//            near one another go to 64 bits more often than they have to
// Adding the bias rounds by half a unit of c, and a key gives up the bits that hold
// its slot (below VPL units).  Two choices whose gap exceeds twice the sum of both errors
// stand in the same order in 64 bits.  size: |c| + |d|, and for group scores, sums of
// two choices that may cancel, twice the largest members' magnitudes; times: 2 there.
template <int VPL>
__device__ __forceinline__ bool far_apart(float c, float d, float size, bool sigmoid, float times) {
    const float score = sigmoid ? 0x1p-19f : 0x1p-16f, rel = 2.0f * (VPL + 2) * 0x1p-23f;
    return c - d > times * (score + rel * size);  // false for a NaN (inf - inf)
}
template <int VPL>
__device__ __forceinline__ bool far_apart(float c, float d, bool sigmoid) {
    return far_apart<VPL>(c, d, fabsf(c) + fabsf(d), sigmoid, 1.0f);
}
__device__ __forceinline__ uint32_t key32(float c) {  // of a number that is not NaN; never 0
    const uint32_t b = __float_as_uint(c + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float choice32(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// Lane l holds experts l V .. l V + V-1, V = ceil(E / 32) <= VPL.  Compares, selects and
// minima are most of a token's instructions, so a key holds its slot in its
// lowest bits: the best of a lane is VPL - 1 maxima, the warp's best one reduction and
// one vote, and equal choices, which this order would get wrong, are never far apart.
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
    float c[VPL], b[VPL];
    // whole 16-byte pieces where every lane's experts are aligned ones
    if (VPL >= 4 && a.E == 32 * VPL && (((uintptr_t)a.logits | (uintptr_t)a.bias) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < VPL / 4; ++i) {
            const float4 u = __ldg(reinterpret_cast<const float4 *>(row + e0) + i);
            const float4 w = a.bias ? __ldg(reinterpret_cast<const float4 *>(a.bias + e0) + i)
                                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float us[4] = {u.x, u.y, u.z, u.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[4 * i + j < VPL ? 4 * i + j : 0] = us[j];
                b[4 * i + j < VPL ? 4 * i + j : 0] = ws[j];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool in = i < V && e0 + i < a.E;
            c[i] = in ? __ldg(row + e0 + i) : -INFINITY;
            b[i] = in && a.bias ? __ldg(a.bias + e0 + i) : 0.0f;
        }
    }
    uint32_t key[VPL];
    float m = 0.0f;
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const float v = __fdividef(1.0f, 1.0f + __expf(-c[i])) + b[i];
            key[i] = is_live(c[i]) && is_live(b[i]) ? (key32(v) & ~(uint32_t)(VPL - 1)) | (uint32_t)i : 0u;
        }
    } else {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = is_live(c[i]) ? fmaxf(m, c[i]) : m;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
        float z = 0.0f, x[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            x[i] = is_live(c[i]) ? (c[i] == m ? 1.0f : __expf(c[i] - m)) : 0.0f;
            z += x[i];
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(kAll, z, off);
        const float rz = __fdividef(1.0f, z);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            key[i] = is_live(c[i]) && is_live(b[i]) ? (key32(x[i] * rz + b[i]) & ~(uint32_t)(VPL - 1)) | (uint32_t)i : 0u;
    }

    if (a.n_group > 1) {
        uint32_t k1 = 0, k2 = 0;
        int g, per;
        const bool whole = a.E == 32 * V && (a.n_group & (a.n_group - 1)) == 0;
        if (whole) {  // a group is a power of two of whole lanes
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
        float size = 0.0f;
        if (lane % per == 0 && k1 != 0) {
            const float c1 = choice32(k1), c2 = a.group_top > 1 && k2 != 0 ? choice32(k2) : 0.0f;
            gk = c1 + c2 == c1 + c2 ? key32(c1 + c2) : 0xffffffffu;  // (inf - inf: first, and not far from any)
            size = fabsf(c1) + fabsf(c2);
        }
        // the largest members of any group: a sum that cancels carries their errors
        const float most = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(size)));
        uint32_t kept = 0, last = 0;
        for (int r = 0; r <= a.topk_group; ++r) {
            const uint32_t best = __reduce_max_sync(kAll, gk);
            if (best == 0) break;
            const int win = __ffs(__ballot_sync(kAll, gk == best)) - 1;  // equal groups are not far apart
            if (r == a.topk_group) {
                if (!far_apart<VPL>(choice32(last), choice32(best), 2.0f * most, a.sigmoid, 2.0f))
                    kept = groups_exact<VPL>(a, row, m, sk);
                break;
            }
            if (lane == win) gk = 0;
            kept |= 1u << (win / per);
            last = best;
        }
        if (whole) {
            const bool on = (kept >> g) & 1u;
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = on ? key[i] : 0u;
        } else {
            const uint32_t mul = group_mul(a.group_size);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (!((kept >> (((uint32_t)(e0 + i) * mul) >> 22)) & 1u)) key[i] = 0;
        }
    }

    // k rounds, and more until a gap separates the candidates from the rest: lane j
    // holds the j-th best key and the expert it stands for
    uint32_t my_key = 0, last = 0;
    int mine = -1, n = 0;  // n candidates
    bool sure = true;
    for (;; ++n) {
        uint32_t bk = key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) bk = max(bk, key[i]);
        const uint32_t best = __reduce_max_sync(kAll, bk);
        if (best == 0) break;  // every live expert of the kept groups is taken
        if (n >= a.k && far_apart<VPL>(choice32(last), choice32(best), a.sigmoid)) break;
        if (n == 32) {
            sure = false;
            break;
        }
        if (n == a.k - 1) last = best;  // (a later candidate has to be far from place k, not from the one before)
        const int win = __ffs(__ballot_sync(kAll, bk == best)) - 1, slot = (int)(best & (VPL - 1));
        if (lane == n) {
            my_key = best;
            mine = win * V + slot;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (slot == i) key[i] = lane == win ? 0u : key[i];  // one slot, the same on all lanes
    }
    // the softmax denominator in 64 bits, where a choice or a weight needs it
    double z = 1.0;
    bool have_z = a.sigmoid != 0;
    double s = 0.0;
    if (!sure) {
        mine = route_exact<VPL>(a, row, m, sk);
    } else {
        const uint32_t after = __shfl_down_sync(kAll, my_key, 1);
        const bool ordered = lane >= min(n, a.k) - 1 || far_apart<VPL>(choice32(my_key), choice32(after), a.sigmoid);
        if (n > a.k || !__all_sync(kAll, ordered)) {
            // the candidates' order in 64 bits, one to a lane
            if (!have_z) z = denominator(a, row, m);
            have_z = true;
            uint64_t ck = 0;
            if (mine >= 0)
                ck = choice_key(score_of(__ldg(row + mine), a.sigmoid, m, z) + (double)(a.bias ? __ldg(a.bias + mine) : 0.0f));
            int won = -1;
            for (int j = 0; j < min(n, a.k); ++j) {
                const uint64_t best = warp_max_key(ck);
                const int win = __reduce_min_sync(kAll, ck == best ? mine : 0x7fffffff);
                if (mine == win) ck = 0;
                if (lane == j) won = win;
            }
            mine = won;
        }
    }
    if (lane >= a.k) mine = -1;

    // weights.  The softmax denominator cancels where they are renormalised
    if (!a.renorm && !have_z) z = denominator(a, row, m);
    if (mine >= 0) s = score_of(__ldg(row + mine), a.sigmoid, m, a.renorm ? 1.0 : z);
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
