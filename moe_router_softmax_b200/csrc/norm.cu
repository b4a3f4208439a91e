// norm.cu -- the norms around a block: the block's output (dense, or combined
// from the experts' rows) is normalised, gated and added to the residual, and
// the sum is normalised again for the next block, whose int8 products may take
// it as codes.  The row is held in registers throughout.
//
//   z  = dense z[t], or sum_j w[t][j] rows[route_pos[t k + j]]      (fp32)
//   zn = z * rsqrt(mean(z^2) + eps) * (offset + post_w)
//   y  = residual_scale * residual + block_scale * gate_t[t] * gate_h[h] * zn
//   xn = y * rsqrt(mean(y^2) + eps) * (offset + next_w)             (y as stored)
//   sx = max |xn| / 127,  xq = rint(xn / sx)                        (xn before its rounding)
// In xn / sx = 127 xn / max |xn| the row's norm cancels, and any factor of it does.  The
// codes are formed from p = y f (offset + next_w), f = 127 times a power of two: without an
// offset p is exact (8 bits of y, 7 of 127, 8 of the weight), and so is max |p| / 127, so that a code
// carries neither the rounding of the sum of squares nor those of xn and sx: it is the
// definition's, halves included.
#include <cuda_bf16.h>

#include "i8_math.cuh"
#include "ops.cuh"

namespace moe {
namespace {

enum { kSrcNone = 0, kSrcDense = 1, kSrcRows = 2 };

__device__ __forceinline__ void unpack8(uint4 u, float v[8]) {
    const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(p[i]);
        v[2 * i + 1] = bf16_hi(p[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float v[8]) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        p[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(p[0], p[1], p[2], p[3]);
}

// Sum or maximum over a row's threads, the same on every one (fixed order: the
// lanes' butterfly, then the warps in turn).  Each reduction of a kernel has its own
// partials, so one barrier serves it.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float *s_part) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? max_nan(v, o) : v + o;
    }
    const int nw = (int)(blockDim.x >> 5);
    if (nw == 1) return v;
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    // four partials a load, added in turn
    v = MAX ? 0.0f : -0.0f;
    for (int i = 0; i < nw; i += 4) {
        const float4 u = *reinterpret_cast<const float4 *>(s_part + i);
        const float w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < nw) v = MAX ? max_nan(v, w[j]) : v + w[j];
    }
    return v;
}

__device__ __forceinline__ void load8(const float *p, float v[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// A row on blockDim.x threads (blockDim.y rows per CTA, more than one only when a
// row is a warp's), CH chunks of 8 columns per thread (chunk c of the row on thread
// c % blockDim.x).  The rows are read once and written once.  FEW rows are bound by the
// chain of loads and reductions: everything that a row needs is requested before its
// first reduction, and the rows of eight routes at a time.  Many are bound by HBM, where
// more rows in flight (fewer registers) hide a row's chain.
constexpr int kMaxThreads = 512;
template <int SRC, int CH, bool FEW>
__global__ void __launch_bounds__(kMaxThreads, FEW || CH > 1 ? 1 : 2) k_norm(const NormArgs a) {
    constexpr bool EARLY = (FEW || SRC != kSrcRows) && CH <= 2;
    // routes at a time (many rows: 2, 148 us; 1, 157; 3, 176; 4, 188)
    constexpr int B = FEW ? (CH == 1 ? 8 : 4) : 2;
    __shared__ __align__(16) float s_part[3][32];
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x * blockDim.y + threadIdx.y, nch = a.H / 8;
    if (t >= a.T) return;
    const size_t base = (size_t)t * a.H;
    const bool post = SRC != kSrcNone && a.post_w != nullptr, next = a.next_w != nullptr;
    float v[CH][8];
    uint4 res[CH], pw[CH], nw[CH];
    float gh[CH][8];
    // the block's weights for chunk c of this thread
    auto load_block = [&](int c, int ch) {
        res[c] = reinterpret_cast<const uint4 *>(a.residual + base)[ch];  // a plain load: y may be this row
        if (post) pw[c] = __ldg(reinterpret_cast<const uint4 *>(a.post_w) + ch);
        if (a.gate_h) load8(a.gate_h + ch * 8, gh[c]);
    };
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = threadIdx.x + c * blockDim.x;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = 0.0f;
        if (ch >= nch) continue;
        if (SRC == kSrcRows) {
            for (int j0 = 0; j0 < a.k; j0 += B) {
                int p[B];
                float wj[B], r[B][8];
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    p[j] = j0 + j < a.k ? __ldg(a.route_pos + (size_t)t * a.k + j0 + j) : -1;
                    wj[j] = j0 + j < a.k ? __ldg(a.w + (size_t)t * a.k + j0 + j) : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < B; ++j)
                    if ((unsigned)p[j] < (unsigned)(a.T * a.k)) load8(a.rows + (size_t)p[j] * a.H + ch * 8, r[j]);
                if (EARLY && j0 == 0) {
                    load_block(c, ch);
                    if (next) nw[c] = __ldg(reinterpret_cast<const uint4 *>(a.next_w) + ch);
                }
#pragma unroll
                for (int j = 0; j < B; ++j)
                    if ((unsigned)p[j] < (unsigned)(a.T * a.k)) {  // not a dropped route
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[c][i] = __fmaf_rn(wj[j], r[j][i], v[c][i]);
                    }
            }
        } else {
            const uint16_t *src = SRC == kSrcDense ? a.z : a.residual;
            const uint4 u = reinterpret_cast<const uint4 *>(src + base)[ch];
            if (EARLY) {
                if (SRC == kSrcDense) load_block(c, ch);
                if (next) nw[c] = __ldg(reinterpret_cast<const uint4 *>(a.next_w) + ch);
            }
            unpack8(u, v[c]);
        }
    }
    if (SRC != kSrcNone) {
        const float bs = a.gate_t ? a.block_scale * __ldg(a.gate_t + t) : a.block_scale;
        float r = 1.0f;
        if (post) {
            float ss = 0.0f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = __fmaf_rn(v[c][i], v[c][i], ss);
            r = __frsqrt_rn(__fmaf_rn(row_reduce<false>(ss, s_part[0]), a.inv_h, a.eps));
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = threadIdx.x + c * blockDim.x;
            if (ch >= nch) continue;
            if (!EARLY) load_block(c, ch);
            float rv[8], wv[8];
            unpack8(res[c], rv);
            if (post) unpack8(pw[c], wv);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float zn = v[c][i];
                // (roundings spelled out: the same in every instantiation)
                if (post) zn = __fmul_rn(__fmul_rn(zn, r), __fadd_rn(a.offset, wv[i]));
                if (a.gate_h) zn = __fmul_rn(zn, gh[c][i]);
                v[c][i] = __fmaf_rn(bs, zn, __fmul_rn(a.residual_scale, rv[i]));
            }
            const uint4 o = pack8(v[c]);
            reinterpret_cast<uint4 *>(a.y + base)[ch] = o;
            unpack8(o, v[c]);  // the next norm reads what is stored
        }
    }
    if (!next) return;
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __fmaf_rn(v[c][i], v[c][i], ss);
    const float r = __frsqrt_rn(__fmaf_rn(row_reduce<false>(ss, s_part[1]), a.inv_h, a.eps));
    if (a.xq == nullptr) {  // without codes: xn alone, by the same operations
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = threadIdx.x + c * blockDim.x;
            if (ch >= nch) continue;
            if (!EARLY) nw[c] = __ldg(reinterpret_cast<const uint4 *>(a.next_w) + ch);
            float wv[8];
            unpack8(nw[c], wv);
#pragma unroll
            for (int i = 0; i < 8; ++i) wv[i] = __fmul_rn(__fmul_rn(v[c][i], r), __fadd_rn(a.offset, wv[i]));
            reinterpret_cast<uint4 *>(a.xn + base)[ch] = pack8(wv);
        }
        return;
    }
    // r = f rr, f = 127/128 of a power of two, 1 <= rr < 2.02: p has the range of n = p rr
    const uint32_t r_exp = __float_as_uint(r) & 0x7f800000u;
    const float f = __fmul_rn(__uint_as_float(r_exp), 127.0f / 128.0f);
    const float rr = __fmul_rn(__fmul_rn(r, __uint_as_float(0x7f000000u - r_exp)), 128.0f / 127.0f);
    float amax = 0.0f;  // of p
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = threadIdx.x + c * blockDim.x;
        if (ch >= nch) continue;
        if (!EARLY) nw[c] = __ldg(reinterpret_cast<const uint4 *>(a.next_w) + ch);
        float wv[8];
        unpack8(nw[c], wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float w = __fadd_rn(a.offset, wv[i]);
            wv[i] = __fmul_rn(__fmul_rn(v[c][i], r), w);
            v[c][i] = __fmul_rn(__fmul_rn(v[c][i], f), w);
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) amax = max_nan(amax, fabsf(v[c][i]), fabsf(v[c][i + 1]));
        if (a.xn) reinterpret_cast<uint4 *>(a.xn + base)[ch] = pack8(wv);
    }
    amax = row_reduce<true>(amax, s_part[2]);
    CodeScale sc = code_scale(amax);
    float sx = __fmul_rn(sc.s, rr);
    if (sx < 0x1p-126f) {  // a subnormal scale has few bits: the codes are those of n at it
        sc = code_scale(__fmul_rn(amax, rr));
        sx = sc.s;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = __fmul_rn(v[c][i], rr);
    }
    if (threadIdx.x == 0) a.sx[t] = sx;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = threadIdx.x + c * blockDim.x;
        if (ch >= nch) continue;
        reinterpret_cast<uint2 *>(a.xq + base)[ch] =
            make_uint2(sc.code4(make_float4(v[c][0], v[c][1], v[c][2], v[c][3])),
                       sc.code4(make_float4(v[c][4], v[c][5], v[c][6], v[c][7])));
    }
}

// Rows up to 1024 wide: a warp each, four to a CTA.  Wider ones: a CTA each, up to
// 512 threads.  A row's layout, and so the order of its sums, depends on its width
// alone: a row's result is the same in any batch, and whether the norm before the next
// block runs here or by itself.
// Measured, 2816 wide: one token of 8 routes 3.7 us (with codes 4.4); 8192 tokens of 8 routes
// 146 us, 6.0 TB/s of 876 MB; a dense block's 8192 tokens 52 us (71), 3.6 TB/s; moe_norm of
// 1023 rows 4.7 us (7.5), of 16384 rows 53 us (85), 3.5 TB/s.  Without the routes' loads HBM
// does not bound it: the schedulers issue in 67% of the cycles (78% with codes), 27 (52)
// instructions a value for unpacking, rounding and packing and a thread's share of the
// reductions; for the rest of the cycles the four CTAs that an SM holds, a row each, wait for their
// loads and barriers.  Four rows on the same threads, for more loads in flight, were no faster.
constexpr int kFewRows = 256;

template <int SRC, bool FEW>
cudaError_t launch_rows(const NormArgs &a, cudaStream_t s) {
    const int nch = a.H / 8, y = nch <= 128 && a.T >= 4 ? 4 : 1, x_max = nch <= 128 ? 32 : kMaxThreads;
    int ch = 1;
    while (ch * x_max < nch) ch *= 2;  // 1, 2 or 4 (H <= 16384)
    const int x = ((nch + ch - 1) / ch + 31) / 32 * 32;
    const dim3 grid((unsigned)((a.T + y - 1) / y)), block((unsigned)x, (unsigned)y);
    if (ch == 1) return launch_pdl(k_norm<SRC, 1, FEW>, grid, block, 0, s, a);
    if (ch == 2) return launch_pdl(k_norm<SRC, 2, FEW>, grid, block, 0, s, a);
    return launch_pdl(k_norm<SRC, 4, FEW>, grid, block, 0, s, a);
}

template <int SRC>
cudaError_t launch_src(const NormArgs &a, cudaStream_t s) {
    return a.T <= kFewRows ? launch_rows<SRC, true>(a, s) : launch_rows<SRC, false>(a, s);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    if (a.rows) return launch_src<kSrcRows>(a, s);
    if (a.z) return launch_src<kSrcDense>(a, s);
    return launch_src<kSrcNone>(a, s);
}

}  // namespace moe
