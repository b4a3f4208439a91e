// norm.cu -- the norms around a block: the block's output (dense, or combined
// from the experts' rows) is normalised, gated and added to the residual, and
// the sum is normalised again for the next block, whose int8 products may take
// it as codes.  One CTA per token, the row held in registers throughout.
//
//   z  = dense z[t], or sum_j w[t][j] rows[route_pos[t k + j]]      (fp32)
//   zn = z * rsqrt(mean(z^2) + eps) * (offset + post_w)
//   y  = residual_scale * residual + block_scale * gate_t[t] * gate_h[h] * zn
//   xn = y * rsqrt(mean(y^2) + eps) * (offset + next_w)             (y as stored)
//   sx = max |xn| / 127,  xq = rint(xn / sx)                        (xn before its rounding)
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
    for (int i = 0; i < 4; ++i)
        p[i] = (uint32_t)f32_to_bf16_rne(v[2 * i]) | ((uint32_t)f32_to_bf16_rne(v[2 * i + 1]) << 16);
    return make_uint4(p[0], p[1], p[2], p[3]);
}

// Sum or maximum over the CTA, the same on every thread (fixed order: the
// lanes' butterfly, then the warps in turn).
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float *s_part) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    const int nw = (int)(blockDim.x >> 5);
    if (nw == 1) return v;
    __syncthreads();  // the previous reduction's partials have been read
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s_part[0];
    for (int i = 1; i < nw; ++i) v = MAX ? fmaxf(v, s_part[i]) : v + s_part[i];
    return v;
}

// CH chunks of 8 columns per thread (chunk c on thread c % blockDim).
template <int SRC, int CH>
__global__ void __launch_bounds__(1024) k_norm(const NormArgs a) {
    __shared__ float s_part[32];
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x, nch = a.H / 8;
    const size_t base = (size_t)t * a.H;
    float v[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = threadIdx.x + c * blockDim.x;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = 0.0f;
        if (ch >= nch) continue;
        if (SRC == kSrcRows) {
            for (int j = 0; j < a.k; ++j) {
                const int p = __ldg(a.route_pos + (size_t)t * a.k + j);
                if ((unsigned)p >= (unsigned)(a.T * a.k)) continue;  // a dropped route
                const float wj = __ldg(a.w + (size_t)t * a.k + j);
                const float4 *r = reinterpret_cast<const float4 *>(a.rows + (size_t)p * a.H + ch * 8);
                const float4 r0 = __ldg(r), r1 = __ldg(r + 1);
                const float rv[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) v[c][i] = __fmaf_rn(wj, rv[i], v[c][i]);
            }
        } else {
            const uint16_t *src = SRC == kSrcDense ? a.z : a.residual;
            unpack8(reinterpret_cast<const uint4 *>(src + base)[ch], v[c]);  // a plain load: y may be this row
        }
    }
    if (SRC != kSrcNone) {
        float r = 1.0f;
        if (a.post_w) {
            float ss = 0.0f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = __fmaf_rn(v[c][i], v[c][i], ss);
            r = __frsqrt_rn(block_reduce<false>(ss, s_part) / (float)a.H + a.eps);
        }
        const float bs = a.gate_t ? a.block_scale * __ldg(a.gate_t + t) : a.block_scale;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = threadIdx.x + c * blockDim.x;
            if (ch >= nch) continue;
            float res[8], pw[8];
            unpack8(reinterpret_cast<const uint4 *>(a.residual + base)[ch], res);
            if (a.post_w) unpack8(__ldg(reinterpret_cast<const uint4 *>(a.post_w) + ch), pw);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float zn = v[c][i];
                if (a.post_w) zn = zn * r * (a.offset + pw[i]);
                if (a.gate_h) zn *= __ldg(a.gate_h + ch * 8 + i);
                v[c][i] = a.residual_scale * res[i] + bs * zn;
            }
            const uint4 o = pack8(v[c]);
            reinterpret_cast<uint4 *>(a.y + base)[ch] = o;
            unpack8(o, v[c]);  // the next norm reads what is stored
        }
    }
    if (a.next_w == nullptr) return;
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __fmaf_rn(v[c][i], v[c][i], ss);
    const float r = __frsqrt_rn(block_reduce<false>(ss, s_part) / (float)a.H + a.eps);
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = threadIdx.x + c * blockDim.x;
        if (ch >= nch) continue;
        float nw[8];
        unpack8(__ldg(reinterpret_cast<const uint4 *>(a.next_w) + ch), nw);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[c][i] = v[c][i] * r * (a.offset + nw[i]);
            amax = fmaxf(amax, fabsf(v[c][i]));
        }
        if (a.xn) reinterpret_cast<uint4 *>(a.xn + base)[ch] = pack8(v[c]);
    }
    if (a.xq == nullptr) return;
    const CodeScale sc = code_scale(block_reduce<true>(amax, s_part));
    if (threadIdx.x == 0) a.sx[t] = sc.s;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int ch = threadIdx.x + c * blockDim.x;
        if (ch >= nch) continue;
        reinterpret_cast<uint2 *>(a.xq + base)[ch] =
            make_uint2(sc.code4(make_float4(v[c][0], v[c][1], v[c][2], v[c][3])),
                       sc.code4(make_float4(v[c][4], v[c][5], v[c][6], v[c][7])));
    }
}

template <int SRC>
cudaError_t launch_src(const NormArgs &a, cudaStream_t s) {
    const int nch = a.H / 8;
    const int ch = (nch + 1023) / 1024;                       // 1 or 2 (H <= 16384)
    const int threads = (((nch + ch - 1) / ch) + 31) / 32 * 32;
    if (ch == 1) return launch_pdl(k_norm<SRC, 1>, dim3((unsigned)a.T), dim3((unsigned)threads), 0, s, a);
    return launch_pdl(k_norm<SRC, 2>, dim3((unsigned)a.T), dim3((unsigned)threads), 0, s, a);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    if (a.rows) return launch_src<kSrcRows>(a, s);
    if (a.z) return launch_src<kSrcDense>(a, s);
    return launch_src<kSrcNone>(a, s);
}

}  // namespace moe
