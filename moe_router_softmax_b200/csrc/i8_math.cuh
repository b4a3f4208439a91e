// i8_math.cuh -- device arithmetic shared by the int8 kernels: the scales'
// products, the gate, and the codes of a row.
#pragma once

#include "common.cuh"

namespace moe {

// The scales' products and the gate, in a fixed order of roundings: every kernel
// that takes a shape gives the same bits.
__device__ __forceinline__ float scaled(int sum, float s_token, float s_row) {
    return __fmul_rn(__fmul_rn((float)sum, s_token), s_row);
}
__device__ __forceinline__ float gate_up(int g_sum, int u_sum, float s_token, float s_gate, float s_up) {
    const float v = scaled(g_sum, s_token, s_gate), u = scaled(u_sum, s_token, s_up);
    const float cube = __fmul_rn(__fmul_rn(v, v), v);
    const float t = tanhf(__fmul_rn(0.7978845608028654f, __fmaf_rn(0.044715f, cube, v)));  // sqrt(2/pi)
    return __fmul_rn(__fmul_rn(__fmul_rn(0.5f, v), __fadd_rn(1.0f, t)), u);
}

// Maximum of magnitudes that a NaN takes part in (and wins): the codes of a row hold
// none, so it is the row's scale that has to carry one on.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// The codes rint(v / s) of a row whose largest magnitude is amax, s = amax / 127; 0 where s
// is 0, infinite or NaN.  The quotient is the correctly rounded one, so that a value
// halfway between two codes goes to the even one and every other to the nearest; a product with
// 1 / s alone is up to one and a half steps off, which gives every eighth of the values next to
// a half its neighbour's code.  A division per value costs more than the rest of a code;
// one residual, exact in fp32, corrects the product (Markstein's final step).
struct CodeScale {
    float s, inv;  // inv: 1 / s, or 0 where every code is
    // The rounding to an integer is that of an addition: the quotient is at most 127, and
    // 1.5 * 2^23 + q has q, to the nearest even, in its lowest bits (the converting
    // instruction runs at a quarter of the rate).
    __device__ __forceinline__ uint32_t pack(float4 q) const {
        const uint32_t x = __float_as_uint(__fadd_rn(q.x, 12582912.0f)), y = __float_as_uint(__fadd_rn(q.y, 12582912.0f));
        const uint32_t z = __float_as_uint(__fadd_rn(q.z, 12582912.0f)), w = __float_as_uint(__fadd_rn(q.w, 12582912.0f));
        return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
    }
    __device__ __forceinline__ float quotient(float v) const {
        const float q = __fmul_rn(v, inv);
        return __fmaf_rn(__fmaf_rn(-q, s, v), inv, q);
    }
    // The division itself where the residual would be subnormal or 1 / s may overflow (a scale of
    // few bits may leave the quotient a little over 127).
    __device__ __noinline__ uint32_t code4_tiny(float4 v) const {
        float q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
        for (int i = 0; i < 4; ++i) q[i] = fminf(fmaxf(__fdiv_rn(q[i], s), -127.0f), 127.0f);
        return pack(make_float4(q[0], q[1], q[2], q[3]));
    }
    __device__ __forceinline__ uint32_t code4(float4 v) const {
        if (inv > 0x1p100f) return code4_tiny(v);
        const uint32_t c = pack(make_float4(quotient(v.x), quotient(v.y), quotient(v.z), quotient(v.w)));
        return inv != 0.0f ? c : 0u;
    }
};
__device__ __forceinline__ CodeScale code_scale(float amax) {
    CodeScale c;
    c.s = __fdiv_rn(amax, 127.0f);
    c.inv = c.s > 0.0f ? __frcp_rn(c.s) : 0.0f;
    return c;
}

}  // namespace moe
