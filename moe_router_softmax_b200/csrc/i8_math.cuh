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
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Scale of a row from its largest magnitude, and the codes at it: rint(v / s) by a
// multiplication with 1 / s (a division per value costs more than the rest of a
// code); 0 where s is 0 or NaN and for a NaN.  Where 1 / s overflows (s below 2^-128, a
// scale of few bits), v / s itself, kept to +-127.
struct CodeScale {
    float s, inv;
    // The rounding to an integer is that of an addition: v / s is at most 127 and a
    // rounding, and 1.5 * 2^23 + q has q, to the nearest even, in its lowest bits (the
    // converting instruction runs at a quarter of the rate).
    __device__ __forceinline__ uint32_t code_bits(float v) const {  // the code in the lowest byte
        const float q = inv <= 3.402823466e+38f ? __fmul_rn(v, inv) : fminf(fmaxf(__fdiv_rn(v, s), -127.0f), 127.0f);
        return q == q ? __float_as_uint(__fadd_rn(q, 12582912.0f)) : 0u;
    }
    __device__ __forceinline__ uint32_t code4(float4 v) const {
        const uint32_t lo = __byte_perm(code_bits(v.x), code_bits(v.y), 0x0040);
        const uint32_t hi = __byte_perm(code_bits(v.z), code_bits(v.w), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
};
__device__ __forceinline__ CodeScale code_scale(float amax) {
    CodeScale c;
    c.s = __fdiv_rn(amax, 127.0f);
    c.inv = c.s > 0.0f ? __fdiv_rn(1.0f, c.s) : 0.0f;
    return c;
}

}  // namespace moe
