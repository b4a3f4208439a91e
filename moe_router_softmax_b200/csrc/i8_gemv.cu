// i8_gemv.cu -- int8 x int8 products for few tokens: dot products of codes with
// dp4a (four multiply-adds per lane and instruction, int32 sums, exact), the
// scales applied once per output.
//
//   linear  y[t][n] = sx[t] sw[n] sum_k xq[t][k] wq[n][k]
//   ffn     g = s13 sx (Q13 xq);  h_i = gelu_tanh(g_i) g_{I+i}   (fp32)
//           sh = max |h| / 127,  hq = rint(h / sh);  rows = s2 sh (Q2 hq)
//
// A weight row is read once (by the FFN once per route), 16 bytes per lane, so the weights'
// bytes bound these kernels.
#include <math.h>

#include <algorithm>

#include "i8_math.cuh"
#include "ops.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 4;

// These kernels up to here, then the tensor cores.  Measured on B200, these / those:
//   linear: 2816 x 2816, 2 tokens 4.4 / 5.2 us, 4 tokens 6.9 / 5.2; 8192 x 2816, 2
//   tokens 7.7 / 9.4, 4 tokens 12.8 / 9.4; 1408 x 704, 4 tokens 3.5 / 4.8 (every warp
//   reads the tokens' codes again, from L1)
//   ffn: these kernels read an expert's weights once for every route of it, those once,
//   behind two more launches.  What counts is the bytes that are read again (routes less the
//   distinct experts of a uniform choice, times 3 H I):
//     128 experts of 2816 x 704, top-8   40 routes, 28 MB again: 47.0 / 49.0 us; 48, 42 MB: 53.6 / 56.7; 96: 93 / 79
//     64 of 2048 x 1024, top-6           30, 32 MB: 42.4 / 43.3; 36, 47 MB: 47.2 / 43.8
//     8 of 1024 x 512, top-2             24, 26 MB: 12.2 / 15.2; 32, 38 MB: 16.4 / 15.2
//     4 of 4096 x 2048, top-2            8, 128 MB: 38 / 28; 40, 906 MB: 133 / 31
//     2 of 4096 x 4096, top-1            8, 303 MB: 70 / 32; 40, 1.9 GB: 268 / 35
//   and, for small experts, the routes (16 of 512 x 256, top-4: 40 routes 9.7 / 14.0, 96 routes 18.8 / 14.1).
constexpr int kGemvTokens = 2;
constexpr int kGemvTokensSmall = 4;
constexpr int64_t kGemvProducts = 20000000;  // T N K, past kGemvTokens
constexpr int kGemvRoutes = 40;
constexpr double kGemvAgainBytes = 35e6;

// First problem a kernel of this file recorded (0 = none), read and cleared by
// moe_take_device_errors(): 0x2005 a slot past the pool, 0x2007 a route out of range.
__device__ unsigned int g_i8_error;
__device__ unsigned int g_i8_error_info;
__device__ __forceinline__ void record_error(unsigned code, unsigned info) {
    if (atomicCAS(&g_i8_error, 0u, code) == 0u) g_i8_error_info = info;
}

__device__ __forceinline__ int dot16(uint4 w, uint4 x, int acc) {
    acc = __dp4a((int)w.x, (int)x.x, acc);
    acc = __dp4a((int)w.y, (int)x.y, acc);
    acc = __dp4a((int)w.z, (int)x.z, acc);
    return __dp4a((int)w.w, (int)x.w, acc);
}

// One warp per output row n and up to TB tokens.
template <int TB, bool FP32>
__global__ void __launch_bounds__(32 * kWarps) k_linear_i8(const LinearArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int n = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (n >= a.N) return;
    const int nch = a.K / 16;
    const uint4 *wr = reinterpret_cast<const uint4 *>(a.wq + (size_t)n * a.K);
    // a lane's loads of the weight row go out together, ahead of the tokens' (from L1/L2)
    constexpr int U = 6;
    int acc[TB] = {};
    for (int c0 = lane; c0 < nch; c0 += 32 * U) {
        uint4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            w[u] = c0 + 32 * u < nch ? ld_stream_v4(wr + c0 + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * u < nch)
#pragma unroll
                for (int t = 0; t < TB; ++t)
                    if (t < a.T)
                        acc[t] = dot16(w[u], __ldg(reinterpret_cast<const uint4 *>(a.xq + (size_t)t * a.K) + c0 + 32 * u),
                                       acc[t]);
    }
    const float sw = __ldg(a.sw + n);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        const int sum = __reduce_add_sync(kAll, acc[t]);
        if (lane != t || t >= a.T) continue;
        const float v = scaled(sum, __ldg(a.sx + t), sw);
        const size_t at = (size_t)t * a.N + n;
        if (FP32) static_cast<float *>(a.y)[at] = v;
        else static_cast<uint16_t *>(a.y)[at] = f32_to_bf16_rne(v);
    }
}

// Expert of sorted row s < offsets[E] (the number of experts whose rows end at
// or before s), by one warp.
__device__ __forceinline__ int expert_of_row(const int32_t *offsets, int E, int s) {
    int n = 0;
    for (int e = threadIdx.x & 31; e < E; e += 32) n += __ldg(offsets + e + 1) <= s;
    return __reduce_add_sync(kAll, n);
}

// Blob of the expert that sorted row s belongs to, or null where there is nothing
// to compute (past the last route, or a slot past the pool).
__device__ __forceinline__ const uint8_t *blob_of_row(const FfnI8Args &a, int s) {
    if (s >= min(__ldg(a.offsets + a.L.E), a.T * a.k)) return nullptr;
    const int e = expert_of_row(a.offsets, a.L.E, s);
    const uint8_t *blob = expert_blob(a.L, e);
    if (blob == nullptr && (threadIdx.x & 31) == 0) record_error(0x2005u, (unsigned)__ldg(a.L.slot_table + e));
    return blob;
}

constexpr int kU = 12;  // 16-byte loads of a lane in flight

// Phase 1: one warp per sorted row and intermediate column: lanes 0..15 take the
// gate row of W13, lanes 16..31 its up row, 16 bytes a lane and load.  All of a
// 2816-wide pair's loads are issued before the first product, so the launch is about one
// round trip to HBM wide.
__global__ void __launch_bounds__(32 * kWarps, 7) k_ffn_i8_gemv1(const FfnI8Args a, float *__restrict__ h) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, l16 = lane & 15, I = a.L.I, H = a.L.H, per = I / kWarps;
    const int s = blockIdx.x / per, i = (blockIdx.x % per) * kWarps + (threadIdx.x >> 5);
    const int R = a.T * a.k;
    const int route = a.T == 1 ? s : __ldg(a.sorted_route + s);
    const uint8_t *blob = blob_of_row(a, s);
    if (blob == nullptr) return;
    if (route < 0 || route >= R) {
        if (lane == 0) record_error(0x2007u, (unsigned)s);
        return;
    }
    const int t = a.T == 1 ? 0 : route / a.k;
    const int row = lane < 16 ? i : I + i, nch = H / 16;
    const uint4 *w = reinterpret_cast<const uint4 *>(blob + a.L.off.q13 + (size_t)row * H) + l16;
    const uint4 *x = reinterpret_cast<const uint4 *>(a.xq + (size_t)t * H) + l16;
    const float sw = __ldg(reinterpret_cast<const float *>(blob + a.L.off.s13) + row), sx = __ldg(a.sx + t);
    int acc = 0;
    for (int c0 = l16; c0 < nch; c0 += 16 * kU, w += 16 * kU, x += 16 * kU) {
        uint4 u[kU];
#pragma unroll
        for (int j = 0; j < kU; ++j)
            u[j] = c0 + 16 * j < nch ? ld_stream_v4(w + 16 * j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < kU; ++j)
            if (c0 + 16 * j < nch) acc = dot16(u[j], __ldg(x + 16 * j), acc);
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) acc += __shfl_xor_sync(kAll, acc, off);
    const int up = __shfl_xor_sync(kAll, acc, 16);
    const float su = __shfl_xor_sync(kAll, sw, 16);
    if (lane == 0) h[(size_t)s * I + i] = gate_up(acc, up, sx, sw, su);
}

// Phase 2: a CTA takes 32 output rows of one sorted row, four lanes a row.  A lane's
// first weights are requested before the wait for h (phase 1 has waited for all
// launches before it, and writes no weights), then the CTA forms the codes of the
// row's h in shared memory.
constexpr int kRows2 = 8 * kWarps;
__global__ void __launch_bounds__(32 * kWarps, 6) k_ffn_i8_gemv2(const FfnI8Args a, const float *__restrict__ h) {
    extern __shared__ __align__(16) int8_t s_hq[];  // [I]
    __shared__ float s_part[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, I = a.L.I, H = a.L.H;
    const int per = H / kRows2, nch = I / 16;
    const int s = blockIdx.x / per, n = (blockIdx.x % per) * kRows2 + (threadIdx.x >> 2), l4 = lane & 3;
    const uint8_t *blob = blob_of_row(a, s);
    if (blob == nullptr) {
        pdl_wait();
        return;
    }
    const uint4 *w = reinterpret_cast<const uint4 *>(blob + a.L.off.q2 + (size_t)n * I) + l4;
    uint4 u[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j)
        u[j] = l4 + 4 * j < nch ? ld_stream_v4(w + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
    const float sw = __ldg(reinterpret_cast<const float *>(blob + a.L.off.s2) + n);
    pdl_wait();
    pdl_launch_dependents();
    const float4 *hr = reinterpret_cast<const float4 *>(h + (size_t)s * I);
    float amax = 0.0f;
    for (int i = threadIdx.x; i < I / 4; i += 32 * kWarps) {
        const float4 v = hr[i];
        amax = max_nan(amax, max_nan(max_nan(fabsf(v.x), fabsf(v.y)), max_nan(fabsf(v.z), fabsf(v.w))));
    }
    amax = warp_max(amax);
    if (lane == 0) s_part[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) amax = max_nan(amax, s_part[i]);
    const CodeScale sc = code_scale(amax);
    for (int i = threadIdx.x; i < I / 4; i += 32 * kWarps) reinterpret_cast<uint32_t *>(s_hq)[i] = sc.code4(hr[i]);
    __syncthreads();
    const uint4 *x = reinterpret_cast<const uint4 *>(s_hq);
    int acc = 0;
    for (int c0 = l4;;) {
#pragma unroll
        for (int j = 0; j < kU; ++j)
            if (c0 + 4 * j < nch) acc = dot16(u[j], x[c0 + 4 * j], acc);
        c0 += 4 * kU;
        w += 4 * kU;
        if (c0 >= nch) break;
#pragma unroll
        for (int j = 0; j < kU; ++j)
            u[j] = c0 + 4 * j < nch ? ld_stream_v4(w + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
    }
    acc += __shfl_xor_sync(kAll, acc, 1);
    acc += __shfl_xor_sync(kAll, acc, 2);
    if (l4 == 0) a.rows[(size_t)s * H + n] = scaled(acc, sc.s, sw);
}

}  // namespace

cudaError_t launch_linear_i8(const LinearArgs &a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    if (a.T > kGemvTokens && (a.T > kGemvTokensSmall || (int64_t)a.T * a.N * a.K > kGemvProducts))
        return launch_linear_i8_tc(a, s);
    const dim3 block(32 * kWarps);
    auto go = [&](auto kern) {
        return launch_pdl(kern, dim3((unsigned)((a.N + kWarps - 1) / kWarps)), block, 0, s, a);
    };
    if (a.T == 1) return a.fp32 ? go(k_linear_i8<1, true>) : go(k_linear_i8<1, false>);
    if (a.T == 2) return a.fp32 ? go(k_linear_i8<2, true>) : go(k_linear_i8<2, false>);
    return a.fp32 ? go(k_linear_i8<4, true>) : go(k_linear_i8<4, false>);
}

// Whether the kernels of this file take the FFN (by sizes alone: the workspace is asked
// for before the routes are known; with more tokens it turns false once).
static bool ffn_i8_gemv(int E, int H, int I, int T, int k) {
    const double R = (double)T * k;
    if (R > kGemvRoutes) return false;
    const double distinct = E * (1.0 - pow(1.0 - (double)std::min(k, E) / E, T));
    return (R - distinct) * 3.0 * H * I <= kGemvAgainBytes;
}

size_t ffn_i8_workspace(int E, int H, int I, int T, int k) {
    return ffn_i8_gemv(E, H, I, T, k) ? (size_t)T * k * I * 4 : ffn_i8_tc_workspace(H, I, T, k);
}

cudaError_t launch_ffn_i8(const FfnI8Args &a, cudaStream_t s) {
    const int64_t R = (int64_t)a.T * a.k;
    if (R == 0) return cudaSuccess;
    if (!ffn_i8_gemv(a.L.E, a.L.H, a.L.I, a.T, a.k)) return launch_ffn_i8_tc(a, s);
    float *h = static_cast<float *>(a.ws);
    const int64_t b1 = R * (a.L.I / kWarps), b2 = R * (a.L.H / kRows2);
    if (b1 > INT32_MAX || b2 > INT32_MAX) return cudaErrorInvalidValue;
    const cudaError_t err = launch_pdl(k_ffn_i8_gemv1, dim3((unsigned)b1), dim3(32 * kWarps), 0, s, a, h);
    if (err != cudaSuccess) return err;
    return launch_pdl(k_ffn_i8_gemv2, dim3((unsigned)b2), dim3(32 * kWarps), (size_t)a.L.I, s, a, (const float *)h);
}

cudaError_t i8_take_error(unsigned *code, unsigned *info) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_i8_error, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(info, g_i8_error_info, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_i8_error, &zero, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_i8_error_info, &zero, sizeof(unsigned));
    return e;
}

}  // namespace moe
