// What sits between the experts' products when they run as operators of their own: SwiGLU with its
// gradient, and the row quantiser of the INT8 products (alone, and of SwiGLU's output).
//   h = g sigma(g) u
//   dg = dh u sigma(g) (1 + g (1 - sigma(g))),  du = dh g sigma(g)
//   scale[r] = max_k |x[r, k]| / 127,  q[r, k] = rint(x[r, k] / scale[r])  (ties to even; 0 where scale is 0)
// bf16, fp16 or fp32 in memory, FP32 arithmetic.  All are bound by HBM: 16-byte loads and stores (32
// bytes of fp32), eight elements per thread and step.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace beam {

// Plain loads: the outputs of a call may be its inputs' buffers.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <>
__device__ __forceinline__ void load8(const __half *p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 b = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// sigma(g): for 16-bit data with the fast exponential and division (a few FP32 ulp, far below the result's
// rounding), for fp32 with the accurate ones.  g -> -inf: exp overflows to +inf and the quotient is 0.
template <typename T>
__device__ __forceinline__ float sigmoid_of(float g) {
    if constexpr (sizeof(T) == 2) return __fdividef(1.0f, 1.0f + __expf(-g));
    else return __fdiv_rn(1.0f, 1.0f + expf(-g));
}

struct SwigluParams {
    const void *dh, *g, *u;  // dh: backward only
    void *h, *dg, *du;       // h: forward; dg, du: backward (may be g and u themselves)
    int64_t ld_dh, ld_g, ld_u, ld_h, ld_dg, ld_du;
    int64_t R;
    int I;
};

// Threads (x, y): eight columns each, rows y, y + gridDim.y blockDim.y, ...
template <typename T, bool BACKWARD>
__global__ void __launch_bounds__(256) swiglu_kernel(const SwigluParams p) {
    const int c = (blockIdx.x * blockDim.x + threadIdx.x) * 8;
    if (c >= p.I) return;
    const T *gp = reinterpret_cast<const T *>(p.g), *up = reinterpret_cast<const T *>(p.u);
    for (int64_t r = static_cast<int64_t>(blockIdx.y) * blockDim.y + threadIdx.y; r < p.R;
         r += static_cast<int64_t>(gridDim.y) * blockDim.y) {
        float g[8], u[8], a[8];
        load8(gp + r * p.ld_g + c, g);
        load8(up + r * p.ld_u + c, u);
        if constexpr (BACKWARD) {
            float d[8], b[8];
            load8(reinterpret_cast<const T *>(p.dh) + r * p.ld_dh + c, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = sigmoid_of<T>(g[i]);
                a[i] = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
                b[i] = d[i] * (g[i] * s);
            }
            store8(reinterpret_cast<T *>(p.dg) + r * p.ld_dg + c, a);
            store8(reinterpret_cast<T *>(p.du) + r * p.ld_du + c, b);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = g[i] * sigmoid_of<T>(g[i]) * u[i];
            store8(reinterpret_cast<T *>(p.h) + r * p.ld_h + c, a);
        }
    }
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct QuantParams {
    const void *x, *u;  // SWIGLU: x is g
    int64_t ld_x, ld_u;
    int8_t *q;          // [R, K]
    float *scale;       // [R]
    int64_t R;
    int K;
};

template <typename T, bool SWIGLU>
__device__ __forceinline__ void quant_values(const QuantParams &p, int64_t r, int c, float (&v)[8]) {
    load8(reinterpret_cast<const T *>(p.x) + r * p.ld_x + c, v);
    if constexpr (SWIGLU) {
        float u[8];
        load8(reinterpret_cast<const T *>(p.u) + r * p.ld_u + c, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * sigmoid_of<T>(v[i]) * u[i];
    }
}
__device__ __forceinline__ void quant_store(int8_t *q, const float (&v)[8], float s) {
    uint32_t w[2] = {0u, 0u};
    if (s > 0.0f && s < INFINITY) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // a scale among the subnormals can round the quotient past 127
            const int c = max(-127, min(127, __float2int_rn(__fdiv_rn(v[i], s))));
            w[i >> 2] |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * (i & 3));
        }
    }
    *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
}

constexpr int kQuantCached = 4;  // steps whose values stay in registers between the two passes

// One row per warp (WARP_ROW: short rows, 8 rows per CTA) or per CTA: the largest magnitude of the row,
// then its codes.  Values past the cached steps (K > 16384) are read again.
template <typename T, bool SWIGLU, bool WARP_ROW>
__global__ void __launch_bounds__(512) quant_i8_kernel(const QuantParams p) {
    __shared__ float part[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = WARP_ROW ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
    if (WARP_ROW && r >= p.R) return;
    const int me = WARP_ROW ? lane : threadIdx.x, all = WARP_ROW ? 32 : blockDim.x;
    float v[kQuantCached][8];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kQuantCached; ++i) {
        const int c = (me + i * all) * 8;
        if (c < p.K) {
            quant_values<T, SWIGLU>(p, r, c, v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[i][j]));
        }
    }
    for (int c = (me + kQuantCached * all) * 8; c < p.K; c += all * 8) {
        float t[8];
        quant_values<T, SWIGLU>(p, r, c, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(t[j]));
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    if constexpr (!WARP_ROW) {
        if (lane == 0) part[warp] = m;
        __syncthreads();
        m = part[0];
        for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) m = max_nan(m, part[w]);
    }
    const float s = __fdiv_rn(m, 127.0f);
    if (me == 0) p.scale[r] = s;
    int8_t *q = p.q + r * static_cast<int64_t>(p.K);
#pragma unroll
    for (int i = 0; i < kQuantCached; ++i) {
        const int c = (me + i * all) * 8;
        if (c < p.K) quant_store(q + c, v[i], s);
    }
    for (int c = (me + kQuantCached * all) * 8; c < p.K; c += all * 8) {
        float t[8];
        quant_values<T, SWIGLU>(p, r, c, t);
        quant_store(q + c, t, s);
    }
}

}  // namespace beam
