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
#include "launch.cuh"

namespace beam {

// Eight elements as loaded, and as FP32.  Plain loads: the outputs of a call may be its inputs' buffers.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T *p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}
__device__ __forceinline__ void unpack(const Raw8<float> &r, float (&v)[8]) {
    const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void unpack(const Raw8<__nv_bfloat16> &r, float (&v)[8]) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const Raw8<__half> &r, float (&v)[8]) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    unpack(load_raw(p), v);
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

// 2^x to within a few 2^-23 (the hardware's approximation; overflows to +inf, underflows to 0).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// sigma(g) = 1 / (1 + e^-g).  16-bit data: the fast exponential and quotient, whose error (|g| 2^-24 from the
// rounded product with log2 e) is far below the result's rounding.  fp32 data: that product's rounding error is
// kept and applied to first order, e^x = 2^p (1 + r ln 2) with p + r = x log2 e, which leaves a few 2^-23; the
// argument is clamped so that r stays small and e^x finite (an infinite one plus a negative correction would be NaN).
// Both give 0 for a sigma below 2^-126, g < -87.34: the quotient is 0 for a divisor above 2^126, which e^88 is.
template <typename T>
__device__ __forceinline__ float sigmoid_of(float g) {
    if constexpr (sizeof(T) == 2) {
        return __fdividef(1.0f, 1.0f + __expf(-g));
    } else {
        constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147181f;
        const float x = g != g ? g : fminf(fmaxf(-g, -126.0f), 88.0f);
        const float p = x * kLog2e;
        const float r = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -p));
        const float e = exp2_fast(p);
        return __fdividef(1.0f, 1.0f + fmaf(e, r * kLn2, e));
    }
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
    let_next_launch();
    wait_for_stream();
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

// Largest magnitude of eight values as an unsigned pattern: magnitudes compare like their bits, with infinity above
// every number and NaN above infinity.  16-bit data stay packed, two to an instruction; `magnitude` turns the
// pattern (for packed ones, of the two halves) into a float.
template <typename T>
__device__ __forceinline__ uint32_t most_bits(uint32_t m, const Raw8<T> &r) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
        const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m = sizeof(T) == 4 ? max(m, w[j] & 0x7FFFFFFFu) : __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    }
    return m;
}
template <typename T>
__device__ __forceinline__ float magnitude(uint32_t m) {
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(m);
    } else {
        Raw8<T> r{};
        r.w[0].x = max(m & 0xFFFFu, m >> 16);
        float v[8];
        unpack(r, v);
        return v[0];
    }
}
__device__ __forceinline__ uint32_t most_of(uint32_t m, const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    return m;
}

struct QuantParams {
    const void *x, *u;  // SWIGLU: x is g
    int64_t ld_x, ld_u;
    int8_t *q;          // [R, K]
    float *scale;       // [R]
    int64_t R;
    int K;
};

// Eight values of a row as loaded (SWIGLU: of both operands), and what is quantised of them.
template <typename T, bool SWIGLU>
struct QuantRaw {
    Raw8<T> x[SWIGLU ? 2 : 1];
    __device__ __forceinline__ void load(const QuantParams &p, int64_t r, int c) {
        x[0] = load_raw(reinterpret_cast<const T *>(p.x) + r * p.ld_x + c);
        if constexpr (SWIGLU) x[1] = load_raw(reinterpret_cast<const T *>(p.u) + r * p.ld_u + c);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        unpack(x[0], v);
        if constexpr (SWIGLU) {
            float u[8];
            unpack(x[1], u);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * sigmoid_of<T>(v[i]) * u[i];
        }
    }
};
// Codes of eight values: the integers nearest to the FP32 quotients v / s, with inv = 1 / s to nearest.  The
// quotient comes from v * inv by two of Markstein's corrections (P. W. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990): the first leaves it within a unit of its last
// place, and from there the second gives the quotient to nearest, as long as the residuals v - q s are exact,
// which they are for s >= 2^-100.  No element needs a branch (a bf16 row often holds half of its own largest
// magnitude, whose quotient 63.5 is a tie, so a test for nearby halves sent a quarter of all warps through the
// divisions).  Adding 1.5 x 2^23 rounds to an integer, ties to even, and leaves its two's complement in the low bits.
__device__ __forceinline__ void quant_store(int8_t *q, const float (&v)[8], float s, float inv) {
    uint32_t w[2] = {0u, 0u};
    if (s > 0.0f && s < INFINITY) {
        constexpr float kMagic = 12582912.0f;
        float y[8];
        if (s >= 0x1p-100f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float t = v[i] * inv;
                t = fmaf(fmaf(-t, s, v[i]), inv, t);
                t = fmaf(fmaf(-t, s, v[i]), inv, t);
                y[i] = t + kMagic;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)  // a subnormal s can round the quotient past 127
                y[i] = fminf(fmaxf(__fdiv_rn(v[i], s), -127.0f), 127.0f) + kMagic;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __byte_perm(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]), 0x0040);
            const uint32_t hi = __byte_perm(__float_as_uint(y[4 * i + 2]), __float_as_uint(y[4 * i + 3]), 0x0040);
            w[i] = __byte_perm(lo, hi, 0x5410);
        }
    }
    *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
}

// Steps of eight elements that a thread keeps in registers between the two passes (x as loaded, or SwiGLU's
// FP32 values).
constexpr int kQuantCached = 4;

// One row per warp (WARP_ROW: short rows, 8 rows per CTA) or per CTA: the largest magnitude of the row, then its
// codes.  All of a thread's loads are issued before the first is used, and CTAs are kept small, so that enough
// rows are in flight per SM.  8192 x 5120 bf16: 30 us (4.2 TB/s; 32768 rows 5.0); 38 to 45 us with 96 threads of
// seven steps, 44 with 320 of two, 71 with a warp of twenty, 54 with CTAs that walk over the rows.
// Values past the cached steps are read again.
template <typename T, bool SWIGLU, bool WARP_ROW>
__global__ void __launch_bounds__(512) quant_i8_kernel(const QuantParams p) {
    let_next_launch();
    wait_for_stream();
    constexpr int kSteps = kQuantCached;
    __shared__ uint32_t part[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = WARP_ROW ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
    if (WARP_ROW && r >= p.R) return;
    const int me = WARP_ROW ? lane : threadIdx.x, all = WARP_ROW ? 32 : blockDim.x;
    QuantRaw<T, SWIGLU> raw[kSteps];
    float h[SWIGLU ? kSteps : 1][8];
    uint32_t m = 0u;  // pattern of the largest magnitude: of T as loaded, or of SwiGLU's FP32 values
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        if ((me + i * all) * 8 < p.K) raw[i].load(p, r, (me + i * all) * 8);
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        if ((me + i * all) * 8 < p.K) {
            if constexpr (SWIGLU) {
                raw[i].values(h[i]);
                m = most_of(m, h[i]);
            } else {
                m = most_bits(m, raw[i].x[0]);
            }
        }
    for (int c = (me + kSteps * all) * 8; c < p.K; c += all * 8) {
        QuantRaw<T, SWIGLU> more;
        more.load(p, r, c);
        if constexpr (SWIGLU) {
            float t[8];
            more.values(t);
            m = most_of(m, t);
        } else {
            m = most_bits(m, more.x[0]);
        }
    }
    m = __float_as_uint(SWIGLU ? __uint_as_float(m) : magnitude<T>(m));  // of FP32
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (!WARP_ROW) {
        if (lane == 0) part[warp] = m;
        __syncthreads();
        m = part[0];
        for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w) m = max(m, part[w]);
    }
    const float s = __fdiv_rn(__uint_as_float(m), 127.0f), inv = __fdiv_rn(1.0f, s);
    if (me == 0) p.scale[r] = s;
    int8_t *q = p.q + r * static_cast<int64_t>(p.K);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int c = (me + i * all) * 8;
        if (c < p.K) {
            if constexpr (SWIGLU) {
                quant_store(q + c, h[i], s, inv);
            } else {
                float t[8];
                raw[i].values(t);
                quant_store(q + c, t, s, inv);
            }
        }
    }
    for (int c = (me + kSteps * all) * 8; c < p.K; c += all * 8) {
        QuantRaw<T, SWIGLU> more;
        float t[8];
        more.load(p, r, c);
        more.values(t);
        quant_store(q + c, t, s, inv);
    }
}

}  // namespace beam
