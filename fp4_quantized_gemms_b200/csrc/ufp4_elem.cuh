// ufp4_elem.cuh -- element access and the activations of the operators that
// work on plain bf16 / fp32 tensors (GEMM epilogue, norms, router, clipping).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ufp4_internal.h"

namespace ufp4 {

// Two kernels of one call: the second is launched while the first still runs
// (launch_early) and waits for its results before it reads them; the first
// says as early as it likes that its blocks are all placed.
__device__ __forceinline__ void let_next_kernel_launch() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t stream, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 values to bf16, each rounded to nearest even; `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float load_elem(const void *p, int64_t i, bool bf16) {
    return bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16)
                : static_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_elem(void *p, int64_t i, bool bf16, float v) {
    if (bf16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(p)[i] = v;
}

// Four consecutive elements from index i: one 8- or 16-byte access when `vec`
// (the address allows it), else element by element; elements at or beyond
// `valid` are not touched (read as 0).
__device__ __forceinline__ float4 load_quad(const void *p, int64_t i, bool bf16, bool vec, int valid) {
    if (vec && valid >= 4) {
        if (bf16) {
            const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
            return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
        }
        return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    }
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < valid ? load_elem(p, i + e, bf16) : 0.0f;
    return make_float4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ void store_quad(void *p, int64_t i, bool bf16, bool vec, int valid, float4 v) {
    if (vec && valid >= 4) {
        if (bf16)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) =
                make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = v;
        return;
    }
    const float e4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < valid) store_elem(p, i + e, bf16, e4[e]);
}

// ---------------------------------------------------------------------------
// Eight consecutive elements at any element alignment (odd widths and pitches,
// views that start anywhere), as fast as the alignment allows: whole 16-byte
// granules are moved, and a funnel shift lines them up.

// Moves words [shift, ..) of w to its front; shift in 0 .. 3, the same for the
// warp's lanes.
template <int N>
__device__ __forceinline__ void drop_words(uint32_t (&w)[N], int shift) {
    if (shift & 2) {
#pragma unroll
        for (int k = 0; k + 2 < N; ++k) w[k] = w[k + 2];
    }
    if (shift & 1) {
#pragma unroll
        for (int k = 0; k + 1 < N; ++k) w[k] = w[k + 1];
    }
}

// Elements p[i .. i + 7] (global or shared memory) as stored, those at or
// beyond `valid` as 0.  A granule is read only when it holds a valid element
// (so never outside that element's page); what else it holds is not used.
template <bool BF16>
__device__ __forceinline__ void load8_raw(const void *p, int64_t i, int valid, uint32_t (&o)[BF16 ? 4 : 8]) {
    constexpr int kSize = BF16 ? 2 : 4, kGranules = BF16 ? 2 : 3;
    const uintptr_t addr = reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(i * kSize);
    const int s = static_cast<int>(addr & 15u);
    const uint4 *g = reinterpret_cast<const uint4 *>(addr - static_cast<uintptr_t>(s));
    const int bytes = (valid < 8 ? valid : 8) * kSize + s;
    uint32_t w[4 * kGranules];
#pragma unroll
    for (int k = 0; k < kGranules; ++k) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (valid > 0 && 16 * k < bytes) q = g[k];
        w[4 * k] = q.x, w[4 * k + 1] = q.y, w[4 * k + 2] = q.z, w[4 * k + 3] = q.w;
    }
    drop_words(w, s >> 2);
    if constexpr (BF16) {
        const int bits = (s & 2) * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __funnelshift_r(w[k], w[k + 1], bits);
        if (valid < 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = 2 * k >= valid ? 0u : 2 * k + 1 >= valid ? o[k] & 0xFFFFu : o[k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = k < valid ? w[k] : 0u;
    }
}

template <bool BF16>
__device__ __forceinline__ void load8_any(const void *p, int64_t i, int valid, float (&v)[8]) {
    uint32_t o[BF16 ? 4 : 8];
    load8_raw<BF16>(p, i, valid, o);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = BF16 ? ((k & 1) ? bf16_hi(o[k / 2]) : bf16_lo(o[k / 2])) : __uint_as_float(o[BF16 ? 0 : k]);
}

// Stores eight elements per lane, lane l's right behind lane l - 1's (p[i]
// differs by 8 from lane to lane); `rest`: elements of the row from this
// lane's first on (any number; none are stored beyond it).  All 32 lanes take
// part.  A granule that two lanes share is written by the second, from the
// first one's last words; what the warp does not fill whole is written
// element by element.
template <bool BF16>
__device__ __forceinline__ void store8_any(void *p, int64_t i, int rest, const float (&v)[8]) {
    constexpr int kSize = BF16 ? 2 : 4, kWords = BF16 ? 4 : 8;
    const uintptr_t addr = reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(i * kSize);
    const int s = static_cast<int>(addr & 15u);           // the same in all lanes
    const int lane = threadIdx.x & 31;
    if (rest + 8 * lane <= 0) return;                      // nothing for the whole warp
    uint32_t w[4 + kWords];                                // the last 16 bytes of the lane before, then this one's
#pragma unroll
    for (int k = 0; k < kWords; ++k)
        w[4 + k] = BF16 ? pack_bf16(v[(2 * k) % 8], v[(2 * k + 1) % 8]) : __float_as_uint(v[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __shfl_up_sync(0xFFFFFFFFu, w[kWords + k], 1);
    // bytes [16 - s, ..) of the 16 + 4 kWords: the granules from addr - s on
    const int head = s == 0 ? 0 : (16 - s) / kSize;        // this lane's elements in the shared granule
    const int have = rest < 8 ? rest : 8;
    const bool shared = s != 0 && lane > 0 && rest >= head;
    const bool next = s != 0 && lane < 31 && rest - 8 >= head;   // the next lane writes this one's end
    uint32_t o[4 + kWords];
#pragma unroll
    for (int k = 0; k < 4 + kWords; ++k) o[k] = w[k];
    drop_words(o, s == 0 ? 0 : (16 - s) >> 2);
    if constexpr (BF16) {
        const int bits = (s & 2) * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __funnelshift_r(o[k], o[k + 1], bits);
    }
    uint4 *g = reinterpret_cast<uint4 *>(addr - static_cast<uintptr_t>(s));
    int done_to = 0, done_from = 0;                        // elements [done_from, done_to) are in granules
    if (s == 0) {
        constexpr int kOwn = BF16 ? 1 : 2;
#pragma unroll
        for (int q = 0; q < kOwn; ++q) {
            if (have >= (q + 1) * 16 / kSize) {
                g[q] = make_uint4(w[4 + 4 * q], w[5 + 4 * q], w[6 + 4 * q], w[7 + 4 * q]);
                done_to = (q + 1) * 16 / kSize;
            }
        }
    } else {
        done_from = head;
        if (shared) {
            g[0] = make_uint4(o[0], o[1], o[2], o[3]);
            done_from = 0;
        }
        done_to = head;
        if constexpr (!BF16) {                             // one granule is the lane's own
            if (have >= head + 4) {
                g[1] = make_uint4(o[4], o[5], o[6], o[7]);
                done_to = head + 4;
            }
        }
        if (next) done_to = 8;
    }
    if (done_from > 0 || done_to < have) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < have && (k < done_from || k >= done_to)) store_elem(p, i + k, BF16, v[k]);
    }
}

// Eight elements of a row as loaded, bf16 or fp32 (load: 16-byte aligned, read
// once, evict first).
template <bool BF16>
struct Raw8 {
    uint4 w[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const uint4 *q = BF16 ? reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i)
                              : reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
        w[0] = __ldcs(q);
        if constexpr (!BF16) w[1] = __ldcs(q + 1);
    }
    // any alignment; elements at or beyond `valid` as 0
    __device__ __forceinline__ void load_any(const void *p, int64_t i, int valid) {
        uint32_t o[BF16 ? 4 : 8];
        load8_raw<BF16>(p, i, valid, o);
        w[0] = make_uint4(o[0], o[1], o[2], o[3]);
        if constexpr (!BF16) w[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    __device__ __forceinline__ void zero() {
        w[0] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (!BF16) w[1] = w[0];
    }
    __device__ __forceinline__ void get2(float2 (&v)[4]) const {
        float f[8];
        get(f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = make_float2(f[2 * j], f[2 * j + 1]);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (BF16) {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = bf16_lo(u[j]);
                v[2 * j + 1] = bf16_hi(u[j]);
            }
        } else {
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(u[j]);
        }
    }
};

// ---------------------------------------------------------------------------
// Activations (ufp4_act_t) on the hardware's ex2 and reciprocal (ex2.approx and
// rcp.approx: 2^-22 and 1 ulp): every value below is within a few 1e-7 of
// max(|z|, 1).  Where values get small, far left, they keep a relative accuracy
// of (5 |x| ln 2 + 24) 2^-24, x the binary logarithm of the exponential (the
// argument's roundings), 3e-5 at worst; below 2^-126 the exponential's side is
// flushed to 0.

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// z within [-m, m]; NaN stays NaN.
__device__ __forceinline__ float clamp_nan(float z, float m) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(z), "f"(-m));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(y), "f"(m));
    return y;
}

// GELU in its tanh form, z (1 + tanh u) / 2 = z / (1 + exp(-2u)),
// u = sqrt(2 / pi) (z + 0.044715 z^3); exp(-2u) = 2^(-z (A + B z^2)).
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu2A = 2.0f * 0.79788456080286536f;          // 2 sqrt(2 / pi)
constexpr float kGelu2B = kGelu2A * 0.044715f;

// The normal distribution's tail beyond a >= 0 as a product e r, so with its
// relative accuracy wherever it is a normal number: e = exp(-a^2 / 2) and
// r = erfcx(a / sqrt 2) / 2 = t P(t), t = 1 / (1 + 0.3 a).  P is a polynomial of
// degree 7 fitted to equal relative error over a in [0, 14] (Lawson's iterated
// least squares): 1.7e-7, 4.5e-7 in fp32 arithmetic.
struct NormalTail {
    float e, r;
};
__device__ __forceinline__ NormalTail normal_tail(float a) {
    const float t = rcp_approx(fmaf(0.3f, a, 1.0f));
    float p = fmaf(0.03567476198077202f, t, -0.15720301866531372f);
    p = fmaf(p, t, 0.20635341107845306f);
    p = fmaf(p, t, -0.05368354544043541f);
    p = fmaf(p, t, 0.1285615712404251f);
    p = fmaf(p, t, 0.09991350769996643f);
    p = fmaf(p, t, 0.1207539513707161f);
    p = fmaf(p, t, 0.11962930113077164f);
    return {ex2_approx(-0.5f * kLog2e * a * a), p * t};
}

__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case UFP4_ACT_RELU: return z < 0.0f ? 0.0f : z;          // NaN stays NaN
        case UFP4_ACT_GELU: {
            const float p = fmaf(-kGelu2B * kLog2e, z * z, -kGelu2A * kLog2e);
            return z * rcp_approx(1.0f + ex2_approx(z * p));
        }
        case UFP4_ACT_GELU_ERF: {
            const NormalTail n = normal_tail(fabsf(z));
            return z * (z < 0.0f ? n.e * n.r : fmaf(-n.e, n.r, 1.0f));
        }
        case UFP4_ACT_SILU: return z * rcp_approx(1.0f + ex2_approx(-kLog2e * z));
        default: return z;
    }
}

__device__ __forceinline__ float4 act_quad(float4 z, int act) {
    if (act == UFP4_ACT_NONE) return z;
    return make_float4(act_value(z.x, act), act_value(z.y, act), act_value(z.z, act), act_value(z.w, act));
}

// Two lanes of one packed fp32x2 operation each (the same IEEE results).
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// Derivative of the activation, two at a time.  With t = exp(-2u) (GELU) or exp(-z) (SiLU)
// and s = 1 / (1 + t): d = s + z u2' (t s) s, where t s = 1 - s without
// cancellation and u2' = d(2u)/dz.  (t s first: it is at most 1 and s a normal
// number, while s^2 would underflow left of z = -43.)  The clamp, |z| = 9.9
// (GELU) or 87 (SiLU), keeps t finite and s normal; beyond it the derivative is
// within 3e-35 of 0 or 1.  GELU_ERF: the tail beyond |z| less |z| times the
// density there (no cancellation but at its zero, |z| = 0.75), or 1 less that;
// within 2e-36 beyond |z| = 13.
template <int ACT>
__device__ __forceinline__ float2 act_slope2(float2 z) {
    if constexpr (ACT == UFP4_ACT_RELU) {
        return make_float2(z.x > 0.0f ? 1.0f : 0.0f, z.y > 0.0f ? 1.0f : 0.0f);
    } else if constexpr (ACT == UFP4_ACT_GELU || ACT == UFP4_ACT_SILU) {
        constexpr bool kGelu = ACT == UFP4_ACT_GELU;
        const float lim = kGelu ? 9.9f : 87.0f;
        const float2 c = make_float2(clamp_nan(z.x, lim), clamp_nan(z.y, lim));
        float2 arg, du = c;                              // log2 t; z d(2u)/dz
        if constexpr (kGelu) {
            const float2 c2 = mul2(c, c);
            arg = mul2(c, fma2(splat(-kGelu2B * kLog2e), c2, splat(-kGelu2A * kLog2e)));
            du = mul2(c, fma2(splat(3.0f * kGelu2B), c2, splat(kGelu2A)));
        } else {
            arg = mul2(splat(-kLog2e), c);
        }
        const float2 t = make_float2(ex2_approx(arg.x), ex2_approx(arg.y));
        const float2 d = add2(splat(1.0f), t);
        const float2 s = make_float2(rcp_approx(d.x), rcp_approx(d.y));
        return fma2(du, mul2(mul2(t, s), s), s);
    } else if constexpr (ACT == UFP4_ACT_GELU_ERF) {
        auto one = [](float v) {
            const float c = clamp_nan(v, 13.0f), a = fabsf(c);
            const NormalTail n = normal_tail(a);
            const float d = fmaf(-0.39894228040143268f, a, n.r);      // tail and density over e
            return c < 0.0f ? n.e * d : fmaf(-n.e, d, 1.0f);
        };
        return make_float2(one(z.x), one(z.y));
    } else {
        return splat(1.0f);
    }
}

// ---------------------------------------------------------------------------
// The GEMM epilogue: z = product + bias; pre = z; out = act(z) + residual,
// all in fp32, each stored value rounded once.

__device__ __forceinline__ float4 add_quad(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Finishes columns col .. col + valid - 1 (valid <= 4) of a row: z without
// its bias, the bias and the residual already loaded.
__device__ __forceinline__ void epilogue_quad(const EpiArgs &e, int64_t row, int64_t col, int valid, float4 z,
                                              float4 bias, float4 res) {
    z = add_quad(z, bias);
    if (e.pre != nullptr) store_quad(e.pre, row * e.ld_pre + col, e.pre_bf16, e.vec_pre, valid, z);
    const float4 v = add_quad(act_quad(z, e.act), res);
    store_quad(e.out, row * e.ld_out + col, e.out_bf16, e.vec_out, valid, v);
}

__device__ __forceinline__ float4 epilogue_bias(const EpiArgs &e, int64_t col, int valid) {
    if (e.bias == nullptr || valid <= 0) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    return load_quad(e.bias, col, e.bias_bf16, e.vec_bias, valid);
}

__device__ __forceinline__ float4 epilogue_residual(const EpiArgs &e, int64_t row, int64_t col, int valid) {
    if (e.residual == nullptr || valid <= 0) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    return load_quad(e.residual, row * e.ld_res + col, e.res_bf16, e.vec_res, valid);
}

}  // namespace ufp4
