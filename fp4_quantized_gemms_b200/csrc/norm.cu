// norm.cu -- root-mean-square norm of a residual stream, forward and backward.
//
// Forward, per row:   h = x + residual (rounded to the stream's type and
// stored), r = 1 / sqrt(mean(h^2) + eps), y = h r w.  y leaves as bf16, or as
// an 8-bit GEMM operand: per 32 elements X = the smallest integer with
// amax <= 448 2^X, elements E4M3(y 2^-X), scale byte X + 127.
// Backward, with g = dy w and xhat = h r:
//     dx = r (g - xhat mean(g xhat)) + dh      (dh: gradient arriving at h itself)
//     dw = sum over rows of dy xhat
// The 8-bit rounding passes its gradient straight through.
//
// One pass: a row is read once, held in registers while its sum is reduced,
// and written once, so HBM is the bound (forward 7 bytes per element for a
// bf16 stream with residual and 8-bit output, backward 8).  Row sums, r and
// the weight gradient are fp32.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ufp4.h"
#include "ufp4_elem.cuh"
#include "ufp4_internal.h"

namespace ufp4 {

namespace {

// Eight consecutive elements starting at p[i]: 16-byte accesses (VEC), or one
// by one, those at or beyond `valid` read as 0 and left alone.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void *p, int64_t i, int valid, float (&v)[8]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < valid ? load_elem(p, i + j, BF16) : 0.0f;
    } else if (valid <= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    } else if constexpr (BF16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_lo(w[j]);
            v[2 * j + 1] = bf16_hi(w[j]);
        }
    } else {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void put8(void *p, int64_t i, int valid, const float (&v)[8]) {
    if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < valid) store_elem(p, i + j, BF16, v[j]);
    } else if (valid > 0) {
        if constexpr (BF16) {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        } else {
            float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
}

__device__ __forceinline__ void load_weight8(const void *w, bool bf16, int64_t i, int valid, bool vec, float (&v)[8]) {
    if (vec) {
        if (bf16)
            load8<true, true>(w, i, valid, v);
        else
            load8<false, true>(w, i, valid, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < valid ? load_elem(w, i + j, bf16) : 0.0f;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the W warps that share a row; every thread gets it.  `slot` holds
// W floats of shared memory that no earlier sum still uses.
template <int W>
__device__ __forceinline__ float row_sum(float v, float *slot) {
    v = warp_sum(v);
    if constexpr (W > 1) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) slot[warp] = v;
        __syncthreads();
        v = slot[lane % W];
        // the W sums, each the same number of times in the 32 lanes
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    }
    return v;
}

// The block exponent of amax (E4M3 maximum 448 = 1.75 * 2^8): the smallest X
// with amax <= 448 2^X, within [-127, 127].  Zero and anything below 448 *
// 2^-127 give -127.
__device__ __forceinline__ int block_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int x = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return x < -127 ? -127 : x;
}

// 2^-X for X in [-127, 120]: a normal fp32 number.
__device__ __forceinline__ float exp2_neg(int x) { return __uint_as_float(static_cast<uint32_t>(127 - x) << 23); }

// E4M3 bytes with every zero +0 (zeros carry no sign in an operand): the sign
// bit is kept only beside a magnitude that is not 0.
__device__ __forceinline__ uint32_t plain_zeros(uint32_t w) {
    const uint32_t mag = w & 0x7F7F7F7Fu;
    return mag | (w & (mag + 0x7F7F7F7Fu) & 0x80808080u);
}

// Rows of W warps, R = kWarps / W rows per block (R > 1 only with W = 1); a
// thread holds NV vectors of eight elements, vector j at element
// 8 (t + 32 W j) of its row.
template <int W>
struct RowShape {
    static constexpr int kRowThreads = 32 * W;
    static constexpr int kRows = W == 1 ? 4 : 1;
    static constexpr int kThreads = kRowThreads * kRows;
};

template <int W, int NV, bool SBF16, bool XBF16, bool RES, bool OUT8, bool VEC>
__global__ void __launch_bounds__(RowShape<W>::kThreads) rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    using S = RowShape<W>;
    __shared__ float s_sum[W];
    const int t = W == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * S::kRows + (W == 1 ? threadIdx.x >> 5 : 0);
    if (W == 1 && row >= a.rows) return;               // whole warps
    float h[NV][8];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t col = 8 * (t + S::kRowThreads * j);
        const int valid = col + 8 <= a.cols ? 8 : static_cast<int>(a.cols - col);
        load8<XBF16, VEC>(a.x, row * a.ld_x + col, valid, h[j]);
        if constexpr (RES) {
            float r[8];
            load8<SBF16, VEC>(a.residual, row * a.ld_res + col, valid, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[j][e] += r[e];
                if constexpr (SBF16) h[j][e] = __bfloat162float(__float2bfloat16_rn(h[j][e]));
            }
            put8<SBF16, VEC>(a.h, row * a.ld_h + col, valid, h[j]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(h[j][e], h[j][e], sum);
    }
    sum = row_sum<W>(sum, s_sum);
    const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.cols) + a.eps);
    if (t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t col = 8 * (t + S::kRowThreads * j);
        const int valid = col + 8 <= a.cols ? 8 : static_cast<int>(a.cols - col);
        float w[8];
        load_weight8(a.weight, a.weight_bf16, col, valid, a.vec_weight, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] = h[j][e] * rstd * w[e];
        if constexpr (!OUT8) {
            put8<true, VEC>(a.y, row * a.ld_y + col, valid, h[j]);
        } else {
            // blocks of 32 elements: four neighbouring lanes (all lanes of the
            // warp take part; elements beyond the row are 0)
            float amax = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(h[j][e]));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            const int x = block_exponent(amax);
            const float inv = exp2_neg(x);
            if (col < a.kpad) {
                uint32_t p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p[e] = __nv_cvt_float2_to_fp8x2(make_float2(h[j][2 * e] * inv, h[j][2 * e + 1] * inv),
                                                    __NV_SATFINITE, __NV_E4M3);
                *reinterpret_cast<uint2 *>(a.elems8 + row * a.kpad + col) =
                    make_uint2(plain_zeros(p[0] | (p[1] << 16)), plain_zeros(p[2] | (p[3] << 16)));
                if ((t & 3) == 0) {
                    const int64_t b = col / 32;
                    const uint8_t byte = static_cast<uint8_t>(x + 127);
                    a.scales[b * a.scale_ld + row] = byte;
                    if (a.sf_atoms != nullptr)
                        a.sf_atoms[((row / 128) * a.atoms_k + b / 4) * 512 + 16 * (row % 32) + 4 * ((row / 32) % 4) +
                                   b % 4] = byte;
                }
            }
        }
    }
}

// Backward: a block takes rows blockIdx.x * R + its row slot, + gridDim.x * R,
// ..., and keeps the weight gradient of its columns in registers; the slots'
// sums go to one partial row per block and slot.
template <int W, int NV, bool SBF16, bool DYBF16, bool DXBF16, bool VEC>
__global__ void __launch_bounds__(RowShape<W>::kThreads) rmsnorm_backward_kernel(const __grid_constant__ NormBwdArgs a) {
    using S = RowShape<W>;
    __shared__ float s_sum[2][W];
    const int t = W == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * S::kRows + (W == 1 ? threadIdx.x >> 5 : 0);
    const int64_t nslots = static_cast<int64_t>(gridDim.x) * S::kRows;
    float dw[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    int phase = 0;
    for (int64_t row = slot; row < a.rows; row += nslots, phase ^= 1) {
        const float r = a.rstd[row];
        float xh[NV][8], g[NV][8];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = 8 * (t + S::kRowThreads * j);
            const int valid = col + 8 <= a.cols ? 8 : static_cast<int>(a.cols - col);
            float w[8];
            load8<SBF16, VEC>(a.h, row * a.ld_h + col, valid, xh[j]);
            load8<DYBF16, VEC>(a.dy, row * a.ld_dy + col, valid, g[j]);
            load_weight8(a.weight, a.weight_bf16, col, valid, a.vec_weight, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[j][e] *= r;
                dw[j][e] = fmaf(g[j][e], xh[j][e], dw[j][e]);
                g[j][e] *= w[e];
                dot = fmaf(g[j][e], xh[j][e], dot);
            }
        }
        // two slots in turn: a warp may still read the last row's sums
        dot = row_sum<W>(dot, s_sum[phase]) * inv_cols;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = 8 * (t + S::kRowThreads * j);
            const int valid = col + 8 <= a.cols ? 8 : static_cast<int>(a.cols - col);
            float d[8];
            if (a.dh != nullptr) {
                load8<SBF16, VEC>(a.dh, row * a.ld_dh + col, valid, d);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = fmaf(r, g[j][e] - xh[j][e] * dot, d[e]);
            put8<DXBF16, VEC>(a.dx, row * a.ld_dx + col, valid, d);
        }
    }
    if (a.dweight != nullptr) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = 8 * (t + S::kRowThreads * j);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + e < a.cols) a.partial[slot * a.cols + col + e] = dw[j][e];
        }
    }
}

template <int W, int NV, bool SBF16, bool XBF16, bool RES, bool OUT8>
cudaError_t launch_fwd_vec(const NormArgs &a, cudaStream_t stream) {
    using S = RowShape<W>;
    const unsigned grid = static_cast<unsigned>((a.rows + S::kRows - 1) / S::kRows);
    if (a.vec)
        rmsnorm_kernel<W, NV, SBF16, XBF16, RES, OUT8, true><<<grid, S::kThreads, 0, stream>>>(a);
    else
        rmsnorm_kernel<W, NV, SBF16, XBF16, RES, OUT8, false><<<grid, S::kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int W, int NV>
cudaError_t launch_fwd_shape(const NormArgs &a, cudaStream_t stream) {
    const bool out8 = a.elems8 != nullptr;
    if (a.residual == nullptr) {     // the stream is x itself
        if (a.x_bf16)
            return out8 ? launch_fwd_vec<W, NV, true, true, false, true>(a, stream)
                        : launch_fwd_vec<W, NV, true, true, false, false>(a, stream);
        return out8 ? launch_fwd_vec<W, NV, false, false, false, true>(a, stream)
                    : launch_fwd_vec<W, NV, false, false, false, false>(a, stream);
    }
    switch ((a.stream_bf16 ? 4 : 0) | (a.x_bf16 ? 2 : 0) | (out8 ? 1 : 0)) {
        case 0: return launch_fwd_vec<W, NV, false, false, true, false>(a, stream);
        case 1: return launch_fwd_vec<W, NV, false, false, true, true>(a, stream);
        case 2: return launch_fwd_vec<W, NV, false, true, true, false>(a, stream);
        case 3: return launch_fwd_vec<W, NV, false, true, true, true>(a, stream);
        case 4: return launch_fwd_vec<W, NV, true, false, true, false>(a, stream);
        case 5: return launch_fwd_vec<W, NV, true, false, true, true>(a, stream);
        case 6: return launch_fwd_vec<W, NV, true, true, true, false>(a, stream);
        default: return launch_fwd_vec<W, NV, true, true, true, true>(a, stream);
    }
}

template <int W, int NV, bool SBF16, bool DYBF16, bool DXBF16>
cudaError_t launch_bwd_vec(const NormBwdArgs &a, int64_t blocks, cudaStream_t stream) {
    using S = RowShape<W>;
    const unsigned grid = static_cast<unsigned>(blocks);
    if (a.vec)
        rmsnorm_backward_kernel<W, NV, SBF16, DYBF16, DXBF16, true><<<grid, S::kThreads, 0, stream>>>(a);
    else
        rmsnorm_backward_kernel<W, NV, SBF16, DYBF16, DXBF16, false><<<grid, S::kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int W, int NV>
cudaError_t launch_bwd_shape(const NormBwdArgs &a, int64_t blocks, cudaStream_t stream) {
    switch ((a.stream_bf16 ? 4 : 0) | (a.dy_bf16 ? 2 : 0) | (a.dx_bf16 ? 1 : 0)) {
        case 0: return launch_bwd_vec<W, NV, false, false, false>(a, blocks, stream);
        case 1: return launch_bwd_vec<W, NV, false, false, true>(a, blocks, stream);
        case 2: return launch_bwd_vec<W, NV, false, true, false>(a, blocks, stream);
        case 3: return launch_bwd_vec<W, NV, false, true, true>(a, blocks, stream);
        case 4: return launch_bwd_vec<W, NV, true, false, false>(a, blocks, stream);
        case 5: return launch_bwd_vec<W, NV, true, false, true>(a, blocks, stream);
        case 6: return launch_bwd_vec<W, NV, true, true, false>(a, blocks, stream);
        default: return launch_bwd_vec<W, NV, true, true, true>(a, blocks, stream);
    }
}

// Rows per block and blocks of the backward pass (a function of the shape
// alone): enough blocks for every SM to hold two to four.
int64_t bwd_blocks(int64_t rows, int64_t cols) {
    const int64_t per = cols <= 1024 ? 4 : 1;
    const int64_t need = (rows + per - 1) / per;
    const int64_t most = int64_t(148) * (cols <= 4096 ? 4 : cols <= 8192 ? 2 : 1);
    return need < most ? need : most;
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs &a, cudaStream_t stream) {
    const int64_t width = a.elems8 != nullptr ? a.kpad : a.cols;
    if (width <= 256) return launch_fwd_shape<1, 1>(a, stream);
    if (width <= 1024) return launch_fwd_shape<1, 4>(a, stream);
    if (width <= 4096) return launch_fwd_shape<4, 4>(a, stream);
    if (width <= 8192) return launch_fwd_shape<8, 4>(a, stream);
    if (width <= 16384) return launch_fwd_shape<16, 4>(a, stream);
    return launch_fwd_shape<32, 4>(a, stream);
}

int64_t rmsnorm_backward_slots(int64_t rows, int64_t cols) {
    return rows <= 0 ? 0 : bwd_blocks(rows, cols) * (cols <= 1024 ? 4 : 1);
}

cudaError_t launch_rmsnorm_backward(const NormBwdArgs &a, cudaStream_t stream) {
    const int64_t blocks = bwd_blocks(a.rows, a.cols);
    cudaError_t e;
    if (a.cols <= 256)
        e = launch_bwd_shape<1, 1>(a, blocks, stream);
    else if (a.cols <= 1024)
        e = launch_bwd_shape<1, 4>(a, blocks, stream);
    else if (a.cols <= 4096)
        e = launch_bwd_shape<4, 4>(a, blocks, stream);
    else if (a.cols <= 8192)
        e = launch_bwd_shape<8, 4>(a, blocks, stream);
    else if (a.cols <= 16384)
        e = launch_bwd_shape<16, 4>(a, blocks, stream);
    else
        e = launch_bwd_shape<32, 4>(a, blocks, stream);
    if (e != cudaSuccess || a.dweight == nullptr) return e;
    return launch_column_sums(a.partial, rmsnorm_backward_slots(a.rows, a.cols), a.cols, a.dweight, stream);
}

}  // namespace ufp4
