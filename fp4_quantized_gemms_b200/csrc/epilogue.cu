// epilogue.cu -- the GEMM epilogue's companions: its backward pass, the
// epilogue of a product without a reduction dimension, and column sums.
//
// Forward (in the GEMM kernels): z = (1/n) A B^T + bias, out = act(z) +
// residual.  Backward, with dout = dL/dout and z as the forward stored it:
//     dL/dz        = dout * act'(z)       (dpre; feeds the quantizer of DGRAD and WGRAD)
//     dL/dbias     = sum over rows of dL/dz
//     dL/dresidual = dout                 (nothing to compute)
//
// epilogue_backward_kernel reads dout and z once and writes dpre once; HBM is
// its bound (6 bytes per element in bf16, about 15 flops).  A block covers 256
// columns x a chunk of rows: a lane owns eight columns (one 16-byte bf16
// access), the eight warps take rows in turn and keep the column sums in fp32
// registers, so the bias gradient costs no second pass over dpre.  The sums
// of a chunk go to a partial row, and column_sums_kernel adds the partial
// rows: no atomics, the same bits every time.
#include <cuda_runtime.h>
#include <stdint.h>

#include "ufp4.h"
#include "ufp4_elem.cuh"
#include "ufp4_internal.h"

namespace ufp4 {

namespace {

constexpr int kBwdThreads = 256;
constexpr int kBwdWarps = kBwdThreads / 32;
constexpr int kBwdCols = 256;      // columns of a block
// Rows of a warp in flight: 128 to 192 bytes per lane, within the registers of
// three blocks per SM.
template <bool DOUT_BF16, bool PRE_BF16>
constexpr int kBwdUnroll = DOUT_BF16 && PRE_BF16 ? 4 : DOUT_BF16 || PRE_BF16 ? 3 : 2;

template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t i, const float2 (&v)[4]) {
    if constexpr (BF16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
            make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y),
                       pack_bf16(v[3].x, v[3].y));
    } else {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    }
}

// Sums of a warp row of columns over the block's warps, written to the
// chunk's partial row.
__device__ __forceinline__ void store_partial(const EpiBwdArgs &a, const float (&sum)[8], int64_t col0) {
    __shared__ float s_sum[kBwdWarps][kBwdCols];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < 8; ++j) s_sum[warp][8 * lane + j] = sum[j];
    __syncthreads();
    const int64_t col = col0 + threadIdx.x;
    if (col < a.n) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kBwdWarps; ++w) t += s_sum[w][threadIdx.x];
        a.partial[blockIdx.y * a.n + col] = t;
    }
}

template <int ACT, bool DOUT_BF16, bool PRE_BF16, bool DPRE_BF16>
__global__ void __launch_bounds__(kBwdThreads, 3) epilogue_backward_kernel(const __grid_constant__ EpiBwdArgs a) {
    let_next_kernel_launch();
    constexpr int U = kBwdUnroll<DOUT_BF16, PRE_BF16>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * kBwdCols;
    const int64_t col = col0 + 8 * lane;
    const bool col_ok = col < a.n;                     // n % 8 == 0: all eight or none
    const int64_t r_first = blockIdx.y * a.rows_per_chunk + warp;
    const int64_t r_end = min(a.m, (blockIdx.y + 1) * a.rows_per_chunk);
    float2 sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = splat(0.0f);
    if (col_ok) {
        for (int64_t r0 = r_first; r0 < r_end; r0 += kBwdWarps * U) {
            Raw8<DOUT_BF16> g[U];
            Raw8<PRE_BF16> z[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = r0 + kBwdWarps * u;
                if (r < r_end) {
                    g[u].load(a.dout, r * a.ld_dout + col);
                    if constexpr (ACT != UFP4_ACT_NONE) z[u].load(a.pre, r * a.ld_pre + col);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = r0 + kBwdWarps * u;
                if (r < r_end) {
                    float2 d[4], zv[4];
                    g[u].get2(d);
                    if constexpr (ACT != UFP4_ACT_NONE) {
                        z[u].get2(zv);
#pragma unroll
                        for (int j = 0; j < 4; ++j) d[j] = mul2(d[j], act_slope2<ACT>(zv[j]));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[j] = add2(sum[j], d[j]);
                    if (a.dpre != nullptr) store8<DPRE_BF16>(a.dpre, r * a.ld_dpre + col, d);
                }
            }
        }
    }
    const float sums[8] = {sum[0].x, sum[0].y, sum[1].x, sum[1].y, sum[2].x, sum[2].y, sum[3].x, sum[3].y};
    if (a.dbias != nullptr) store_partial(a, sums, col0);
}

// Any width, row pitch and alignment: the same by whole granules (load8_raw,
// store8_any).
template <int ACT, bool DOUT_BF16, bool PRE_BF16>
__global__ void __launch_bounds__(kBwdThreads, 2) epilogue_backward_any_kernel(const __grid_constant__ EpiBwdArgs a) {
    let_next_kernel_launch();
    constexpr int U = kBwdUnroll<DOUT_BF16, PRE_BF16>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * kBwdCols;
    const int64_t col = col0 + 8 * lane;
    const int64_t left = a.n - col;
    const int rest = left > 1024 ? 1024 : left < -8 ? -8 : static_cast<int>(left);
    const int64_t r_first = blockIdx.y * a.rows_per_chunk + warp;
    const int64_t r_end = min(a.m, (blockIdx.y + 1) * a.rows_per_chunk);
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    for (int64_t r0 = r_first; r0 < r_end; r0 += kBwdWarps * U) {     // whole warps
        Raw8<DOUT_BF16> g[U];
        Raw8<PRE_BF16> z[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + kBwdWarps * u;
            const int valid = r < r_end ? rest : 0;
            g[u].load_any(a.dout, r * a.ld_dout + col, valid);
            if constexpr (ACT != UFP4_ACT_NONE) z[u].load_any(a.pre, r * a.ld_pre + col, valid);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + kBwdWarps * u;
            float d[8];
            g[u].get(d);
            if constexpr (ACT != UFP4_ACT_NONE) {
                float2 zv[4];
                z[u].get2(zv);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 q = mul2(make_float2(d[2 * j], d[2 * j + 1]), act_slope2<ACT>(zv[j]));
                    d[2 * j] = q.x;
                    d[2 * j + 1] = q.y;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += d[j];
            if (a.dpre != nullptr && r < r_end) {
                if (a.dpre_bf16)
                    store8_any<true>(a.dpre, r * a.ld_dpre + col, rest, d);
                else
                    store8_any<false>(a.dpre, r * a.ld_dpre + col, rest, d);
            }
        }
    }
    if (a.dbias != nullptr) store_partial(a, sum, col0);
}

// out[c] = sum of the partial rows: 32 columns per block, its 32 warps take
// every 32nd row, then the 32 sums in a tree.  (With eight warps the 592 partial
// rows of a 16384 x 2048 norm took 13 us, a fifth of that call.)
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) column_sums_kernel(const float *partial, int64_t rows, int64_t cols,
                                                                     float *out) {
    __shared__ float s_sum[kSumWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    wait_for_previous_kernel();
    float t = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t r = warp; r < rows; r += kSumWarps) t += partial[r * cols + c];
    }
    s_sum[warp][lane] = t;
    __syncthreads();
    // warp w finishes column w
    float s = s_sum[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const int64_t cw = static_cast<int64_t>(blockIdx.x) * 32 + warp;
    if (lane == 0 && cw < cols) out[cw] = s;
}

__global__ void __launch_bounds__(256) epilogue_only_kernel(const __grid_constant__ EpiArgs e, int64_t m, int64_t n) {
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
        for (int64_t col = 4 * threadIdx.x; col < n; col += 4 * 256) {
            const int valid = col + 4 <= n ? 4 : static_cast<int>(n - col);
            epilogue_quad(e, row, col, valid, make_float4(0.0f, 0.0f, 0.0f, 0.0f), epilogue_bias(e, col, valid),
                          epilogue_residual(e, row, col, valid));
        }
    }
}

template <int ACT>
cudaError_t launch_bwd_act(const EpiBwdArgs &a, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((a.n + kBwdCols - 1) / kBwdCols), static_cast<unsigned>(a.chunks));
    if (!a.vec) {
        switch ((a.dout_bf16 ? 2 : 0) | (a.pre_bf16 ? 1 : 0)) {
            case 0: epilogue_backward_any_kernel<ACT, false, false><<<grid, kBwdThreads, 0, stream>>>(a); break;
            case 1: epilogue_backward_any_kernel<ACT, false, true><<<grid, kBwdThreads, 0, stream>>>(a); break;
            case 2: epilogue_backward_any_kernel<ACT, true, false><<<grid, kBwdThreads, 0, stream>>>(a); break;
            default: epilogue_backward_any_kernel<ACT, true, true><<<grid, kBwdThreads, 0, stream>>>(a); break;
        }
    } else {
        const int types = (a.dout_bf16 ? 4 : 0) | (a.pre_bf16 ? 2 : 0) | (a.dpre_bf16 ? 1 : 0);
        switch (types) {
            case 0: epilogue_backward_kernel<ACT, false, false, false><<<grid, kBwdThreads, 0, stream>>>(a); break;
            case 1: epilogue_backward_kernel<ACT, false, false, true><<<grid, kBwdThreads, 0, stream>>>(a); break;
            case 2: epilogue_backward_kernel<ACT, false, true, false><<<grid, kBwdThreads, 0, stream>>>(a); break;
            case 3: epilogue_backward_kernel<ACT, false, true, true><<<grid, kBwdThreads, 0, stream>>>(a); break;
            case 4: epilogue_backward_kernel<ACT, true, false, false><<<grid, kBwdThreads, 0, stream>>>(a); break;
            case 5: epilogue_backward_kernel<ACT, true, false, true><<<grid, kBwdThreads, 0, stream>>>(a); break;
            case 6: epilogue_backward_kernel<ACT, true, true, false><<<grid, kBwdThreads, 0, stream>>>(a); break;
            default: epilogue_backward_kernel<ACT, true, true, true><<<grid, kBwdThreads, 0, stream>>>(a); break;
        }
    }
    return cudaGetLastError();
}

}  // namespace

// Row chunks: about 24 blocks for each of the GPU's 148 SMs over the whole
// matrix (several waves, so the last one is a small share), at least 32 rows
// each.  A function of the shape alone: so are the workspace and the order of
// the sums.
int64_t epilogue_backward_chunks(int64_t m, int64_t n) {
    if (m <= 0 || n <= 0) return 1;
    const int64_t blocks_n = (n + kBwdCols - 1) / kBwdCols;
    int64_t chunks = int64_t(148) * 24 / blocks_n;
    const int64_t most = (m + 31) / 32;
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    const int64_t per = ((m + chunks - 1) / chunks + 7) / 8 * 8;
    return (m + per - 1) / per;
}

cudaError_t launch_epilogue_backward(const EpiBwdArgs &args, cudaStream_t stream) {
    EpiBwdArgs a = args;
    a.rows_per_chunk = ((a.m + a.chunks - 1) / a.chunks + 7) / 8 * 8;
    if (a.dbias != nullptr && a.chunks == 1) a.partial = a.dbias;   // the only partial row is the result
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.act) {
        case UFP4_ACT_NONE: e = launch_bwd_act<UFP4_ACT_NONE>(a, stream); break;
        case UFP4_ACT_RELU: e = launch_bwd_act<UFP4_ACT_RELU>(a, stream); break;
        case UFP4_ACT_GELU: e = launch_bwd_act<UFP4_ACT_GELU>(a, stream); break;
        case UFP4_ACT_GELU_ERF: e = launch_bwd_act<UFP4_ACT_GELU_ERF>(a, stream); break;
        case UFP4_ACT_SILU: e = launch_bwd_act<UFP4_ACT_SILU>(a, stream); break;
    }
    if (e != cudaSuccess || a.dbias == nullptr || a.chunks == 1) return e;
    return launch_column_sums(a.partial, a.chunks, a.n, a.dbias, stream);
}

cudaError_t launch_column_sums(const float *partial, int64_t rows, int64_t cols, float *out, cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>((cols + 31) / 32);
    return launch_early(column_sums_kernel, dim3(blocks), dim3(32 * kSumWarps), stream, partial, rows, cols, out);
}

cudaError_t launch_epilogue_only(const EpiArgs &e, int64_t m, int64_t n, int num_sms, cudaStream_t stream) {
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    epilogue_only_kernel<<<static_cast<unsigned>(m < cap ? m : cap), 256, 0, stream>>>(e, m, n);
    return cudaGetLastError();
}

}  // namespace ufp4
