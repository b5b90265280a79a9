// clip.cu -- global norm of many gradient tensors, and clipping by it.
//
//     N = sqrt(sum over all tensors of g^2),   out = g * min(1, max_norm / N)
//
// Two passes: square_sums_kernel reads every tensor and leaves one fp64 sum
// per block; the second kernel's blocks add those sums (all in the same
// order, so all get the same N and no counter or atomic is needed) and scale.
// HBM bounds both.  The second pass visits the chunks in the opposite order:
// what the first one read last is still in L2.
//
// Squares are added in fp32 eight at a time and then in fp64 (so the norm is
// within 6 * 2^-24 of its value); where eight squares leave fp32's comfortable
// range they are taken in fp64, so this holds for gradients of any size.  The
// factor max_norm / N is fp32; below fp32's normal numbers, where it would lose
// bits that the products still have, it stays fp64 and so do the products.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "ufp4.h"
#include "ufp4_elem.cuh"
#include "ufp4_internal.h"

namespace ufp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                         // elements per thread and step
// Elements of a chunk: 8 steps of a block, or fewer where that leaves SMs
// without one (300,000 elements: 22 chunks of 8 steps took 8 us a pass, 148
// of one step 4).
constexpr int64_t kChunkMax = 16384, kChunkMin = kVec * kThreads;

// Eight elements from p[i]; `vec`: 16-byte accesses are allowed.
__device__ __forceinline__ void get8(const void *p, int64_t i, bool bf16, bool vec, int valid, float (&v)[8]) {
    if (vec && valid >= 8) {
        if (bf16) {
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
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < valid ? load_elem(p, i + j, bf16) : 0.0f;
}

__device__ __forceinline__ void put8(void *p, int64_t i, bool bf16, bool vec, int valid, const float (&v)[8]) {
    if (vec && valid >= 8) {
        if (bf16) {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        } else {
            float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < valid) store_elem(p, i + j, bf16, v[j]);
}

__device__ __forceinline__ double squares8(const float (&v)[8]) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
    if (s >= 1e-25f && s <= 1e37f) return static_cast<double>(s);
    // zeros, squares that may have underflowed or overflowed, NaN
    double d = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) d = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), d);
    return d;
}

// The same value in every thread of the block, added in one order.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double s_part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += s_part[w];
    return s;
}

// Tensor of a chunk: the last one whose first chunk is not beyond it.
template <int MAX>
__device__ __forceinline__ int tensor_of(const ClipTable<MAX> &t, int64_t chunk) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.e[mid].chunk0 <= chunk)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

template <int MAX>
__global__ void __launch_bounds__(kThreads) square_sums_kernel(const __grid_constant__ ClipTable<MAX> t, double *sums) {
    let_next_kernel_launch();
    double acc = 0.0;
    for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const ClipEntry &e = t.e[tensor_of(t, c)];
        const int64_t first = (c - e.chunk0) * t.chunk;
        const int64_t end = first + t.chunk < e.n ? first + t.chunk : e.n;
#pragma unroll 2
        for (int64_t i = first + kVec * threadIdx.x; i < end; i += kVec * kThreads) {
            float v[8];
            get8(e.src, i, e.src_bf16, e.vec, static_cast<int>(end - i < 8 ? end - i : 8), v);
            acc += squares8(v);
        }
    }
    acc = block_sum(acc);
    if (threadIdx.x == 0) sums[blockIdx.x] = acc;
}

__device__ __forceinline__ double total_norm(const double *sums, int64_t count) {
    wait_for_previous_kernel();
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < count; i += kThreads) s += sums[i];
    return sqrt(block_sum(s));
}

template <int MAX>
__global__ void __launch_bounds__(kThreads)
    scale_kernel(const __grid_constant__ ClipTable<MAX> t, const double *sums, int64_t count, float max_norm, float *norm) {
    const double n = total_norm(sums, count);
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(n);
    // A norm that is not finite leaves the values as they are.
    const bool scale = n > static_cast<double>(max_norm) && n < static_cast<double>(CUDART_INF);
    const double ratio = scale ? static_cast<double>(max_norm) / n : 1.0;
    const float coef = static_cast<float>(ratio);
    const bool tiny = ratio < 1.1754943508222875e-38 && ratio > 0.0;      // 2^-126
    for (int64_t k = blockIdx.x; k < t.chunks; k += gridDim.x) {
        const int64_t c = t.chunks - 1 - k;
        const ClipEntry &e = t.e[tensor_of(t, c)];
        if (!scale && e.dst == e.src) continue;         // in place and nothing to change
        const int64_t first = (c - e.chunk0) * t.chunk;
        const int64_t end = first + t.chunk < e.n ? first + t.chunk : e.n;
#pragma unroll 2
        for (int64_t i = first + kVec * threadIdx.x; i < end; i += kVec * kThreads) {
            const int valid = static_cast<int>(end - i < 8 ? end - i : 8);
            float v[8];
            get8(e.src, i, e.src_bf16, e.vec, valid, v);
            if (tiny) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = static_cast<float>(v[j] * ratio);
            } else if (scale) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= coef;
            }
            put8(e.dst, i, e.dst_bf16, e.vec, valid, v);
        }
    }
}

__global__ void __launch_bounds__(kThreads) norm_only_kernel(const double *sums, int64_t count, float *norm) {
    const double n = total_norm(sums, count);
    if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

int64_t blocks_of(int64_t chunks) {
    const int64_t most = kClipBlocks;
    return chunks < most ? chunks : most;
}

// Tables of at most MAX tensors, filled from tensors[first ..); returns how many were taken.
template <int MAX>
int32_t fill(const ufp4_tensor_t *tensors, int32_t first, int32_t n, ClipTable<MAX> *t) {
    t->n = 0;
    t->chunks = 0;
    int32_t i = first;
    for (; i < n && t->n < MAX; ++i) {
        const ufp4_tensor_t &s = tensors[i];
        if (s.n == 0) continue;
        ClipEntry &e = t->e[t->n++];
        e.src = s.src;
        e.dst = s.dst;
        e.n = s.n;
        e.chunk0 = t->chunks;
        e.src_bf16 = s.src_dtype == UFP4_DTYPE_BF16;
        e.dst_bf16 = s.dst_dtype == UFP4_DTYPE_BF16;
        e.vec = ((reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst)) & 15u) == 0;
        t->chunks += (s.n + t->chunk - 1) / t->chunk;
    }
    return i - first;
}

template <int MAX>
cudaError_t run(const ufp4_tensor_t *tensors, int32_t n, double *sums, bool scale, float max_norm, float *norm,
                cudaStream_t stream) {
    ClipTable<MAX> t;
    int64_t total = 0;
    for (int32_t i = 0; i < n; ++i) total += tensors[i].n;
    t.chunk = kChunkMax;
    while (t.chunk > kChunkMin && total < t.chunk * kClipBlocks) t.chunk /= 2;
    int64_t count = 0;
    for (int32_t i = 0; i < n;) {
        i += fill(tensors, i, n, &t);
        if (t.chunks == 0) continue;
        const int64_t b = blocks_of(t.chunks);
        square_sums_kernel<MAX><<<static_cast<unsigned>(b), kThreads, 0, stream>>>(t, sums + count);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        count += b;
    }
    if (!scale || count == 0) {
        return launch_early(norm_only_kernel, dim3(1), dim3(kThreads), stream, sums, count, norm);
    }
    for (int32_t i = 0; i < n;) {
        i += fill(tensors, i, n, &t);
        if (t.chunks == 0) continue;
        const cudaError_t e = launch_early(scale_kernel<MAX>, dim3(static_cast<unsigned>(blocks_of(t.chunks))),
                                           dim3(kThreads), stream, t, sums, count, max_norm, norm);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_grad_clip(const ufp4_tensor_t *tensors, int32_t n, double *sums, bool scale, float max_norm,
                             float *norm, cudaStream_t stream) {
    return n <= 64 ? run<64>(tensors, n, sums, scale, max_norm, norm, stream)
                   : run<kClipTable>(tensors, n, sums, scale, max_norm, norm, stream);
}

}  // namespace ufp4
