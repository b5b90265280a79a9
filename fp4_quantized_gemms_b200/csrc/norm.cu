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
// the weight gradient are fp32.  The forward mean divides: with a rounded
// 1 / cols elements crossed borders of the 8-bit rounding.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ufp4.h"
#define UFP4_PIPELINE_KERNELS 1
#include "ufp4_device.cuh"
#include "ufp4_elem.cuh"
#include "ufp4_internal.h"

namespace ufp4 {

namespace {

// Eight consecutive elements starting at p[i], lane l's behind lane l - 1's;
// `rest`: elements of the row from there on (any number; those beyond it are
// read as 0 and not written).  VEC: rows are 16-byte aligned and a multiple of
// eight long.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void *p, int64_t i, int rest, float (&v)[8]) {
    if constexpr (!VEC) {
        load8_any<BF16>(p, i, rest, v);
    } else if (rest <= 0) {
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
__device__ __forceinline__ void put8(void *p, int64_t i, int rest, const float (&v)[8]) {
    if constexpr (!VEC) {
        store8_any<BF16>(p, i, rest, v);                   // all 32 lanes
    } else if (rest > 0) {
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

__device__ __forceinline__ void load_weight8(const void *w, bool bf16, int64_t i, int rest, bool vec, float (&v)[8]) {
    if (vec) {
        if (bf16)
            load8<true, true>(w, i, rest, v);
        else
            load8<false, true>(w, i, rest, v);
    } else {
        if (bf16)
            load8_any<true>(w, i, rest, v);
        else
            load8_any<false>(w, i, rest, v);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the W warps that share a row; every thread gets it.  `slot` holds
// W floats of shared memory that no earlier sum still uses.  `bad` leaves as
// true in every thread when it came as true in any.
template <int W>
__device__ __forceinline__ float row_sum(float v, float *slot, bool *bad = nullptr) {
    v = warp_sum(v);
    if constexpr (W > 1) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) slot[warp] = v;
        if (bad == nullptr)
            __syncthreads();
        else
            *bad = __syncthreads_or(*bad) != 0;
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

// max(|a|, |b|, |c|)
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float m;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// Where a row's scale bytes and atom bytes go; block b of the row is at
// scales[b * scale_ld] and atoms[b / 4 * 512 + b % 4].
struct RowFactors {
    uint8_t *scales, *atoms;
    __device__ __forceinline__ RowFactors(const NormArgs &a, int64_t row) {
        scales = a.scales + row;
        atoms = a.sf_atoms == nullptr ? nullptr
                                      : a.sf_atoms + (row / 128) * a.atoms_k * 512 + 16 * (row % 32) + 4 * ((row / 32) % 4);
    }
};

// Writes eight columns of a row's output, y = h r w: bf16, or E4M3 elements and
// their blocks' factors (all lanes of the warp take part: a block of 32
// elements is four neighbouring lanes; elements beyond the row are 0).
template <bool OUT8, bool VEC>
__device__ __forceinline__ void write_y(const NormArgs &a, const RowFactors &f, int64_t row, int col, int rest,
                                        const float (&v)[8]) {
    if constexpr (!OUT8) {
        put8<true, VEC>(a.y, row * a.ld_y + col, rest, v);
    } else {
        float u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = v[e];
        if (rest < 8) {                                   // padding: 0 in rows that are not finite, too
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = e < rest ? u[e] : 0.0f;
        }
        float amax = max_abs3(max_abs3(max_abs3(u[0], u[1], u[2]), u[3], u[4]), max_abs3(u[5], u[6], u[7]), 0.0f);
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const int x = block_exponent(amax);
        const float inv = exp2_neg(x);
        if (col < a.kpad) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[e] = __nv_cvt_float2_to_fp8x2(mul2(make_float2(u[2 * e], u[2 * e + 1]), splat(inv)), __NV_SATFINITE,
                                                __NV_E4M3);
            *reinterpret_cast<uint2 *>(a.elems8 + row * a.kpad + col) =
                make_uint2(plain_zeros(p[0] | (p[1] << 16)), plain_zeros(p[2] | (p[3] << 16)));
            if ((threadIdx.x & 3) == 0) {
                const int b = col >> 5;
                f.scales[b * a.scale_ld] = static_cast<uint8_t>(x + 127);
                if (f.atoms != nullptr) f.atoms[(b >> 2) * 512 + (b & 3)] = static_cast<uint8_t>(x + 127);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Rows through a ring in shared memory: bulk copies bring the next rows of the
// block's tensors while the current one is reduced, so the reduction's
// barriers and the second half of the row's work never leave HBM idle.  The
// row sum's barrier is also what frees a stage: every thread has moved its
// part of the row into registers by then, and thread 0 refills the stage.
constexpr int kMaxStages = 8;

__device__ __forceinline__ void bulk_load(void *smem_dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(smem_dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

struct RingState {
    uint64_t full[kMaxStages];
    uint32_t abort;
};

// Waits (with a limit) for copies [from, to) to land, so that none is in
// flight when the block ends early.
__device__ __forceinline__ void drain_ring(RingState &s, int64_t from, int64_t to, int stages) {
    uint32_t dummy = 0;
    for (int64_t k = from; k < to; ++k)
        mbar_wait(&s.full[k % stages], static_cast<uint32_t>(k / stages) & 1u, kErrTimeoutDrain, &dummy);
}

// A row of a tensor in a stage: the 16-byte granules that hold it, so with
// `shift` bytes of something else in front when the row is not aligned.
template <bool BF16, bool VEC>
struct StagedRow {
    const uint8_t *src;        // first granule
    uint32_t shift, bytes;     // of its first element; of the granules
    __device__ __forceinline__ StagedRow(const void *base, int64_t row, int64_t ld, int cols) {
        src = static_cast<const uint8_t *>(base) + row * ld * (BF16 ? 2 : 4);
        shift = VEC ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
        src -= shift;
        bytes = (shift + static_cast<uint32_t>(cols) * (BF16 ? 2u : 4u) + 15u) / 16u * 16u;
    }
    // shared memory that a row of the tensor takes at most
    static __host__ __device__ __forceinline__ uint32_t room(int cols) {
        return (static_cast<uint32_t>(cols) * (BF16 ? 2u : 4u) + 15u) / 16u * 16u + (VEC ? 0u : 16u);
    }
};

// Eight elements of a staged row (at `p`, its shift included) as pairs.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8s(const uint8_t *p, int col, int rest, float2 (&v)[4]) {
    float f[8];
    load8<BF16, VEC>(p, col, rest, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float2(f[2 * e], f[2 * e + 1]);
}

template <int W, int NV, bool SBF16, bool XBF16, bool RES, bool OUT8, bool VEC>
__global__ void __launch_bounds__(32 * W, 32 / W) rmsnorm_ring_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ RingState st;
    __shared__ float s_sum[2][W];
    const int t = threadIdx.x;
    const int cols = static_cast<int>(a.cols);
    using XRow = StagedRow<XBF16, VEC>;
    using RRow = StagedRow<SBF16, VEC>;
    const uint32_t x_room = XRow::room(cols);
    const int64_t n = (a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x;      // rows of this block
    auto issue = [&](int64_t k) {
        const int s = static_cast<int>(k % a.stages);
        const int64_t row = blockIdx.x + k * gridDim.x;
        uint8_t *buf = ring + s * a.stage_bytes;
        const XRow x(a.x, row, a.ld_x, cols);
        const RRow r(a.residual, row, a.ld_res, cols);
        mbar_arrive_expect_tx(&st.full[s], x.bytes + (RES ? r.bytes : 0u));
        bulk_load(buf, x.src, x.bytes, &st.full[s]);
        if constexpr (RES) bulk_load(buf + x_room, r.src, r.bytes, &st.full[s]);
    };
    if (t == 0) {
        for (int s = 0; s < a.stages; ++s) mbar_init(&st.full[s], 1);
        st.abort = 0u;
        fence_barrier_init();
    }
    __syncthreads();
    if (t == 0)
        for (int64_t k = 0; k < a.stages && k < n; ++k) issue(k);
    float2 w[NV][4];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = 8 * (t + 32 * W * j);
        float v[8];
        load_weight8(a.weight, a.weight_bf16, col, cols - col, a.vec_weight, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[j][e] = make_float2(v[2 * e], v[2 * e + 1]);
    }
    const float count = static_cast<float>(a.cols);
    int s = 0;
    uint32_t parity = 0;
    bool bad = false;
    int64_t k = 0;
    for (; k < n; ++k) {
        const int64_t row = blockIdx.x + k * gridDim.x;
        bad = !mbar_wait(&st.full[s], parity, kErrTimeoutTransform, &st.abort);
        const uint8_t *x_row = ring + s * a.stage_bytes + XRow(a.x, row, a.ld_x, cols).shift;
        const uint8_t *r_row = ring + s * a.stage_bytes + x_room + RRow(a.residual, row, a.ld_res, cols).shift;
        float2 h[NV][4], sq = splat(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = 8 * (t + 32 * W * j);
            load8s<XBF16, VEC>(x_row, col, cols - col, h[j]);
            if constexpr (RES) {
                float2 r[4];
                load8s<SBF16, VEC>(r_row, col, cols - col, r);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = add2(h[j][e], r[e]);
                if constexpr (SBF16) {                    // the stream as it is stored
                    uint32_t hw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        hw[e] = pack_bf16(h[j][e].x, h[j][e].y);
                        h[j][e] = make_float2(bf16_lo(hw[e]), bf16_hi(hw[e]));
                    }
                    if (VEC && col < cols)
                        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.h) + row * a.ld_h + col) =
                            make_uint4(hw[0], hw[1], hw[2], hw[3]);
                }
                if constexpr (!SBF16 || !VEC) {
                    const float hv[8] = {h[j][0].x, h[j][0].y, h[j][1].x, h[j][1].y,
                                         h[j][2].x, h[j][2].y, h[j][3].x, h[j][3].y};
                    put8<SBF16, VEC>(a.h, row * a.ld_h + col, cols - col, hv);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sq = fma2(h[j][e], h[j][e], sq);
        }
        float sum = sq.x + sq.y;
        sum = row_sum<W>(sum, s_sum[k & 1], &bad);
        if (bad) break;
        if (t == 0 && k + a.stages < n) issue(k + a.stages);
        const float rstd = 1.0f / sqrtf(sum / count + a.eps);
        if (t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
        const RowFactors factors(a, row);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = 8 * (t + 32 * W * j);
            float y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = mul2(mul2(h[j][e], splat(rstd)), w[j][e]);
                y[2 * e] = v.x;
                y[2 * e + 1] = v.y;
            }
            write_y<OUT8, VEC>(a, factors, row, col, cols - col, y);
        }
        if (++s == a.stages) {
            s = 0;
            parity ^= 1u;
        }
    }
    if (bad && t == 0) drain_ring(st, k, n < k + a.stages ? n : k + a.stages, a.stages);
}

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
        const int rest = static_cast<int>(a.cols - col);
        load8<XBF16, VEC>(a.x, row * a.ld_x + col, rest, h[j]);
        if constexpr (RES) {
            float r[8];
            load8<SBF16, VEC>(a.residual, row * a.ld_res + col, rest, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[j][e] += r[e];
                if constexpr (SBF16) h[j][e] = __bfloat162float(__float2bfloat16_rn(h[j][e]));
            }
            put8<SBF16, VEC>(a.h, row * a.ld_h + col, rest, h[j]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(h[j][e], h[j][e], sum);
    }
    sum = row_sum<W>(sum, s_sum);
    const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.cols) + a.eps);
    if (t == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
    const RowFactors factors(a, row);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = 8 * (t + S::kRowThreads * j);
        const int rest = static_cast<int>(a.cols - col);
        float w[8];
        load_weight8(a.weight, a.weight_bf16, col, rest, a.vec_weight, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] = h[j][e] * rstd * w[e];
        write_y<OUT8, VEC>(a, factors, row, col, rest, h[j]);
    }
}

// The weight gradient of a block's rows, to its partial row.
template <int W, int NV>
__device__ __forceinline__ void write_partial(const NormBwdArgs &a, const float (&dw)[NV][8]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t col = 8 * (threadIdx.x + 32 * W * j);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < a.cols) a.partial[blockIdx.x * a.cols + col + e] = dw[j][e];
    }
}

// Backward of rows that do not fit the ring: a block takes rows blockIdx.x, +
// gridDim.x, ..., and keeps the weight gradient of its columns in registers;
// its sums go to its partial row.  1024 threads hold four vectors of h, dy and
// the gradient each in 64 registers, so it spills 424 to 864 bytes a thread:
// 4096 x 32768 bf16 912 us (164 at the copy rate), 4096 x 12288 fp32 404 (123).
//
// (The mean of all three backward kernels is a product with 1 / cols: one
// rounding more of one term of dx; a division by every thread cost 2%, 177 ->
// 181 us at 16384 x 8192.)
template <int W, int NV, bool SBF16, bool DYBF16, bool DXBF16, bool VEC>
__global__ void __launch_bounds__(32 * W) rmsnorm_backward_kernel(const __grid_constant__ NormBwdArgs a) {
    let_next_kernel_launch();
    __shared__ float s_sum[2][W];
    const int t = threadIdx.x;
    float dw[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    int phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, phase ^= 1) {
        const float r = a.rstd[row];
        float xh[NV][8], g[NV][8];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = 8 * (t + 32 * W * j);
            const int rest = static_cast<int>(a.cols - col);
            float w[8];
            load8<SBF16, VEC>(a.h, row * a.ld_h + col, rest, xh[j]);
            load8<DYBF16, VEC>(a.dy, row * a.ld_dy + col, rest, g[j]);
            load_weight8(a.weight, a.weight_bf16, col, rest, a.vec_weight, w);
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
            const int64_t col = 8 * (t + 32 * W * j);
            const int rest = static_cast<int>(a.cols - col);
            float d[8];
            if (a.dh != nullptr) {
                load8<SBF16, VEC>(a.dh, row * a.ld_dh + col, rest, d);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = fmaf(r, g[j][e] - xh[j][e] * dot, d[e]);
            put8<DXBF16, VEC>(a.dx, row * a.ld_dx + col, rest, d);
        }
    }
    if (a.dweight != nullptr) write_partial<W, NV>(a, dw);
}

// Backward of short rows: a warp takes U rows at a time (U NV <= 4
// vectors of each tensor in flight per lane), all loads before the dot
// product, the elements kept as loaded so that 16 warps fit an SM; the weight
// is read again for each row (from L1).  128 registers are not enough for every
// type: up to 372 bytes a thread are spilled with fp32 tensors (513 to 1024
// columns), 108 with bf16.  65536 x 1024: 104 us in bf16 (82 at the copy rate),
// 195 in fp32 (164).
template <int NV, int U, bool SBF16, bool DYBF16, bool DXBF16, bool VEC>
__global__ void __launch_bounds__(128, 4) rmsnorm_backward_short_kernel(const __grid_constant__ NormBwdArgs a) {
    let_next_kernel_launch();
    __shared__ float s_dw[4][256 * NV];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cols = static_cast<int>(a.cols);
    const bool has_dh = a.dh != nullptr;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    float dw[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 4 * U;
    for (int64_t row0 = (static_cast<int64_t>(blockIdx.x) * 4 + warp) * U; row0 < a.rows; row0 += step) {
        Raw8<SBF16> h[U][NV], d[U][NV];
        Raw8<DYBF16> g[U][NV];
        float r[U], dot[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u;
            const bool in = row < a.rows;
            r[u] = in ? a.rstd[row] : 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = 8 * (lane + 32 * j);
                if constexpr (VEC) {
                    h[u][j].zero();
                    g[u][j].zero();
                    d[u][j].zero();
                    if (in && col < cols) {
                        h[u][j].load(a.h, row * a.ld_h + col);
                        g[u][j].load(a.dy, row * a.ld_dy + col);
                        if (has_dh) d[u][j].load(a.dh, row * a.ld_dh + col);
                    }
                } else {
                    const int rest = in ? cols - col : 0;
                    h[u][j].load_any(a.h, row * a.ld_h + col, rest);
                    g[u][j].load_any(a.dy, row * a.ld_dy + col, rest);
                    d[u][j].load_any(a.dh, row * a.ld_dh + col, has_dh ? rest : 0);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) dot[u] = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = 8 * (lane + 32 * j);
            float w[8];
            load_weight8(a.weight, a.weight_bf16, col, cols - col, a.vec_weight, w);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[8], y[8];
                h[u][j].get(x);
                g[u][j].get(y);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= r[u];
                    dw[j][e] = fmaf(y[e], x[e], dw[j][e]);
                    dot[u] = fmaf(y[e] * w[e], x[e], dot[u]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) dot[u] = warp_sum(dot[u]) * inv_cols;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = 8 * (lane + 32 * j);
            float w[8];
            load_weight8(a.weight, a.weight_bf16, col, cols - col, a.vec_weight, w);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[8], y[8], o[8];
                h[u][j].get(x);
                g[u][j].get(y);
                d[u][j].get(o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = fmaf(r[u], y[e] * w[e] - x[e] * r[u] * dot[u], o[e]);
                if (row0 + u < a.rows) put8<DXBF16, VEC>(a.dx, (row0 + u) * a.ld_dx + col, cols - col, o);
            }
        }
    }
    if (a.dweight == nullptr) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s_dw[warp][8 * (lane + 32 * j) + e] = dw[j][e];
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += 128)
        a.partial[blockIdx.x * a.cols + c] = (s_dw[0][c] + s_dw[1][c]) + (s_dw[2][c] + s_dw[3][c]);
}

// Backward through the ring: h, dy and dh of the next rows are on their way
// while a row's dot product is reduced.  Up to 8192 columns nothing is spilled;
// 1024 threads (wider rows) have 64 registers each and spill 200 to 300 bytes
// (8192 x 16384 bf16: 331 us, 164 at the copy rate).
template <int W, int NV, bool SBF16, bool DYBF16, bool DXBF16, bool VEC>
__global__ void __launch_bounds__(32 * W) rmsnorm_backward_ring_kernel(const __grid_constant__ NormBwdArgs a) {
    let_next_kernel_launch();
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ RingState st;
    __shared__ float s_sum[2][W];
    const int t = threadIdx.x;
    const int cols = static_cast<int>(a.cols);
    const bool has_dh = a.dh != nullptr;
    using HRow = StagedRow<SBF16, VEC>;
    using GRow = StagedRow<DYBF16, VEC>;
    const uint32_t g_at = HRow::room(cols), d_at = g_at + GRow::room(cols);
    const int64_t n = (a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x;
    auto issue = [&](int64_t k) {
        const int s = static_cast<int>(k % a.stages);
        const int64_t row = blockIdx.x + k * gridDim.x;
        uint8_t *buf = ring + s * a.stage_bytes;
        const HRow h(a.h, row, a.ld_h, cols), d(a.dh, row, a.ld_dh, cols);
        const GRow g(a.dy, row, a.ld_dy, cols);
        mbar_arrive_expect_tx(&st.full[s], h.bytes + g.bytes + (has_dh ? d.bytes : 0u));
        bulk_load(buf, h.src, h.bytes, &st.full[s]);
        bulk_load(buf + g_at, g.src, g.bytes, &st.full[s]);
        if (has_dh) bulk_load(buf + d_at, d.src, d.bytes, &st.full[s]);
    };
    if (t == 0) {
        for (int s = 0; s < a.stages; ++s) mbar_init(&st.full[s], 1);
        st.abort = 0u;
        fence_barrier_init();
    }
    __syncthreads();
    if (t == 0)
        for (int64_t k = 0; k < a.stages && k < n; ++k) issue(k);
    // 1024 threads have 64 registers each: they read the weight again for each
    // row (from L1)
    constexpr bool kHoldWeight = W < 32;
    float w[NV][8], dw[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = 8 * (t + 32 * W * j);
        if constexpr (kHoldWeight) load_weight8(a.weight, a.weight_bf16, col, cols - col, a.vec_weight, w[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    }
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    int s = 0;
    uint32_t parity = 0;
    bool bad = false;
    int64_t k = 0;
    for (; k < n; ++k) {
        const int64_t row = blockIdx.x + k * gridDim.x;
        const float r = a.rstd[row];
        bad = !mbar_wait(&st.full[s], parity, kErrTimeoutTransform, &st.abort);
        const uint8_t *buf = ring + s * a.stage_bytes;
        const uint8_t *h_row = buf + HRow(a.h, row, a.ld_h, cols).shift;
        const uint8_t *g_row = buf + g_at + GRow(a.dy, row, a.ld_dy, cols).shift;
        const uint8_t *d_row = buf + d_at + HRow(a.dh, row, a.ld_dh, cols).shift;
        float xh[NV][8], g[NV][8], d[NV][8];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = 8 * (t + 32 * W * j);
            load8<SBF16, VEC>(h_row, col, cols - col, xh[j]);
            load8<DYBF16, VEC>(g_row, col, cols - col, g[j]);
            load8<SBF16, VEC>(d_row, col, has_dh ? cols - col : 0, d[j]);
            if constexpr (!kHoldWeight) load_weight8(a.weight, a.weight_bf16, col, cols - col, a.vec_weight, w[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[j][e] *= r;
                dw[j][e] = fmaf(g[j][e], xh[j][e], dw[j][e]);
                g[j][e] *= w[j][e];
                dot = fmaf(g[j][e], xh[j][e], dot);
            }
        }
        dot = row_sum<W>(dot, s_sum[k & 1], &bad) * inv_cols;
        if (bad) break;
        if (t == 0 && k + a.stages < n) issue(k + a.stages);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = 8 * (t + 32 * W * j);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[j][e] = fmaf(r, g[j][e] - xh[j][e] * dot, d[j][e]);
            put8<DXBF16, VEC>(a.dx, row * a.ld_dx + col, cols - col, d[j]);
        }
        if (++s == a.stages) {
            s = 0;
            parity ^= 1u;
        }
    }
    if (bad && t == 0) drain_ring(st, k, n < k + a.stages ? n : k + a.stages, a.stages);
    if (a.dweight != nullptr) write_partial<W, NV>(a, dw);
}

// The stream's, dy's and dx's types as compile-time choices.
template <typename F>
cudaError_t with_bwd_types(const NormBwdArgs &a, F f) {
    using T = std::true_type;
    using N = std::false_type;
    switch ((a.stream_bf16 ? 4 : 0) | (a.dy_bf16 ? 2 : 0) | (a.dx_bf16 ? 1 : 0)) {
        case 0: return f(N(), N(), N());
        case 1: return f(N(), N(), T());
        case 2: return f(N(), T(), N());
        case 3: return f(N(), T(), T());
        case 4: return f(T(), N(), N());
        case 5: return f(T(), N(), T());
        case 6: return f(T(), T(), N());
        default: return f(T(), T(), T());
    }
}

template <int W, int NV>
cudaError_t launch_bwd_rows(const NormBwdArgs &a, int64_t blocks, cudaStream_t stream) {
    const unsigned n = static_cast<unsigned>(blocks);
    return with_bwd_types(a, [&](auto s, auto g, auto d) {
        constexpr bool S = decltype(s)::value, G = decltype(g)::value, D = decltype(d)::value;
        if (a.vec)
            rmsnorm_backward_kernel<W, NV, S, G, D, true><<<n, 32 * W, 0, stream>>>(a);
        else
            rmsnorm_backward_kernel<W, NV, S, G, D, false><<<n, 32 * W, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

template <int NV, int U>
cudaError_t launch_bwd_short(const NormBwdArgs &a, int64_t blocks, cudaStream_t stream) {
    const unsigned n = static_cast<unsigned>(blocks);
    return with_bwd_types(a, [&](auto s, auto g, auto d) {
        constexpr bool S = decltype(s)::value, G = decltype(g)::value, D = decltype(d)::value;
        if (a.vec)
            rmsnorm_backward_short_kernel<NV, U, S, G, D, true><<<n, 128, 0, stream>>>(a);
        else
            rmsnorm_backward_short_kernel<NV, U, S, G, D, false><<<n, 128, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

// Width of the rings: warps per row with two vectors per thread.
template <typename F>
cudaError_t with_ring_shape(int64_t width, F f) {
    if (width <= 2048) return f(std::integral_constant<int, 4>());
    if (width <= 4096) return f(std::integral_constant<int, 8>());
    if (width <= 8192) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

// Blocks per SM: 1024 threads in all forward (at most 64 registers each), 512
// backward (128: the weight gradient stays in registers).
int fwd_blocks_per_sm(int64_t width) { return width <= 2048 ? 8 : width <= 4096 ? 4 : width <= 8192 ? 2 : 1; }
int bwd_blocks_per_sm(int64_t width) { return width <= 2048 ? 4 : width <= 4096 ? 2 : 1; }

constexpr int64_t kRingSmem = 216 * 1024;      // of the SM's shared memory, over its blocks

// Stages of a ring whose rows take row_bytes; below 2 it is not used.
int ring_stages(int64_t row_bytes, int blocks_per_sm) {
    const int64_t s = kRingSmem / blocks_per_sm / ((row_bytes + 127) / 128 * 128);
    return static_cast<int>(s < kMaxStages ? s : kMaxStages);
}

// Blocks of the backward pass (a function of the shape alone: so are the
// workspace and the order of the sums).
int64_t bwd_blocks(int64_t rows, int64_t cols) {
    const int64_t per = cols <= 1024 ? 4 : 1;
    const int64_t need = (rows + per - 1) / per;
    const int64_t most = int64_t(148) * (cols <= 1024 ? 4 : bwd_blocks_per_sm(cols));
    return need < most ? need : most;
}

template <int W, bool SBF16, bool XBF16, bool RES, bool OUT8, bool VEC>
cudaError_t launch_fwd_ring_kernel(const NormArgs &a, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const int smem = a.stages * static_cast<int>(a.stage_bytes);
    auto *kernel = rmsnorm_ring_kernel<W, 2, SBF16, XBF16, RES, OUT8, VEC>;
    const cudaError_t e = allow_smem(kernel, kRingSmem, done);
    if (e != cudaSuccess) return e;
    const int64_t most = int64_t(148) * fwd_blocks_per_sm(a.kpad);
    kernel<<<static_cast<unsigned>(a.rows < most ? a.rows : most), 32 * W, smem, stream>>>(a);
    return cudaGetLastError();
}

// x's and the stream's types, the residual and the output as compile-time choices.
template <typename F>
cudaError_t with_fwd_types(const NormArgs &a, F f) {
    using T = std::true_type;
    using N = std::false_type;
    const bool out8 = a.elems8 != nullptr;
    if (a.residual == nullptr) {     // the stream is x itself
        if (a.x_bf16) return out8 ? f(T(), T(), N(), T()) : f(T(), T(), N(), N());
        return out8 ? f(N(), N(), N(), T()) : f(N(), N(), N(), N());
    }
    switch ((a.stream_bf16 ? 4 : 0) | (a.x_bf16 ? 2 : 0) | (out8 ? 1 : 0)) {
        case 0: return f(N(), N(), T(), N());
        case 1: return f(N(), N(), T(), T());
        case 2: return f(N(), T(), T(), N());
        case 3: return f(N(), T(), T(), T());
        case 4: return f(T(), N(), T(), N());
        case 5: return f(T(), N(), T(), T());
        case 6: return f(T(), T(), T(), N());
        default: return f(T(), T(), T(), T());
    }
}

template <int W>
cudaError_t launch_fwd_ring(const NormArgs &a, cudaStream_t stream) {
    return with_fwd_types(a, [&](auto s, auto x, auto r, auto o) {
        constexpr bool S = decltype(s)::value, X = decltype(x)::value, R = decltype(r)::value, O = decltype(o)::value;
        return a.vec ? launch_fwd_ring_kernel<W, S, X, R, O, true>(a, stream)
                     : launch_fwd_ring_kernel<W, S, X, R, O, false>(a, stream);
    });
}

template <int W, int NV>
cudaError_t launch_fwd_rows(const NormArgs &a, cudaStream_t stream) {
    using S = RowShape<W>;
    const unsigned grid = static_cast<unsigned>((a.rows + S::kRows - 1) / S::kRows);
    return with_fwd_types(a, [&](auto s, auto x, auto r, auto o) {
        constexpr bool SB = decltype(s)::value, X = decltype(x)::value, R = decltype(r)::value, O = decltype(o)::value;
        if (a.vec)
            rmsnorm_kernel<W, NV, SB, X, R, O, true><<<grid, S::kThreads, 0, stream>>>(a);
        else
            rmsnorm_kernel<W, NV, SB, X, R, O, false><<<grid, S::kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

template <int W, bool SBF16, bool DYBF16, bool DXBF16, bool VEC>
cudaError_t launch_bwd_ring_kernel(const NormBwdArgs &a, int64_t blocks, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const int smem = a.stages * static_cast<int>(a.stage_bytes);
    auto *kernel = rmsnorm_backward_ring_kernel<W, 2, SBF16, DYBF16, DXBF16, VEC>;
    const cudaError_t e = allow_smem(kernel, kRingSmem, done);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(blocks), 32 * W, smem, stream>>>(a);
    return cudaGetLastError();
}

template <int W>
cudaError_t launch_bwd_ring(const NormBwdArgs &a, int64_t blocks, cudaStream_t stream) {
    return with_bwd_types(a, [&](auto s, auto g, auto d) {
        constexpr bool S = decltype(s)::value, G = decltype(g)::value, D = decltype(d)::value;
        return a.vec ? launch_bwd_ring_kernel<W, S, G, D, true>(a, blocks, stream)
                     : launch_bwd_ring_kernel<W, S, G, D, false>(a, blocks, stream);
    });
}

// Shared memory of a row of `cols` elements of `size` bytes in a stage.
int64_t staged_room(int64_t cols, int64_t size, bool vec) { return (cols * size + 15) / 16 * 16 + (vec ? 0 : 16); }

}  // namespace

// Rows of 1025 to 16384 elements go through the ring once an SM gets more than
// one of them and two stages fit its shared memory (fp32 x with an fp32
// residual: not at 1729-2048, 3457-4096, 6913-8192 and above 13824 elements;
// other types always); short rows have a warp each, and few or very long rows
// a block each.
cudaError_t launch_rmsnorm(const NormArgs &args, cudaStream_t stream) {
    NormArgs a = args;
    const int64_t width = a.kpad;
    if (width > 1024 && width <= 16384 && a.rows > 148) {
        int64_t bytes = staged_room(a.cols, a.x_bf16 ? 2 : 4, a.vec);
        if (a.residual != nullptr) bytes += staged_room(a.cols, a.stream_bf16 ? 2 : 4, a.vec);
        a.stages = ring_stages(bytes, fwd_blocks_per_sm(width));
        a.stage_bytes = (bytes + 127) / 128 * 128;
        if (a.stages >= 2)
            return with_ring_shape(width, [&](auto w) { return launch_fwd_ring<decltype(w)::value>(a, stream); });
    }
    if (width <= 256) return launch_fwd_rows<1, 1>(a, stream);
    if (width <= 512) return launch_fwd_rows<1, 2>(a, stream);
    if (width <= 1024) return launch_fwd_rows<1, 4>(a, stream);
    // one vector per thread (one token of 8192: 8.0 us with four, 4.3 with one)
    if (width <= 2048) return launch_fwd_rows<8, 1>(a, stream);
    if (width <= 8192) return launch_fwd_rows<32, 1>(a, stream);
    return launch_fwd_rows<32, 4>(a, stream);
}

int64_t rmsnorm_backward_slots(int64_t rows, int64_t cols) { return rows <= 0 ? 0 : bwd_blocks(rows, cols); }

// The backward ring likewise wants two stages: up to 16384 elements in bf16 with
// dh, 9216 with three fp32 tensors, 11059 with an fp32 stream and bf16 dy.
cudaError_t launch_rmsnorm_backward(const NormBwdArgs &args, cudaStream_t stream) {
    NormBwdArgs a = args;
    const int64_t blocks = bwd_blocks(a.rows, a.cols);
    cudaError_t e = cudaErrorInvalidValue;
    bool ring = false;
    if (a.cols > 1024 && a.cols <= 16384) {
        const int64_t st = staged_room(a.cols, a.stream_bf16 ? 2 : 4, a.vec);
        const int64_t bytes = (a.dh == nullptr ? st : 2 * st) + staged_room(a.cols, a.dy_bf16 ? 2 : 4, a.vec);
        a.stages = ring_stages(bytes, bwd_blocks_per_sm(a.cols));
        a.stage_bytes = (bytes + 127) / 128 * 128;
        ring = a.stages >= 2;
    }
    if (ring)
        e = with_ring_shape(a.cols, [&](auto w) { return launch_bwd_ring<decltype(w)::value>(a, blocks, stream); });
    else if (a.cols <= 256)
        e = launch_bwd_short<1, 4>(a, blocks, stream);
    else if (a.cols <= 512)
        e = launch_bwd_short<2, 2>(a, blocks, stream);
    else if (a.cols <= 1024)
        e = launch_bwd_short<4, 1>(a, blocks, stream);
    else
        e = launch_bwd_rows<32, 4>(a, blocks, stream);
    if (e != cudaSuccess || a.dweight == nullptr) return e;
    return launch_column_sums(a.partial, blocks, a.cols, a.dweight, stream);
}

// Host side of ufp4_check_device_status for this translation unit's waits.
cudaError_t norm_read_and_clear_error_word(uint32_t *out) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_error_word, sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_error_word, &zero, sizeof(uint32_t));
}

}  // namespace ufp4
