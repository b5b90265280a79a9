// router.cu -- balance loss of a mixture-of-experts router, with per-expert
// counts and the gradient of the logits.
//
// For T valid tokens, E experts, k choices per token, p = softmax(logits):
//     c_e = number of choices of expert e,   f_e = c_e / (k T),   P_e = (sum over tokens of p_te) / T
//     loss = coef * E * sum_e f_e P_e
//     dloss/dlogits_te = p_te (g_e - sum_j p_tj g_j),   g_e = coef * E * f_e / T    (f is a constant)
//
// balance_partial_kernel reads logits and choices once: G lanes share a token
// and hold its E / G logits in registers (max, exp, sum by shuffles), the
// probabilities are added up in fp32 registers over a lane's tokens, then over
// the block, and each block writes one partial row; balance_finish_kernel adds
// the rows in a fixed order, so the loss has the same bits every time (the
// counts are integers).  balance_backward_kernel recomputes p from the logits
// (one read, one write): HBM is the bound of both.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "ufp4.h"
#include "ufp4_elem.cuh"
#include "ufp4_internal.h"

namespace ufp4 {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// Experts of a token: lane g of its G lanes holds J of them, in vectors of V
// consecutive ones: expert V (g + G (j / V)) + j % V.
template <int G, int V>
__device__ __forceinline__ int expert_of(int g, int j) {
    return V * (g + G * (j / V)) + j % V;
}

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Tokens that a group of lanes works on at a time: their loads and their
// shuffle chains overlap.
template <int J>
constexpr int kTokensAtOnce = J <= 4 ? 4 : J <= 16 ? 2 : 1;

// exp(x - max) of U tokens' logits in registers, and each token's reciprocal
// sum; experts beyond E and tokens that do not count (`live` false) give 0.
// -inf logits give 0; a row of nothing but -inf gives 0 everywhere.  NaN
// stays NaN.
//
// Fewer bits than expf and a division would give, by choice: ex2.approx is
// within 2^-22, the product with log2 e within 2^-24 per unit of max - x, and
// __fdividef within 2 ulp.  At 131072 x 256 fp32 the gradient is 8.7e-8 from 64
// bits (relative norm); carrying the product's rounding along left that as it is
// and cost 9% forward, 3% backward (bf16: 16 and 20%), an exact division gave
// 8.6e-8 and cost 255 experts 3%.
template <int G, int J, int V, bool BF16, int U>
__device__ __forceinline__ void token_exp(const BalanceArgs &a, const int64_t (&token)[U], const bool (&live)[U], int g,
                                          float (&p)[U][J], float (&inv)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t base = token[u] * a.ld;
#pragma unroll
        for (int j = 0; j < J; j += V) {
            const int e = expert_of<G, V>(g, j);
            const bool in = live[u] && e < a.experts;
            if constexpr (V == 4) {
                const float4 q = in ? load_quad(a.logits, base + e, BF16, true, 4)
                                    : make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F);
                p[u][j] = q.x, p[u][j + 1] = q.y, p[u][j + 2] = q.z, p[u][j + 3] = q.w;
            } else {
                p[u][j] = in ? load_elem(a.logits, base + e, BF16) : -CUDART_INF_F;
            }
        }
    }
    float m[U], s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        m[u] = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < J; ++j) m[u] = fmaxf(m[u], p[u][j]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) m[u] = group_max<G>(m[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        // the difference first (exact near the maximum), then its base-2 exponent
        const float shift = m[u] == -CUDART_INF_F ? 0.0f : m[u];
        if constexpr (J % 2 == 0) {
            float2 sum = splat(0.0f);
#pragma unroll
            for (int j = 0; j < J; j += 2) {
                const float2 x = mul2(add2(make_float2(p[u][j], p[u][j + 1]), splat(-shift)), splat(kLog2e));
                p[u][j] = ex2_approx(x.x);
                p[u][j + 1] = ex2_approx(x.y);
                sum = add2(sum, make_float2(p[u][j], p[u][j + 1]));
            }
            s[u] = sum.x + sum.y;
        } else {
            s[u] = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                p[u][j] = ex2_approx((p[u][j] - shift) * kLog2e);
                s[u] += p[u][j];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = group_sum<G>(s[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) inv[u] = s[u] == 0.0f ? 0.0f : __fdividef(1.0f, s[u]);
}

// The token count and the loss from sum_e c_e (sum of p_e) and the count.
__device__ __forceinline__ void write_loss(const BalanceArgs &a, double dot, int64_t tokens) {
    const double n = static_cast<double>(tokens);
    *a.valid_tokens = tokens;
    *a.loss = tokens == 0 ? 0.0f : static_cast<float>(static_cast<double>(a.coef) * a.experts * dot / (n * n * a.topk));
}

template <int G, int J, int V, bool BF16>
__global__ void __launch_bounds__(kThreads, J <= 16 ? 2 : 1) balance_partial_kernel(const __grid_constant__ BalanceArgs a) {
    extern __shared__ uint32_t s_mem[];
    const int E = a.experts;
    int32_t *s_count = reinterpret_cast<int32_t *>(s_mem);          // [E]
    float *s_prob = reinterpret_cast<float *>(s_mem + E);           // [kWarps][E]
    __shared__ int32_t s_tokens;
    let_next_kernel_launch();
    for (int i = threadIdx.x; i < E; i += kThreads) s_count[i] = 0;
    if (threadIdx.x == 0) s_tokens = 0;
    __syncthreads();
    constexpr int kGroups = kThreads / G;                           // tokens of a block at a time
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = threadIdx.x % G;
    float acc[J];
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] = 0.0f;
    int32_t mine = 0;
    constexpr int U = kTokensAtOnce<J>;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    // whole warps go round together (the shuffles need all lanes)
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kGroups; t0 < a.tokens; t0 += U * step) {
        int64_t t[U];
        bool live[U];
        int first[U];           // this lane's first choice of each token
#pragma unroll
        for (int u = 0; u < U; ++u) {
            t[u] = t0 + u * step + threadIdx.x / G;
            live[u] = t[u] < a.tokens && (a.mask == nullptr || a.mask[t[u]] != 0);
            first[u] = live[u] && g < a.topk ? a.choices[t[u] * a.topk + g] : -1;
        }
        float p[U][J], inv[U];
        token_exp<G, J, V, BF16, U>(a, t, live, g, p, inv);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < J; ++j) acc[j] = fmaf(p[u][j], inv[u], acc[j]);
            mine += live[u] && g == 0;
            if (first[u] >= 0 && first[u] < E) atomicAdd(&s_count[first[u]], 1);
            if (live[u])
                for (int i = g + G; i < a.topk; i += G) {
                    const int e = a.choices[t[u] * a.topk + i];
                    if (e >= 0 && e < E) atomicAdd(&s_count[e], 1);
                }
        }
    }
    // over the warp's token groups, then (in order) over the warps
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int o = G; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
        const int e = expert_of<G, V>(g, j);
        if (lane < G && e < E) s_prob[warp * E + e] = acc[j];
    }
    if (mine != 0) atomicAdd(&s_tokens, mine);
    __syncthreads();
    const bool alone = gridDim.x == 1;          // few tokens: the results themselves
    double dot = 0.0;
    for (int e = threadIdx.x; e < E; e += kThreads) {
        float s = 0.0f;
        for (int w = 0; w < kWarps; ++w) s += s_prob[w * E + e];
        if (alone) {
            a.counts[e] = s_count[e];
            dot += static_cast<double>(s_count[e]) * static_cast<double>(s);
        } else {
            a.part_prob[static_cast<int64_t>(blockIdx.x) * E + e] = s;
            a.part_count[static_cast<int64_t>(blockIdx.x) * E + e] = s_count[e];
        }
    }
    if (!alone) {
        if (threadIdx.x == 0) a.part_tokens[blockIdx.x] = s_tokens;
        return;
    }
    __shared__ double s_dot[kWarps];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
    if (lane == 0) s_dot[warp] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        double d = 0.0;
        for (int w = 0; w < kWarps; ++w) d += s_dot[w];
        write_loss(a, d, s_tokens);
    }
}

// Adds the partial rows; writes counts, the token count and the loss.  One
// cluster of eight blocks (one block took 17 us for 296 rows of 256 experts):
// block r takes experts r * share .., `width` (a power of two, at least the
// share) threads side by side, and 1024 / width slices every so-many-th row
// each.  Slices and blocks are added in order.
constexpr int kFinishBlocks = 8;
__global__ void __cluster_dims__(kFinishBlocks) __launch_bounds__(1024)
    balance_finish_kernel(const __grid_constant__ BalanceArgs a, int blocks, int share, int width) {
    __shared__ float s_prob[1024];
    __shared__ int64_t s_count[1024];
    __shared__ double s_red[32];
    __shared__ int64_t s_tok[32];
    __shared__ double s_dot;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = blockIdx.x;
    const int col = threadIdx.x & (width - 1), slice = threadIdx.x / width, slices = 1024 / width;
    const int e = rank * share + col;
    const bool mine = col < share && e < a.experts;
    int64_t tok = 0;
    wait_for_previous_kernel();
    if (rank == 0)
        for (int b = threadIdx.x; b < blocks; b += 1024) tok += a.part_tokens[b];
    float s = 0.0f;
    int64_t c = 0;
    if (mine) {
#pragma unroll 8
        for (int b = slice; b < blocks; b += slices) {
            s += a.part_prob[static_cast<int64_t>(b) * a.experts + e];
            c += a.part_count[static_cast<int64_t>(b) * a.experts + e];
        }
    }
    s_prob[threadIdx.x] = s;
    s_count[threadIdx.x] = c;
    __syncthreads();
    // halve the slices until one is left
    for (int n = slices / 2; n > 0; n /= 2) {
        if (slice < n) {
            s_prob[threadIdx.x] += s_prob[threadIdx.x + n * width];
            s_count[threadIdx.x] += s_count[threadIdx.x + n * width];
        }
        __syncthreads();
    }
    double dot = 0.0;       // c_e * sum of p_e
    if (slice == 0 && mine) {
        c = s_count[threadIdx.x];
        a.counts[e] = c;
        dot = static_cast<double>(c) * static_cast<double>(s_prob[threadIdx.x]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        tok += __shfl_xor_sync(0xFFFFFFFFu, tok, o);
    }
    if (lane == 0) {
        s_red[warp] = dot;
        s_tok[warp] = tok;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double d = 0.0;
        for (int w = 0; w < 32; ++w) d += s_red[w];
        s_dot = d;
    }
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    cluster.sync();
    if (rank == 0 && threadIdx.x == 0) {
        double d = 0.0;
        int64_t n = 0;
        for (int r = 0; r < kFinishBlocks; ++r) d += *cluster.map_shared_rank(&s_dot, r);
        for (int w = 0; w < 32; ++w) n += s_tok[w];
        write_loss(a, d, n);
    }
    cluster.sync();         // the other blocks' sums stay until they are read
}

// dloss coef E / (k T^2), what makes g of a count.
__device__ __forceinline__ float balance_scale(const BalanceArgs &a) {
    const double n = static_cast<double>(*a.valid_tokens_in);
    return n == 0.0 ? 0.0f
                    : static_cast<float>(static_cast<double>(*a.dloss) * a.coef * a.experts / (n * n * a.topk));
}

// Tokens that do not count have p = 0, and 0 (g - dot) is 0 unless g is not
// finite: then their zeros are written once more, by the lanes that stored
// there.  (A choice in the backward kernel's loop, or this inlined behind it,
// cost 256 bf16 experts 5 to 15%.)
template <int G, int J, int V, bool BF16>
__device__ __noinline__ void zero_masked(const BalanceArgs &a) {
    if (a.mask == nullptr || fabsf(balance_scale(a)) < 1e25f) return;      // |g| <= 2^36 scale
    const int64_t groups = kThreads / G;
    for (int64_t t = blockIdx.x * groups + threadIdx.x / G; t < a.tokens; t += gridDim.x * groups) {
        for (int j = 0; j < J && a.mask[t] == 0; ++j) {
            const int e = expert_of<G, V>(threadIdx.x % G, j);
            if (e < a.experts) store_elem(a.dlogits, t * a.ld_d + e, BF16, 0.0f);
        }
    }
}

template <int G, int J, int V, bool BF16>
__global__ void __launch_bounds__(kThreads, J <= 16 ? 2 : 1) balance_backward_kernel(const __grid_constant__ BalanceArgs a) {
    constexpr int kGroups = kThreads / G;
    const int g = threadIdx.x % G;
    const int E = a.experts;
    const float scale = balance_scale(a);
    // g relative to the mean count's (p sums to 1, so the gradient is the same):
    // a balanced router's small differences come from whole numbers, not from
    // the cancellation of large products.
    const int64_t mean = *a.valid_tokens_in * a.topk / E;
    float ge[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = expert_of<G, V>(g, j);
        ge[j] = e < E ? scale * static_cast<float>(a.counts_in[e] - mean) : 0.0f;
    }
    constexpr int U = kTokensAtOnce<J>;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kGroups; t0 < a.tokens; t0 += U * step) {
        int64_t t[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            t[u] = t0 + u * step + threadIdx.x / G;
            live[u] = t[u] < a.tokens && (a.mask == nullptr || a.mask[t[u]] != 0);
        }
        float p[U][J], inv[U], dot[U];
        token_exp<G, J, V, BF16, U>(a, t, live, g, p, inv);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            dot[u] = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) dot[u] = fmaf(p[u][j], ge[j], dot[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) dot[u] = group_sum<G>(dot[u]) * inv[u];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < J; ++j) p[u][j] *= inv[u];
#pragma unroll
            for (int j = 0; j < J; j += V) {
                const int e = expert_of<G, V>(g, j);
                if (t[u] < a.tokens && e < E) {
                    if constexpr (V == 4)
                        store_quad(a.dlogits, t[u] * a.ld_d + e, BF16, true, 4,
                                   make_float4(p[u][j] * (ge[j] - dot[u]), p[u][j + 1] * (ge[j + 1] - dot[u]),
                                               p[u][j + 2] * (ge[j + 2] - dot[u]), p[u][j + 3] * (ge[j + 3] - dot[u])));
                    else
                        store_elem(a.dlogits, t[u] * a.ld_d + e, BF16, p[u][j] * (ge[j] - dot[u]));
                }
            }
        }
    }
    zero_masked<G, J, V, BF16>(a);
}

template <int G, int J, int V, bool BF16>
cudaError_t launch_shape(const BalanceArgs &a, bool backward, cudaStream_t stream) {
    const int64_t groups = kThreads / G;
    const int64_t need = (a.tokens + groups - 1) / groups;
    if (backward) {
        const int64_t most = int64_t(148) * 4;
        balance_backward_kernel<G, J, V, BF16>
            <<<static_cast<unsigned>(need < most ? need : most), kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    // four blocks' worth of tokens or fewer: one block and no second kernel
    // (512 tokens, 8 experts: 31 -> 29 us for both passes, launches included)
    const int blocks = need <= 4 ? 1 : static_cast<int>(need < kBalanceBlocks ? need : kBalanceBlocks);
    const int smem = a.experts * 4 * (1 + kWarps);
    static std::atomic<uint64_t> done{0};
    if (smem > 48 * 1024 - 256) {
        const cudaError_t e = allow_smem(balance_partial_kernel<G, J, V, BF16>, 4 * kBalanceMaxExperts * (1 + kWarps), done);
        if (e != cudaSuccess) return e;
    }
    balance_partial_kernel<G, J, V, BF16><<<blocks, kThreads, smem, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || blocks == 1) return e;
    const int share = (a.experts + kFinishBlocks - 1) / kFinishBlocks;
    int width = 1;
    while (width < share) width *= 2;
    return launch_early(balance_finish_kernel, dim3(kFinishBlocks), dim3(1024), stream, a, blocks, share, width);
}

// Experts to lanes.  Rows that allow vectors of four: 16 experts per lane where
// there are enough of them (a token's sums then take the fewest shuffles per
// expert; two blocks per SM leave 64 registers, of which 44 to 60 bytes forward
// and 24 to 36 backward are spilled), else a few lanes per token; other rows one
// expert at a time.
template <bool BF16>
cudaError_t launch_type(const BalanceArgs &a, bool backward, cudaStream_t stream) {
    const int E = a.experts;
    if (a.vec) {
        if (E <= 8) return launch_shape<2, 4, 4, BF16>(a, backward, stream);
        if (E <= 32) return launch_shape<4, 8, 4, BF16>(a, backward, stream);
        if (E <= 64) return launch_shape<4, 16, 4, BF16>(a, backward, stream);
        if (E <= 128) return launch_shape<8, 16, 4, BF16>(a, backward, stream);
        if (E <= 256) return launch_shape<16, 16, 4, BF16>(a, backward, stream);
        if (E <= 512) return launch_shape<32, 16, 4, BF16>(a, backward, stream);
        return launch_shape<32, 32, 4, BF16>(a, backward, stream);
    }
    if (E <= 8) return launch_shape<8, 1, 1, BF16>(a, backward, stream);
    if (E <= 32) return launch_shape<32, 1, 1, BF16>(a, backward, stream);
    if (E <= 128) return launch_shape<32, 4, 1, BF16>(a, backward, stream);
    if (E <= 256) return launch_shape<32, 8, 1, BF16>(a, backward, stream);
    return launch_shape<32, 32, 1, BF16>(a, backward, stream);
}

}  // namespace

cudaError_t launch_moe_balance(const BalanceArgs &a, bool backward, cudaStream_t stream) {
    return a.bf16 ? launch_type<true>(a, backward, stream) : launch_type<false>(a, backward, stream);
}

}  // namespace ufp4
