// ep_balance_loss and ep_balance_loss_backward: the router's sequence-wise
// balance loss, its per-expert counts and the gradient for the logits.
//
// One warp scores one token with its E logits in registers. The mean scores
// need sums over all tokens of a sequence: each CTA sums a chunk of tokens
// and writes one partial row per (chunk, sequence) pair, and a second kernel
// adds a sequence's rows in chunk order, so the results do not depend on the
// order in which CTAs run.
//
// Pairs that share a token form a staircase: from one to the next the chunk or
// the sequence (or both) grows. So chunk + sequence is a row index that no two
// pairs share, the rows of one sequence are contiguous, and chunks + S rows
// are enough.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "ep.h"
#include "internal.h"

namespace ep {
namespace {

constexpr int kWarps = 8;

struct BalanceParams {
    int64_t N;
    int E, K, S, score;
    int chunk;        // tokens per CTA
    int64_t nchunks;
    const float* logits;
    const int32_t* idx;
    const int32_t* off;
    float coef;
    float* loss;
    int32_t* counts;
    float* prob;
    float* part_p;    // [nchunks + S][E]
    int32_t* part_c;  // [nchunks + S][E]
    float* part_l;    // [S][column blocks]
    uint32_t* err;
    // backward
    const int32_t* in_counts;
    const float* grad_loss;
    int accumulate;
    float* dlogits;
};

// Sequence s as [lo, hi), clamped into [0, N]; hi >= lo.
__device__ __forceinline__ void sequence(const BalanceParams& p, int s, int64_t& lo, int64_t& hi) {
    if (!p.off) {
        lo = 0;
        hi = p.N;
        return;
    }
    lo = min(max((int64_t)p.off[s], (int64_t)0), p.N);
    hi = min(max((int64_t)p.off[s + 1], lo), p.N);
}

// The first sequence that ends after token t (S if none).
__device__ __forceinline__ int first_sequence(const BalanceParams& p, int64_t t) {
    if (!p.off) return 0;
    int a = 0, b = p.S;
    while (a < b) {
        const int m = (a + b) >> 1;
        if ((int64_t)p.off[m + 1] > t) b = m;
        else a = m + 1;
    }
    return a;
}

// Expert of lane register i: 4 neighbours per lane where rows load as float4.
template <bool VEC>
__device__ __forceinline__ int expert_of(int i, int lane) {
    return VEC ? (i >> 2) * 128 + lane * 4 + (i & 3) : i * 32 + lane;
}

template <int EPL, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float (&z)[EPL]) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
            const int e = expert_of<true>(i, lane);
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e < E) v = __ldcs(reinterpret_cast<const float4*>(row + e));
            z[i] = v.x;
            z[i + 1] = v.y;
            z[i + 2] = v.z;
            z[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = expert_of<false>(i, lane);
            z[i] = e < E ? __ldcs(row + e) : -INFINITY;
        }
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
    return v;
}

// z becomes the unnormalised scores a (0 at -inf); returns 1 / sum(a). For
// the sigmoid, c becomes 1 - sigmoid(z) where WANT_C.
template <int EPL, bool WANT_C>
__device__ __forceinline__ float score_row(int score, float (&z)[EPL], float (&c)[EPL]) {
    float sum = 0.f;
    bool soft = score == EP_SCORE_SOFTMAX;
    if (!soft) {
        float tot = 0.f, a[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float t = __expf(-fabsf(z[i]));
            const float r = __fdividef(1.0f, 1.0f + t);
            a[i] = z[i] >= 0.f ? r : t * r;
            if (WANT_C) c[i] = z[i] >= 0.f ? t * r : r;
            tot += a[i];
        }
        sum = warp_sum(tot);
        // All sigmoids below 1e-17: there sigmoid(z) = exp(z) to fp32, and
        // the softmax below gives the quotient without underflow.
        soft = sum < 1e-17f;
        if (!soft) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) z[i] = a[i];
        }
    }
    if (soft) {
        float m = -INFINITY, tot = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) m = fmaxf(m, z[i]);
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            z[i] = __expf(z[i] - m);
            if (WANT_C) c[i] = 1.0f;
            tot += z[i];
        }
        sum = warp_sum(tot);
    }
    return 1.0f / sum;
}

template <int EPL, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) balance_partial_kernel(BalanceParams p) {
    extern __shared__ float sm[];
    float* red = sm;                                             // [kWarps][E]
    int32_t* cnt = reinterpret_cast<int32_t*>(sm + kWarps * p.E);  // [E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = blockIdx.x, clo = c * p.chunk, chi = min(clo + p.chunk, p.N);
    uint32_t bad = 0;
    for (int s = first_sequence(p, clo); s < p.S; ++s) {
        int64_t lo, hi;
        sequence(p, s, lo, hi);
        if (lo >= chi) break;
        lo = max(lo, clo);
        hi = min(hi, chi);
        if (lo >= hi) continue;
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) cnt[e] = 0;
        __syncthreads();
        for (int64_t i = lo * p.K + threadIdx.x; i < hi * p.K; i += blockDim.x) {
            const int e = p.idx[i];
            if (e >= 0 && e < p.E) atomicAdd(&cnt[e], 1);
            else if (e != -1) bad = EP_DEVERR_EXPERT_ID;
        }
        float acc[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] = 0.f;
        for (int64_t t = lo + warp; t < hi; t += kWarps) {
            float z[EPL], unused[EPL];
            load_row<EPL, VEC>(p.logits + t * p.E, p.E, lane, z);
            const float r = score_row<EPL, false>(p.score, z, unused);
#pragma unroll
            for (int i = 0; i < EPL; ++i) acc[i] = fmaf(z[i], r, acc[i]);
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = expert_of<VEC>(i, lane);
            if (e < p.E) red[warp * p.E + e] = acc[i];
        }
        __syncthreads();
        const int64_t slot = (c + s) * p.E;
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) a += red[w * p.E + e];
            p.part_p[slot + e] = a;
            p.part_c[slot + e] = cnt[e];
        }
    }
    if (bad) set_error(p.err, bad);
}

// One CTA per (sequence, 32 experts): the sequence's partial rows in 32
// strides, then the strides in order.
__global__ void __launch_bounds__(1024) balance_reduce_kernel(BalanceParams p) {
    __shared__ float sp[32][33];
    __shared__ int32_t sc[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int s = blockIdx.x, e = blockIdx.y * 32 + lane;
    int64_t lo, hi;
    sequence(p, s, lo, hi);
    if (p.off && threadIdx.x == 0 && blockIdx.y == 0) {
        const int a = p.off[s], b = p.off[s + 1];
        if (a < 0 || b < a || b > p.N) set_error(p.err, EP_DEVERR_ROW_BOUNDS);
    }
    float a = 0.f;
    int32_t n = 0;
    if (hi > lo && e < p.E) {
        const int64_t last = (hi - 1) / p.chunk + s;
        for (int64_t r = lo / p.chunk + s + w; r <= last; r += 32) {
            a += p.part_p[r * p.E + e];
            n += p.part_c[r * p.E + e];
        }
    }
    sp[w][lane] = a;
    sc[w][lane] = n;
    __syncthreads();
    if (w != 0) return;
    for (int i = 1; i < 32; ++i) {
        a += sp[i][lane];
        n += sc[i][lane];
    }
    const float inv_t = hi > lo ? 1.0f / (float)(hi - lo) : 0.f;
    const float pr = a * inv_t;
    const float term = e < p.E ? (float)n * ((float)p.E / (float)p.K) * inv_t * pr : 0.f;
    if (e < p.E) {
        p.counts[(int64_t)s * p.E + e] = n;
        if (p.prob) p.prob[(int64_t)s * p.E + e] = pr;
    }
    const float l = warp_sum(term);
    if (lane == 0) p.part_l[(int64_t)s * gridDim.y + blockIdx.y] = l;
}

__global__ void __launch_bounds__(1024) balance_loss_kernel(const float* part, int64_t n, float scale, float* loss) {
    __shared__ double sd[32];
    double a = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 1024) a += part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(FULL, a, o);
    if ((threadIdx.x & 31) == 0) sd[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 32; ++i) a += sd[i];
        *loss = (float)(a * scale);
    }
}

template <int EPL, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) balance_backward_kernel(BalanceParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a warp's consecutive tokens
    const int64_t per = p.chunk / kWarps;
    const int64_t wlo = (int64_t)blockIdx.x * p.chunk + warp * per, whi = min(wlo + per, p.N);
    if (wlo >= whi) return;
    const float g0 = (p.grad_loss ? *p.grad_loss : 1.0f) * p.coef / (float)p.S;
    for (int s = first_sequence(p, wlo); s < p.S; ++s) {
        int64_t lo, hi;
        sequence(p, s, lo, hi);
        if (lo >= whi) break;
        const float inv_t = hi > lo ? 1.0f / (float)(hi - lo) : 0.f;
        lo = max(lo, wlo);
        hi = min(hi, whi);
        if (lo >= hi) continue;
        float f[EPL];
        const float fs = (float)p.E / (float)p.K * inv_t;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = expert_of<VEC>(i, lane);
            f[i] = e < p.E ? (float)p.in_counts[(int64_t)s * p.E + e] * fs : 0.f;
        }
        const float g = g0 * inv_t;
        for (int64_t t = lo; t < hi; ++t) {
            float z[EPL], c[EPL];
            load_row<EPL, VEC>(p.logits + t * p.E, p.E, lane, z);
            const float r = score_row<EPL, true>(p.score, z, c);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) dot = fmaf(f[i], z[i], dot);
            dot = warp_sum(dot) * r;
            const float gr = g * r;
#pragma unroll
            for (int i = 0; i < EPL; ++i) z[i] = gr * z[i] * c[i] * (f[i] - dot);
            float* out = p.dlogits + t * p.E;
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < EPL; i += 4) {
                    const int e = expert_of<true>(i, lane);
                    if (e >= p.E) continue;
                    float4 v = make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]);
                    float4* o = reinterpret_cast<float4*>(out + e);
                    if (p.accumulate) {
                        const float4 w = *o;
                        v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
                    }
                    *o = v;
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = expert_of<false>(i, lane);
                    if (e < p.E) out[e] = p.accumulate ? out[e] + z[i] : z[i];
                }
            }
        }
    }
}

// Tokens per CTA: a multiple of the CTA's warps, about 1184 CTAs (8 on each
// of 148 SMs) on large batches.
int chunk_of(int64_t N) {
    const int64_t c = (N + 1183) / 1184;
    return (int)((c + kWarps - 1) / kWarps * kWarps);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Space {
    size_t p, c, l, total;
};
Space space_of(int64_t N, int E, int S) {
    const int64_t chunk = N > 0 ? chunk_of(N) : 1;
    const size_t rows = (size_t)((N + chunk - 1) / chunk + S);
    Space s;
    s.p = 0;
    s.c = align256(rows * E * 4);
    s.l = s.c + align256(rows * E * 4);
    s.total = s.l + align256((size_t)S * ((E + 31) / 32) * 4);
    return s;
}

ep_status_t check(int64_t N, int E, int K, int S, const int32_t* off) {
    if (N < 0) return fail(EP_ERR_INVALID, "N must be >= 0");
    if (N >= (int64_t)1 << 31) return fail(EP_ERR_UNSUPPORTED, "N must be < 2^31 (int32 offsets)");
    if (E < 1 || E > 1024) return fail(EP_ERR_UNSUPPORTED, "E must be in [1, 1024]");
    if (K < 1 || K > 32 || K > E) return fail(EP_ERR_INVALID, "K must be in [1, min(32, E)]");
    if (S < 1) return fail(EP_ERR_INVALID, "S must be >= 1");
    if (S > 1 << 24) return fail(EP_ERR_UNSUPPORTED, "S must be <= 2^24");
    if (!off && S != 1) return fail(EP_ERR_INVALID, "S > 1 needs d_seq_off");
    if ((uintptr_t)off % 4 != 0) return fail(EP_ERR_INVALID, "d_seq_off must be 4-byte aligned");
    return EP_OK;
}

template <int EPL, bool VEC>
void launch_partial(const BalanceParams& p, cudaStream_t s) {
    balance_partial_kernel<EPL, VEC><<<(unsigned)p.nchunks, kWarps * 32, (kWarps + 1) * p.E * 4, s>>>(p);
}
template <int EPL, bool VEC>
void launch_backward(const BalanceParams& p, cudaStream_t s) {
    balance_backward_kernel<EPL, VEC><<<(unsigned)p.nchunks, kWarps * 32, 0, s>>>(p);
}

ep_status_t launched(const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    set_last_error("");
    return EP_OK;
}

}  // namespace
}  // namespace ep

extern "C" {

ep_status_t ep_balance_loss_workspace_bytes(int64_t N, int E, int S, size_t* bytes) {
    using namespace ep;
    if (ep_status_t st = check(N, E, 1, S, reinterpret_cast<const int32_t*>(16))) return st;
    if (!bytes) return fail(EP_ERR_INVALID, "bytes is NULL");
    *bytes = space_of(N, E, S).total;
    set_last_error("");
    return EP_OK;
}

ep_status_t ep_balance_loss(int64_t N, int E, int K, int score, const float* d_logits, const int32_t* d_topk_idx,
                            int S, const int32_t* d_seq_off, float coef, float* d_loss, int32_t* d_counts,
                            float* d_prob, void* d_workspace, size_t workspace_bytes, uint32_t* d_error_word,
                            void* stream) {
    using namespace ep;
    if (ep_status_t st = check(N, E, K, S, d_seq_off)) return st;
    if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID) return fail(EP_ERR_INVALID, "unknown score %d", score);
    if (N > 0 && (!d_logits || !d_topk_idx)) return fail(EP_ERR_INVALID, "d_logits and d_topk_idx must be non-NULL");
    if (!d_loss || !d_counts || !d_error_word)
        return fail(EP_ERR_INVALID, "d_loss, d_counts and d_error_word must be non-NULL");
    if (((uintptr_t)d_logits | (uintptr_t)d_topk_idx | (uintptr_t)d_loss | (uintptr_t)d_counts | (uintptr_t)d_prob |
         (uintptr_t)d_error_word) % 4 != 0)
        return fail(EP_ERR_INVALID, "every array must be 4-byte aligned");
    if (!d_workspace || (uintptr_t)d_workspace % 256 != 0)
        return fail(EP_ERR_INVALID, "d_workspace must be non-NULL and 256-byte aligned");
    const Space sp = space_of(N, E, S);
    if (workspace_bytes < sp.total)
        return fail(EP_ERR_OOM, "workspace has %zu bytes, the call needs %zu", workspace_bytes, sp.total);
    uint8_t* ws = static_cast<uint8_t*>(d_workspace);
    BalanceParams p{};
    p.N = N;
    p.E = E;
    p.K = K;
    p.S = S;
    p.score = score;
    p.chunk = N > 0 ? chunk_of(N) : 1;
    p.nchunks = (N + p.chunk - 1) / p.chunk;
    p.logits = d_logits;
    p.idx = d_topk_idx;
    p.off = d_seq_off;
    p.coef = coef;
    p.loss = d_loss;
    p.counts = d_counts;
    p.prob = d_prob;
    p.part_p = reinterpret_cast<float*>(ws + sp.p);
    p.part_c = reinterpret_cast<int32_t*>(ws + sp.c);
    p.part_l = reinterpret_cast<float*>(ws + sp.l);
    p.err = d_error_word;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = E % 4 == 0 && (uintptr_t)d_logits % 16 == 0;
    if (p.nchunks > 0) {
        if (E <= 32) launch_partial<1, false>(p, s);
        else if (vec) {
            if (E <= 128) launch_partial<4, true>(p, s);
            else if (E <= 256) launch_partial<8, true>(p, s);
            else if (E <= 512) launch_partial<16, true>(p, s);
            else launch_partial<32, true>(p, s);
        } else {
            if (E <= 128) launch_partial<4, false>(p, s);
            else if (E <= 256) launch_partial<8, false>(p, s);
            else if (E <= 512) launch_partial<16, false>(p, s);
            else launch_partial<32, false>(p, s);
        }
        if (ep_status_t st = launched("balance partial")) return st;
    }
    const unsigned cb = (unsigned)((E + 31) / 32);
    balance_reduce_kernel<<<dim3((unsigned)S, cb), 1024, 0, s>>>(p);
    if (ep_status_t st = launched("balance reduce")) return st;
    balance_loss_kernel<<<1, 1024, 0, s>>>(p.part_l, (int64_t)S * cb, coef / (float)S, d_loss);
    return launched("balance loss");
}

ep_status_t ep_balance_loss_backward(int64_t N, int E, int K, int score, const float* d_logits, int S,
                                     const int32_t* d_seq_off, const int32_t* d_counts, float coef,
                                     const float* d_grad_loss, int accumulate, float* d_dlogits, void* stream) {
    using namespace ep;
    if (ep_status_t st = check(N, E, K, S, d_seq_off)) return st;
    if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID) return fail(EP_ERR_INVALID, "unknown score %d", score);
    if (N > 0 && (!d_logits || !d_counts || !d_dlogits))
        return fail(EP_ERR_INVALID, "d_logits, d_counts and d_dlogits must be non-NULL");
    if (((uintptr_t)d_logits | (uintptr_t)d_counts | (uintptr_t)d_grad_loss | (uintptr_t)d_dlogits) % 4 != 0)
        return fail(EP_ERR_INVALID, "every array must be 4-byte aligned");
    set_last_error("");
    if (N == 0) return EP_OK;
    BalanceParams p{};
    p.N = N;
    p.E = E;
    p.K = K;
    p.S = S;
    p.score = score;
    p.chunk = chunk_of(N);
    p.nchunks = (N + p.chunk - 1) / p.chunk;
    p.logits = d_logits;
    p.off = d_seq_off;
    p.coef = coef;
    p.in_counts = d_counts;
    p.grad_loss = d_grad_loss;
    p.accumulate = accumulate;
    p.dlogits = d_dlogits;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = E % 4 == 0 && ((uintptr_t)d_logits | (uintptr_t)d_dlogits) % 16 == 0;
    if (E <= 32) launch_backward<1, false>(p, s);
    else if (vec) {
        if (E <= 128) launch_backward<4, true>(p, s);
        else if (E <= 256) launch_backward<8, true>(p, s);
        else if (E <= 512) launch_backward<16, true>(p, s);
        else launch_backward<32, true>(p, s);
    } else {
        if (E <= 128) launch_backward<4, false>(p, s);
        else if (E <= 256) launch_backward<8, false>(p, s);
        else if (E <= 512) launch_backward<16, false>(p, s);
        else launch_backward<32, false>(p, s);
    }
    return launched("balance backward");
}

}  // extern "C"
