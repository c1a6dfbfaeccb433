// ep_balance_loss and ep_balance_loss_backward: the router's sequence-wise
// balance loss, its per-expert counts and the gradient for the logits.
//
// LT lanes score a token, with up to 16 of its E logits each (32 where E is
// over 512), so a warp takes 32 / LT tokens at once and a reduction over the
// experts is log2(LT) shuffles for all of them. A lane loads its logits of the
// next tokens into its own part of shared memory with cp.async while it scores
// the present ones: registers for two rows left too few warps and bytes in
// flight to fill HBM (131072 x 256: 42 us for the sums, 48 us for the gradient).
//
// Now 36 and 47 us: bound by instruction issue (59 and 63%) and latency.
//
// The mean scores need sums over all tokens of a sequence: each CTA sums a
// chunk of tokens and writes one partial row per (chunk, sequence) pair, and a
// second kernel adds a sequence's rows in chunk order, so the results do not
// depend on the order in which CTAs run.
//
// Pairs that share a token form a staircase: from one to the next the chunk or
// the sequence (or both) grows. So chunk + sequence is a row index that no two
// pairs share, the rows of one sequence are contiguous, and chunks + S rows
// are enough.
#include <cuda_runtime.h>
#include <stdint.h>

#include "block.h"
#include "common.cuh"
#include "ep.h"
#include "internal.h"

namespace ep {
namespace {

constexpr int kWarps = 8;

struct BalanceParams {
    int64_t N;
    int E, K, S, score;
    int lt;           // lanes per token
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
    uint32_t* done;   // CTAs of the reduction that have written their part_l
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

// Expert of register i of lane `lane` of LT: 4 neighbours per lane where rows load as float4.
template <bool VEC>
__device__ __forceinline__ int expert_of(int i, int lane, int lt) {
    return VEC ? ((i >> 2) * lt + lane) * 4 + (i & 3) : i * lt + lane;
}

// The rows of logits that a warp's lanes will score next, LT lanes to a row. A
// lane reads back only what it loaded itself.
template <int VPL, bool VEC>
struct Rows {
    static constexpr int kDepth = VPL > 16 ? 3 : 4;
    static constexpr int kWarpBytes = kDepth * VPL * 32 * 4;
    const float* base;   // the lane's first logit of token 0
    float* slots;        // [kDepth][VPL / 4][32 lanes][4], or [VPL][32] where scalar
    int E, lane, lt;
    int64_t ahead, hi, step;
    int stage = 0;
    const float* now = nullptr;

    // Places beyond E stay -inf.
    __device__ __forceinline__ void clear() {
#pragma unroll 4
        for (int i = 0; i < kDepth * VPL; ++i) {
            if constexpr (VEC) slots[(i >> 2) * 128 + (i & 3)] = -INFINITY;
            else slots[i * 32] = -INFINITY;
        }
    }
    // Token t of lane group 0 first, then every `step` tokens, up to hi.
    __device__ __forceinline__ void start(int64_t t, int64_t end, int stride) {
        ahead = t;
        hi = end;
        step = stride;
        stage = 0;
#pragma unroll
        for (int d = 0; d < kDepth - 1; ++d) fetch(d);
    }
    __device__ __forceinline__ void fetch(int d) {
        if (ahead < hi) {
            const float* row = base + ahead * E;
            float* dst = slots + d * (VPL * 32);
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < VPL / 4; ++i)
                    if ((i * lt + lane) * 4 < E) copy<16>(dst + i * 128, row + i * lt * 4);
            } else {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (i * lt + lane < E) copy<4>(dst + i * 32, row + i * lt);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ahead += step;
    }
    // The next row (-inf beyond E; of no meaning beyond hi), and a fetch behind it.
    __device__ __forceinline__ void next(float (&z)[VPL]) {
        fetch(stage == 0 ? kDepth - 1 : stage - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        now = slots + stage * (VPL * 32);
        stage = stage == kDepth - 1 ? 0 : stage + 1;
        read(z);
    }
    // The row that next() gave last, again.
    __device__ __forceinline__ void read(float (&z)[VPL]) const {
        const float* src = now;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < VPL / 4; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(src + i * 128);
                z[4 * i] = v.x;
                z[4 * i + 1] = v.y;
                z[4 * i + 2] = v.z;
                z[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) z[i] = src[i * 32];
        }
    }
    template <int BYTES>
    static __device__ __forceinline__ void copy(float* dst, const float* src) {
        const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
        if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
    }
};

template <int VPL, bool VEC>
__device__ __forceinline__ Rows<VPL, VEC> rows_of(const BalanceParams& p, uint8_t* ring, int lane, int group, int lt) {
    Rows<VPL, VEC> r;
    r.base = p.logits + (int64_t)group * p.E + lane * (VEC ? 4 : 1);
    r.slots = reinterpret_cast<float*>(ring + (threadIdx.x >> 5) * r.kWarpBytes) + (threadIdx.x & 31) * (VEC ? 4 : 1);
    r.E = p.E;
    r.lane = lane;
    r.lt = lt;
    r.clear();
    return r;
}

// Over the LT lanes of a token; every lane of the warp takes part.
__device__ __forceinline__ float group_sum(float v, int lt) {
    for (int o = lt >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
__device__ __forceinline__ float group_max(float v, int lt) {
    for (int o = lt >> 1; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
    return v;
}

// z becomes exp(z - max), 0 at -inf; returns the sum.
template <int VPL>
__device__ __forceinline__ float softmax_row(float (&z)[VPL], int lt) {
    float m = -INFINITY, tot = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, z[i]);
    m = group_max(m, lt);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        z[i] = __expf(z[i] - m);
        tot += z[i];
    }
    return group_sum(tot, lt);
}

// The next row's unnormalised scores a (0 at -inf); returns 1 / sum(a). For
// the sigmoid, c becomes 1 - sigmoid(z) where WANT_C.
template <int VPL, bool VEC, bool SOFT, bool WANT_C>
__device__ __forceinline__ float score_next(Rows<VPL, VEC>& rows, int lt, float (&a)[VPL], float (&c)[VPL]) {
    rows.next(a);
    if constexpr (SOFT) return 1.0f / softmax_row<VPL>(a, lt);
    float tot = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const float z = a[i];
        const float t = __expf(-fabsf(z));
        const float r = __fdividef(1.0f, 1.0f + t);
        a[i] = z >= 0.f ? r : t * r;
        if (WANT_C) c[i] = z >= 0.f ? t * r : r;
        tot += a[i];
    }
    float sum = group_sum(tot, lt);
    // All sigmoids below 1e-17: there sigmoid(z) = exp(z) to fp32, and the
    // softmax gives the quotient without underflow.
    const bool tiny = sum < 1e-17f;
    if (__any_sync(FULL, tiny)) {
        float b[VPL];
        rows.read(b);
        const float sb = softmax_row<VPL>(b, lt);
        if (tiny) {
            sum = sb;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                a[i] = b[i];
                if (WANT_C) c[i] = 1.0f;
            }
        }
    }
    return 1.0f / sum;
}

template <int LT_, int VPL, bool VEC, bool SOFT>
__global__ void __launch_bounds__(kWarps * 32, VPL > 16 ? 2 : 3) balance_partial_kernel(BalanceParams p) {
    extern __shared__ __align__(16) uint8_t sm[];                 // rows | red | cnt
    float* red = reinterpret_cast<float*>(sm + kWarps * Rows<VPL, VEC>::kWarpBytes);  // [kWarps][E]
    int32_t* cnt = reinterpret_cast<int32_t*>(red + kWarps * p.E);                    // [E]
    const int lt = LT_ ? LT_ : p.lt;
    const int warp = threadIdx.x >> 5, lane = (threadIdx.x & 31) & (lt - 1), group = (threadIdx.x & 31) / lt;
    const int per_warp = 32 / lt;
    const int64_t c = blockIdx.x, clo = c * p.chunk, chi = min(clo + p.chunk, p.N);
    if (c == 0 && threadIdx.x == 0) *p.done = 0;
    Rows<VPL, VEC> rows = rows_of<VPL, VEC>(p, sm, lane, group, lt);
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
        uint64_t acc[VPL / 2];  // fp32 pairs
#pragma unroll
        for (int i = 0; i < VPL / 2; ++i) acc[i] = 0;
        const int step = kWarps * per_warp;
        int64_t t = lo + warp * per_warp;  // of the warp's first group
        rows.start(t, hi - group, step);
        for (; t < hi; t += step) {
            float a[VPL], unused[VPL];
            const float r = score_next<VPL, VEC, SOFT, false>(rows, lt, a, unused);
            if (t + group < hi) {
                const uint64_t rr = f32x2_pack(r, r);
#pragma unroll
                for (int i = 0; i < VPL / 2; ++i) acc[i] = f32x2_fma_rn(f32x2_pack(a[2 * i], a[2 * i + 1]), rr, acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const float2 pair = f32x2_unpack(acc[i / 2]);
            float v = i & 1 ? pair.y : pair.x;
            for (int o = lt; o < 32; o <<= 1) v += __shfl_xor_sync(FULL, v, o);
            const int e = expert_of<VEC>(i, lane, lt);
            if (group == 0 && e < p.E) red[warp * p.E + e] = v;
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

// One CTA per (sequence, 32 experts): the sequence's partial rows in one stride
// per warp, then the strides in order. The CTA that finishes last adds the loss
// up, in the order of the parts. (`done` is 0: the kernel before set it.)
__global__ void __launch_bounds__(1024) balance_reduce_kernel(BalanceParams p) {
    __shared__ float sp[32][33];
    __shared__ int32_t sc[32][33];
    __shared__ double sd[32];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
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
        const int64_t end = (hi - 1) / p.chunk + s;
        for (int64_t r = lo / p.chunk + s + w; r <= end; r += nw) {
            a += p.part_p[r * p.E + e];
            n += p.part_c[r * p.E + e];
        }
    }
    sp[w][lane] = a;
    sc[w][lane] = n;
    __syncthreads();
    if (w == 0) {
        for (int i = 1; i < nw; ++i) {
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
        const float l = group_sum(term, 32);
        if (lane == 0) {
            p.part_l[(int64_t)s * gridDim.y + blockIdx.y] = l;
            __threadfence();
            last = atomicAdd(p.done, 1u) == gridDim.x * gridDim.y - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    const int64_t parts = (int64_t)gridDim.x * gridDim.y;
    double total = 0.0;
    for (int64_t i = threadIdx.x; i < parts; i += blockDim.x) total += *(volatile float*)(p.part_l + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(FULL, total, o);
    if (lane == 0) sd[w] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < nw; ++i) total += sd[i];
        *p.loss = (float)(total * (p.coef / (float)p.S));
    }
}

template <int LT_, int VPL, bool VEC, bool SOFT>
__global__ void __launch_bounds__(kWarps * 32, VPL > 16 ? 2 : 3) balance_backward_kernel(BalanceParams p) {
    const int lt = LT_ ? LT_ : p.lt;
    const int warp = threadIdx.x >> 5, lane = (threadIdx.x & 31) & (lt - 1), group = (threadIdx.x & 31) / lt;
    const int per_warp = 32 / lt;
    const int64_t clo = (int64_t)blockIdx.x * p.chunk, chi = min(clo + p.chunk, p.N);
    extern __shared__ __align__(16) uint8_t sm[];
    Rows<VPL, VEC> rows = rows_of<VPL, VEC>(p, sm, lane, group, lt);
    const float g0 = (p.grad_loss ? *p.grad_loss : 1.0f) * p.coef / (float)p.S;
    for (int s = first_sequence(p, clo); s < p.S; ++s) {
        int64_t lo, hi;
        sequence(p, s, lo, hi);
        if (lo >= chi) break;
        const float inv_t = hi > lo ? 1.0f / (float)(hi - lo) : 0.f;
        lo = max(lo, clo);
        hi = min(hi, chi);
        if (lo >= hi) continue;
        const int step = kWarps * per_warp;
        int64_t t = lo + warp * per_warp;  // of the warp's first group
        if (t >= hi) continue;
        rows.start(t, hi - group, step);
        uint64_t f[VPL / 2];  // fp32 pairs
        const float fs = (float)p.E / (float)p.K * inv_t;
#pragma unroll
        for (int i = 0; i < VPL / 2; ++i) {
            float v[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int e = expert_of<VEC>(2 * i + q, lane, lt);
                v[q] = e < p.E ? (float)p.in_counts[(int64_t)s * p.E + e] * fs : 0.f;
            }
            f[i] = f32x2_pack(v[0], v[1]);
        }
        const float g = g0 * inv_t;
        for (; t < hi; t += step) {
            const bool live = t + group < hi;
            float a[VPL], c[VPL];
            const float r = score_next<VPL, VEC, SOFT, true>(rows, lt, a, c);
            uint64_t dots = 0;
#pragma unroll
            for (int i = 0; i < VPL / 2; ++i) dots = f32x2_fma_rn(f[i], f32x2_pack(a[2 * i], a[2 * i + 1]), dots);
            const float2 pair = f32x2_unpack(dots);
            const float dot = group_sum(pair.x + pair.y, lt) * r, gr = g * r;
            const uint64_t gg = f32x2_pack(gr, gr), one = f32x2_pack(1.f, 1.f), minus = f32x2_pack(-dot, -dot);
#pragma unroll
            for (int i = 0; i < VPL / 2; ++i) {
                uint64_t v = f32x2_mul_rn(f32x2_pack(a[2 * i], a[2 * i + 1]), gg);
                if (!SOFT) v = f32x2_mul_rn(v, f32x2_pack(c[2 * i], c[2 * i + 1]));
                const float2 o = f32x2_unpack(f32x2_mul_rn(v, f32x2_fma_rn(f[i], one, minus)));
                a[2 * i] = o.x;
                a[2 * i + 1] = o.y;
            }
            if (live) {
                float* out = p.dlogits + (t + group) * p.E;
                if constexpr (VEC) {
#pragma unroll
                    for (int i = 0; i < VPL; i += 4) {
                        const int e = expert_of<true>(i, lane, lt);
                        if (e >= p.E) continue;
                        float4 v = make_float4(a[i], a[i + 1], a[i + 2], a[i + 3]);
                        float4* o = reinterpret_cast<float4*>(out + e);
                        if (p.accumulate) {
                            const float4 w = *o;
                            v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
                        }
                        *o = v;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < VPL; ++i) {
                        const int e = expert_of<false>(i, lane, lt);
                        if (e < p.E) out[e] = p.accumulate ? out[e] + a[i] : a[i];
                    }
                }
            }
        }
    }
}

// Lanes per token for E experts: a power of two that leaves each at most 16.
int lanes_of(int E) {
    int lt = 1;
    while (lt < 32 && lt * 16 < E) lt *= 2;
    return lt;
}

// Tokens per CTA: 3 CTAs on each of 148 SMs on large batches, whole steps of a
// CTA's warps; fewer tokens where a batch is small.
int chunk_of(int64_t N, int E) {
    const int64_t c = (N + 443) / 444, step = kWarps * 32 / lanes_of(E);
    return (int)(c <= step ? (c + kWarps - 1) / kWarps * kWarps : (c + step - 1) / step * step);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Space {
    size_t p, c, l, done, total;
};
Space space_of(int64_t N, int E, int S) {
    const int64_t chunk = N > 0 ? chunk_of(N, E) : 1;
    const size_t rows = (size_t)((N + chunk - 1) / chunk + S);
    Space s;
    s.p = 0;
    s.c = align256(rows * E * 4);
    s.l = s.c + align256(rows * E * 4);
    s.done = s.l + align256((size_t)S * ((E + 31) / 32) * 4);
    s.total = s.done + 256;
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

template <int LT, int VPL, bool VEC>
void launch_as(const BalanceParams& p, bool backward, cudaStream_t s) {
    const bool soft = p.score == EP_SCORE_SOFTMAX;
    constexpr int ring = kWarps * Rows<VPL, VEC>::kWarpBytes;
    // The kernel's limit is what the most experts that it serves need, in every
    // call: another host thread's call, of other experts, may come between this
    // one's limit and its launch.
    constexpr int most = ring + (kWarps + 1) * (LT ? LT : 32) * VPL * 4;
    static_assert(most <= 227 * 1024, "shared memory");
    const int smem = ring + (backward ? 0 : (kWarps + 1) * p.E * 4);
    const auto kernel =
        backward ? (soft ? balance_backward_kernel<LT, VPL, VEC, true> : balance_backward_kernel<LT, VPL, VEC, false>)
                 : (soft ? balance_partial_kernel<LT, VPL, VEC, true> : balance_partial_kernel<LT, VPL, VEC, false>);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) kernel<<<(unsigned)p.nchunks, kWarps * 32, smem, s>>>(p);
}

void launch_tokens(BalanceParams& p, bool vec, bool backward, cudaStream_t s) {
    p.lt = lanes_of(p.E);
    if (p.E > 512) return vec ? launch_as<32, 32, true>(p, backward, s) : launch_as<32, 32, false>(p, backward, s);
    if (!vec) return launch_as<0, 16, false>(p, backward, s);
    switch (p.lt) {
        case 1: return launch_as<1, 16, true>(p, backward, s);
        case 2: return launch_as<2, 16, true>(p, backward, s);
        case 4: return launch_as<4, 16, true>(p, backward, s);
        case 8: return launch_as<8, 16, true>(p, backward, s);
        case 16: return launch_as<16, 16, true>(p, backward, s);
        default: return launch_as<32, 16, true>(p, backward, s);
    }
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
    p.chunk = N > 0 ? chunk_of(N, E) : 1;
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
    p.done = reinterpret_cast<uint32_t*>(ws + sp.done);
    p.err = d_error_word;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = E % 4 == 0 && (uintptr_t)d_logits % 16 == 0;
    if (p.nchunks > 0) {
        launch_tokens(p, vec, false, s);
    } else {
        const cudaError_t e = cudaMemsetAsync(p.done, 0, sizeof(uint32_t), s);
        if (e != cudaSuccess) return fail(EP_ERR_CUDA, "memset: %s", cudaGetErrorString(e));
    }
    if (ep_status_t st = launched("balance partial")) return st;
    // a warp for every 4 partial rows that a sequence has in the mean
    const int64_t rows = p.nchunks / S + 1;
    int warps = 1;
    while (warps < 32 && warps * 4 < rows) warps *= 2;
    balance_reduce_kernel<<<dim3((unsigned)S, (unsigned)((E + 31) / 32)), warps * 32, 0, s>>>(p);
    return launched("balance reduce");
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
    p.chunk = chunk_of(N, E);
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
    launch_tokens(p, vec, true, s);
    return launched("balance backward");
}

}  // extern "C"
