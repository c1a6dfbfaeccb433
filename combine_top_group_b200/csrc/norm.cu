// ep_rmsnorm and ep_rmsnorm_backward: residual addition, RMS norm and the
// e4m3 cast in one pass over the row, and the gradient.
//
// Both are bound by HBM where rows are many: 32768 x 7168 with residual, bf16
// and e4m3 out takes 351 us from a graph and 364 call by call (5.8 to 6.0 TB/s,
// 89 to 92% of a copy's rate), the gradient of 16384 x 7168 156 and 161 us (the
// same rates). The row stays in registers between the reduction and the outputs,
// so each input is read once and each output written once. Rows over 16384
// channels do not stream: 2048 x 32768 takes 123 us forward (93 at a copy's
// rate) and 282 backward (82), 1024 x 65536 158 and 447; the backward's 96 and
// 192 values of a thread do not fit its 64 registers.
#include <cuda_runtime.h>
#include <stdint.h>

#include "block.h"
#include "common.cuh"
#include "ep.h"
#include "internal.h"

namespace ep {
namespace {

// A thread holds VPT vectors of 16 channels; `tpr` threads (whole warps) hold
// a row, and a CTA holds blockDim.x / tpr rows. Vector j of thread t covers
// channels 16 * (t + j * tpr) .. +15, so 8 neighbouring lanes hold one
// 128-channel scale block.
constexpr int kVec = 16;

struct NormParams {
    int64_t N;
    int H, nv, tpr;
    const uint16_t* x;
    const uint16_t* res;
    const void* gamma;
    int gamma_fp32;
    float eps, inv_h;
    uint16_t* h;
    uint16_t* y;
    uint8_t* q;
    float* q_scale;
    float* rstd;
};

__device__ __forceinline__ u32x8 ld256(const void* p) {
    u32x8 a;
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(a.v[0]), "=r"(a.v[1]), "=r"(a.v[2]), "=r"(a.v[3]), "=r"(a.v[4]), "=r"(a.v[5]),
                   "=r"(a.v[6]), "=r"(a.v[7])
                 : "l"(p));
    return a;
}

__device__ __forceinline__ void load_gamma(const void* gamma, int fp32, int c, float* g) {
    if (fp32) {
        const u32x8 a = ld256(static_cast<const float*>(gamma) + c);
        const u32x8 b = ld256(static_cast<const float*>(gamma) + c + 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i] = __uint_as_float(a.v[i]);
            g[8 + i] = __uint_as_float(b.v[i]);
        }
    } else {
        const u32x8 a = ld256(static_cast<const uint16_t*>(gamma) + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[2 * i] = bf16lo(a.v[i]);
            g[2 * i + 1] = bf16hi(a.v[i]);
        }
    }
}

// Sum over the tpr threads of the caller's row, the same bits in each. red
// holds 32 floats. Every thread of the CTA calls it.
__device__ __forceinline__ float row_sum(float v, int tpr, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, wpr = tpr >> 5, first = (int)threadIdx.x / tpr * wpr;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    v = (int)(threadIdx.x & 31) < wpr ? red[first + (threadIdx.x & 31)] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

template <int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(NormParams p) {
    __shared__ float red[32];
    const int rpc = blockDim.x / p.tpr;
    const int sub = threadIdx.x / p.tpr, t = threadIdx.x - sub * p.tpr;
    const int64_t row = (int64_t)blockIdx.x * rpc + sub;
    const bool live = row < p.N;
    const int64_t base = live ? row * p.H : 0;
    float v[VPT][kVec];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int k = t + j * p.tpr;
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[j][i] = 0.f;
        if (live && k < p.nv) {
            const u32x8 a = ld256_stream(p.x + base + k * kVec);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[j][2 * i] = bf16lo(a.v[i]);
                v[j][2 * i + 1] = bf16hi(a.v[i]);
            }
            if (p.res) {
                const u32x8 b = ld256_stream(p.res + base + k * kVec);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[j][2 * i] += bf16lo(b.v[i]);
                    v[j][2 * i + 1] += bf16hi(b.v[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i) ss = fmaf(v[j][i], v[j][i], ss);
        }
    }
    ss = row_sum(ss, p.tpr, red);
    const float rstd = rsqrtf(ss * p.inv_h + p.eps);
    if (live && t == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int k = t + j * p.tpr;
        const bool on = live && k < p.nv;  // a multiple of 8 lanes: nv is
        u32x8 o;
        if (on && p.h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o.v[i] = pack_bf16x2(v[j][2 * i], v[j][2 * i + 1]);
            st256(p.h + base + k * kVec, o);
        }
        float g[kVec];
        if (on) {
            load_gamma(p.gamma, p.gamma_fp32, k * kVec, g);
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[j][i] = v[j][i] * rstd * g[i];
        }
        if (on && p.y) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o.v[i] = pack_bf16x2(v[j][2 * i], v[j][2 * i + 1]);
            st256(p.y + base + k * kVec, o);
        }
        if (p.q) {
            float amax = 1e-4f;
#pragma unroll
            for (int i = 0; i < kVec; ++i) amax = fmaxf(amax, fabsf(v[j][i]));
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, off));
            if (on) {
                const float s = 448.0f / amax;
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = pack_e4m3x2(v[j][4 * i] * s, v[j][4 * i + 1] * s) |
                           pack_e4m3x2(v[j][4 * i + 2] * s, v[j][4 * i + 3] * s) << 16;
                *reinterpret_cast<uint4*>(p.q + base + k * kVec) = make_uint4(w[0], w[1], w[2], w[3]);
                if ((k & 7) == 0) p.q_scale[row * (p.H / 128) + k / 8] = amax / 448.0f;
            }
        }
    }
}

// ---- streams of rows -----------------------------------------------------------
// A call with rows for every CTA several times over runs persistent CTAs. Each
// group of up to 32 lanes loads its own part of the next rows into shared
// memory with cp.async while it works on one: loads stay in flight across the
// reduction and the stores, no warp reads what another loaded, and gamma and
// the dgamma sums stay in registers. A thread holds 16 neighbouring channels
// (8 lanes to a scale block); the arithmetic runs on pairs of fp32 values,
// since the instruction rate bounds the e4m3 cast and the gradient otherwise
// (77% of issue slots with scalar arithmetic on 8 channels per thread).

__device__ __forceinline__ uint32_t smem_of(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of the thread's groups are in flight.
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint64_t f32x2_add_rn(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t widen(uint32_t u) { return f32x2_pack(bf16lo(u), bf16hi(u)); }
__device__ __forceinline__ uint32_t narrow(uint64_t v) {
    const float2 f = f32x2_unpack(v);
    return pack_bf16x2(f.x, f.y);
}
// 16 channels of bf16 as 8 fp32 pairs, and back.
__device__ __forceinline__ void widen16(const uint4 (&a)[2], uint64_t (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[4 * i] = widen(a[i].x);
        v[4 * i + 1] = widen(a[i].y);
        v[4 * i + 2] = widen(a[i].z);
        v[4 * i + 3] = widen(a[i].w);
    }
}
__device__ __forceinline__ void store16(uint16_t* p, const uint64_t (&v)[8]) {
    u32x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = narrow(v[i]);
    st256(p, o);
}

// Rows of a slot in shared memory: as many as leave room for VPT vectors of
// each array for 512 threads.
__host__ __device__ constexpr int depth_of(int vpt, int arrays) { return vpt == 1 ? 4 : arrays < 3 ? 3 : 2; }

// Where a thread stands: its row of the CTA's and its place in it; what it
// loads (chunks of 16 bytes: its lane's, and one group further) and reads (two
// neighbouring chunks) of a vector, as byte offsets.
struct Place {
    int rpc, sub, t;
    uint32_t load, load_step, read;
    uint32_t plane;   // bytes from one vector, array or ring position to the next
    int from, next;   // first channels of the two chunks it loads, within its vector
};
__device__ __forceinline__ Place place_of(int tpr) {
    Place q;
    q.rpc = blockDim.x / tpr;
    q.sub = threadIdx.x / tpr;
    q.t = threadIdx.x - q.sub * tpr;
    const int group = tpr < 32 ? tpr : 32, lane = q.t & (group - 1), first = (q.t - lane) * 2;
    const uint32_t row = q.sub * tpr * 2;
    q.load = (row + first + lane) * 16;
    q.load_step = group * 16;
    // Lanes 4-7 of each 8 take their second half first: otherwise lanes 4
    // apart would meet in the same banks.
    q.read = (row + 2 * q.t + ((lane >> 2) & 1)) * 16;
    q.plane = blockDim.x * 32;
    q.from = (first + lane) * 8;
    q.next = q.from + group * 8;
    return q;
}
// Loads the thread's chunks of a row into the planes from dst on.
template <int VPT>
__device__ __forceinline__ void load_ahead(uint32_t dst, const Place& q, int tpr, int H, const uint16_t* row) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int at = j * tpr * kVec;
        if (at + q.from < H) cp_async16(dst + j * q.plane + q.load, row + at + q.from);
        if (at + q.next < H) cp_async16(dst + j * q.plane + q.load + q.load_step, row + at + q.next);
    }
}
// The thread's 16 channels of a plane.
__device__ __forceinline__ void read16(const uint8_t* plane, const Place& q, uint64_t (&v)[8]) {
    const bool second = q.read & 16;
    const uint4 x = *reinterpret_cast<const uint4*>(plane + q.read),
                y = *reinterpret_cast<const uint4*>(plane + (q.read ^ 16));
    const uint4 b[2] = {second ? y : x, second ? x : y};
    widen16(b, v);
}

__device__ __forceinline__ void load_gamma_pairs(const void* gamma, int fp32, int c, uint64_t (&g)[8]) {
    float f[kVec];
    load_gamma(gamma, fp32, c, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = f32x2_pack(f[2 * i], f[2 * i + 1]);
}

// Sum over the row's threads: shuffles within a group, shared memory beyond.
__device__ __forceinline__ float stream_sum(uint64_t pairs, int tpr, float* red) {
    const float2 f = f32x2_unpack(pairs);
    float v = f.x + f.y;
    if (tpr >= 32) return row_sum(v, tpr, red);
    for (int o = tpr >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

template <int VPT, bool RES>
__global__ void __launch_bounds__(512) rmsnorm_stream_kernel(NormParams p) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][32];
    constexpr int A = RES ? 2 : 1, kDepth = depth_of(VPT, A);
    const Place q = place_of(p.tpr);
    const int64_t step = (int64_t)gridDim.x * q.rpc, row_first = (int64_t)blockIdx.x * q.rpc;
    const uint32_t base = smem_of(ring), stage_bytes = A * VPT * q.plane;
    int64_t ahead = row_first + q.sub;  // the next row to load
    const uint16_t *x = p.x + ahead * p.H, *res = RES ? p.res + ahead * p.H : nullptr;
    const int64_t stride = step * p.H;
    auto issue = [&](uint32_t at) {
        if (ahead < p.N) {
            load_ahead<VPT>(base + at, q, p.tpr, p.H, x);
            if (RES) load_ahead<VPT>(base + at + VPT * q.plane, q, p.tpr, p.H, res);
        }
        cp_commit();
        ahead += step;
        x += stride;
        if (RES) res += stride;
    };
    uint64_t g[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (q.t + j * p.tpr < p.nv) load_gamma_pairs(p.gamma, p.gamma_fp32, (q.t + j * p.tpr) * kVec, g[j]);
#pragma unroll
    for (int s = 0; s < kDepth - 1; ++s) issue(s * stage_bytes);
    uint32_t at = 0, fill = (kDepth - 1) * stage_bytes;
    int flip = 0;
    for (int64_t row0 = row_first; row0 < p.N; row0 += step, flip ^= 1) {
        __syncwarp();  // the slot filled next was read by the whole group
        issue(fill);
        fill = at;
        cp_wait<kDepth - 1>();
        __syncwarp();  // every lane's copies of this row are done
        const int64_t row = row0 + q.sub;
        const bool live = row < p.N;
        uint64_t v[VPT][8], ss = 0;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = 0;
            if (live && q.t + j * p.tpr < p.nv) {
                read16(ring + at + j * q.plane, q, v[j]);
                if (RES) {
                    uint64_t r[8];
                    read16(ring + at + (VPT + j) * q.plane, q, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = f32x2_add_rn(v[j][i], r[i]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = f32x2_fma_rn(v[j][i], v[j][i], ss);
            }
        }
        at = at == (kDepth - 1) * stage_bytes ? 0 : at + stage_bytes;
        const float rstd = rsqrtf(stream_sum(ss, p.tpr, red[flip]) * p.inv_h + p.eps);
        if (live && q.t == 0 && p.rstd) p.rstd[row] = rstd;
        const uint64_t rr = f32x2_pack(rstd, rstd);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int k = q.t + j * p.tpr;
            const bool on = live && k < p.nv;
            const int64_t to = row * p.H + k * kVec;
            if (on && p.h) store16(p.h + to, v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = f32x2_mul_rn(f32x2_mul_rn(v[j][i], rr), g[j][i]);
            if (on && p.y) store16(p.y + to, v[j]);
            if (p.q) {
                float amax = 1e-4f;
                if (on) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = f32x2_unpack(v[j][i]);
                        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
#pragma unroll
                for (int off = 1; off < 8; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, off));
                if (on) {
                    const float s = 448.0f / amax;
                    const uint64_t s2 = f32x2_pack(s, s);
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 a = f32x2_unpack(f32x2_mul_rn(v[j][2 * i], s2)),
                                     b = f32x2_unpack(f32x2_mul_rn(v[j][2 * i + 1], s2));
                        w[i] = pack_e4m3x2(a.x, a.y) | pack_e4m3x2(b.x, b.y) << 16;
                    }
                    *reinterpret_cast<uint4*>(p.q + to) = make_uint4(w[0], w[1], w[2], w[3]);
                    if ((k & 7) == 0) p.q_scale[row * (p.H / 128) + k / 8] = amax / 448.0f;
                }
            }
        }
    }
}

struct NormBwdParams {
    int64_t N;
    int H, nv, tpr;
    const uint16_t* h;
    const float* rstd;
    const void* gamma;
    int gamma_fp32;
    float inv_h;
    const uint16_t* dy;
    const uint16_t* dh;
    uint16_t* dx;
    float* part;  // [CTAs][H]
};

// Rows over 16384 channels, one at a time per CTA: CTA b takes rows b, b + CTAs,
// ... and keeps its dgamma sums in registers until the end.
template <int VPT>
__global__ void __launch_bounds__(1024, 1) rmsnorm_bwd_kernel(NormBwdParams p) {
    __shared__ float red[2][32];
    const int t = threadIdx.x;
    float dg[VPT][kVec];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) dg[j][i] = 0.f;
    int flip = 0;
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x, flip ^= 1) {
        const int64_t base = row * p.H;
        const float rstd = p.rstd[row];
        float n[VPT][kVec], dt[VPT][kVec];
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int k = t + j * p.tpr;
            if (k < p.nv) {
                const u32x8 a = ld256_stream(p.h + base + k * kVec), b = ld256_stream(p.dy + base + k * kVec);
                float g[kVec];
                load_gamma(p.gamma, p.gamma_fp32, k * kVec, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    n[j][2 * i] = bf16lo(a.v[i]) * rstd;
                    n[j][2 * i + 1] = bf16hi(a.v[i]) * rstd;
                    dt[j][2 * i] = bf16lo(b.v[i]);
                    dt[j][2 * i + 1] = bf16hi(b.v[i]);
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    dg[j][i] = fmaf(dt[j][i], n[j][i], dg[j][i]);
                    dt[j][i] *= g[i];
                    dot = fmaf(dt[j][i], n[j][i], dot);
                }
            }
        }
        const float m = row_sum(dot, p.tpr, red[flip]) * p.inv_h;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int k = t + j * p.tpr;
            if (k < p.nv) {
                u32x8 c;
                if (p.dh) c = ld256_stream(p.dh + base + k * kVec);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float lo = rstd * (dt[j][2 * i] - n[j][2 * i] * m);
                    float hi = rstd * (dt[j][2 * i + 1] - n[j][2 * i + 1] * m);
                    if (p.dh) {
                        lo += bf16lo(c.v[i]);
                        hi += bf16hi(c.v[i]);
                    }
                    c.v[i] = pack_bf16x2(lo, hi);
                }
                st256(p.dx + base + k * kVec, c);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int k = t + j * p.tpr;
        if (k < p.nv) {
            float4* o = reinterpret_cast<float4*>(p.part + (int64_t)blockIdx.x * p.H + k * kVec);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = make_float4(dg[j][4 * i], dg[j][4 * i + 1], dg[j][4 * i + 2], dg[j][4 * i + 3]);
        }
    }
}

// The gradient on a stream of rows. At the end a CTA adds its rows-per-CTA
// dgamma sums through shared memory, in row order, and writes one partial row.
template <int VPT, bool DH>
__global__ void __launch_bounds__(512) rmsnorm_bwd_stream_kernel(NormBwdParams p) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][32];
    constexpr int A = DH ? 3 : 2, kDepth = depth_of(VPT, A);
    const Place q = place_of(p.tpr);
    const int64_t step = (int64_t)gridDim.x * q.rpc, row_first = (int64_t)blockIdx.x * q.rpc;
    const uint32_t base = smem_of(ring), stage_bytes = A * VPT * q.plane;
    int64_t ahead = row_first + q.sub;  // the next row to load
    int64_t from = ahead * p.H;
    const int64_t stride = step * p.H;
    auto issue = [&](uint32_t at) {
        if (ahead < p.N) {
            load_ahead<VPT>(base + at, q, p.tpr, p.H, p.h + from);
            load_ahead<VPT>(base + at + VPT * q.plane, q, p.tpr, p.H, p.dy + from);
            if (DH) load_ahead<VPT>(base + at + 2 * VPT * q.plane, q, p.tpr, p.H, p.dh + from);
        }
        cp_commit();
        ahead += step;
        from += stride;
    };
    uint64_t g[VPT][8], dg[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (q.t + j * p.tpr < p.nv) load_gamma_pairs(p.gamma, p.gamma_fp32, (q.t + j * p.tpr) * kVec, g[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[j][i] = 0;
    }
#pragma unroll
    for (int s = 0; s < kDepth - 1; ++s) issue(s * stage_bytes);
    uint32_t at = 0, fill = (kDepth - 1) * stage_bytes;
    int flip = 0;
    float rstd_next = row_first + q.sub < p.N ? p.rstd[row_first + q.sub] : 0.f;
    for (int64_t row0 = row_first; row0 < p.N; row0 += step, flip ^= 1) {
        __syncwarp();  // the slot filled next was read by the whole group
        issue(fill);
        fill = at;
        const int64_t row = row0 + q.sub;
        const bool live = row < p.N;
        const float rstd = rstd_next;
        if (row + step < p.N) rstd_next = p.rstd[row + step];
        cp_wait<kDepth - 1>();
        __syncwarp();  // every lane's copies of this row are done
        const uint64_t rr = f32x2_pack(rstd, rstd);
        uint64_t n[VPT][8], dt[VPT][8], dot = 0;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (live && q.t + j * p.tpr < p.nv) {
                read16(ring + at + j * q.plane, q, n[j]);
                read16(ring + at + (VPT + j) * q.plane, q, dt[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    n[j][i] = f32x2_mul_rn(n[j][i], rr);
                    dg[j][i] = f32x2_fma_rn(dt[j][i], n[j][i], dg[j][i]);
                    dt[j][i] = f32x2_mul_rn(dt[j][i], g[j][i]);
                    dot = f32x2_fma_rn(dt[j][i], n[j][i], dot);
                }
            }
        }
        const float m = -stream_sum(dot, p.tpr, red[flip]) * p.inv_h;
        const uint64_t mm = f32x2_pack(m, m);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int k = q.t + j * p.tpr;
            if (live && k < p.nv) {
                uint64_t o[8];
                if (DH) {
                    read16(ring + at + (2 * VPT + j) * q.plane, q, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = 0;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = f32x2_fma_rn(f32x2_fma_rn(n[j][i], mm, dt[j][i]), rr, o[i]);
                store16(p.dx + row * p.H + k * kVec, o);
            }
        }
        at = at == (kDepth - 1) * stage_bytes ? 0 : at + stage_bytes;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    float* sums = reinterpret_cast<float*>(ring);  // [rpc][H]
    float* out = p.part + (int64_t)blockIdx.x * p.H;
    if (q.rpc > 1) __syncthreads();  // every thread is done with its slots
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int k = q.t + j * p.tpr;
        if (k < p.nv) {
            float4* o = reinterpret_cast<float4*>((q.rpc > 1 ? sums + (int64_t)q.sub * p.H : out) + k * kVec);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = f32x2_unpack(dg[j][2 * i]), b = f32x2_unpack(dg[j][2 * i + 1]);
                o[i] = make_float4(a.x, a.y, b.x, b.y);
            }
        }
    }
    if (q.rpc > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
            float a = sums[c];
            for (int i = 1; i < q.rpc; ++i) a += sums[i * p.H + c];
            out[c] = a;
        }
    }
}

// dgamma[c] = sum of the partial rows, in slot order within each of 32
// strides, then over the strides.
__global__ void __launch_bounds__(1024) dgamma_kernel(const float* part, int slots, int H, float* dgamma) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float a = 0.f;
    for (int i = w; i < slots; i += 32) a += part[(int64_t)i * H + c];
    s[w][lane] = a;
    __syncthreads();
    if (w == 0) {
#pragma unroll
        for (int i = 1; i < 32; ++i) a += s[i][lane];
        dgamma[c] = a;
    }
}

// Threads per row (whole warps) and vectors per thread: one vector each up to
// 512 threads, then two, then four.
void shape_of(int H, int* nv, int* tpr, int* vpt) {
    *nv = H / kVec;
    *vpt = *nv <= 512 ? 1 : *nv <= 2048 ? 2 : 4;
    *tpr = ((*nv + *vpt - 1) / *vpt + 31) / 32 * 32;
}

int rows_per_cta(int tpr) { return tpr >= 256 ? 1 : 256 / tpr; }

// The stream kernels: a power of two of lanes up to a warp, or whole warps.
bool stream_shape(int H, int* nv, int* tpr, int* vpt) {
    if (H > 16384) return false;
    *nv = H / kVec;
    *vpt = *nv <= 512 ? 1 : 2;
    const int n = (*nv + *vpt - 1) / *vpt;
    *tpr = n <= 8 ? 8 : n <= 16 ? 16 : (n + 31) / 32 * 32;
    return true;
}
int stream_rows(int tpr) { return 512 / tpr; }

// Partial dgamma rows of a backward call, at most.
constexpr int64_t kMaxSlots = 592;

// A stream kernel runs from this many row groups on.
constexpr int64_t kStreamRows = 592;

int64_t bwd_slots(int64_t N) { return N < kMaxSlots ? N : kMaxSlots; }

constexpr int kMaxStreamSmem = 226 * 1024;  // beside the reduction's static 256 bytes

// CTAs of a stream kernel that the current device holds at once (per SM, on its
// SMs). Sets the kernel's shared-memory limit. The host thread's last counts
// are kept, since asking takes longer than the launch; the limit is set by every
// call, always to the same value: a reset of the device forgets it. On an error
// the call fails: another kernel in its place would add up in another order, and
// the same call would not give the same bits.
ep_status_t resident(const void* kernel, int threads, int smem, int* per, int* sms) {
    struct Known {
        const void* kernel;
        int threads, smem, dev, per, sms;
    };
    static thread_local Known known{};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxStreamSmem);
    if (e == cudaSuccess &&
        (known.kernel != kernel || known.threads != threads || known.smem != smem || known.dev != dev)) {
        known.kernel = nullptr;
        e = cudaDeviceGetAttribute(&known.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&known.per, kernel, threads, smem);
        if (e == cudaSuccess) known = {kernel, threads, smem, dev, known.per, known.sms};
    }
    if (e == cudaSuccess && known.per < 1) e = cudaErrorInvalidConfiguration;
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(EP_ERR_CUDA, "resident CTAs of the norm's kernel: %s", cudaGetErrorString(e));
    }
    *per = known.per;
    *sms = known.sms;
    return EP_OK;
}

ep_status_t check_shape(int64_t N, int H, int gamma_type) {
    if (N < 0) return fail(EP_ERR_INVALID, "N must be >= 0");
    if (H < 128 || H % 128 != 0 || H > 65536)
        return fail(EP_ERR_UNSUPPORTED, "H must be a multiple of 128 in [128, 65536]");
    if (N > ((int64_t)1 << 31) - 1) return fail(EP_ERR_UNSUPPORTED, "N must be < 2^31");
    if (gamma_type != EP_DTYPE_BF16 && gamma_type != EP_DTYPE_FP32)
        return fail(EP_ERR_INVALID, "gamma_type must be EP_DTYPE_BF16 or EP_DTYPE_FP32");
    return EP_OK;
}

bool misaligned(const void* p, unsigned n) { return (uintptr_t)p % n != 0; }

ep_status_t launched(const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    set_last_error("");
    return EP_OK;
}

}  // namespace
}  // namespace ep

extern "C" {

ep_status_t ep_rmsnorm(int64_t N, int H, const void* d_x, const void* d_residual, const void* d_gamma, int gamma_type,
                       float eps, void* d_h, void* d_y, void* d_q, float* d_q_scale, float* d_rstd, void* stream) {
    using namespace ep;
    if (ep_status_t st = check_shape(N, H, gamma_type)) return st;
    if (!(eps > 0.f)) return fail(EP_ERR_INVALID, "eps must be > 0");
    if ((d_q == nullptr) != (d_q_scale == nullptr)) return fail(EP_ERR_INVALID, "d_q and d_q_scale go together");
    if (N > 0 && !d_h && !d_y && !d_q && !d_rstd) return fail(EP_ERR_INVALID, "no output is given");
    if (N > 0 && d_y && d_y == d_h) return fail(EP_ERR_INVALID, "d_h and d_y are the same array");
    if (N > 0 && (!d_x || !d_gamma)) return fail(EP_ERR_INVALID, "d_x and d_gamma must be non-NULL");
    if (misaligned(d_x, 32) || misaligned(d_residual, 32) || misaligned(d_gamma, 32) || misaligned(d_h, 32) ||
        misaligned(d_y, 32))
        return fail(EP_ERR_INVALID, "d_x, d_residual, d_gamma, d_h and d_y must be 32-byte aligned");
    if (misaligned(d_q, 16)) return fail(EP_ERR_INVALID, "d_q must be 16-byte aligned");
    if (misaligned(d_q_scale, 4) || misaligned(d_rstd, 4))
        return fail(EP_ERR_INVALID, "d_q_scale and d_rstd must be 4-byte aligned");
    set_last_error("");
    if (N == 0) return EP_OK;
    NormParams p{};
    int vpt;
    shape_of(H, &p.nv, &p.tpr, &vpt);
    p.N = N;
    p.H = H;
    p.x = static_cast<const uint16_t*>(d_x);
    p.res = static_cast<const uint16_t*>(d_residual);
    p.gamma = d_gamma;
    p.gamma_fp32 = gamma_type == EP_DTYPE_FP32;
    p.eps = eps;
    p.inv_h = 1.0f / (float)H;
    p.h = static_cast<uint16_t*>(d_h);
    p.y = static_cast<uint16_t*>(d_y);
    p.q = static_cast<uint8_t*>(d_q);
    p.q_scale = d_q_scale;
    p.rstd = d_rstd;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    NormParams ps = p;
    int svpt;
    if (stream_shape(H, &ps.nv, &ps.tpr, &svpt)) {
        const int rps = stream_rows(ps.tpr), threads = rps * ps.tpr;
        const int arrays = ps.res ? 2 : 1, smem = depth_of(svpt, arrays) * arrays * svpt * threads * 32;
        const auto kernel = svpt == 1 ? (ps.res ? rmsnorm_stream_kernel<1, true> : rmsnorm_stream_kernel<1, false>)
                                      : (ps.res ? rmsnorm_stream_kernel<2, true> : rmsnorm_stream_kernel<2, false>);
        const int64_t groups = (N + rps - 1) / rps;
        if (groups >= kStreamRows) {
            int per = 0, sms = 0;
            if (ep_status_t st = resident((const void*)kernel, threads, smem, &per, &sms)) return st;
            int ctas = per * sms;
            // HBM bounds a stream with a residual, and one CTA per SM then reads
            // and writes faster than two (32768 x 7168: 6.44 against 5.57 TB/s);
            // instructions bound one without (153 against 185 us), and the
            // reduction's latency a few rows per SM.
            if (per > 1 && ps.res && groups >= 16 * sms) ctas = sms;
            kernel<<<(unsigned)(groups < ctas ? groups : ctas), threads, smem, s>>>(ps);
            return launched("rmsnorm");
        }
    }
    const int rpc = rows_per_cta(p.tpr);
    const unsigned grid = (unsigned)((N + rpc - 1) / rpc);
    if (vpt == 1) rmsnorm_kernel<1><<<grid, p.tpr * rpc, 0, s>>>(p);
    else if (vpt == 2) rmsnorm_kernel<2><<<grid, p.tpr * rpc, 0, s>>>(p);
    else rmsnorm_kernel<4><<<grid, p.tpr * rpc, 0, s>>>(p);
    return launched("rmsnorm");
}

ep_status_t ep_rmsnorm_backward_workspace_bytes(int64_t N, int H, size_t* bytes) {
    using namespace ep;
    if (ep_status_t st = check_shape(N, H, EP_DTYPE_BF16)) return st;
    if (!bytes) return fail(EP_ERR_INVALID, "bytes is NULL");
    *bytes = (size_t)(N > 0 ? bwd_slots(N) : 1) * H * sizeof(float);
    set_last_error("");
    return EP_OK;
}

ep_status_t ep_rmsnorm_backward(int64_t N, int H, const void* d_h, const float* d_rstd, const void* d_gamma,
                                int gamma_type, const void* d_dy, const void* d_dh, void* d_dx, float* d_dgamma,
                                void* d_workspace, size_t workspace_bytes, void* stream) {
    using namespace ep;
    if (ep_status_t st = check_shape(N, H, gamma_type)) return st;
    if (!d_dgamma) return fail(EP_ERR_INVALID, "d_dgamma must be non-NULL");
    if (N > 0 && (!d_h || !d_rstd || !d_gamma || !d_dy || !d_dx))
        return fail(EP_ERR_INVALID, "d_h, d_rstd, d_gamma, d_dy and d_dx must be non-NULL");
    if (misaligned(d_h, 32) || misaligned(d_gamma, 32) || misaligned(d_dy, 32) || misaligned(d_dh, 32) ||
        misaligned(d_dx, 32))
        return fail(EP_ERR_INVALID, "d_h, d_gamma, d_dy, d_dh and d_dx must be 32-byte aligned");
    if (misaligned(d_rstd, 4) || misaligned(d_dgamma, 4))
        return fail(EP_ERR_INVALID, "d_rstd and d_dgamma must be 4-byte aligned");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) {
        const cudaError_t e = cudaMemsetAsync(d_dgamma, 0, (size_t)H * sizeof(float), s);
        if (e != cudaSuccess) return fail(EP_ERR_CUDA, "memset: %s", cudaGetErrorString(e));
        set_last_error("");
        return EP_OK;
    }
    size_t need = 0;
    if (ep_status_t st = ep_rmsnorm_backward_workspace_bytes(N, H, &need)) return st;
    if (!d_workspace || misaligned(d_workspace, 256))
        return fail(EP_ERR_INVALID, "d_workspace must be non-NULL and 256-byte aligned");
    if (workspace_bytes < need)
        return fail(EP_ERR_OOM, "workspace has %zu bytes, the call needs %zu", workspace_bytes, need);
    NormBwdParams p{};
    int vpt;
    shape_of(H, &p.nv, &p.tpr, &vpt);
    p.N = N;
    p.H = H;
    p.h = static_cast<const uint16_t*>(d_h);
    p.rstd = d_rstd;
    p.gamma = d_gamma;
    p.gamma_fp32 = gamma_type == EP_DTYPE_FP32;
    p.inv_h = 1.0f / (float)H;
    p.dy = static_cast<const uint16_t*>(d_dy);
    p.dh = static_cast<const uint16_t*>(d_dh);
    p.dx = static_cast<uint16_t*>(d_dx);
    p.part = static_cast<float*>(d_workspace);
    NormBwdParams ps = p;
    int svpt;
    if (stream_shape(H, &ps.nv, &ps.tpr, &svpt)) {
        const int rps = stream_rows(ps.tpr), threads = rps * ps.tpr;
        const int arrays = ps.dh ? 3 : 2, smem = depth_of(svpt, arrays) * arrays * svpt * threads * 32;
        const auto kernel =
            svpt == 1 ? (ps.dh ? rmsnorm_bwd_stream_kernel<1, true> : rmsnorm_bwd_stream_kernel<1, false>)
                      : (ps.dh ? rmsnorm_bwd_stream_kernel<2, true> : rmsnorm_bwd_stream_kernel<2, false>);
        const int64_t groups = (N + rps - 1) / rps;
        int per = 0, sms = 0;
        if (ep_status_t st = resident((const void*)kernel, threads, smem, &per, &sms)) return st;
        int64_t ctas = (int64_t)per * sms;
        const int64_t rows = bwd_slots(N);  // what the workspace holds
        if (ctas > rows) ctas = rows;
        if (groups < ctas) ctas = groups;
        kernel<<<(unsigned)ctas, threads, smem, s>>>(ps);
        if (ep_status_t st = launched("rmsnorm backward")) return st;
        dgamma_kernel<<<H / 32, 1024, 0, s>>>(p.part, (int)ctas, H, d_dgamma);
        return launched("dgamma");
    }
    const int slots = (int)bwd_slots(N);
    if (vpt == 2) rmsnorm_bwd_kernel<2><<<slots, p.tpr, 0, s>>>(p);
    else rmsnorm_bwd_kernel<4><<<slots, p.tpr, 0, s>>>(p);
    if (ep_status_t st = launched("rmsnorm backward")) return st;
    dgamma_kernel<<<H / 32, 1024, 0, s>>>(p.part, slots, H, d_dgamma);
    return launched("dgamma");
}

}  // extern "C"
