// What the kernels of ep_linear and ep_expert_linear share: parameters, the walk
// over the groups' tiles, the epilogue's arithmetic.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "ep.h"
#include "tcgen05.cuh"

namespace ep {
namespace linear {


struct LinearParams {
    const void* x;
    const float* x_scale;
    const void* w;
    const float* w_scale;
    const float* bias;
    const uint16_t* res;
    void* out;
    float* out_scale;
    int K, N, wide, parts;  // in_features, out_features, rows per weight matrix, wide / N
    int act, out_type;
    // groups of rows: group g holds rows [start, start + count)
    int G;                 // groups
    int R;                 // groups per weight matrix
    const int32_t* off;    // [G + 1], or NULL
    const int32_t* cnt;    // low latency: cnt[(g % R) * (G / R) + g / R] rows from g * region
    int64_t region;
    int64_t rows;          // dense: the one group's rows
    int64_t row_limit;     // rows the arrays hold
    uint32_t* err;
    // shape of the launch
    int bn;        // rows of x per tile: 32, 64 or 128; 256 with pairs of CTAs
    int na;        // 128-channel weight tiles per CTA tile: gate and up, or neighbours
    int nt;        // channel tiles: out_features over 128 (swiglu) or 128 * na
    int stages;    // of the shared-memory ring
    int kblocks;   // 128-byte blocks of in_features
    int splits;    // CTAs of a cluster that share a tile's in_features
    int flush;     // blocks summed in tensor memory at a time
    int acc_log;   // log2 of the accumulator sets
    uint32_t cols; // tensor-memory columns
    int vec;       // rows of out and residual allow 4-channel accesses
};

// Rows [start, start + count) of group g; none, and an error bit, where they
// leave [0, row_limit).
__device__ __forceinline__ void group_rows(const LinearParams& p, int g, int64_t& start, int& count) {
    int64_t n;
    if (p.off) {
        start = p.off[g];
        n = p.off[g + 1] - start;
    } else if (p.cnt) {
        start = (int64_t)g * p.region;
        n = min((int64_t)p.cnt[(int64_t)(g % p.R) * (p.G / p.R) + g / p.R], p.region);
    } else {
        start = 0;
        n = p.rows;
    }
    if (n > 0 && (start < 0 || start + n > p.row_limit)) {
        set_error(p.err, EP_DEVERR_ROW_BOUNDS);
        n = 0;
    }
    count = (int)max(n, (int64_t)0);
}

__device__ __forceinline__ float activate(int act, float z) {
    if (act == EP_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));
    if (act == EP_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    return z;
}


constexpr int kEpiWarps = 8;
// Three warpgroups: two of the epilogue, one of loads, products, e4m3 scales
// and an idle warp. The launch gives each thread 168 registers; the epilogue's
// fp32 sums need more: 2 * 128 * 216 + 128 * 72 = 384 * 168.
constexpr int kThreads = 384;
constexpr int kEpiRegs = 216, kOtherRegs = 72;
static_assert(2 * 128 * kEpiRegs + 128 * kOtherRegs == kThreads * 168, "register split");
constexpr int kSub = 128 * 128;                 // bytes of a 128-channel weight tile of one stage
constexpr int kMaxStages = 10;
// Shared memory: ring | staging, or inboxes | barriers and scales.
constexpr int kStaging = 32 * 256 * 4;
constexpr int kInbox = 2 * 36 * 256 * 4;        // a cluster's: 2 x at most 36 rows (splits x rows of each)
constexpr int kMaxAcc = 8;                      // accumulator sets in tensor memory
constexpr int kScales = 512 * 4;                // [sets][2][bn]: sets * bn is at most 256
constexpr int kControl = 512 + kScales;
constexpr int kSmemMax = 227 * 1024;

__host__ __device__ constexpr int stage_bytes(int na, int bn) { return na * kSub + bn * 128; }

constexpr int64_t kMaxTiles = (int64_t)1 << 30;

// Walks the tiles of all groups in order: a group's channel tiles, and within
// one the row tiles, so that CTAs running together share weights through L2.
// One warp holds 32 groups at a time.
struct Cursor {
    int g0 = -32;
    int base = 0, total = 0;  // tiles before the window, and in it
    int incl = 0, mine = 0;   // of the lane's group: tiles up to and with it, its own
    int64_t start = 0;
    int count = 0;
};
struct Tile {
    int group, n;          // group, channel tile
    int64_t row;           // first row of x
    int rows;              // valid rows, at most bn
};

// Tiles of bn rows that `count` rows take; count + bn - 1 may not fit 31 bits.
__device__ __forceinline__ int row_tiles(int count, int bn) { return count > 0 ? (count - 1) / bn + 1 : 0; }

__device__ __forceinline__ bool find_tile(const LinearParams& p, Cursor& c, int id, Tile& t) {
    const int lane = threadIdx.x & 31;
    while (id >= c.base + c.total) {
        c.base += c.total;
        c.g0 += 32;
        if (c.g0 >= p.G) return false;
        c.start = 0;
        c.count = 0;
        if (c.g0 + lane < p.G) group_rows(p, c.g0 + lane, c.start, c.count);
        int64_t incl = (int64_t)row_tiles(c.count, p.bn) * p.nt;
        c.mine = (int)incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += v;
        }
        c.incl = (int)incl;
        const int64_t total = __shfl_sync(FULL, incl, 31);
        c.total = (int)total;
        // Rows that overlap can give more tiles than the host allowed for.
        if (c.base + total > kMaxTiles) {
            set_error(p.err, EP_DEVERR_ROW_BOUNDS);
            return false;
        }
    }
    const int in_window = id - c.base;
    const int src = __ffs(__ballot_sync(FULL, in_window < c.incl)) - 1;
    const int at = in_window - (__shfl_sync(FULL, c.incl, src) - __shfl_sync(FULL, c.mine, src));
    const int count = __shfl_sync(FULL, c.count, src);
    const int64_t start = __shfl_sync(FULL, c.start, src);
    const int tt = row_tiles(count, p.bn);
    t.group = c.g0 + src;
    t.n = at / tt;
    const int r = (at - t.n * tt) * p.bn;
    t.row = start + r;
    t.rows = min(p.bn, count - r);
    return true;
}

// Weight tiles of a CTA tile that hold channels.
__device__ __forceinline__ int subs_of(const LinearParams& p, const Tile& t) {
    if (p.parts == 2) return 2;
    return p.na == 2 && (t.n * 2 + 1) * 128 < p.N ? 2 : 1;
}
// First channel of sub-tile `sub` within its half.
__device__ __forceinline__ int channel_of(const LinearParams& p, const Tile& t, int sub) {
    return p.parts == 2 ? t.n * 128 : (t.n * p.na + sub) * 128;
}

struct Bias {
    float v[2][4];
};
__device__ __forceinline__ void load_bias(const LinearParams& p, const Tile& t, int subs, Bias& b) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b.v[s][i] = 0.f;
            const int n = channel_of(p, t, s) + lane * 4 + i;
            if (p.bias && s < subs && n < p.N)
                b.v[s][i] = p.bias[(int64_t)(t.group / p.R) * p.wide + (p.parts == 2 ? s * p.N : 0) + n];
        }
}

__device__ __forceinline__ void activate4(int act, float (&z)[4]) {
    if (act == EP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = activate(EP_ACT_SILU, z[i]);
    } else if (act == EP_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = activate(EP_ACT_GELU, z[i]);
    }
}

// Four channels of a row, rounded and stored at `at`; e4m3: the warp holds a
// block of 128, whose scale goes to *scale.
template <int OUT>
__device__ __forceinline__ void store4(const LinearParams& p, int64_t at, const float (&z)[4], float* scale) {
    if (OUT == EP_DTYPE_E4M3) {
        float amax = fmaxf(fmaxf(fabsf(z[0]), fabsf(z[1])), fmaxf(fabsf(z[2]), fabsf(z[3])));
        amax = fmaxf(amax, 1e-4f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, o));
        const float s = 448.0f / amax;
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + at) =
            pack_e4m3x2(z[0] * s, z[1] * s) | pack_e4m3x2(z[2] * s, z[3] * s) << 16;
        if ((threadIdx.x & 31) == 0) *scale = amax / 448.0f;
    } else if (OUT == EP_DTYPE_FP32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(z[0], z[1], z[2], z[3]);
    } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
            make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
    }
}
__device__ __forceinline__ void add_residual(const LinearParams& p, int64_t at, float (&z)[4]) {
    const uint2 r = *reinterpret_cast<const uint2*>(p.res + at);
    z[0] += bf16lo(r.x);
    z[1] += bf16hi(r.x);
    z[2] += bf16lo(r.y);
    z[3] += bf16hi(r.y);
}

// Staged rows i = first, first + kEpiWarps, ... < own, which are rows
// row + (i - first) * gap of the output, 4 channels of each tile to a lane:
// gate and up of 128 channels, or one or two neighbouring tiles. load(i, s)
// gives the lane's 4 sums of row i, tile s. What is the same for all rows is
// settled outside the loop (choosing per row took half of the epilogue). VEC:
// rows of out and residual allow 4-channel accesses (out_features % 4 == 0).
template <int OUT, bool GATED, bool VEC, typename Load>
__device__ __forceinline__ void emit_rows(const LinearParams& p, const Tile& t, int subs, const Bias& b, int first, int own,
                                          int64_t row, int gap, Load load) {
    const int lane4 = (threadIdx.x & 31) * 4;
    const int n0 = channel_of(p, t, 0) + lane4, n1 = channel_of(p, t, 1) + lane4;
    const bool two = !GATED && subs == 2, on0 = n0 < p.N, on1 = two && n1 < p.N;
    int64_t at = row * p.N;
    const int64_t stride = (int64_t)gap * kEpiWarps * p.N;
    const int blocks = p.N / 128;
    float* scale = OUT == EP_DTYPE_E4M3 ? p.out_scale + row * blocks + channel_of(p, t, 0) / 128 : nullptr;
#pragma unroll 1
    for (int i = first; i < own; i += kEpiWarps, at += stride) {
        const float4 v = load(i, 0), w = GATED || two ? load(i, 1) : make_float4(0.f, 0.f, 0.f, 0.f);
        float z[4] = {v.x + b.v[0][0], v.y + b.v[0][1], v.z + b.v[0][2], v.w + b.v[0][3]};
        float u[4] = {w.x + b.v[1][0], w.y + b.v[1][1], w.z + b.v[1][2], w.w + b.v[1][3]};
        if (GATED) {
#pragma unroll
            for (int k = 0; k < 4; ++k) z[k] = activate(EP_ACT_SILU, z[k]) * u[k];
        } else {
            activate4(p.act, z);
            if (two) activate4(p.act, u);
        }
        if (VEC) {
            if (p.res) {
                if (on0) add_residual(p, at + n0, z);
                if (on1) add_residual(p, at + n1, u);
            }
            // e4m3: out_features is a multiple of 128, so on0 and on1 hold for whole warps
            if (on0) store4<OUT>(p, at + n0, z, scale);
            if (on1) store4<OUT>(p, at + n1, u, scale + 1);
            if (OUT == EP_DTYPE_E4M3) scale += (int64_t)gap * kEpiWarps * blocks;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int n = (s ? n1 : n0) + k;
                    if (n >= p.N || (s && !two)) continue;
                    float y = s ? u[k] : z[k];
                    if (p.res) y += __uint_as_float((uint32_t)p.res[at + n] << 16);
                    if (OUT == EP_DTYPE_FP32) static_cast<float*>(p.out)[at + n] = y;
                    else static_cast<uint16_t*>(p.out)[at + n] = (uint16_t)(pack_bf16x2(y, 0.f) & 0xffff);
                }
            }
        }
    }
}

template <typename Load>
__device__ __forceinline__ void emit_chunk(const LinearParams& p, const Tile& t, int subs, const Bias& b, int first, int own,
                                           int64_t row, int gap, Load load) {
    const bool gated = p.parts == 2;
    auto as = [&](auto out) {
        constexpr int OUT = decltype(out)::value;
        if (OUT == EP_DTYPE_E4M3 || p.vec) {
            if (gated) emit_rows<OUT, true, true>(p, t, subs, b, first, own, row, gap, load);
            else emit_rows<OUT, false, true>(p, t, subs, b, first, own, row, gap, load);
        } else {
            if (gated) emit_rows<OUT, true, false>(p, t, subs, b, first, own, row, gap, load);
            else emit_rows<OUT, false, false>(p, t, subs, b, first, own, row, gap, load);
        }
    };
    if (p.out_type == EP_DTYPE_BF16) as(std::integral_constant<int, EP_DTYPE_BF16>());
    else if (p.out_type == EP_DTYPE_FP32) as(std::integral_constant<int, EP_DTYPE_FP32>());
    else as(std::integral_constant<int, EP_DTYPE_E4M3>());
}

// Barrier of the epilogue warps; the _and form tells whether all of them are ok.
__device__ __forceinline__ bool epi_sync_and(bool ok) {
    uint32_t r;
    asm volatile(
        "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.and.pred q, 1, %2, p; selp.u32 %0, 1, 0, q; }"
        : "=r"(r)
        : "r"((uint32_t)ok), "n"(kEpiWarps * 32)
        : "memory");
    return r != 0;
}
// Every warp of the CTA is through with its tiles: from here on the stop flag
// is final. (A barrier of its own, as the warps come to it from two branches:
// with one after both, what drains needs stayed in the epilogue's registers, and
// an e4m3 layer of 4096 x 8192 -> 8192 took 406 us instead of 394.)
__device__ __forceinline__ void all_done() { asm volatile("bar.sync 6, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory"); }

// Pairs of CTAs.
constexpr int kPairEpiRegs = 224, kPairOtherRegs = 56;  // as kEpiRegs and kOtherRegs: no e4m3 scales warp here
static_assert(2 * 128 * kPairEpiRegs + 128 * kPairOtherRegs == kThreads * 168, "register split");
constexpr int kPairStage = 2 * kSub;
constexpr int kPairStages = 7;
constexpr int kPairSmem = kPairStages * kPairStage + 256 + 2 * 128 * 4 + 1024;
static_assert(kPairSmem <= kSmemMax, "shared memory");

using Kernel = void (*)(CUtensorMap, CUtensorMap, LinearParams);
// The kernel for tiles of bn rows (32, 64, 128; 256: pairs of CTAs, whose sums
// leave tensor memory in parts or whole), for bf16 and for e4m3 operands.
Kernel bf16_kernel(bool pair, bool split, int bn, bool parts);
Kernel e4m3_kernel(bool pair, bool split, int bn);

}  // namespace linear
}  // namespace ep
