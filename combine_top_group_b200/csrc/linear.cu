// ep_linear and ep_expert_linear: out = act(x W^T + bias) + residual on dense
// rows or on the experts' receive rows, bf16 or e4m3 with scales.
//
// The product is taken as W x^T: output channels are the 128 lanes of a
// tensor-memory tile, rows of x its columns. Experts get any number of rows,
// and the column count of a tcgen05 product can be any multiple of 16, so a
// ragged last tile costs only its own columns, and a decode batch of a few
// rows per expert wastes no lanes. Rows of W are never ragged across experts.
//
// One persistent CTA per SM: a warp loads tiles with TMA into a ring of shared
// memory stages, a warp issues the products, eight warps read finished
// accumulators out of tensor memory, where a second set fills meanwhile.
//  - e4m3: each block of 128 channels is summed on its own in tensor memory
//    and leaves it times its scales (row scale x weight block scale, fp32)
//    into fp32 registers, since the scales differ from block to block.
//  - bf16: the whole sum, or for fp32 and e4m3 outputs every 8 blocks of 64
//    channels, leaves tensor memory the same way. Sums there lose about 1.5e-8
//    of their size with each step of 16 channels (they are cut, not rounded:
//    7e-6 over 7168 channels). That is nothing beside a bf16 output's 2^-8; 32
//    steps keep it below the roundings of an fp32 sum of that length (4.8e-7
//    measured for 512 to 7168 channels), at the price of 8 to 20% of the time.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "ep.h"
#include "internal.h"
#include "tcgen05.cuh"

namespace ep {
namespace {

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
    int bn;        // rows of x per tile: 32, 64 or 128
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

// Rows [start, start + count) of group g, kept inside [0, row_limit).
__device__ __forceinline__ void group_rows(const LinearParams& p, int g, int64_t& start, int& count) {
    if (p.off) {
        start = p.off[g];
        count = p.off[g + 1] - (int)start;
    } else if (p.cnt) {
        start = (int64_t)g * p.region;
        count = min(p.cnt[(int64_t)(g % p.R) * (p.G / p.R) + g / p.R], (int)p.region);
    } else {
        start = 0;
        count = (int)p.rows;
    }
    if (start < 0 || count <= 0 || start + count > p.row_limit) count = 0;
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
constexpr int kScales = 1024 * 4;               // [sets][2][bn]
constexpr int kControl = 512 + kScales;
constexpr int kSmemMax = 227 * 1024;

__host__ __device__ constexpr int stage_bytes(int na, int bn) { return na * kSub + bn * 128; }

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

__device__ __forceinline__ bool find_tile(const LinearParams& p, Cursor& c, int id, Tile& t) {
    const int lane = threadIdx.x & 31;
    while (id >= c.base + c.total) {
        c.base += c.total;
        c.g0 += 32;
        if (c.g0 >= p.G) return false;
        c.start = 0;
        c.count = 0;
        if (c.g0 + lane < p.G) group_rows(p, c.g0 + lane, c.start, c.count);
        c.mine = (c.count + p.bn - 1) / p.bn * p.nt;
        c.incl = c.mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL, c.incl, o);
            if (lane >= o) c.incl += v;
        }
        c.total = __shfl_sync(FULL, c.incl, 31);
    }
    const int in_window = id - c.base;
    const int src = __ffs(__ballot_sync(FULL, in_window < c.incl)) - 1;
    const int at = in_window - (__shfl_sync(FULL, c.incl, src) - __shfl_sync(FULL, c.mine, src));
    const int count = __shfl_sync(FULL, c.count, src);
    const int64_t start = __shfl_sync(FULL, c.start, src);
    const int tt = (count + p.bn - 1) / p.bn;
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
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory"); }

// BN: rows of x per tile (p.bn).
template <bool F8, bool SPLIT, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, LinearParams p) {
    extern __shared__ uint8_t smem_raw[];
    const int sb = stage_bytes(p.na, BN);
    // swizzled tiles start on 1024 bytes (the same offset in every CTA of a cluster)
    const uint32_t ring = (tc::smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t* smem = smem_raw + (ring - tc::smem_u32(smem_raw));
    uint8_t* after = smem + (size_t)p.stages * sb;
    float* staging = reinterpret_cast<float*>(after);
    uint8_t* control = after + (SPLIT ? kInbox : kStaging);
    float* scales = reinterpret_cast<float*>(control + 512);  // [sets][2][bn]
    volatile uint32_t* stop = reinterpret_cast<uint32_t*>(control + 500);
    const uint32_t bars = tc::smem_u32(control);
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (kMaxStages + s); };
    auto acc_full = [&](int s) { return bars + 8 * (2 * kMaxStages + s); };
    auto acc_empty = [&](int s) { return bars + 8 * (2 * kMaxStages + kMaxAcc + s); };
    auto scale_full = [&](int s) { return bars + 8 * (2 * kMaxStages + 2 * kMaxAcc + s); };
    const uint32_t drained = bars + 8 * (2 * kMaxStages + 3 * kMaxAcc);
    auto inbox_full = [&](int b) { return drained + 8 + 8 * b; };
    auto inbox_free = [&](int b) { return drained + 24 + 8 * b; };
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(control + 496);
    const int sets = 1 << p.acc_log;
    // set of the acc-th use, the parity of that use's phase, and of the one before it
    auto set_of = [&](int acc) { return acc & (sets - 1); };
    auto phase_of = [&](int acc) { return (uint32_t)(acc >> p.acc_log) & 1; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            tc::bar_init(full(s), 1);
            tc::bar_init(empty(s), 1);
        }
        for (int s = 0; s < sets; ++s) {
            tc::bar_init(acc_full(s), 1);
            tc::bar_init(acc_empty(s), kEpiWarps);
            tc::bar_init(scale_full(s), 32);
        }
        tc::bar_init(drained, 1);
        for (int b = 0; b < 2; ++b) {
            tc::bar_init(inbox_full(b), 1);
            tc::bar_init(inbox_free(b), p.splits);
        }
        *stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kEpiWarps + 1) tc::tmem_alloc(tc::smem_u32(tmem_at), p.cols);
    tc::fence_before();
    __syncthreads();
    if (SPLIT) tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = *tmem_at;

    // the CTAs of a cluster take the same tiles, each its part of in_features
    const int rank = SPLIT ? (int)tc::cluster_rank() : 0;
    const int first = SPLIT ? blockIdx.x / p.splits : blockIdx.x;
    const int step = SPLIT ? gridDim.x / p.splits : gridDim.x;
    const int k_lo = SPLIT ? (int)((int64_t)p.kblocks * rank / p.splits) : 0;
    const int k_hi = SPLIT ? (int)((int64_t)p.kblocks * (rank + 1) / p.splits) : p.kblocks;
    constexpr int kElems = F8 ? 128 : 64;  // in_features of a block
    Cursor cur;
    Tile t;

    // The loads and products warps run their loops whole and converged; one
    // elected lane issues.
    if (warp == kEpiWarps) {  // loads
        tc::fewer_registers<kOtherRegs>();
        int i = 0, s = 0;
        uint32_t wrap = 0;
        bool ok = true;
        for (int id = first; ok && find_tile(p, cur, id, t); id += step) {
            const int subs = subs_of(p, t);
            const uint32_t bytes = subs * kSub + BN * 128;
            for (int k = k_lo; k < k_hi; ++k, ++i) {
                if (wrap > 0) ok = __all_sync(FULL, tc::bar_wait(empty(s), (wrap - 1) & 1, stop));
                if (!ok) break;
                if (tc::elect()) {
                    const uint32_t at = ring + s * sb;
                    tc::bar_expect(full(s), bytes);
                    tc::tma_4d(at, &map_w, full(s), k * kElems, channel_of(p, t, 0), 0, t.group / p.R);
                    if (subs == 2)
                        tc::tma_4d(at + kSub, &map_w, full(s), k * kElems, channel_of(p, t, 1), p.parts == 2 ? 1 : 0,
                                   t.group / p.R);
                    tc::tma_2d(at + p.na * kSub, &map_x, full(s), k * kElems, (int)t.row);
                }
                __syncwarp();
                if (++s == p.stages) {
                    s = 0;
                    ++wrap;
                }
            }
            if (!ok && lane == 0)  // copies in flight land before the CTA leaves
                for (int j = i > p.stages ? i - p.stages : 0; j < i; ++j)
                    tc::bar_drain(full(j % p.stages), (j / p.stages) & 1);
        }
    } else if (warp == kEpiWarps + 1) {  // products
        tc::fewer_registers<kOtherRegs>();
        int s = 0, acc = 0;
        uint32_t wrap = 0;
        bool ok = true;
        for (int id = first; ok && find_tile(p, cur, id, t); id += step) {
            const int subs = subs_of(p, t);
            const uint32_t idesc = tc::instr_desc(F8, 128, (t.rows + 15) / 16 * 16);
            int in_set = 0;  // blocks summed in this set so far
            for (int k = k_lo; k < k_hi; ++k) {
                if (in_set == 0 && acc >= sets)
                    ok = __all_sync(FULL, tc::bar_wait(acc_empty(set_of(acc)), phase_of(acc) ^ 1, stop));
                if (ok) ok = __all_sync(FULL, tc::bar_wait(full(s), wrap & 1, stop));
                if (!ok) break;
                tc::fence_after();
                const uint32_t at = ring + s * sb;
                const uint64_t b = tc::smem_desc(at + p.na * kSub), w = tc::smem_desc(at);
                const uint32_t d = tmem + set_of(acc) * p.na * BN;
                const uint32_t keep = in_set > 0 ? 1u : 0u;
                const bool last = F8 || in_set == p.flush - 1 || k == k_hi - 1;
                if (tc::elect()) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)  // 32 bytes of K each
                        tc::mma<F8>(d, w + 2 * q, b + 2 * q, idesc, q > 0 ? 1u : keep);
                    if (subs == 2) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tc::mma<F8>(d + BN, w + kSub / 16 + 2 * q, b + 2 * q, idesc, q > 0 ? 1u : keep);
                    }
                    tc::commit(empty(s));
                    if (last) tc::commit(acc_full(set_of(acc)));
                }
                __syncwarp();
                acc += last;
                    in_set = last ? 0 : in_set + 1;
                if (++s == p.stages) {
                    s = 0;
                    ++wrap;
                }
            }
            if (!ok) {  // products in flight end before the CTA leaves
                if (tc::elect()) tc::commit(drained);
                tc::bar_drain(drained, 0);
            }
        }
    } else if (warp == kEpiWarps + 2) {  // e4m3: row scale x weight block scale of each block and column
        tc::fewer_registers<kOtherRegs>();
        if (F8) {
            int acc = 0;
            bool ok = true;
            const int nb = (p.N + 127) / 128;
            for (int id = first; ok && find_tile(p, cur, id, t); id += step) {
                const int subs = subs_of(p, t);
                const float* ws[2];
#pragma unroll
                for (int a = 0; a < 2; ++a)
                    ws[a] = p.w_scale + ((int64_t)(t.group / p.R * p.parts + (p.parts == 2 ? a : 0)) * nb +
                                         min(channel_of(p, t, a) / 128, nb - 1)) * p.kblocks;
                // four blocks at a time, loaded four ahead: one load per block
                // would hold each block up by its latency
                float xn[BN / 32][4], wn[2][4];
                auto fetch = [&](int k) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const bool in = k + q < k_hi;
                        wn[0][q] = in ? ws[0][k + q] : 0.f;
                        wn[1][q] = in && subs == 2 ? ws[1][k + q] : 0.f;
#pragma unroll
                        for (int j = 0; j < BN / 32; ++j)
                            xn[j][q] = in && lane + 32 * j < t.rows
                                           ? p.x_scale[(t.row + lane + 32 * j) * p.kblocks + k + q] : 0.f;
                    }
                };
                fetch(k_lo);
#pragma unroll 1
                for (int k = k_lo; ok && k < k_hi; k += 4) {
                    float x4[BN / 32][4], w4[2][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        w4[0][q] = wn[0][q];
                        w4[1][q] = wn[1][q];
#pragma unroll
                        for (int j = 0; j < BN / 32; ++j) x4[j][q] = xn[j][q];
                    }
                    fetch(k + 4);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (!ok || k + q >= k_hi) continue;
                        if (acc >= sets) ok = __all_sync(FULL, tc::bar_wait(acc_empty(set_of(acc)), phase_of(acc) ^ 1, stop));
                        if (!ok) continue;
                        float* dst = scales + set_of(acc) * 2 * BN;
#pragma unroll
                        for (int j = 0; j < BN / 32; ++j)
                            if (32 * j < BN) {
                                dst[lane + 32 * j] = x4[j][q] * w4[0][q];
                                dst[BN + lane + 32 * j] = x4[j][q] * w4[1][q];
                            }
                        tc::bar_arrive(scale_full(set_of(acc)));
                        ++acc;
                    }
                }
            }
        }
    } else if (warp < kEpiWarps) {  // epilogue: warps 0-3 read sub-tile 0, warps 4-7 sub-tile 1
        tc::more_registers<kEpiRegs>();
        const int sub = warp >> 2;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const int col = sub * 128 + (warp & 3) * 32 + lane;  // channel within a staged row
        int acc = 0, use = 0;  // accumulator sets, inboxes
        bool ok = true;
        for (int id = first; ok && find_tile(p, cur, id, t); id += step) {
            const int subs = subs_of(p, t);
            Bias bias;
            load_bias(p, t, subs, bias);
            uint64_t sum[BN / 2];  // fp32 pairs: columns 2i, 2i + 1
#pragma unroll
            for (int i = 0; i < BN / 2; ++i) sum[i] = 0;
            for (int k = k_lo; ok && k < k_hi; k += F8 ? 1 : p.flush, ++acc) {
                ok = tc::bar_wait(acc_full(set_of(acc)), phase_of(acc), stop);
                if (F8) ok = ok && tc::bar_wait(scale_full(set_of(acc)), phase_of(acc), stop);
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                tc::fence_after();
                if (sub < subs) {
                    const ulonglong2* sc = reinterpret_cast<const ulonglong2*>(scales + (set_of(acc) * 2 + sub) * BN);
                    const uint32_t at = tmem + lane_base + (set_of(acc) * p.na + sub) * BN;
                    const uint64_t one = f32x2_pack(1.f, 1.f);
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        if (c * 32 >= t.rows) continue;
                        uint32_t v[32];
                        tc::tmem_ld32(at + c * 32, v);
                        tc::tmem_ld_wait(v);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            ulonglong2 s2 = make_ulonglong2(one, one);
                            if (F8) s2 = sc[c * 8 + j];
                            sum[c * 16 + 2 * j] =
                                f32x2_fma_rn(f32x2_pack(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1])), s2.x,
                                             sum[c * 16 + 2 * j]);
                            sum[c * 16 + 2 * j + 1] =
                                f32x2_fma_rn(f32x2_pack(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3])),
                                             s2.y, sum[c * 16 + 2 * j + 1]);
                        }
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::bar_arrive(acc_empty(set_of(acc)));
            }
            const int width = subs * 128;
            // all warps leave after the same tile: none may wait below for one that left
            ok = epi_sync_and(ok);
            // the rows of a chunk that are this CTA's: rank, rank + splits, ...
            const int slots = (32 + p.splits - 1) / p.splits;  // of a CTA, at most
#pragma unroll 1
            for (int c = 0; c * 32 < t.rows; ++c) {
                const int rows = min(32, t.rows - c * 32), b = use & 1;
                const int own = SPLIT ? (rows + p.splits - 1 - rank) / p.splits : rows;  // this CTA's
                const float* box = staging + (SPLIT ? b * (kInbox / 8) : 0);
                if (SPLIT) {
                    // Row r of the chunk belongs to CTA r % splits. All CTAs push
                    // their sums of it into that one's inbox, which adds them in
                    // the order of the CTAs. Two inboxes alternate.
                    if (use >= 2) ok = tc::bar_wait(inbox_free(b), (use / 2 - 1) & 1, stop) && ok;
                    if (threadIdx.x == 0)
                        tc::bar_expect(inbox_full(b), own * p.splits * width * 4);
                } else if (c > 0) {
                    epi_sync();  // staging is free
                }
                if (ok && sub < subs) {
                    const uint32_t to = tc::smem_u32(box) + ((SPLIT ? rank * slots * width : 0) + col) * 4;
                    int owner = 0;
                    uint32_t at = to;
#pragma unroll
                    for (int q = 0; q < BN / 32; ++q) {
                        if (c != q) continue;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float2 f = f32x2_unpack(sum[q * 16 + j / 2]);
                            const float v = j & 1 ? f.y : f.x;
                            if (!SPLIT) {
                                staging[j * width + col] = v;
                                continue;
                            }
                            if (j < rows)
                                tc::push(tc::peer_smem(at, owner), __float_as_uint(v), tc::peer_smem(inbox_full(b), owner));
                            if (++owner == p.splits) {
                                owner = 0;
                                at += width * 4;
                            }
                        }
                    }
                }
                if (SPLIT) {
                    ok = tc::bar_wait(inbox_full(b), (use / 2) & 1, stop) && ok;
                    ok = epi_sync_and(ok);
                } else {
                    epi_sync();
                }
                if (ok)
                    emit_chunk(p, t, subs, bias, warp, own, t.row + c * 32 + (SPLIT ? rank + warp * p.splits : warp),
                               SPLIT ? p.splits : 1, [&](int i, int s) {
                                   const float* from = box + i * width + s * 128 + lane * 4;
                                   float4 a = *reinterpret_cast<const float4*>(from);
                                   if (SPLIT)
                                       for (int q = 1; q < p.splits; ++q) {
                                           const float4 w = *reinterpret_cast<const float4*>(from + q * slots * width);
                                           a = make_float4(a.x + w.x, a.y + w.y, a.z + w.z, a.w + w.w);
                                       }
                                   return a;
                               });
                if (SPLIT) {
                    epi_sync();
                    if (threadIdx.x < p.splits) tc::bar_arrive_at(tc::peer_smem(inbox_free(b), threadIdx.x));
                    ++use;
                }
            }
        }
    } else {
        tc::fewer_registers<kOtherRegs>();
    }
    __syncwarp();
    __syncthreads();
    if (SPLIT) tc::cluster_sync();  // no CTA leaves while another may push into its inbox
    if (threadIdx.x == 0 && *stop) set_error(p.err, EP_DEVERR_TIMEOUT);
    if (warp == kEpiWarps + 1) tc::tmem_free(tmem, p.cols);
}

// ---- many rows per group: pairs of CTAs ------------------------------------------
// The product the other way round, x W^T: 256 rows of x are the lanes (128 in
// each CTA of the pair), 256 rows of W the columns (gate and up of 128
// channels, or 256 channels; each CTA loads 128 of them and both use all). A
// CTA then moves 32 KB into shared memory for 256 x 128 sums of a 64-channel
// block and the tensor cores read 8 KB per 16 channels, half of what they
// read for two products of 128 x 128; shared memory is what bounds those. A
// thread owns a row: its e4m3 scale is one register, and the epilogue needs no
// exchange but the amax of an e4m3 row between two warps.

constexpr int kPairEpiRegs = 224, kPairOtherRegs = 56;  // as kEpiRegs and kOtherRegs: no e4m3 scales warp here
static_assert(2 * 128 * kPairEpiRegs + 128 * kPairOtherRegs == kThreads * 168, "register split");
constexpr int kPairStage = 2 * kSub;
constexpr int kPairStages = 6;
constexpr int kPairSmem = kPairStages * kPairStage + kEpiWarps * 4096 + 256 + 2 * 128 * 4 + 1024;
static_assert(kPairSmem <= kSmemMax, "shared memory");

// A warp's outputs go through 4 KB of shared memory: each lane puts 16-byte
// pieces of its row there (32 rows of 128 bytes), and the warp stores whole
// rows' pieces together. Lanes that store their own rows touch 32 lines with
// each instruction, which took 2.5 to 6.6 us for a tile.
// Pieces of a row are swapped by row & 7, so that neither side meets in banks.
__device__ __forceinline__ void stage_pieces(uint4* box, int r, int at, int out_type, const float (&y)[16], float scale) {
    uint4* row = box + r * 8;
    const int x = r & 7;
    if (out_type == EP_DTYPE_E4M3) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = pack_e4m3x2(y[4 * j] * scale, y[4 * j + 1] * scale) |
                   pack_e4m3x2(y[4 * j + 2] * scale, y[4 * j + 3] * scale) << 16;
        row[at ^ x] = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (out_type == EP_DTYPE_FP32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            row[(at + i) ^ x] = make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]),
                                           __float_as_uint(y[4 * i + 2]), __float_as_uint(y[4 * i + 3]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            row[(at + i) ^ x] = make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]), pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                                           pack_bf16x2(y[8 * i + 4], y[8 * i + 5]), pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
    }
}
// Stores `pieces` of each of the warp's first `rows` rows, channels from n;
// rows start at `row`. size: bytes of a channel; size * out_features is a multiple of 16.
__device__ __forceinline__ void flush_pieces(const LinearParams& p, const uint4* box, int pieces, int rows, int64_t row,
                                             int n, int size) {
    const int lane = threadIdx.x & 31, piece = lane & 7;
    __syncwarp();
    const bool on = piece < pieces && n + piece * (16 / size) < p.N;
    uint8_t* out = static_cast<uint8_t*>(p.out) + ((row + lane / 8) * p.N + n) * size + piece * 16;
    const int64_t step = (int64_t)4 * p.N * size;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + lane / 8;
        if (on && r < rows) *reinterpret_cast<uint4*>(out + i * step) = box[r * 8 + (piece ^ (r & 7))];
    }
    __syncwarp();
}
// The same values one by one, for rows that are no multiple of 16 bytes.
__device__ __forceinline__ void store_scalars(const LinearParams& p, int64_t row, int n, const float (&y)[16]) {
    const int64_t at = row * p.N + n;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (n + i >= p.N) continue;
        if (p.out_type == EP_DTYPE_FP32) static_cast<float*>(p.out)[at + i] = y[i];
        else static_cast<uint16_t*>(p.out)[at + i] = (uint16_t)(pack_bf16x2(y[i], 0.f) & 0xffff);
    }
}

// Bias, activation and residual of 16 channels from n of a row: y, with u its
// other half where gated. WHOLE: rows are multiples of 8 channels.
template <int ACT, bool WHOLE>
__device__ __forceinline__ void finish16(const LinearParams& p, int g, int64_t row, int n, float (&y)[16], const float (&u)[16]) {
    const float* bias = p.bias ? p.bias + (int64_t)g * p.wide + n : nullptr;
    if (bias) {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] += n + i < p.N ? bias[i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (ACT == EP_ACT_SWIGLU)
            y[i] = activate(EP_ACT_SILU, y[i]) * (u[i] + (bias && n + i < p.N ? bias[p.N + i] : 0.f));
        else
            y[i] = activate(ACT, y[i]);
    }
    if (p.res) {
        const uint16_t* r = p.res + row * p.N + n;
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
            if (WHOLE) {
                if (n + i >= p.N) continue;
                const uint4 v = *reinterpret_cast<const uint4*>(r + i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y[i + 2 * j] += bf16lo(w[j]);
                    y[i + 2 * j + 1] += bf16hi(w[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (n + i + j < p.N) y[i + j] += __uint_as_float((uint32_t)r[i + j] << 16);
            }
        }
    }
}

// SUM: the sums leave tensor memory in parts, into registers; otherwise whole,
// by the chunk that the epilogue works on (p.flush is then kblocks).
template <bool F8, bool SUM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       LinearParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (tc::smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t* boxes = smem_raw + (ring - tc::smem_u32(smem_raw)) + kPairStages * kPairStage;
    uint8_t* control = boxes + kEpiWarps * 4096;
    float* row_amax = reinterpret_cast<float*>(control + 256);  // [2][128]
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(control + 240);
    volatile uint32_t* stop = reinterpret_cast<uint32_t*>(control + 244);
    const uint32_t bars = tc::smem_u32(control);
    auto full = [&](int s) { return bars + 8 * s; };  // the leader's are used
    auto empty = [&](int s) { return bars + 8 * (kPairStages + s); };
    auto acc_full = [&](int s) { return bars + 8 * (2 * kPairStages + s); };
    auto acc_empty = [&](int s) { return bars + 8 * (2 * kPairStages + 2 + s); };  // the leader's are used
    const uint32_t drained = bars + 8 * (2 * kPairStages + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            tc::bar_init(full(s), 1);
            tc::bar_init(empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::bar_init(acc_full(s), 1);
            tc::bar_init(acc_empty(s), 2 * kEpiWarps);
        }
        tc::bar_init(drained, 1);
        *stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kEpiWarps + 1) tc::pair_tmem_alloc(tc::smem_u32(tmem_at), 512);
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = *tmem_at;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
    constexpr int kElems = F8 ? 128 : 64;
    Cursor cur;
    Tile t;

    if (warp == kEpiWarps) {  // loads, each CTA its halves
        tc::fewer_registers<kPairOtherRegs>();
        int i = 0, s = 0;
        uint32_t wrap = 0;
        bool ok = true;
        for (int id = first; ok && find_tile(p, cur, id, t); id += step) {
            const int ch = p.parts == 2 ? t.n * 128 : t.n * 256 + rank * 128, part = p.parts == 2 ? rank : 0;
            for (int k = 0; k < p.kblocks; ++k, ++i) {
                if (wrap > 0) ok = __all_sync(FULL, tc::bar_wait(empty(s), (wrap - 1) & 1, stop));
                if (!ok) break;
                if (tc::elect()) {
                    const uint32_t at = ring + s * kPairStage, bar = tc::peer_smem(full(s), 0);
                    if (rank == 0) tc::bar_expect(full(s), 2 * kPairStage);
                    tc::pair_tma_2d(at, &map_x, bar, k * kElems, (int)t.row + rank * 128);
                    tc::pair_tma_4d(at + kSub, &map_w, bar, k * kElems, ch, part, t.group / p.R);
                }
                __syncwarp();
                if (++s == kPairStages) {
                    s = 0;
                    ++wrap;
                }
            }
            if (!ok && lane == 0 && rank == 0)  // the pair's copies in flight land before it leaves
                for (int j = i > kPairStages ? i - kPairStages : 0; j < i; ++j)
                    tc::bar_drain(full(j % kPairStages), (j / kPairStages) & 1);
        }
    } else if (warp == kEpiWarps + 1) {  // products, by the leader
        tc::fewer_registers<kPairOtherRegs>();
        if (rank == 0) {
            int s = 0, acc = 0;
            uint32_t wrap = 0;
            bool ok = true;
            const uint32_t idesc = tc::instr_desc(F8, 256, 256);
            for (int id = first; ok && find_tile(p, cur, id, t); id += step) {
                int in_set = 0;  // blocks summed in this set so far
                for (int k = 0; k < p.kblocks; ++k) {
                    if (in_set == 0 && acc >= 2)
                        ok = __all_sync(FULL, tc::bar_wait(acc_empty(acc & 1), (acc / 2 - 1) & 1, stop));
                    if (ok) ok = __all_sync(FULL, tc::bar_wait(full(s), wrap & 1, stop));
                    if (!ok) break;
                    tc::fence_after();
                    const uint32_t at = ring + s * kPairStage;
                    const uint64_t a = tc::smem_desc(at), w = tc::smem_desc(at + kSub);
                    const uint32_t d = tmem + (acc & 1) * 256;
                    const uint32_t keep = in_set > 0 ? 1u : 0u;
                    const bool last = F8 || in_set == p.flush - 1 || k == p.kblocks - 1;
                    if (tc::elect()) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)  // 32 bytes of K each
                            tc::pair_mma<F8>(d, a + 2 * q, w + 2 * q, idesc, q > 0 ? 1u : keep);
                        tc::pair_commit(empty(s));
                        if (last) tc::pair_commit(acc_full(acc & 1));
                    }
                    __syncwarp();
                    acc += last;
                    in_set = last ? 0 : in_set + 1;
                    if (++s == kPairStages) {
                        s = 0;
                        ++wrap;
                    }
                }
                if (!ok) {  // products in flight end before the pair leaves
                    if (tc::elect()) tc::pair_commit(drained);
                    tc::bar_drain(drained, 0);
                }
            }
        }
    } else if (warp < kEpiWarps) {  // epilogue: warps w and w + 4 share 32 rows, half of the channels each
        tc::more_registers<kPairEpiRegs>();
        const int half = warp >> 2;
        const int r = (warp & 3) * 32 + lane;  // row of the CTA's 128
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const bool gated = p.parts == 2;
        // column of chunk c: two chunks of gate and two of up, or four neighbours
        auto column = [&](int c) { return gated ? (c >> 1) * 128 + half * 64 + (c & 1) * 32 : half * 128 + c * 32; };
        const uint32_t empty_at[2] = {tc::peer_smem(acc_empty(0), 0), tc::peer_smem(acc_empty(1), 0)};
        int acc = 0;
        bool ok = true;
        for (int id = first; ok && find_tile(p, cur, id, t); id += step) {
            const int rows = min(max(t.rows - rank * 128, 0), 128);  // of this CTA
            const int64_t row = t.row + rank * 128 + r;
            const bool live = r < rows;
            const int g = t.group / p.R;
            const int n0 = gated ? t.n * 128 + half * 64 : t.n * 256 + half * 128;  // the thread's first channel
            uint64_t sum[SUM ? 64 : 1];  // fp32 pairs: 32 columns of each chunk
#pragma unroll
            for (int i = 0; i < (SUM ? 64 : 1); ++i) sum[i] = 0;
            // a set's sums, times p0 (first two chunks) or p1, from tensor memory
            auto take = [&](uint64_t p0, uint64_t p1) {
                tc::fence_after();
                if (rows > (warp & 3) * 32) {
                    const uint32_t at = tmem + lane_base + (acc & 1) * 256;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tc::tmem_ld32(at + column(c), v);
                        tc::tmem_ld_wait(v);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            sum[SUM ? c * 16 + j : 0] = f32x2_fma_rn(
                                f32x2_pack(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])),
                                c < 2 ? p0 : p1, sum[SUM ? c * 16 + j : 0]);
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::bar_arrive_at(empty_at[acc & 1]);
                ++acc;
            };
            if (F8) {
                const int nb = (p.N + 127) / 128;
                const float* xs = p.x_scale + (live ? row : t.row) * p.kblocks;
                const float* w0 = p.w_scale + ((int64_t)g * p.parts * nb + (gated ? t.n : min(t.n * 2 + half, nb - 1))) * p.kblocks;
                const float* w1 = gated ? w0 + (int64_t)nb * p.kblocks : w0;
                // row scales four blocks at a time, and four ahead: a load that
                // its own block waited for cost more than the block's products
                float x4[4], x_next[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) x_next[q] = q < p.kblocks ? xs[q] : 0.f;
#pragma unroll 1
                for (int k0 = 0; ok && k0 < p.kblocks; k0 += 4) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        x4[q] = x_next[q];
                        x_next[q] = k0 + 4 + q < p.kblocks ? xs[k0 + 4 + q] : 0.f;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (!ok || k0 + q >= p.kblocks) continue;
                        const float s0 = x4[q] * w0[k0 + q], s1 = x4[q] * w1[k0 + q];
                        ok = __all_sync(FULL, tc::bar_wait(acc_full(acc & 1), (acc / 2) & 1, stop));
                        if (!ok) continue;
                        take(f32x2_pack(s0, s0), f32x2_pack(s1, s1));
                    }
                }
            } else if (!SUM) {
                ok = __all_sync(FULL, tc::bar_wait(acc_full(acc & 1), (acc / 2) & 1, stop));
                tc::fence_after();
            } else {
                const uint64_t one = f32x2_pack(1.f, 1.f);
                for (int k = 0; k < p.kblocks; k += p.flush) {
                    ok = __all_sync(FULL, tc::bar_wait(acc_full(acc & 1), (acc / 2) & 1, stop));
                    if (!ok) break;
                    take(one, one);
                }
            }
            // all warps leave after the same tile: none may wait below for one that left
            ok = epi_sync_and(ok);
            const bool e4m3 = p.out_type == EP_DTYPE_E4M3;
            const int size = e4m3 ? 1 : p.out_type == EP_DTYPE_FP32 ? 4 : 2;  // bytes of a channel
            uint4* box = reinterpret_cast<uint4*>(boxes + warp * 4096);
            float amax = 1e-4f, scale = 0.f;
            // 16 channels, chunk c of the thread's: for the amax (pass 0) or to store
            auto chunk = [&](auto act, auto whole, int pass, int c, float(&y)[16], const float(&u)[16]) {
                constexpr int ACT = decltype(act)::value;
                constexpr bool WHOLE = decltype(whole)::value;
                const int n = n0 + c * 16;
                if (n >= p.N) return;
                if (live) finish16<ACT, WHOLE>(p, g, row, n, y, u);
                if (pass == 0) {
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(y[i]));
                    }
                } else if (WHOLE) {
                    const int at = c * size & 7;  // first piece of the chunk
                    if (live) stage_pieces(box, lane, at, p.out_type, y, scale);
                    if (at + size == 8 || c == (gated ? 3 : 7) || n + 16 >= p.N)
                        flush_pieces(p, box, at + size, rows - (warp & 3) * 32, t.row + rank * 128 + (warp & 3) * 32,
                                     n - at * 16 / size, size);
                } else if (live) {
                    store_scalars(p, row, n, y);
                }
            };
            auto chunks = [&](auto act, auto whole, int pass) {
                if (SUM) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if (c >= (gated ? 4 : 8)) continue;
                        float y[16], u[16];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 v = f32x2_unpack(sum[SUM ? c * 8 + j : 0]),
                                         w = f32x2_unpack(sum[SUM ? (c + 4) % 8 * 8 + j : 0]);
                            y[2 * j] = v.x;
                            y[2 * j + 1] = v.y;
                            u[2 * j] = w.x;
                            u[2 * j + 1] = w.y;
                        }
                        chunk(act, whole, pass, c, y, u);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < (gated ? 4 : 8); ++c) {
                        float y[16], u[16];
                        uint32_t v[16];
                        const uint32_t at = tmem + lane_base + (acc & 1) * 256;
                        tc::tmem_read16(at + (gated ? half * 64 : half * 128) + c * 16, v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(v[j]);
                        if (gated) {
                            tc::tmem_read16(at + 128 + half * 64 + c * 16, v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) u[j] = __uint_as_float(v[j]);
                        }
                        chunk(act, whole, pass, c, y, u);
                    }
                }
            };
            // What the epilogue does is chosen here and not for each chunk, and
            // sums in tensor memory take one loop for all chunks: code that is
            // run over with most of it skipped waits for instructions (4 of 6 us
            // of a tile's epilogue).
            auto pass_of = [&](int pass) {
                auto with = [&](auto act) {
                    if (p.N * size % 16 == 0 && p.N % 8 == 0) chunks(act, std::true_type(), pass);
                    else chunks(act, std::false_type(), pass);
                };
                if (p.act == EP_ACT_NONE) with(std::integral_constant<int, EP_ACT_NONE>());
                else if (p.act == EP_ACT_SILU) with(std::integral_constant<int, EP_ACT_SILU>());
                else if (p.act == EP_ACT_GELU) with(std::integral_constant<int, EP_ACT_GELU>());
                else with(std::integral_constant<int, EP_ACT_SWIGLU>());
            };
            if (ok && rows > (warp & 3) * 32) {
                // e4m3 goes over the row twice: for its amax, then to store it
#pragma unroll 1
                for (int pass = e4m3 ? 0 : 1; pass < 2; ++pass) {
                    if (pass == 1 && e4m3 && gated) {  // the row's other 64 channels are warp +-4's
                        row_amax[half * 128 + r] = amax;
                        asm volatile("bar.sync %0, 64;" ::"r"(2 + (warp & 3)) : "memory");
                        amax = fmaxf(amax, row_amax[(half ^ 1) * 128 + r]);
                    }
                    if (pass == 1 && e4m3 && live && (!gated || half == 0) && n0 < p.N)
                        p.out_scale[row * (p.N / 128) + n0 / 128] = amax / 448.0f;
                    scale = 448.0f / amax;
                    pass_of(pass);
                }
            }
            if (!SUM) {
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::bar_arrive_at(empty_at[acc & 1]);
                ++acc;
            }
        }
    } else {
        tc::fewer_registers<kPairOtherRegs>();
    }
    __syncwarp();
    __syncthreads();
    tc::cluster_sync();
    if (threadIdx.x == 0 && *stop) set_error(p.err, EP_DEVERR_TIMEOUT);
    if (warp == kEpiWarps + 1) tc::pair_tmem_free(tmem, 512);
}

// ---- host ----------------------------------------------------------------------

using encode_t = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime (libep links no libcuda); NULL if the driver lacks it.
encode_t encoder() {
    static const encode_t f = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<encode_t>(fn);
    }();
    return f;
}

// A row-major array as tiles of 128 bytes x box_rows, 128-byte swizzled, zeros outside.
bool encode(CUtensorMap* map, bool f8, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            int box_rows) {
    const cuuint32_t box[4] = {f8 ? 128u : 64u, (cuuint32_t)box_rows, 1, 1}, one[4] = {1, 1, 1, 1};
    return encoder()(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                     const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

ep_status_t check_linear(const ep_linear_t* q, int64_t rows) {
    if (!q) return fail(EP_ERR_INVALID, "p is NULL");
    if (q->in_features < 1 || q->out_features < 1)
        return fail(EP_ERR_INVALID, "in_features and out_features must be >= 1");
    if (q->in_features > 1 << 20 || q->out_features > 1 << 20)
        return fail(EP_ERR_UNSUPPORTED, "in_features and out_features must be <= 2^20");
    if (q->act < EP_ACT_NONE || q->act > EP_ACT_SWIGLU) return fail(EP_ERR_INVALID, "unknown act %d", q->act);
    if (q->out_type < EP_DTYPE_BF16 || q->out_type > EP_DTYPE_E4M3)
        return fail(EP_ERR_INVALID, "unknown out_type %d", q->out_type);
    if ((q->x_scale == nullptr) != (q->w_scale == nullptr))
        return fail(EP_ERR_INVALID, "x_scale and w_scale go together (both e4m3, or both bf16)");
    if (q->x_scale ? q->in_features % 128 != 0 : q->in_features % 8 != 0)
        return fail(EP_ERR_UNSUPPORTED, "in_features must be a multiple of %d", q->x_scale ? 128 : 8);
    if (q->out_type == EP_DTYPE_E4M3 && q->out_features % 128 != 0)
        return fail(EP_ERR_UNSUPPORTED, "e4m3 out needs out_features a multiple of 128");
    if (rows > 0 && (q->out_type == EP_DTYPE_E4M3) != (q->out_scale != nullptr))
        return fail(EP_ERR_INVALID, "out_scale goes with EP_DTYPE_E4M3 out, and only with it");
    if (rows > 0 && (!q->x || !q->w || !q->out)) return fail(EP_ERR_INVALID, "x, w and out must be non-NULL");
    if (q->out && q->out == q->residual && q->out_type != EP_DTYPE_BF16)
        return fail(EP_ERR_INVALID, "out can be residual itself only as bf16");
    if (((uintptr_t)q->x | (uintptr_t)q->w | (uintptr_t)q->out | (uintptr_t)q->residual) % 16 != 0)
        return fail(EP_ERR_INVALID, "x, w, residual and out must be 16-byte aligned");
    if (((uintptr_t)q->x_scale | (uintptr_t)q->w_scale | (uintptr_t)q->bias | (uintptr_t)q->out_scale) % 4 != 0)
        return fail(EP_ERR_INVALID, "scales and bias must be 4-byte aligned");
    return EP_OK;
}

LinearParams params_of(const ep_linear_t& q) {
    LinearParams p{};
    p.x = q.x;
    p.x_scale = q.x_scale;
    p.w = q.w;
    p.w_scale = q.w_scale;
    p.bias = q.bias;
    p.res = static_cast<const uint16_t*>(q.residual);
    p.out = q.out;
    p.out_scale = q.out_scale;
    p.K = q.in_features;
    p.N = q.out_features;
    p.parts = q.act == EP_ACT_SWIGLU ? 2 : 1;
    p.wide = p.N * p.parts;
    p.act = q.act;
    p.out_type = q.out_type;
    p.R = 1;
    return p;
}

constexpr int kMaxSplits = 8;

template <bool F8>
auto kernel_of(bool split, int bn) {
    if (split) return bn == 32 ? linear_kernel<F8, true, 32> : bn == 64 ? linear_kernel<F8, true, 64> : linear_kernel<F8, true, 128>;
    return bn == 32 ? linear_kernel<F8, false, 32> : bn == 64 ? linear_kernel<F8, false, 64> : linear_kernel<F8, false, 128>;
}

// Clusters of n CTAs, one CTA per SM, that device b can hold at once: fewer
// than SMs / n, since a cluster stays within a GPC (15 of 8, not 18).
int clusters_of(const ep_buffer& b, int n) {
    static std::atomic<int> known[64][kMaxSplits + 1];
    std::atomic<int>* at = b.device >= 0 && b.device < 64 ? &known[b.device][n] : nullptr;
    int count = at ? at->load(std::memory_order_relaxed) : 0;
    if (count > 0) return count - 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(n * b.sm_count));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemMax;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const auto kernel = linear_kernel<false, true, 128>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&count, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        count = 0;
    }
    if (at) at->store(count + 1, std::memory_order_relaxed);
    return count;
}

// How a call is tiled.
struct Shape {
    bool pair;
    int bn, na, nt, splits;
    int64_t bound;  // row tiles there can be
};

// Takes the kernel with the least time by this estimate, in microseconds as
// measured on large layers. A 128-byte block of in_features takes 0.28 (bf16)
// or 0.62 (e4m3) for a pair's 256 x 256 tile; 0.25 or 0.51 for 128 rows and
// each weight tile of a CTA; 0.16 + 0.10 or 0.25 + 0.12 for each of them where
// its rows are few (it then waits for weights). A tile's epilogue takes 4.5 or 11 with pairs, else 0.7 for each 32 rows
// and weight tile; with bf16 it runs beside the next tile's products. Among
// groups, the last of a group's tiles is half empty in the mean.
Shape shape_of(const ep_buffer& b, const LinearParams& p, int64_t avg, int64_t most) {
    const bool f8 = p.x_scale != nullptr;
    const int64_t groups = most < p.G ? most : p.G;
    auto row_tiles = [&](int rows) {
        if (p.G == 1) return (double)((avg + rows - 1) / rows);
        return groups * fmax(1.0, (double)avg / rows + 0.5);
    };
    auto total = [&](double tiles, int64_t at_once, double products, double epilogue) {
        const double rounds = fmax(1.0, tiles / at_once < 4 ? ceil(tiles / at_once) : tiles / at_once);
        return f8 ? rounds * (products + epilogue) : (rounds - 1) * fmax(products, epilogue) + products + epilogue;
    };
    Shape c{};
    double best = 0;
    for (int bn = avg <= 32 ? 32 : avg <= 64 ? 64 : 128; bn >= 32; bn /= 2) {
        const double likely = row_tiles(bn);
        // two weight tiles per CTA share its rows of x; one where tiles are few
        int na = 2, nt = p.parts == 2 ? (p.N + 127) / 128 : (p.N + 255) / 256;
        if (p.parts == 1 && (p.N <= 128 || likely * nt < b.sm_count)) {
            na = 1;
            nt = (p.N + 127) / 128;
        }
        const double block = bn == 128 ? (f8 ? 0.51 : 0.25) * na : (f8 ? 0.25 : 0.16) + (f8 ? 0.12 : 0.10) * na;
        const double epilogue = bn / 32 * na * 0.7;
        // A cluster can share each tile's in_features: n CTAs finish a tile n
        // times as fast, less the exchange of its sums (1.5 for each 32 rows),
        // and rounds over all tiles come out less ragged.
        for (int n = 1; n <= kMaxSplits && (n == 1 || p.kblocks >= 4 * n); ++n) {
            const int64_t at_once = n == 1 ? b.sm_count : clusters_of(b, n);
            if (at_once < 1) continue;
            const double time =
                total(likely * nt, at_once, (p.kblocks + n - 1) / n * block, epilogue + (n > 1 ? 1.5 * (bn / 32) : 0));
            if (c.splits > 0 && time >= best) continue;
            best = time;
            c.bn = bn;
            c.na = na;
            c.nt = nt;
            c.splits = n;
        }
    }
    c.bound = p.cnt ? (int64_t)p.G * ((p.region + c.bn - 1) / c.bn) : most / c.bn + groups;
    if (avg < 128 || p.wide < 256) return c;
    const int nt = p.parts == 2 ? (p.N + 127) / 128 : (p.N + 255) / 256;
    if (total(row_tiles(256) * nt, b.sm_count / 2, p.kblocks * (f8 ? 0.62 : 0.28), f8 ? 11.0 : 4.5) > best) return c;
    c.pair = true;
    c.bn = 256;
    c.na = 2;
    c.splits = 1;
    c.nt = nt;
    c.bound = p.cnt ? (int64_t)p.G * ((p.region + 255) / 256) : most / 256 + groups;
    return c;
}

// Chooses tile, split and grid and launches. x_rows: rows that x holds;
// weights: matrices in w; avg: rows of a group to expect (any count is right).
ep_status_t launch_on_device(const ep_buffer& b, LinearParams p, int64_t x_rows, int weights, int64_t avg, int64_t most,
                             cudaStream_t stream) {
    const bool f8 = p.x_scale != nullptr;
    const int size = f8 ? 1 : 2;
    p.kblocks = f8 ? p.K / 128 : (p.K + 63) / 64;
    p.vec = p.N % 4 == 0;
    p.flush = f8 ? 1 : p.out_type == EP_DTYPE_BF16 ? p.kblocks : 8;
    const Shape c = shape_of(b, p, avg, most);
    const bool pair = c.pair;
    p.bn = c.bn;
    p.na = c.na;
    p.nt = c.nt;
    p.splits = c.splits;
    const int64_t bound = c.bound;
    if (bound * p.nt >= (int64_t)1 << 30) return fail(EP_ERR_UNSUPPORTED, "too many tiles: rows x out_features");
    const bool split = p.splits > 1;
    const int sb = stage_bytes(p.na, p.bn);
    const int fixed = kControl + (split ? kInbox : kStaging) + 1024;  // 1024: alignment of the ring
    p.stages = (kSmemMax - fixed) / sb;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    const int smem = p.stages * sb + fixed;
    // a set fills while another is read; e4m3 hands one over for each block, and
    // more of them hide the hand-over
    const int sets = p.na * p.bn <= 64 ? 8 : p.na * p.bn <= 128 ? 4 : 2;
    p.acc_log = sets == 8 ? 3 : sets == 4 ? 2 : 1;
    p.cols = sets * p.na * p.bn;

    CUtensorMap map_x, map_w;
    const cuuint64_t K = p.K, N = p.N;
    const cuuint64_t dx[2] = {K, (cuuint64_t)x_rows}, sx[1] = {K * size};
    const cuuint64_t dw[4] = {K, N, (cuuint64_t)p.parts, (cuuint64_t)weights},
                     sw[3] = {K * size, N * K * size, (cuuint64_t)p.wide * K * size};
    if (!encoder()) return fail(EP_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
    if (!encode(&map_x, f8, p.x, 2, dx, sx, pair ? 128 : p.bn) || !encode(&map_w, f8, p.w, 4, dw, sw, 128))
        return fail(EP_ERR_UNSUPPORTED, "x or w is too large for a tensor map");

    const auto kernel = pair ? (f8 ? linear_pair_kernel<true, true> : p.flush < p.kblocks ? linear_pair_kernel<false, true> : linear_pair_kernel<false, false>)
                        : f8 ? kernel_of<true>(split, p.bn) : kernel_of<false>(split, p.bn);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    const int64_t tiles = bound * p.nt, pairs = b.sm_count / 2, clusters = split ? clusters_of(b, p.splits) : 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(pair ? 2 * (tiles < pairs ? tiles : pairs) : split ? p.splits * (tiles < clusters ? tiles : clusters) : tiles < b.sm_count ? tiles : b.sm_count));
    cfg.blockDim = dim3(pair ? kThreads : kThreads);
    cfg.dynamicSmemBytes = pair ? kPairSmem : smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pair ? 0 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, map_x, map_w, p);
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "linear launch: %s", cudaGetErrorString(e));
    set_last_error("");
    return EP_OK;
}

ep_status_t launch(const ep_buffer& b, const LinearParams& p, int64_t x_rows, int weights, int64_t avg, int64_t most,
                   void* stream) {
    int prev = 0;
    cudaError_t e = cudaGetDevice(&prev);
    if (e == cudaSuccess && prev != b.device) e = cudaSetDevice(b.device);
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(e));
    const ep_status_t st = launch_on_device(b, p, x_rows, weights, avg, most, static_cast<cudaStream_t>(stream));
    if (prev != b.device) cudaSetDevice(prev);
    return st;
}

}  // namespace
}  // namespace ep

extern "C" {

ep_status_t ep_linear(ep_buffer_t* b, int64_t rows, const ep_linear_t* q, void* stream) {
    using namespace ep;
    if (!b) return fail(EP_ERR_INVALID, "buffer is NULL");
    if (rows < 0) return fail(EP_ERR_INVALID, "rows must be >= 0");
    if (rows >= (int64_t)1 << 31) return fail(EP_ERR_UNSUPPORTED, "rows must be < 2^31");
    if (ep_status_t st = check_linear(q, rows)) return st;
    set_last_error("");
    if (rows == 0) return EP_OK;
    LinearParams p = params_of(*q);
    p.G = 1;
    p.rows = p.row_limit = rows;
    p.err = b->err;
    return launch(*b, p, rows, 1, rows, rows, stream);
}

ep_status_t ep_expert_linear(ep_buffer_t* b, int T, const ep_linear_t* q, void* stream) {
    using namespace ep;
    if (!b) return fail(EP_ERR_INVALID, "buffer is NULL");
    if (T != b->last_T) return fail(EP_ERR_INVALID, "T=%d does not match the last layout (T=%d)", T, b->last_T);
    const bool sh = (b->cfg.flags & EP_FLAG_SHARD) != 0;
    if (sh && !b->placed) return fail(EP_ERR_INVALID, "call ep_shard_place after ep_shard_layout first");
    const int64_t rows = (int64_t)b->cfg.num_ranks * T * b->cfg.topk;
    if (ep_status_t st = check_linear(q, rows)) return st;
    set_last_error("");
    if (rows == 0) return EP_OK;
    LinearParams p = params_of(*q);
    const int E = b->cfg.num_experts, R = b->cfg.num_ranks;
    p.row_limit = (b->cfg.flags & EP_FLAG_LOW_LATENCY) ? b->m_max : rows;
    p.err = b->err;
    if (b->cfg.flags & EP_FLAG_LOW_LATENCY) {
        p.G = E * R;
        p.R = R;
        p.cnt = b->cnt;
        p.region = b->cfg.max_tokens_per_rank;
    } else {
        p.G = sh ? E / R : E;
        p.off = sh ? b->recv_off : b->expert_off;
    }
    const int64_t avg = (rows + (sh ? E : p.G) - 1) / (sh ? E : p.G);
    return launch(*b, p, p.row_limit, sh ? E / R : E, avg, rows, stream);
}

}  // extern "C"
