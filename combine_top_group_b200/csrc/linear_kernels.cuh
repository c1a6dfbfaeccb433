// The kernels of ep_linear and ep_expert_linear. One source file instantiates
// them for bf16 operands and one for e4m3, so that they compile side by side.
#pragma once

#include <type_traits>

#include "linear.cuh"

namespace ep {
namespace linear {
namespace {

// Output channels as lanes, rows of x as columns, one CTA or a cluster to a
// tile: for few rows. 32 experts of 32 rows, 7168 -> 2 x 2048, e4m3: 184 to 196
// us under the power cap (1.64 GHz), 4.8 to 5.2 TB/s (74 to 79% of a copy's
// rate). BN: rows of x per tile (p.bn).
template <bool F8, bool SPLIT, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w, LinearParams p) {
    extern __shared__ uint8_t smem_raw[];
    const int sb = stage_bytes(p.na, BN);
    // swizzled tiles start on 1024 bytes (the same offset in every CTA of a cluster)
    const uint32_t ring = (tc::smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t* smem = smem_raw + (ring - tc::smem_u32(smem_raw));
    // the host counts on shared memory that starts so; if not, a stage makes room
    const int stages = ring == tc::smem_u32(smem_raw) ? p.stages : p.stages - 1;
    uint8_t* after = smem + (size_t)stages * sb;
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
        for (int s = 0; s < stages; ++s) {
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
    // elected lane issues. A warpgroup changes its registers by one instruction
    // that all its warps execute, before they part.
    if (warp >= kEpiWarps) {
        tc::fewer_registers<kOtherRegs>();
        int loads = 0;  // that the loads warp has issued
        if (warp == kEpiWarps) {  // loads
            int s = 0;
            uint32_t wrap = 0;
            bool ok = true;
            for (int id = first; ok && find_tile(p, cur, id, t); id += step) {
                const int subs = subs_of(p, t);
                const uint32_t bytes = subs * kSub + BN * 128;
                for (int k = k_lo; k < k_hi; ++k, ++loads) {
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
                    if (++s == stages) {
                        s = 0;
                        ++wrap;
                    }
                }
            }
        } else if (warp == kEpiWarps + 1) {  // products
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
                    if (++s == stages) {
                        s = 0;
                        ++wrap;
                    }
                }
            }
        } else if (warp == kEpiWarps + 2) {  // e4m3: row scale x weight block scale of each block and column
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
                    // loaded four blocks ahead: a load that its own block waited
                    // for would hold that block up by its latency
                    float x4[BN / 32][4], w4[2][4];
                    auto fetch = [&](int k, int q) {
                        const bool in = k < k_hi;
                        w4[0][q] = in ? ws[0][k] : 0.f;
                        w4[1][q] = in && subs == 2 ? ws[1][k] : 0.f;
#pragma unroll
                        for (int j = 0; j < BN / 32; ++j)
                            x4[j][q] = in && lane + 32 * j < t.rows
                                           ? p.x_scale[(t.row + lane + 32 * j) * p.kblocks + k] : 0.f;
                    };
#pragma unroll
                    for (int q = 0; q < 4; ++q) fetch(k_lo + q, q);
#pragma unroll 1
                    for (int k = k_lo; ok && k < k_hi; k += 4) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (!ok || k + q >= k_hi) continue;
                            float s0[BN / 32], s1[BN / 32];
#pragma unroll
                            for (int j = 0; j < BN / 32; ++j) {
                                s0[j] = x4[j][q] * w4[0][q];
                                s1[j] = x4[j][q] * w4[1][q];
                            }
                            fetch(k + 4 + q, q);
                            if (acc >= sets)
                                ok = __all_sync(FULL, tc::bar_wait(acc_empty(set_of(acc)), phase_of(acc) ^ 1, stop));
                            if (!ok) continue;
                            float* dst = scales + set_of(acc) * 2 * BN + lane;
#pragma unroll
                            for (int j = 0; j < BN / 32; ++j) {
                                dst[32 * j] = s0[j];
                                dst[BN + 32 * j] = s1[j];
                            }
                            tc::bar_arrive(scale_full(set_of(acc)));
                            ++acc;
                        }
                    }
                }
            }
        }
        __syncwarp();
        all_done();
        // A wait gave up: copies and products in flight end before the CTA leaves.
        // (Otherwise the epilogue has waited for them all.)
        if (*stop) {
            const long long t0 = clock64();
            if (warp == kEpiWarps) {
                for (int j = max(loads - stages, 0); j < loads; ++j) tc::bar_drain(full(j % stages), (j / stages) & 1, t0);
            } else if (warp == kEpiWarps + 1) {
                if (tc::elect()) tc::commit(drained);
                tc::bar_drain(drained, 0, t0);
            }
            __syncwarp();
        }
    } else {  // epilogue: warps 0-3 read sub-tile 0, warps 4-7 sub-tile 1
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
            for (int c = 0; ok && c * 32 < t.rows; ++c) {
                const int rows = min(32, t.rows - c * 32), b = use & 1;
                const int own = SPLIT ? (rows + p.splits - 1 - rank) / p.splits : rows;  // this CTA's
                const float* box = staging + (SPLIT ? b * (kInbox / 8) : 0);
                if (SPLIT) {
                    // Row r of the chunk belongs to CTA r % splits. All CTAs push
                    // their sums of it into that one's inbox, which adds them in
                    // the order of the CTAs. Two inboxes alternate. Their barriers
                    // order shared memory between CTAs, at the cluster's scope:
                    // full after the pushes, free after the reads.
                    if (use >= 2) ok = tc::bar_wait<tc::kCluster>(inbox_free(b), (use / 2 - 1) & 1, stop) && ok;
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
                    ok = tc::bar_wait<tc::kCluster>(inbox_full(b), (use / 2) & 1, stop) && ok;
                    ok = epi_sync_and(ok);
                    if (!ok) break;  // an inbox that was not filled is not armed again
                } else {
                    epi_sync();
                }
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
                    if (threadIdx.x < p.splits)
                        tc::bar_arrive_at<tc::kCluster>(tc::peer_smem(inbox_free(b), threadIdx.x));
                    ++use;
                }
            }
        }
        __syncwarp();
        all_done();
    }
    __syncwarp();
    if (SPLIT) {
        tc::cluster_sync();  // no CTA leaves while another may push into its inbox
        // pushes issued before that into an inbox that nobody waits for any more
        if (*stop) tc::nap(tc::kPushCycles);
        __syncwarp();
    }
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
// exchange but the amax of an e4m3 row between two warps. 4096 x 8192 -> 8192
// in bf16: 371 us in a burst (1.48 PFLOP/s, 92% of a cuBLAS burst), 444 under the
// power cap (1.26 GHz), tensor cores 92% busy while active; in e4m3 394 us (1.40
// PFLOP/s, no faster), bound by the hand-over of each block's sums.


// 16 channels of a row at n, rounded and stored in 16-byte pieces. (A lane
// stores its own row. Going through shared memory, so that the warp's stores
// run along rows, gained 4% on a bf16 layer of 2048 channels and lost 4% on
// the e4m3 and gated ones.)
__device__ __forceinline__ void store_pieces(const LinearParams& p, int64_t row, int n, const float (&y)[16], float scale) {
    const int64_t at = row * p.N + n;
    if (p.out_type == EP_DTYPE_E4M3) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = pack_e4m3x2(y[4 * j] * scale, y[4 * j + 1] * scale) |
                   pack_e4m3x2(y[4 * j + 2] * scale, y[4 * j + 3] * scale) << 16;
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (p.out_type == EP_DTYPE_FP32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + 4 * i < p.N) o[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    } else {
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (n + 8 * i < p.N)
                o[i] = make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]), pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                                  pack_bf16x2(y[8 * i + 4], y[8 * i + 5]), pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
    }
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
    uint8_t* control = smem_raw + (ring - tc::smem_u32(smem_raw)) + kPairStages * kPairStage;
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

    if (warp >= kEpiWarps) {
        tc::fewer_registers<kPairOtherRegs>();
        int loads = 0;  // that the loads warp has issued
        if (warp == kEpiWarps) {  // loads, each CTA its halves
            int s = 0;
            uint32_t wrap = 0;
            bool ok = true;
            for (int id = first; ok && find_tile(p, cur, id, t); id += step) {
                // the CTA's half of the tile; from row_limit on it is zeros
                const int row = (int)min(t.row + rank * 128, p.row_limit);
                const int ch = p.parts == 2 ? t.n * 128 : t.n * 256 + rank * 128, part = p.parts == 2 ? rank : 0;
                for (int k = 0; k < p.kblocks; ++k, ++loads) {
                    if (wrap > 0) ok = __all_sync(FULL, tc::bar_wait(empty(s), (wrap - 1) & 1, stop));
                    if (!ok) break;
                    if (tc::elect()) {
                        const uint32_t at = ring + s * kPairStage, bar = tc::peer_smem(full(s), 0);
                        if (rank == 0) tc::bar_expect(full(s), 2 * kPairStage);
                        tc::pair_tma_2d(at, &map_x, bar, k * kElems, row);
                        tc::pair_tma_4d(at + kSub, &map_w, bar, k * kElems, ch, part, t.group / p.R);
                    }
                    __syncwarp();
                    if (++s == kPairStages) {
                        s = 0;
                        ++wrap;
                    }
                }
            }
        } else if (warp == kEpiWarps + 1) {  // products, by the leader
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
                }
            }
        }
        __syncwarp();
        all_done();
        // A wait gave up: the pair's copies and products in flight end before it
        // leaves. The leader's barriers count both CTAs' copies, and a leader that no
        // wait stopped has seen them all land.
        if (*stop && rank == 0) {
            const long long t0 = clock64();
            if (warp == kEpiWarps) {
                for (int j = max(loads - kPairStages, 0); j < loads; ++j)
                    tc::bar_drain(full(j % kPairStages), (j / kPairStages) & 1, t0);
            } else if (warp == kEpiWarps + 1) {
                if (tc::elect()) tc::pair_commit(drained);
                tc::bar_drain(drained, 0, t0);
            }
            __syncwarp();
        }
    } else {  // epilogue: warps w and w + 4 share 32 rows, half of the channels each
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
                // block scales: 32 blocks' at a time, one to a lane
                float w0_lane = 0.f, w1_lane = 0.f;
#pragma unroll 1
                for (int k0 = 0; ok && k0 < p.kblocks; k0 += 4) {
                    if ((k0 & 31) == 0 && k0 + lane < p.kblocks) {
                        w0_lane = w0[k0 + lane];
                        w1_lane = w1[k0 + lane];
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        x4[q] = x_next[q];
                        x_next[q] = k0 + 4 + q < p.kblocks ? xs[k0 + 4 + q] : 0.f;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (!ok || k0 + q >= p.kblocks) continue;
                        const int at = (k0 & 31) + q;
                        const float s0 = x4[q] * __shfl_sync(FULL, w0_lane, at), s1 = x4[q] * __shfl_sync(FULL, w1_lane, at);
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
                } else if (live) {
                    if (WHOLE) store_pieces(p, row, n, y, scale);
                    else store_scalars(p, row, n, y);
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
                    if (p.N % 8 == 0) chunks(act, std::true_type(), pass);
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
        __syncwarp();
        all_done();
    }
    __syncwarp();
    tc::cluster_sync();
    if (threadIdx.x == 0 && *stop) set_error(p.err, EP_DEVERR_TIMEOUT);
    if (warp == kEpiWarps + 1) tc::pair_tmem_free(tmem, 512);
}

}  // namespace
}  // namespace linear
}  // namespace ep
