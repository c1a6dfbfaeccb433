// ep_linear and ep_expert_linear: out = act(x W^T + bias) + residual on dense
// rows or on the experts' receive rows, bf16 or e4m3 with scales.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "ep.h"
#include "internal.h"

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
    if (act == EP_ACT_SILU) return z / (1.0f + __expf(-z));
    if (act == EP_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    return z;
}

__device__ __forceinline__ float e4m3_value(uint8_t b) { return unpack_e4m3x2(b).x; }

constexpr int kTile = 64;

// 64 rows x 128 out channels of one group per CTA, fp32 on the CUDA cores.
// blockIdx = (out-channel tile, row tile of the group, group); a CTA walks
// the group's row tiles with the stride of the grid.
__global__ void __launch_bounds__(256) linear_kernel(LinearParams p) {
    __shared__ float xs[16][kTile + 1];
    __shared__ float wsm[2][16][128 + 1];
    __shared__ float red[kTile][4];
    int64_t start;
    int count;
    group_rows(p, blockIdx.z, start, count);
    const int g = blockIdx.z / p.R;
    const int n0 = blockIdx.x * 128;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;  // 4 channels tx + 32 j, 8 rows ty + 8 i
    const bool f8 = p.x_scale != nullptr;
    const int kb = p.K / 128, nb = (p.N + 127) / 128;
    for (int r0 = blockIdx.y * kTile; r0 < count; r0 += gridDim.y * kTile) {
        float acc[2][8][4] = {};
        for (int k0 = 0; k0 < p.K; k0 += 16) {
            __syncthreads();
            for (int i = threadIdx.x; i < kTile * 16; i += 256) {
                const int r = i / 16, k = i % 16;
                float v = 0.f;
                if (r0 + r < count && k0 + k < p.K) {
                    const int64_t at = (start + r0 + r) * p.K + k0 + k;
                    v = f8 ? e4m3_value(static_cast<const uint8_t*>(p.x)[at]) *
                                 p.x_scale[(start + r0 + r) * kb + (k0 + k) / 128]
                           : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.x)[at] << 16);
                }
                xs[k][r] = v;
            }
            for (int h = 0; h < p.parts; ++h)
                for (int i = threadIdx.x; i < 128 * 16; i += 256) {
                    const int n = i / 16, k = i % 16;
                    float v = 0.f;
                    if (n0 + n < p.N && k0 + k < p.K) {
                        const int64_t at = ((int64_t)g * p.wide + (int64_t)h * p.N + n0 + n) * p.K + k0 + k;
                        v = f8 ? e4m3_value(static_cast<const uint8_t*>(p.w)[at]) *
                                     p.w_scale[((int64_t)(g * p.parts + h) * nb + blockIdx.x) * kb + (k0 + k) / 128]
                               : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.w)[at] << 16);
                    }
                    wsm[h][k][n] = v;
                }
            __syncthreads();
            for (int k = 0; k < 16; ++k)
                for (int h = 0; h < 2; ++h) {
                    if (h >= p.parts) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[h][i][j] = fmaf(xs[k][ty + 8 * i], wsm[h][k][tx + 32 * j], acc[h][i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = ty + 8 * i;
            const int64_t row = start + r0 + r;
            const bool live = r0 + r < count;
            float v[4], amax = 1e-4f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx + 32 * j;
                v[j] = 0.f;
                if (!live || n >= p.N) continue;
                float z = acc[0][i][j];
                if (p.bias) z += p.bias[(int64_t)g * p.wide + n];
                if (p.act == EP_ACT_SWIGLU) {
                    float u = acc[1][i][j];
                    if (p.bias) u += p.bias[(int64_t)g * p.wide + p.N + n];
                    v[j] = activate(EP_ACT_SILU, z) * u;
                } else {
                    v[j] = activate(p.act, z);
                }
                if (p.res) v[j] += __uint_as_float((uint32_t)p.res[row * p.N + n] << 16);
                amax = fmaxf(amax, fabsf(v[j]));
            }
            if (p.out_type == EP_DTYPE_E4M3) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, o));
                if (live && tx == 0) p.out_scale[row * nb + blockIdx.x] = amax / 448.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx + 32 * j;
                if (!live || n >= p.N) continue;
                const int64_t at = row * p.N + n;
                if (p.out_type == EP_DTYPE_E4M3)
                    static_cast<uint8_t*>(p.out)[at] = (uint8_t)(pack_e4m3x2(v[j] * (448.0f / amax), 0.f) & 0xff);
                else if (p.out_type == EP_DTYPE_FP32)
                    static_cast<float*>(p.out)[at] = v[j];
                else
                    static_cast<uint16_t*>(p.out)[at] = (uint16_t)(pack_bf16x2(v[j], 0.f) & 0xffff);
            }
        }
    }
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

// avg: rows per group to expect (any count is right).
ep_status_t launch(const ep_buffer& b, const LinearParams& p, int64_t avg, void* stream) {
    int prev = 0;
    cudaError_t e = cudaGetDevice(&prev);
    if (e == cudaSuccess && prev != b.device) e = cudaSetDevice(b.device);
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "cudaSetDevice: %s", cudaGetErrorString(e));
    int64_t rt = (avg + kTile - 1) / kTile;
    if (rt < 1) rt = 1;
    if (rt > 65535) rt = 65535;
    const int gmax = 65535;
    e = cudaSuccess;
    if (p.G > gmax) e = cudaErrorInvalidValue;
    if (e == cudaSuccess) {
        linear_kernel<<<dim3((p.N + 127) / 128, (unsigned)rt, (unsigned)p.G), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
        e = cudaGetLastError();
    }
    if (prev != b.device) cudaSetDevice(prev);
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "linear launch: %s", cudaGetErrorString(e));
    set_last_error("");
    return EP_OK;
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
    return launch(*b, p, rows, stream);
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
    const int64_t avg = (int64_t)R * T * b->cfg.topk / (sh ? E : p.G) + 1;
    return launch(*b, p, avg, stream);
}

}  // extern "C"
