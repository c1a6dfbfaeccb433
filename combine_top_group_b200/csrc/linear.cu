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
//  - bf16: the whole sum leaves tensor memory the same way; beyond 8192 channels
//    parts of 2048 do, and for fp32 and e4m3 outputs every 8 blocks of 64. Sums
//    there are cut, not rounded: operands of one sign lose 2.5e-8 (32 steps of
//    16 channels) to 6e-8 (512 steps) of the sum with each step. So bf16 outputs
//    are off by at most 3.2e-5 before their own rounding by up to 2^-9 or 2^-8
//    (in one go 2^19 channels lost 3.6e-4 even split over a cluster), fp32 and
//    e4m3 outputs by 8e-7, about what roundings of an fp32 sum of that length
//    come to. The price is 7% of the time beyond 8192 channels, and 8 to 20% for
//    fp32 and e4m3 outputs.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "block.h"
#include "ep.h"
#include "internal.h"
#include "linear.cuh"

namespace ep {
namespace {

using namespace linear;

// Self-test of the bounded waits: a barrier that expects one arrival nobody
// makes. Warp 0 gives up after the limit; warp 1, whose own limit is far off,
// follows its stop flag; then warp 0 drains. No copy or product is in flight.
__global__ void timeout_selftest_kernel(uint32_t* err, uint32_t* gave_up, long long limit) {
    __shared__ uint64_t bar;
    __shared__ uint32_t stop;
    const uint32_t at = tc::smem_u32(&bar);
    if (threadIdx.x == 0) {
        tc::bar_init(at, 1);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    const bool met = threadIdx.x < 32 ? tc::bar_wait<tc::kCluster>(at, 0, &stop, limit)
                                      : tc::bar_wait(at, 0, &stop, tc::kWaitLimitCycles);
    if (threadIdx.x < 32) tc::bar_drain(at, 0, clock64(), limit / 4);
    const bool any_met = __syncthreads_or(met);
    if (threadIdx.x == 0 && !any_met && stop) {
        *gave_up = 1u;
        set_error(err, EP_DEVERR_TIMEOUT);
    }
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
    const auto kernel = bf16_kernel(false, true, 128, false);
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
// its rows are few (it then waits for weights). A tile's epilogue takes 4 or 9 with pairs, else 0.7 for each 32 rows
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
    if (total(row_tiles(256) * nt, b.sm_count / 2, p.kblocks * (f8 ? 0.62 : 0.28), f8 ? 9.0 : 4.0) > best) return c;
    c.pair = true;
    c.bn = 256;
    c.na = 2;
    c.splits = 1;
    c.nt = nt;
    c.bound = p.cnt ? (int64_t)p.G * ((p.region + 255) / 256) : most / 256 + groups;
    return c;
}

// The register split of the kernels waits forever if a launch brings fewer
// registers than it moves around, so they are counted before the first launch.
bool has_registers(Kernel kernel) {
    static std::atomic<Kernel> known[32];
    for (auto& k : known) {
        const Kernel at = k.load(std::memory_order_relaxed);
        if (at == kernel) return true;
        if (at) continue;
        cudaFuncAttributes a{};
        if (cudaFuncGetAttributes(&a, kernel) != cudaSuccess || a.numRegs < 168) return false;
        k.store(kernel, std::memory_order_relaxed);
        return true;
    }
    return false;
}

// Chooses tile, split and grid and launches. x_rows: rows that x holds;
// weights: matrices in w; avg: rows of a group to expect (any count is right).
ep_status_t launch_on_device(const ep_buffer& b, LinearParams p, int64_t x_rows, int weights, int64_t avg, int64_t most,
                             cudaStream_t stream) {
    const bool f8 = p.x_scale != nullptr;
    const int size = f8 ? 1 : 2;
    p.kblocks = f8 ? p.K / 128 : (p.K + 63) / 64;
    p.vec = p.N % 4 == 0;
    p.flush = f8 ? 1 : p.out_type != EP_DTYPE_BF16 ? 8 : p.kblocks <= 128 ? p.kblocks : 32;
    if (p.flush > p.kblocks) p.flush = p.kblocks;
    const Shape c = shape_of(b, p, avg, most);
    const bool pair = c.pair;
    p.bn = c.bn;
    p.na = c.na;
    p.nt = c.nt;
    p.splits = c.splits;
    const int64_t bound = c.bound;
    if (bound * p.nt > kMaxTiles) return fail(EP_ERR_UNSUPPORTED, "too many tiles: rows x out_features");
    const bool split = p.splits > 1;
    const int sb = stage_bytes(p.na, p.bn);
    const int fixed = kControl + (split ? kInbox : kStaging);
    p.stages = (kSmemMax - fixed) / sb;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    const int smem = p.stages * sb + fixed;
    // a set fills while another is read; e4m3 hands one over for each block, and
    // more of them hide the hand-over
    const int sets = pair ? 2 : 256 / p.bn;
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

    const Kernel kernel = f8 ? e4m3_kernel(pair, split, p.bn) : bf16_kernel(pair, split, p.bn, p.flush < p.kblocks);
    if (!has_registers(kernel)) return fail(EP_ERR_CUDA, "the linear kernel was built with fewer than 168 registers");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return fail(EP_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    const int64_t tiles = bound * p.nt, pairs = b.sm_count / 2, clusters = split ? clusters_of(b, p.splits) : 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(pair ? 2 * (tiles < pairs ? tiles : pairs) : split ? p.splits * (tiles < clusters ? tiles : clusters) : tiles < b.sm_count ? tiles : b.sm_count));
    cfg.blockDim = dim3(kThreads);
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

cudaError_t launch_linear_timeout_selftest(uint32_t* err, uint32_t* gave_up, unsigned long long limit_ns,
                                           cudaStream_t stream) {
    cudaError_t e = cudaMemsetAsync(gave_up, 0, sizeof(uint32_t), stream);
    if (e != cudaSuccess) return e;
    timeout_selftest_kernel<<<1, 64, 0, stream>>>(err, gave_up, 2 * (long long)limit_ns);  // 2 cycles a nanosecond
    return cudaGetLastError();
}

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
    if (T < 0 || T != b->last_T)
        return fail(EP_ERR_INVALID, "T=%d does not match the last layout (T=%d)", T, b->last_T);
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
