// lora.cu -- low-rank adapters of many requests beside a shared projection
// (include/serving.h): Y[m] = X[m] W^T + s_i (X[m] A_i^T) B_i^T, i = adapter[m].
//
// Two launches.  shrink_kernel computes T = s_i X A_i^T for every token's own
// adapter and lays it out per (m block of the product, adapter that occurs in
// it): a [tile rows x rank] matrix whose rows of other adapters are zero.  The
// product's persistent kernel then appends, after a tile's K blocks, one run
// of K = 16 matrix instructions per such adapter, T times B_i, into the same
// fp32 accumulator in tensor memory: Y is written once and rounded once, and
// the adapters cost rank / k of the projection's matrix work per adapter in a
// tile instead of a pass over Y.  The product's launch overlaps shrink_kernel;
// only the appended steps wait for it (programmatic dependent launch).
//
// shrink_kernel: one CTA per (64 rows, range of adapters, range of K).  A row
// is loaded only for its own adapter (rows of others become zeros in shared
// memory, which also makes their T zero), so a decode batch with an adapter
// per token reads every X row and every A_i once, and a prompt of one request
// streams X once.  The CTAs of a cluster split K; their fp32 sums are added
// through distributed shared memory in rank order, scaled, rounded to the
// input type (the tensor core multiplies 16-bit operands; fp32 outputs carry T
// as two such terms) and stored.
#include <algorithm>
#include <cstring>
#include <new>

#include <cuda_runtime.h>

#include "common.cuh"
#include "elem.cuh"
#include "launch.h"
#include "serving.h"
#include "serving_host.h"

namespace dgb {

constexpr int kShrinkThreads = 128;
constexpr int kShrinkRows = 64;              // tokens of one CTA, 16 per warp
constexpr int kMaxAdapters = 4096;           // one bit each in shared memory
constexpr int kMaxTileRows = 256;

struct ShrinkParams {
    lora_args_t a;
    int64_t ldx;
    int32_t M, K, rank, adapters;
    int32_t tile_rows;        // rows of one m block of the product: 128 or 256
    int32_t max_adapters;     // slots per m block
    int32_t rank16;           // rank rounded up to 16
    int32_t cols;             // columns of T: rank16, or 2 rank16 (two terms)
    int32_t chunks_per_cta;   // 64-element chunks of K per CTA of the cluster
    void* t;
    int32_t* counts;
    int32_t* ids;
};

template <int NT>
struct ShrinkShape {
    static constexpr int kStages = NT > 16 ? 3 : 4;
    static constexpr int kStageBytes = (kShrinkRows + NT * 8) * 128;
    static constexpr int kSumPitch = NT * 8 + 4;      // floats
    static constexpr int kSmemBytes = kStages * kStageBytes + kShrinkRows * kSumPitch * 4;
};

__device__ __forceinline__ float4 load_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// NT: 8-column tiles of the rank held (rank <= 8 NT)
template <typename T, int NT>
__global__ void __launch_bounds__(kShrinkThreads) shrink_kernel(const __grid_constant__ ShrinkParams p) {
    using S = ShrinkShape<NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t bits[kMaxAdapters / 32];
    __shared__ int32_t list[kMaxTileRows];
    __shared__ int32_t row_id[kShrinkRows];
    __shared__ int32_t found;
    float* sums = reinterpret_cast<float*>(smem + S::kStages * S::kStageBytes);

    griddep_wait();
    griddep_launch_dependents();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ks = blockIdx.x, num_ks = gridDim.x;            // cluster rank and size: ranges of K
    const int row0 = blockIdx.z * kShrinkRows;
    const int tile = row0 / p.tile_rows;

    // The adapters of this m block, in ascending order.
    for (int i = threadIdx.x; i < kMaxAdapters / 32; i += kShrinkThreads) bits[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < p.tile_rows; i += kShrinkThreads) {
        const int m = tile * p.tile_rows + i;
        const int id = m < p.M ? p.a.adapter[m] : -1;
        const bool valid = id >= 0 && id < p.adapters;
        if (valid) atomicOr(&bits[id >> 5], 1u << (id & 31));
        if (m >= row0 && m < row0 + kShrinkRows) row_id[m - row0] = valid ? id : -1;
    }
    __syncthreads();
    if (warp == 0) {
        constexpr int kWords = kMaxAdapters / 32 / 32;        // words per lane
        int n = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) n += __popc(bits[lane * kWords + w]);
        int at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += t;
        }
        if (lane == 31) found = at;
        at -= n;
#pragma unroll
        for (int w = 0; w < kWords; ++w)
            for (uint32_t word = bits[lane * kWords + w]; word; word &= word - 1) list[at++] = (lane * kWords + w) * 32 + __ffs(word) - 1;
    }
    __syncthreads();
    const int count = found;
    if (ks == 0 && blockIdx.y == 0 && row0 % p.tile_rows == 0) {
        if (threadIdx.x == 0) p.counts[tile] = count;
        for (int i = threadIdx.x; i < count; i += kShrinkThreads) p.ids[(size_t)tile * p.max_adapters + i] = list[i];
    }

    const int chunks = (p.K + 63) / 64;
    const int c_begin = min(ks * p.chunks_per_cta, chunks), c_end = min(c_begin + p.chunks_per_cta, chunks);
    const uint32_t ring = smem_u32(smem);
    const T* X = static_cast<const T*>(p.a.x);
    const T* A = static_cast<const T*>(p.a.a);

    for (int slot = blockIdx.y; slot < count; slot += gridDim.y) {
        const int id = list[slot];
        T* dst = static_cast<T*>(p.t) + (((size_t)tile * p.max_adapters + slot) * p.tile_rows + row0 % p.tile_rows) * p.cols;
        const bool here = __syncthreads_or(threadIdx.x < kShrinkRows && row_id[threadIdx.x] == id);
        if (!here) {
            // none of these rows: zeros, shared by the cluster's CTAs
            uint4* z = reinterpret_cast<uint4*>(dst);
            const int n = kShrinkRows * p.cols / 8;
            for (int i = ks * kShrinkThreads + threadIdx.x; i < n; i += num_ks * kShrinkThreads) z[i] = make_uint4(0, 0, 0, 0);
            continue;
        }
        const bool warp_here = __any_sync(0xffffffffu, lane < 16 && row_id[warp * 16 + (lane & 15)] == id);
        const T* Ai = A + id * p.a.stride_a;
        auto load = [&](int chunk, int stage) {
            const uint32_t sx = ring + stage * S::kStageBytes, sa = sx + kShrinkRows * 128;
            const int c = threadIdx.x & 7;
            const int k = chunk * 64 + c * 8;
            const uint32_t bytes = (uint32_t)min(max(p.K - k, 0), 8) * 2u;
#pragma unroll
            for (int i = 0; i < kShrinkRows / 16; ++i) {
                const int r = (threadIdx.x >> 3) + 16 * i;
                const bool mine = bytes && row_id[r] == id;
                cp_async_16_zfill(sx + r * 128 + ((c ^ (r & 7)) << 4), mine ? X + (int64_t)(row0 + r) * p.ldx + k : X, mine ? bytes : 0u);
            }
#pragma unroll
            for (int i = 0; i < NT / 2; ++i) {
                const int r = (threadIdx.x >> 3) + 16 * i;
                const bool in = bytes && r < p.rank;
                cp_async_16_zfill(sa + r * 128 + ((c ^ (r & 7)) << 4), in ? Ai + (int64_t)r * p.a.lda + k : A, in ? bytes : 0u);
            }
        };
        float acc[NT][4] = {};
#pragma unroll
        for (int s = 0; s < S::kStages - 1; ++s) {
            if (c_begin + s < c_end) load(c_begin + s, s);
            cp_async_commit();
        }
        int stage = 0;
        for (int ch = c_begin; ch < c_end; ++ch) {
            cp_async_wait<S::kStages - 2>();
            __syncthreads();
            const int next = ch + S::kStages - 1;
            const int fill = stage == 0 ? S::kStages - 1 : stage - 1;
            if (next < c_end) load(next, fill);
            cp_async_commit();
            if (warp_here) {
                const uint32_t sx = ring + stage * S::kStageBytes, sa = sx + kShrinkRows * 128;
                const int xr = warp * 16 + (lane & 15), ar = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    uint32_t x[4];
                    ldmatrix_x4(sx + xr * 128 + (((kk * 2 + (lane >> 4)) ^ (xr & 7)) << 4), x);
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t b[4];
                        ldmatrix_x4(sa + (n * 8 + ar) * 128 + (((kk * 2 + ((lane >> 3) & 1)) ^ (ar & 7)) << 4), b);
                        mma_16816<T>(acc[n], x, b[0], b[1]);
                        mma_16816<T>(acc[n + 1], x, b[2], b[3]);
                    }
                }
            }
            if (++stage == S::kStages) stage = 0;
        }
        cp_async_wait<0>();
        // this CTA's sums over its range of K
        {
            const int r = warp * 16 + (lane >> 2), c = (lane & 3) * 2;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<float2*>(sums + r * S::kSumPitch + n * 8 + c) = make_float2(acc[n][0], acc[n][1]);
                *reinterpret_cast<float2*>(sums + (r + 8) * S::kSumPitch + n * 8 + c) = make_float2(acc[n][2], acc[n][3]);
            }
        }
        cluster_sync();
        // the cluster's: CTA ks finishes rows [64 ks / num_ks, 64 (ks + 1) / num_ks)
        const float scale = p.a.scale ? p.a.scale[id] : 1.f;
        const int rows = kShrinkRows / num_ks, groups = p.rank16 / 8;
        const uint32_t mine = smem_u32(sums);
        for (int i = threadIdx.x; i < rows * groups; i += kShrinkThreads) {
            const int r = ks * rows + i / groups, c = (i % groups) * 8;
            float v[8] = {};
            for (int q = 0; q < num_ks; ++q) {
                const uint32_t from = map_to_cta(mine, (uint32_t)q) + (uint32_t)(r * S::kSumPitch + c) * 4u;
                const float4 lo = load_cluster_f4(from), hi = load_cluster_f4(from + 16);
                v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
                v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= scale;
            const uint4 first = round8<T>(v);
            *reinterpret_cast<uint4*>(dst + (size_t)r * p.cols + c) = first;
            if (p.cols > p.rank16) {
                float back[8];
                unpack8<T>(first, back);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] -= back[j];
                *reinterpret_cast<uint4*>(dst + (size_t)r * p.cols + p.rank16 + c) = round8<T>(v);
            }
        }
        cluster_sync();     // the sums are read; the next slot may overwrite them and the ring
    }
}

template <typename T, int NT>
static cudaError_t launch_shrink_typed(const ShrinkParams& p, dim3 grid, cudaStream_t stream) {
    auto kern = shrink_kernel<T, NT>;
    static std::atomic<int> smem_set[kMaxDevices];
    cudaError_t e = ensure_smem_limit(kern, ShrinkShape<NT>::kSmemBytes, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kShrinkThreads);
    cfg.dynamicSmemBytes = ShrinkShape<NT>::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = grid.x;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T>
static cudaError_t launch_shrink(const ShrinkParams& p, dim3 grid, cudaStream_t stream) {
    if (p.rank16 <= 16) return launch_shrink_typed<T, 2>(p, grid, stream);
    if (p.rank16 <= 32) return launch_shrink_typed<T, 4>(p, grid, stream);
    if (p.rank16 <= 64) return launch_shrink_typed<T, 8>(p, grid, stream);
    if (p.rank16 <= 128) return launch_shrink_typed<T, 16>(p, grid, stream);
    return launch_shrink_typed<T, 32>(p, grid, stream);
}

}  // namespace dgb

using namespace dgb;

struct lora_plan_s {
    lora_desc_t desc;
    lora_plan_info_t info;
    gemm_plan_t product = nullptr;
    void* memory = nullptr;       // T, counts, ids
    int64_t t_bytes = 0, count_bytes = 0;
    int32_t m_blocks = 0, rank16 = 0, cols = 0;
    int32_t chunks_per_cta = 0, slot_groups = 0;
};

namespace {

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

gemm_status_t check_desc(const lora_desc_t& d) {
    if (d.tokens < 0 || d.n < 1 || d.k < 1 || d.rank < 1 || d.adapters < 1) return GEMM_ERR_INVALID_ARG;
    if (d.dtype != GEMM_BF16 && d.dtype != GEMM_F16) return GEMM_ERR_UNSUPPORTED;
    if (d.dtype_y != GEMM_F32 && d.dtype_y != GEMM_BF16 && d.dtype_y != GEMM_F16) return GEMM_ERR_UNSUPPORTED;
    if (d.rank % 8 != 0 || d.rank > 256 || d.adapters > kMaxAdapters) return GEMM_ERR_UNSUPPORTED;
    if (d.tokens > 65535ll * kShrinkRows) return GEMM_ERR_UNSUPPORTED;      // the shrink grid's z extent
    const uint32_t known = GEMM_FLAG_CTA_GROUP_1 | GEMM_FLAG_CTA_GROUP_2 | GEMM_FLAG_NO_STREAM_K | GEMM_FLAG_STAGE_K1 | GEMM_FLAG_STAGE_K2;
    if (d.flags & ~known) return GEMM_ERR_UNSUPPORTED;
    if (d.tile_n > 256) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t lora_plan_create(lora_plan_t* out, const lora_desc_t* desc) {
    if (!out || !desc) return GEMM_ERR_INVALID_ARG;
    *out = nullptr;
    const lora_desc_t& d = *desc;
    gemm_status_t s = check_desc(d);
    if (s != GEMM_OK) return s;
    DeviceFacts dev;
    if ((s = device_facts(&dev)) != GEMM_OK) return s;
    gemm_desc_t g{};
    g.M = d.tokens;
    g.N = d.n;
    g.K = d.k;
    g.batch = 1;
    g.dtype_a = g.dtype_b = d.dtype;
    g.dtype_d = d.dtype_y;
    g.lda = d.ldx;
    g.ldb = d.ldw;
    g.ldd = d.ldy;
    g.flags = d.flags | GEMM_FLAG_NO_SINGLE_CTA;
    g.tile_n = d.tile_n;
    g.stages = d.stages;
    g.max_ctas = d.max_ctas;
    g.wait_timeout_ns = d.wait_timeout_ns;
    lora_plan_s* p = new (std::nothrow) lora_plan_s();
    if (!p) return GEMM_ERR_RESOURCES;
    p->desc = d;
    if (p->desc.ldx == 0) p->desc.ldx = d.k;
    s = gemm_plan_create(&p->product, &g);
    gemm_plan_info_t info{};
    if (s == GEMM_OK) s = gemm_plan_info(p->product, &info);
    if (s == GEMM_OK && info.tile_n > 256) {
        // 512-wide tiles hand their accumulator back in halves, the second with the next tile's work under way;
        // the appended steps keep to one accumulator per tile
        gemm_plan_destroy(p->product);
        p->product = nullptr;
        g.tile_n = 256;
        s = gemm_plan_create(&p->product, &g);
        if (s == GEMM_OK) s = gemm_plan_info(p->product, &info);
    }
    if (s != GEMM_OK) {
        lora_plan_destroy(p);
        return s;
    }
    p->info.product = info;
    p->rank16 = (int32_t)up(d.rank, 16);
    p->cols = d.dtype_y == GEMM_F32 ? 2 * p->rank16 : p->rank16;
    p->info.steps_per_adapter = p->cols / 16;
    if (d.tokens > 0) {
        p->m_blocks = (int32_t)((d.tokens + info.tile_m - 1) / info.tile_m);
        const int64_t slots = std::min<int64_t>(d.adapters, std::min<int64_t>(info.tile_m, d.tokens));
        p->info.max_adapters_per_tile = (int32_t)slots;
        // Grid of shrink_kernel: clusters split K while that fills the device twice over and leaves every CTA four
        // chunks of K; then CTAs share out the slots.
        const int64_t row_blocks = (d.tokens + kShrinkRows - 1) / kShrinkRows, chunks = (d.k + 63) / 64;
        int64_t ks = 1;
        while (ks < 8 && row_blocks * ks * 2 <= 2 * dev.sms && chunks >= 4 * ks * 2) ks *= 2;
        p->chunks_per_cta = (int32_t)((chunks + ks - 1) / ks);
        p->slot_groups = (int32_t)std::min<int64_t>(slots, std::max<int64_t>(1, 4 * dev.sms / (row_blocks * ks)));
        p->info.shrink_k_split = (int32_t)ks;
        p->info.shrink_grid = (int32_t)(row_blocks * ks * p->slot_groups);
        p->t_bytes = up((int64_t)p->m_blocks * slots * info.tile_m * p->cols * 2, 256);
        p->count_bytes = up((int64_t)p->m_blocks * 4, 256);
        const int64_t bytes = p->t_bytes + p->count_bytes + (int64_t)p->m_blocks * slots * 4;
        p->info.workspace_bytes = bytes + info.workspace_bytes;
        const cudaError_t e = cudaMalloc(&p->memory, (size_t)bytes);
        if (e != cudaSuccess) {
            lora_plan_destroy(p);
            return status_of(e);
        }
    }
    *out = p;
    return GEMM_OK;
}

gemm_status_t lora_plan_info(lora_plan_t plan, lora_plan_info_t* info) {
    if (!plan || !info) return GEMM_ERR_INVALID_ARG;
    *info = plan->info;
    return GEMM_OK;
}

gemm_status_t lora_run(lora_plan_t plan, const lora_args_t* args, gemm_stream_t stream_) {
    if (!plan || !args) return GEMM_ERR_INVALID_ARG;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const lora_desc_t& d = plan->desc;
    if (d.tokens == 0) return GEMM_OK;
    ShrinkParams q;
    std::memset(&q, 0, sizeof(q));
    q.a = *args;
    lora_args_t& a = q.a;
    if (!a.x || !a.w || !a.a || !a.b || !a.adapter || !a.y) return GEMM_ERR_INVALID_ARG;
    if (a.lda == 0) a.lda = d.k;
    if (a.stride_a == 0) a.stride_a = d.rank * a.lda;
    if (a.ldb == 0) a.ldb = d.rank;
    if (a.stride_b == 0) a.stride_b = d.n * a.ldb;
    if (a.lda < d.k || a.ldb < d.rank || a.stride_a < 0 || a.stride_b < 0) return GEMM_ERR_INVALID_ARG;
    const int64_t ldw = d.ldw ? d.ldw : d.k, ldy = d.ldy ? d.ldy : d.n, y_bytes = d.dtype_y == GEMM_F32 ? 4 : 2;
    if (!all_aligned(16, {a.x, a.w, a.a, a.b, a.y})) return GEMM_ERR_ALIGNMENT;
    if (!all_multiples(8, {d.ldx, ldw, a.lda, a.stride_a, a.ldb, a.stride_b}) || ldy * y_bytes % 16 != 0) return GEMM_ERR_ALIGNMENT;
    const gemm_plan_info_t& info = plan->info.product;
    PersistentParams p;
    gemm_status_t s = product_params(plan->product, a.x, a.w, a.y, &p);
    if (s != GEMM_OK) return s;
    char* mem = static_cast<char*>(plan->memory);
    q.ldx = d.ldx;
    q.M = (int32_t)d.tokens;
    q.K = (int32_t)d.k;
    q.rank = d.rank;
    q.adapters = d.adapters;
    q.tile_rows = info.tile_m;
    q.max_adapters = plan->info.max_adapters_per_tile;
    q.rank16 = plan->rank16;
    q.cols = plan->cols;
    q.chunks_per_cta = plan->chunks_per_cta;
    q.t = mem;
    q.counts = reinterpret_cast<int32_t*>(mem + plan->t_bytes);
    q.ids = reinterpret_cast<int32_t*>(mem + plan->t_bytes + plan->count_bytes);
    LoraTail tail;
    s = encode_steps_map(&tail.tmap_t, d.dtype, q.t, q.cols, q.tile_rows, (int64_t)plan->m_blocks * q.max_adapters, q.cols,
                         (int64_t)q.tile_rows * q.cols, 128);
    if (s != GEMM_OK) return s;
    // one adapter: the stride is never used but has to be a valid one
    const int64_t stride_b = d.adapters > 1 ? a.stride_b : d.n * a.ldb;
    if ((s = encode_steps_map(&tail.tmap_b, d.dtype, a.b, d.rank, d.n, d.adapters, a.ldb, stride_b, info.tile_n / info.cta_group)) != GEMM_OK)
        return s;
    tail.counts = q.counts;
    tail.ids = q.ids;
    tail.max_adapters = q.max_adapters;
    tail.steps = q.cols / 16;
    tail.b_steps = q.rank16 / 16;
    const dim3 grid((unsigned)plan->info.shrink_k_split, (unsigned)plan->slot_groups, (unsigned)((d.tokens + kShrinkRows - 1) / kShrinkRows));
    cudaError_t e = d.dtype == GEMM_BF16 ? launch_shrink<__nv_bfloat16>(q, grid, stream) : launch_shrink<__half>(q, grid, stream);
    if (e != cudaSuccess) return status_of(e);
    return status_of(launch_adapters(p, tail, info.cta_group, d.dtype_y, info.grid, (size_t)info.smem_bytes, stream));
}

gemm_status_t lora_sync_status(lora_plan_t plan, gemm_stream_t stream, gemm_device_error_t* out) {
    if (!plan) return GEMM_ERR_INVALID_ARG;
    return gemm_sync_status(plan->product, stream, out);
}

gemm_status_t lora_plan_destroy(lora_plan_t plan) {
    if (!plan) return GEMM_OK;
    gemm_status_t s = gemm_plan_destroy(plan->product);
    const cudaError_t e = cudaFree(plan->memory);
    delete plan;
    return e == cudaSuccess ? s : status_of(e);
}

}  // extern "C"
