// lora.cu -- low-rank adapters of many requests beside a shared projection
// (include/serving.h): Y[m] = X[m] W^T + s_i (X[m] A_i^T) B_i^T, i = adapter[m].
//
// Two launches.  A first kernel computes T = s_i X A_i^T for every token's own
// adapter and lays it out per m block of the product: [tile rows][slot][rank],
// one slot for each adapter that occurs among the block's rows, rows of other
// adapters zero.  The product's persistent kernel then appends, after a tile's
// K blocks, one run of K = 16 matrix instructions per slot, T times that
// adapter's B, into the same fp32 accumulator in tensor memory: Y is written
// once and rounded once, and the adapters cost rank / k of the projection's
// matrix work per adapter in a tile instead of a pass over Y.  The product's
// launch overlaps the first kernel; only the appended steps wait for it
// (programmatic dependent launch).
//
// T is rounded to the input type before its product (the tensor core
// multiplies 16-bit operands); fp32 outputs carry it as two such terms.  Its
// sums are fp32, added in a fixed order.
//
// Two forms of the first kernel:
//   gather_kernel, for decode batches (each adapter with few rows): a CTA per
//   token, of which every eighth of an adapter goes on, with its row and the
//   adapter's next seven.  Its time is latency, so nothing is staged: eight
//   warps split K and load 16-byte pieces of A_i and of the rows straight into
//   matrix fragments, many at once;
//   stream_kernel, above that (prompts, long runs of one adapter): one CTA per
//   (64 rows, range of slots, range of K); a row is loaded only for its own
//   adapter (others are zeros in shared memory), the CTAs of a cluster split K
//   and add their sums through distributed shared memory.
//
// Bounds, GB300.  Few tokens: the bytes of W and the adapters, 34 MB for 4
// tokens x 4096 x 4096 with two adapters of rank 16: 11.0 us, 3.1 TB/s; 56 MB
// for 96 tokens with 80 adapters: 17.5 us, 3.2 TB/s (8.6 and 10.6 with no
// token's adapter set).  What keeps it from the 6.8 TB/s of a plain copy is the
// chain of steps around the stream: T (7 to 9 us beside the stream of W), the
// adapter steps that wait for it (1.7), the join of the cluster and the stores
// (2 to 3).  Above rank 32 also that the two kernels no longer share an SM (see
// plan_skinny): 96 tokens with 80 adapters of rank 64 take 48 us at a floor of
// 18, of rank 128 72 at 30.  Many tokens: the tensor cores, 8192 x 8192 x 8192
// with prompts of 12 requests and rank 64: 619 us on a cool device, 638 on a warm
// one (power cap), 1.75 to 1.80 PFLOP/s, of which T takes 44; the plain product
// in the same minute 612.  Between those, T is what stands out: it is complete
// before the adapter steps begin and does not shrink with the product (1024 x
// 2048 x 2048 with 8 adapters of rank 16: 19.2 us, 15.4 with no adapter set, the
// plain product 10.8), and where the rows of a 64-row block have many adapters
// the streamed form multiplies all 64 rows for each of them (4096 x 4096 x 4096,
// 32 adapters of rank 16 mixed token by token: 239 us, the plain product 82).
// fp32 outputs run twice the adapter steps and, in the persistent kernel, spill
// (104 bytes stored a thread): 96 tokens 20.2 us, 8192^3 667.
#include <algorithm>
#include <cstring>
#include <new>

#include <cuda_runtime.h>

#include "common.cuh"
#include "elem.cuh"
#include "launch.h"
#include "lora_list.cuh"
#include "lora_skinny.h"
#include "ptx.cuh"
#include "serving.h"
#include "serving_host.h"

namespace dgb {

constexpr int kShrinkThreads = 128;
constexpr int kShrinkRows = 64;              // tokens of one CTA, 16 per warp
constexpr int kGatherTokens = 256;

struct ShrinkParams {
    lora_args_t a;
    int64_t ldx;
    int32_t M, K, rank, adapters;
    int32_t tile_rows;        // rows of one m block of the product: 128 or 256
    int32_t max_adapters;     // slots per m block
    int32_t rank16;           // rank rounded up to 16
    int32_t cols;             // columns of T per slot: rank16, or 2 rank16 (two terms)
    int32_t pitch;            // elements between rows of T: max_adapters * cols
    int32_t chunks_per_cta;   // 64-element chunks of K per CTA of the cluster
    void* t;
    int32_t* counts;
    int32_t* ids;
};

template <int NT>
struct StreamShape {
    static constexpr int kStages = 3;
    static constexpr int kStageBytes = (kShrinkRows + NT * 8) * 128;
    static constexpr int kSumPitch = NT * 8 + 4;      // floats; the sums lie over the ring
    static constexpr int kSmemBytes = kStages * kStageBytes;
    static_assert(kShrinkRows * kSumPitch * 4 <= kSmemBytes, "");
};

__device__ __forceinline__ void publish_adapters(const ShrinkParams& p, int tile, const AdapterList& l, int count) {
    if (threadIdx.x == 0) p.counts[tile] = count;
    for (int i = threadIdx.x; i < count; i += kShrinkThreads) p.ids[(size_t)tile * p.max_adapters + i] = l.list[i];
}

// Eight scaled sums as T's row piece: one term, or for fp32 outputs the rounded value and what the rounding left.  Nothing is
// left of an infinity (an f16 sum past 65504 among them): the difference would be a NaN.
template <typename T>
__device__ __forceinline__ void store_t(const ShrinkParams& p, T* at, float (&v)[8], float scale) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= scale;
    const uint4 first = round8<T>(v);
    *reinterpret_cast<uint4*>(at) = first;
    if (p.cols > p.rank16) {
        float back[8];
        unpack8<T>(first, back);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = back[j] - back[j] == 0.f ? v[j] - back[j] : 0.f;
        *reinterpret_cast<uint4*>(at + p.rank16) = round8<T>(v);
    }
}

constexpr int kGatherWarps = 8, kGatherThreads = 32 * kGatherWarps;
constexpr int kGatherRows = 8;               // tokens of one CTA: the columns of the matrix instruction

// The 16 bytes at elements k .. k + 7 of a row of K elements; elements past the row's end are zeros and not read.
template <typename T>
__device__ __forceinline__ uint4 load_piece(const T* row, int k, int K, bool in) {
    if (in && k + 8 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (in && k < K) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < K) w[e / 2] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(row + k + e)) << (16 * (e & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// MT: 16-row tiles of the rank held (rank <= 16 MT).  The matrix instruction has A_i's rows as its 16 rows and the tokens
// as its 8 columns.  Lane (g, j) = (lane / 4, lane % 4) loads elements 8 j .. 8 j + 7 of every 32 of K of its rows: two
// instructions' worth of fragments, in an order of k that is the same for both operands, so that no data moves between
// lanes.
template <typename T, int MT>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ ShrinkParams p) {
    constexpr int kBatch = MT == 1 ? 8 : (MT == 2 ? 4 : (MT == 4 ? 2 : 1));     // 32-element chunks whose loads are in flight
    constexpr int kSumPitch = MT * 16 + 4;
    __shared__ uint32_t bits[kMaxAdapters / 32];         // adapters that occur in the m block
    __shared__ uint32_t same[kMaxTileRows / 32];         // its rows of this CTA's adapter
    __shared__ __align__(16) float sums[kGatherWarps][kGatherRows][kSumPitch];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.y, lead = blockIdx.x, m0 = tile * p.tile_rows;
    const int words = (p.adapters + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kGatherThreads) bits[i] = 0u;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    auto adapter_of = [&](int i) {       // of row i of the m block; -1: none
        if (i >= p.tile_rows || m0 + i >= p.M) return -1;
        const int a = p.a.adapter[m0 + i];
        return a >= 0 && a < p.adapters ? a : -1;
    };
    static_assert(kGatherThreads == kMaxTileRows, "a thread per row");
    const int id = adapter_of(lead), mine = adapter_of(threadIdx.x);
    if (mine >= 0) atomicOr(&bits[mine >> 5], 1u << (mine & 31));
    const uint32_t ballot = __ballot_sync(0xffffffffu, mine == id);
    if (lane == 0) same[warp] = ballot;
    __syncthreads();
    if (lead == 0 && warp == 0) {
        // the m block's list of adapters, for the product
        const int count = list_bits(bits, words, lane, p.ids + (size_t)tile * p.max_adapters);
        if (lane == 0) p.counts[tile] = count;
    }
    if (id < 0) return;
    // This row leads a group if the number of its adapter's rows before it is a multiple of eight.
    int before = 0;
#pragma unroll
    for (int w = 0; w < kMaxTileRows / 32; ++w)
        before += __popc(same[w] & (w < (lead >> 5) ? 0xffffffffu : (w == (lead >> 5) ? (1u << (lead & 31)) - 1u : 0u)));
    if (before % kGatherRows != 0) return;
    // its slot: adapters of the block with smaller numbers
    int slot = 0;
    for (int w = lane; w < words; w += 32)
        slot += __popc(bits[w] & (w < (id >> 5) ? 0xffffffffu : (w == (id >> 5) ? (1u << (id & 31)) - 1u : 0u)));
    slot = __reduce_add_sync(0xffffffffu, slot);
    // the i-th row of the group, counted from the leader; -1 past the last
    auto row_of = [&](int i) {
        int skip = before + i;
        for (int w = 0; w < kMaxTileRows / 32; ++w) {
            const int here = __popc(same[w]);
            if (skip < here) {
                uint32_t left = same[w];
                for (; skip > 0; --skip) left &= left - 1;
                return w * 32 + __ffs(left) - 1;
            }
            skip -= here;
        }
        return -1;
    };

    const int g = lane >> 2, j = lane & 3;
    const int chunks = (p.K + 31) / 32;
    const int c_end = chunks * (warp + 1) / kGatherWarps;
    const int my_row = row_of(g);
    const bool in_x = my_row >= 0;
    const T* X = static_cast<const T*>(p.a.x) + (int64_t)(m0 + (in_x ? my_row : 0)) * p.ldx;
    const T* A = static_cast<const T*>(p.a.a) + id * p.a.stride_a + (int64_t)g * p.a.lda;
    const int64_t a_step = 8 * p.a.lda;
    float acc[MT][4] = {};
    const int c_begin = chunks * warp / kGatherWarps;
    // A_i comes from DRAM: what the first batch does not load is brought to L2 meanwhile
    for (int c = c_begin + kBatch; c < c_end; c += 2) {
        // 128 bytes of a row: two chunks, one lane in four
        const int k = c * 32 + j * 8;
#pragma unroll
        for (int t = 0; t < 2 * MT; ++t)
            if (j == 0 && t * 8 + g < p.rank && k < p.K) asm volatile("prefetch.global.L2 [%0];" ::"l"(A + t * a_step + k));
    }
    for (int c = c_begin; c < c_end; c += kBatch) {
        uint4 x[kBatch], w[kBatch][2 * MT];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int k = (c + u) * 32 + j * 8;
            const bool in = c + u < c_end;
            x[u] = load_piece(X, k, p.K, in && in_x);
#pragma unroll
            for (int t = 0; t < 2 * MT; ++t) w[u][t] = load_piece(A + t * a_step, k, p.K, in && t * 8 + g < p.rank);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const uint4 &lo = w[u][2 * t], &hi = w[u][2 * t + 1];
                const uint32_t f0[4] = {lo.x, hi.x, lo.y, hi.y}, f1[4] = {lo.z, hi.z, lo.w, hi.w};
                mma_16816<T>(acc[t], f0, x[u].x, x[u].y);
                mma_16816<T>(acc[t], f1, x[u].z, x[u].w);
            }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        sums[warp][2 * j][t * 16 + g] = acc[t][0];
        sums[warp][2 * j + 1][t * 16 + g] = acc[t][1];
        sums[warp][2 * j][t * 16 + g + 8] = acc[t][2];
        sums[warp][2 * j + 1][t * 16 + g + 8] = acc[t][3];
    }
    T* dst = static_cast<T*>(p.t) + (size_t)tile * p.tile_rows * p.pitch + slot * p.cols;
    if (before == 0) {
        // zeros in the other rows (those of tokens that exist)
        const int live = min(p.tile_rows, p.M - m0), pieces = p.cols / 8;
        for (int i = threadIdx.x; i < live * pieces; i += kGatherThreads) {
            const int r = i / pieces;
            if (!((same[r >> 5] >> (r & 31)) & 1u)) *reinterpret_cast<uint4*>(dst + (size_t)r * p.pitch + (i - r * pieces) * 8) = make_uint4(0, 0, 0, 0);
        }
    }
    __syncthreads();
    const float scale = p.a.scale ? p.a.scale[id] : 1.f;
    const int groups = p.rank16 / 8;
    for (int i = threadIdx.x; i < kGatherRows * groups; i += kGatherThreads) {
        const int r = i / groups, c = (i - r * groups) * 8;
        const int row = row_of(r);
        if (row < 0) break;
        float v[8] = {};
#pragma unroll
        for (int q = 0; q < kGatherWarps; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += sums[q][r][c + e];
        store_t<T>(p, dst + (size_t)row * p.pitch + c, v, scale);
    }
}

template <typename T, int NT>
__global__ void __launch_bounds__(kShrinkThreads) stream_kernel(const __grid_constant__ ShrinkParams p) {
    using S = StreamShape<NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ AdapterList adapters;
    __shared__ int32_t row_id[kShrinkRows];
    float* sums = reinterpret_cast<float*>(smem);

    griddep_wait();
    griddep_launch_dependents();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ks = blockIdx.x, num_ks = gridDim.x;            // cluster rank and size: ranges of K
    const int row0 = blockIdx.y * kShrinkRows;
    const int tile = row0 / p.tile_rows, in_tile = row0 % p.tile_rows;
    const int count = find_adapters(p.a.adapter, p.adapters, p.M, tile * p.tile_rows, p.tile_rows, adapters, row_id, in_tile, kShrinkRows,
                                    threadIdx.x, kShrinkThreads, [] { __syncthreads(); });
    if (ks == 0 && blockIdx.z == 0 && in_tile == 0) publish_adapters(p, tile, adapters, count);

    const int chunks = (p.K + 63) / 64;
    const int c_begin = min(ks * p.chunks_per_cta, chunks), c_end = min(c_begin + p.chunks_per_cta, chunks);
    const uint32_t ring = smem_u32(smem);
    const T* X = static_cast<const T*>(p.a.x);
    const T* A = static_cast<const T*>(p.a.a);

    for (int slot = blockIdx.z; slot < count; slot += gridDim.z) {
        const int id = adapters.list[slot];
        T* dst = static_cast<T*>(p.t) + ((size_t)tile * p.tile_rows + in_tile) * p.pitch + slot * p.cols;
        const bool here = __syncthreads_or(threadIdx.x < kShrinkRows && row_id[threadIdx.x] == id);
        if (!here) {
            // none of these rows: zeros, shared by the cluster's CTAs
            const int pieces = p.cols / 8;
            for (int i = ks * kShrinkThreads + threadIdx.x; i < kShrinkRows * pieces; i += num_ks * kShrinkThreads) {
                const int r = i / pieces;
                *reinterpret_cast<uint4*>(dst + (size_t)r * p.pitch + (i - r * pieces) * 8) = make_uint4(0, 0, 0, 0);
            }
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
        __syncthreads();        // the ring is idle
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
            // a row of another adapter has to stay zero, also where A_i holds infinities or NaN
            if (row_id[r] != id) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.f;
            }
            store_t<T>(p, dst + (size_t)r * p.pitch + c, v, row_id[r] == id ? scale : 1.f);
        }
        cluster_sync();     // the sums are read; the next slot may overwrite them and the ring
    }
}

template <typename T, int NT>
static cudaError_t launch_stream_typed(const ShrinkParams& p, dim3 grid, cudaStream_t stream) {
    auto kern = stream_kernel<T, NT>;
    static std::atomic<int> smem_set[kMaxDevices];
    cudaError_t e = ensure_smem_limit(kern, StreamShape<NT>::kSmemBytes, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kShrinkThreads);
    cfg.dynamicSmemBytes = StreamShape<NT>::kSmemBytes;
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

// Whether the plan's first kernel gathers rows (see the top of this file): always for a decode batch; up to 1024 tokens where
// an adapter has few of them on average (GB300, 400 x 4096 x 4096 with 64 adapters: 33 to 34 us against 62 streamed; 777 x 1543 x
// 1001 with 5: 15.6 against 12.9).  A rank above 128 does not fit its registers.
static bool gathers(const lora_desc_t& d) {
    return d.rank <= 128 && (d.tokens <= kGatherTokens || (d.tokens <= 1024 && d.tokens <= 16 * (int64_t)d.adapters));
}

template <typename T>
static cudaError_t launch_shrink(const ShrinkParams& p, bool gather, dim3 grid, cudaStream_t stream) {
    if (gather) {
        const dim3 block(kGatherThreads);
        if (p.rank16 <= 16) return launch_dependent(gather_kernel<T, 1>, grid, block, 0, stream, p);
        if (p.rank16 <= 32) return launch_dependent(gather_kernel<T, 2>, grid, block, 0, stream, p);
        if (p.rank16 <= 64) return launch_dependent(gather_kernel<T, 4>, grid, block, 0, stream, p);
        return launch_dependent(gather_kernel<T, 8>, grid, block, 0, stream, p);
    }
    if (p.rank16 <= 16) return launch_stream_typed<T, 2>(p, grid, stream);
    if (p.rank16 <= 32) return launch_stream_typed<T, 4>(p, grid, stream);
    if (p.rank16 <= 64) return launch_stream_typed<T, 8>(p, grid, stream);
    if (p.rank16 <= 128) return launch_stream_typed<T, 16>(p, grid, stream);
    return launch_stream_typed<T, 32>(p, grid, stream);
}

}  // namespace dgb

using namespace dgb;

struct lora_plan_s {
    lora_desc_t desc;
    lora_plan_info_t info;
    gemm_plan_t product = nullptr;
    int device = 0;
    void* memory = nullptr;       // T, counts, ids
    int64_t t_bytes = 0, count_bytes = 0;
    int32_t m_blocks = 0, rank16 = 0, cols = 0;
    int32_t chunks_per_cta = 0;
    dim3 shrink_grid;
    bool gather = false;
    bool skinny = false;          // few output tiles: lora_skinny.cu instead of the persistent kernel
    int32_t tile_rows = 0;        // rows of an m block
    SkinnyParams sk = {};         // everything but pointers and maps
    dim3 skinny_grid;
    size_t skinny_smem = 0;
};

namespace {

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

gemm_status_t check_desc(const lora_desc_t& d) {
    if (d.tokens < 0 || d.n < 1 || d.k < 1 || d.rank < 1 || d.adapters < 1) return GEMM_ERR_INVALID_ARG;
    if (d.dtype != GEMM_BF16 && d.dtype != GEMM_F16) return GEMM_ERR_UNSUPPORTED;
    if (d.dtype_y != GEMM_F32 && d.dtype_y != GEMM_BF16 && d.dtype_y != GEMM_F16) return GEMM_ERR_UNSUPPORTED;
    if (d.rank % 8 != 0 || d.rank > 256 || d.adapters > kMaxAdapters) return GEMM_ERR_UNSUPPORTED;
    if (d.tokens > 65535ll * kShrinkRows) return GEMM_ERR_UNSUPPORTED;      // the shrink grid's y extent
    const uint32_t known = GEMM_FLAG_CTA_GROUP_1 | GEMM_FLAG_CTA_GROUP_2 | GEMM_FLAG_NO_STREAM_K | GEMM_FLAG_STAGE_K1 | GEMM_FLAG_STAGE_K2;
    if (d.flags & ~known) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// Tiles and K split of the few-tile kernel; false: the persistent kernel.  On GB300 up to 256 tokens ran 1.3 to 1.9 times
// faster in one wave of this kernel than in the persistent one (4 x 4096 x 4096: 11.1 against 21.5 us; 200 x 4096 x 4096:
// 21.1 against 27.3); up to 512 tokens it still pays on long K (300 x 1024 x 4096: 15.9 against 18.8; 512 x 4096 x 4096: 27.3
// against 28.9), and not on short K or with more tiles (777 x 1543 x 1001: 17.7 against 12.7).  Clusters of eight leave SMs
// without a place in one (128 CTAs of 96 x 4096 x 4096: 38.5 us, in fours 24.9), and a second wave costs as much as the
// first.  Within that: the least time a CTA takes to bring in its operands (about 50 bytes a cycle into an SM and 100
// cycles a stage) and, in a cluster, to join (2,000 cycles and a tenth of one per element).
bool plan_skinny(const lora_desc_t& d, const DeviceFacts& dev, lora_plan_s* p) {
    // a forced choice of the persistent kernel's parameters keeps it
    if (d.flags || d.tile_n || d.stages || d.max_ctas) return false;
    const int64_t m_blocks = (d.tokens + 127) / 128, k_blocks = (d.k + 63) / 64;
    if (d.tokens > 256 && (d.tokens > 512 || d.k < 2048 || m_blocks * ((d.n + 127) / 128) > dev.sms)) return false;
    const int64_t box_m = up(std::min<int64_t>(d.tokens, 128), 8);
    double best = 0;
    for (int64_t tile_n = 32; tile_n <= 256; tile_n *= 2)
        for (int64_t ks = 1; ks <= kSkinnyMaxSplit && ks <= k_blocks; ks *= 2) {
            if (m_blocks * ((d.n + tile_n - 1) / tile_n) * ks > dev.sms) continue;
            const double cost = (double)((k_blocks + ks - 1) / ks) * ((box_m + tile_n) * 128 / 50 + 100) +
                                (ks > 1 ? 2000 + 0.1 * (double)(box_m * tile_n) : 0);
            if (best > 0 && cost >= best) continue;
            best = cost;
            p->sk.tile_n = (int32_t)tile_n;
            p->sk.k_split = (int32_t)ks;
        }
    if (best == 0) return false;
    SkinnyParams& q = p->sk;
    q.M = (int32_t)d.tokens;
    q.N = (int32_t)d.n;
    q.k_blocks = (int32_t)k_blocks;
    q.box_m = (int32_t)box_m;
    q.tmem_cols = std::max(32, q.tile_n);
    q.sum_pitch = q.tile_n + 4;
    q.ldy = d.ldy ? d.ldy : d.n;
    q.timeout_ns = d.wait_timeout_ns ? d.wait_timeout_ns : 2000000000ull;
    q.idesc = make_idesc(d.dtype == GEMM_BF16 ? 1u : 0u, 128u, (uint32_t)q.tile_n);
    q.adapters = d.adapters;
    // the last stage's matrix instruction reads 128 rows from its X box on: 16 KB behind the ring
    const int64_t stage = (box_m + q.tile_n) * 128, slack = 128 * 128 + 1024;
    const int64_t most = dev.smem_optin - 4096 - slack;       // 4096: the kernel's static shared memory, rounded up
    // Room beside it for a CTA of gather_kernel, so that the two kernels overlap on an SM: 5.6 KB up to rank 16, 9.6 up to 32.
    // At ranks up to 64 and 128 it takes 17.6 and 33.6 KB, and where the ring fills its share its CTAs come first.
    const int64_t room = most - (12 << 10);
    q.stages = (int32_t)std::min<int64_t>(kSkinnyMaxStages, room / stage);
    const int64_t ring = std::max<int64_t>(q.stages * stage, std::min<int64_t>(d.tokens, 128) * q.sum_pitch * 4);
    if (q.stages < 2 || ring > most) return false;
    p->skinny_smem = (size_t)(ring + slack);
    p->skinny_grid = dim3((unsigned)((d.n + q.tile_n - 1) / q.tile_n * q.k_split), (unsigned)m_blocks);
    p->tile_rows = 128;
    return true;
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
    p->device = dev.device;
    if (p->desc.ldx == 0) p->desc.ldx = d.k;
    p->skinny = d.tokens > 0 && plan_skinny(d, dev, p);
    // the product's plan also holds the device error record, which both kernels use
    if (p->skinny) g.flags |= GEMM_FLAG_NO_STREAM_K;          // ... and then needs no workspace
    s = gemm_plan_create(&p->product, &g);
    gemm_plan_info_t info{};
    if (s == GEMM_OK) s = gemm_plan_info(p->product, &info);
    if (s != GEMM_OK) {
        lora_plan_destroy(p);
        return s;
    }
    if (p->skinny) {
        // what runs instead
        info.cta_group = 1;
        info.tile_m = 128;
        info.tile_n = p->sk.tile_n;
        info.tile_k = 64;
        info.stages = p->sk.stages;
        info.tmem_stages = 1;
        info.tmem_cols = p->sk.tmem_cols;
        info.grid = (int32_t)(p->skinny_grid.x * p->skinny_grid.y);
        info.block_threads = 192;
        info.num_tiles = (int64_t)(p->skinny_grid.x / p->sk.k_split) * p->skinny_grid.y;
        info.stage_bytes = (p->sk.box_m + p->sk.tile_n) * 128;
        info.pipeline_bytes = info.stages * info.stage_bytes + 8 * (2 * info.stages + 2) + 4;
        info.smem_bytes = (int64_t)p->skinny_smem;
        info.epilogue = 1;
    } else {
        p->tile_rows = info.tile_m;
    }
    p->info.product = info;
    p->info.product_k_split = p->skinny ? p->sk.k_split : 1;
    p->rank16 = (int32_t)up(d.rank, 16);
    p->cols = d.dtype_y == GEMM_F32 ? 2 * p->rank16 : p->rank16;
    p->info.steps_per_adapter = p->cols / 16;
    if (d.tokens > 0) {
        p->m_blocks = (int32_t)((d.tokens + p->tile_rows - 1) / p->tile_rows);
        const int64_t slots = std::min<int64_t>(d.adapters, std::min<int64_t>(p->tile_rows, d.tokens));
        p->info.max_adapters_per_tile = (int32_t)slots;
        p->gather = gathers(d);
        if (p->gather) {
            p->info.shrink_k_split = 1;
            p->shrink_grid = dim3((unsigned)std::min<int64_t>(d.tokens, p->tile_rows), (unsigned)p->m_blocks, 1);
        } else {
            // Clusters split K, up to four ways while that fills the device four times over (8192 rows of 8192, rank 64: 44
            // us, two ways 56; the mixed 4096 x 4096 x 4096 above as a whole: 241 so, up to 304 with the other splits tried),
            // up to eight while it does so twice (beyond, starts outweigh it), and every CTA keeps four
            // chunks of K.  Then CTAs share out the slots; those of a block's first slots come first in the grid, as most
            // blocks of prompts have no others.
            const int64_t row_blocks = (d.tokens + kShrinkRows - 1) / kShrinkRows, chunks = (d.k + 63) / 64;
            int64_t ks = 1;
            while (ks < 8 && row_blocks * ks * 2 <= (ks < 4 ? 4 : 2) * dev.sms && chunks >= 4 * ks * 2) ks *= 2;
            p->chunks_per_cta = (int32_t)((chunks + ks - 1) / ks);
            p->info.shrink_k_split = (int32_t)ks;
            p->shrink_grid = dim3((unsigned)ks, (unsigned)row_blocks,
                                  (unsigned)std::min<int64_t>(slots, std::max<int64_t>(1, 8 * dev.sms / (row_blocks * ks))));
        }
        p->info.shrink_grid = (int32_t)(p->shrink_grid.x * p->shrink_grid.y * p->shrink_grid.z);
        p->t_bytes = up((int64_t)p->m_blocks * slots * p->tile_rows * p->cols * 2, 256);
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
    gemm_status_t s;
    if ((s = check_device(plan->device)) != GEMM_OK) return s;
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
    char* mem = static_cast<char*>(plan->memory);
    q.ldx = d.ldx;
    q.M = (int32_t)d.tokens;
    q.K = (int32_t)d.k;
    q.rank = d.rank;
    q.adapters = d.adapters;
    q.tile_rows = plan->tile_rows;
    q.max_adapters = plan->info.max_adapters_per_tile;
    q.rank16 = plan->rank16;
    q.cols = plan->cols;
    q.pitch = q.max_adapters * q.cols;
    q.chunks_per_cta = plan->chunks_per_cta;
    q.t = mem;
    q.counts = reinterpret_cast<int32_t*>(mem + plan->t_bytes);
    q.ids = reinterpret_cast<int32_t*>(mem + plan->t_bytes + plan->count_bytes);
    LoraTail tail;
    const int32_t box_m = plan->skinny ? plan->sk.box_m : 128;
    s = encode_matrices_map(&tail.tmap_t, d.dtype, q.t, q.pitch, q.tile_rows, plan->m_blocks, q.pitch, (int64_t)q.tile_rows * q.pitch,
                            128, box_m);
    if (s != GEMM_OK) return s;
    // one adapter: the stride is never used but has to be a valid one
    const int64_t stride_b = d.adapters > 1 ? a.stride_b : d.n * a.ldb;
    if ((s = encode_matrices_map(&tail.tmap_b, d.dtype, a.b, d.rank, d.n, d.adapters, a.ldb, stride_b, 32, std::min(info.tile_n, 256) / info.cta_group)) != GEMM_OK)
        return s;
    tail.counts = q.counts;
    tail.ids = q.ids;
    tail.max_adapters = q.max_adapters;
    tail.steps = q.cols / 16;
    tail.b_steps = q.rank16 / 16;
    tail.x = a.x;
    tail.w = a.w;
    tail.b = a.b;
    tail.t = q.t;
    tail.adapter = a.adapter;
    tail.ldx = d.ldx;
    tail.ldw = ldw;
    tail.ldb = a.ldb;
    tail.stride_b = a.stride_b;
    tail.k = q.K;
    tail.rank = d.rank;
    tail.bf16 = d.dtype == GEMM_BF16;
    SkinnyParams sk;
    PersistentParams p;
    if (plan->skinny) {
        sk = plan->sk;
        sk.y = a.y;
        sk.status = device_record(plan->product);
        sk.adapter = a.adapter;
        if ((s = encode_rows_map(&sk.tmap_x, d.dtype, a.x, d.k, d.tokens, d.ldx, box_m)) != GEMM_OK) return s;
        if ((s = encode_rows_map(&sk.tmap_w, d.dtype, a.w, d.k, d.n, ldw, sk.tile_n)) != GEMM_OK) return s;
    } else if ((s = product_params(plan->product, a.x, a.w, a.y, &p)) != GEMM_OK) {
        return s;
    }
    cudaError_t e = d.dtype == GEMM_BF16 ? launch_shrink<__nv_bfloat16>(q, plan->gather, plan->shrink_grid, stream)
                                         : launch_shrink<__half>(q, plan->gather, plan->shrink_grid, stream);
    if (e != cudaSuccess) return status_of(e);
    if (plan->skinny) return status_of(launch_skinny(sk, tail, d.dtype_y, plan->skinny_grid, plan->skinny_smem, stream));
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
