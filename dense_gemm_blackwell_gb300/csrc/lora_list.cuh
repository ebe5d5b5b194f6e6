// lora_list.cuh -- which adapters occur among the rows of an m block
// (lora.cu, lora_skinny.cu).
#pragma once

#include <cstdint>

namespace dgb {

constexpr int kMaxAdapters = 4096;           // one bit each in shared memory
constexpr int kMaxTileRows = 256;

struct AdapterList {
    uint32_t bits[kMaxAdapters / 32];
    int32_t list[kMaxTileRows];              // ascending
    int32_t count;
};

// Writes the numbers of the set bits of `words` words to `list`, ascending; returns how many.  Called by a whole warp.
__device__ __forceinline__ int list_bits(const uint32_t* bits, int words, int lane, int32_t* list) {
    int done = 0;
    for (int base = 0; base < words; base += 32) {
        uint32_t word = base + lane < words ? bits[base + lane] : 0u;
        int at = __popc(word);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += t;
        }
        const int all = __shfl_sync(0xffffffffu, at, 31);
        at += done - __popc(word);
        for (; word; word &= word - 1) list[at++] = (base + lane) * 32 + __ffs(word) - 1;
        done += all;
    }
    return done;
}

// Fills `out` from the adapters of rows [row0, row0 + rows) (rows past M and numbers outside [0, adapters) have none), and
// row_ids[i] (-1: none) for the rows i of [first, first + num) among them.  Called by `threads` threads, the first
// warp of them whole, numbered `tid`; `sync` is their barrier.
template <typename Sync>
__device__ __forceinline__ int find_adapters(const int32_t* adapter, int adapters, int M, int row0, int rows, AdapterList& out,
                                             int32_t* row_ids, int first, int num, int tid, int threads, Sync&& sync) {
    const int words = (adapters + 31) / 32, lane = tid & 31;
    for (int i = tid; i < words; i += threads) out.bits[i] = 0u;
    sync();
    for (int i = tid; i < rows; i += threads) {
        int id = row0 + i < M ? adapter[row0 + i] : -1;
        if (id < 0 || id >= adapters) id = -1;
        if (id >= 0) atomicOr(&out.bits[id >> 5], 1u << (id & 31));
        if (i >= first && i < first + num) row_ids[i - first] = id;
    }
    sync();
    if (tid < 32) {
        const int count = list_bits(out.bits, words, lane, out.list);
        if (lane == 0) out.count = count;
    }
    sync();
    return out.count;
}

}  // namespace dgb
