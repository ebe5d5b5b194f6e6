// lora_repair.cuh -- outputs that another token's adapter spoiled
// (kernels_persistent.cu, lora_skinny.cu).
//
// A tile multiplies every row of T by the B of every adapter that occurs among
// its rows, and T is zero in the rows of other adapters.  Where B_j[n] holds an
// infinity or a NaN those zeros become NaN, and column n of every token of the
// tile with them.  The epilogues therefore look at what they store (one
// multiply-add per value), and a value that is not finite is computed again
// from its own token's factors alone, if some other adapter's row n is to
// blame.  Finite adapters never come here.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "elem.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace dgb {

// Zero, or NaN if one of the N values is not finite.
template <int N>
__device__ __forceinline__ float finite_probe(const uint32_t (&v)[N], float z) {
#pragma unroll
    for (int i = 0; i < N; ++i) z = fmaf(__uint_as_float(v[i]), 0.f, z);
    return z;
}

template <typename T>
__device__ __forceinline__ float row_dot(const T* a, const T* b, int n) {
    float s[8] = {};
    int i = 0;
    for (; i + 8 <= n; i += 8) {
        float x[8], y[8];
        unpack8<T>(__ldcg(reinterpret_cast<const uint4*>(a + i)), x);
        unpack8<T>(__ldcg(reinterpret_cast<const uint4*>(b + i)), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = fmaf(x[e], y[e], s[e]);
    }
    for (int e = 0; i < n; ++i, ++e) s[e] = fmaf((float)a[i], (float)b[i], s[e]);
    return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

// Columns [n0, n1) of token m, stored at `out`.
template <int OUT, typename T>
__device__ __forceinline__ void repair_row_typed(const LoraTail& tail, int m, int mb, int n0, int n1, uint8_t* out) {
    constexpr int kBytes = OUT == GEMM_F32 ? 4 : 2;
    griddep_wait();         // T, counts and ids
    const int count = __ldcg(tail.counts + mb);
    const int32_t* ids = tail.ids + (size_t)mb * tail.max_adapters;
    const int id = tail.adapter[m];
    auto row_b = [&](int j, int n) { return static_cast<const T*>(tail.b) + j * tail.stride_b + n * tail.ldb; };
    for (int n = n0; n < n1; ++n) {
        uint8_t* at = out + (n - n0) * kBytes;
        float now;
        if constexpr (OUT == GEMM_F32) now = *reinterpret_cast<const float*>(at);
        else if constexpr (OUT == GEMM_BF16) now = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(at));
        else now = __half2float(*reinterpret_cast<const __half*>(at));
        if (now - now == 0.f) continue;
        int own = -1;
        float others = 0.f;
        for (int s = 0; s < count; ++s) {
            const int j = __ldcg(ids + s);
            if (j == id) {
                own = s;
                continue;
            }
            const T* b = row_b(j, n);
            for (int i = 0; i < tail.rank; ++i) others = fmaf((float)b[i], 0.f, others);
        }
        if (others == 0.f) continue;
        float v = row_dot<T>(static_cast<const T*>(tail.x) + m * tail.ldx, static_cast<const T*>(tail.w) + n * tail.ldw, tail.k);
        if (own >= 0) {
            // T's columns: one term of 16 b_steps, or two
            const T* t = static_cast<const T*>(tail.t) + ((int64_t)m * tail.max_adapters + own) * tail.steps * 16;
            v += row_dot<T>(t, row_b(id, n), tail.rank);
            if (tail.steps > tail.b_steps) v += row_dot<T>(t + tail.b_steps * 16, row_b(id, n), tail.rank);
        }
        if constexpr (OUT == GEMM_F32) *reinterpret_cast<float*>(at) = v;
        else *reinterpret_cast<uint16_t*>(at) = (uint16_t)pack2<OUT>(v, 0.f);
    }
}

template <int OUT>
__device__ __noinline__ void repair_row(const LoraTail& tail, int m, int mb, int n0, int n1, uint8_t* out) {
    if (tail.bf16) repair_row_typed<OUT, __nv_bfloat16>(tail, m, mb, n0, n1, out);
    else repair_row_typed<OUT, __half>(tail, m, mb, n0, n1, out);
}

}  // namespace dgb
