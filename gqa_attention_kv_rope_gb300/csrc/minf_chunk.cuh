// minf_chunk.cuh -- chunks of new tokens over cached sequences: the descriptors that the chunk
// operators share (RoPE + store, read back, attention) and the device helpers that resolve them.
//
// A call packs the new tokens of n_seq sequences into nt rows: sequence s owns rows
// chunk_off[s] .. chunk_off[s+1]-1, and its i-th new token is at cache position n_past[s] + i.
// Both arrays are device data, so a captured call replays with other lengths.  A null chunk_off
// means one token a sequence.  The cached rows are paged (a block table) or contiguous (regions
// or an arena).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "minf_common.cuh"
#include "minf_kernels.h"
#include "minf_q8.cuh"

namespace minf {

// Rows of sequence s's chunk, clamped to [0, nt): valid for any contents of chunk_off.
__device__ __forceinline__ void chunk_rows(const int32_t *chunk_off, int nt, int s, int &lo, int &hi) {
    if (!chunk_off) {
        lo = s < nt ? s : nt;
        hi = s + 1 < nt ? s + 1 : nt;
        return;
    }
    lo = min(max(__ldg(chunk_off + s), 0), nt);
    hi = min(max(__ldg(chunk_off + s + 1), lo), nt);
}

// The sequence that owns packed row t, or -1 (a row of padding).  chunk_off is nondecreasing; with
// any other contents the search still ends and reads inside the array.
__device__ __forceinline__ int chunk_seq_of(const int32_t *chunk_off, int n_seq, int t) {
    if (!chunk_off) return t < n_seq ? t : -1;
    int lo = 0, hi = n_seq;  // the largest s in [0, n_seq] with chunk_off[s] <= t, if any
    if (__ldg(chunk_off) > t) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(chunk_off + mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    return t < __ldg(chunk_off + lo + 1) ? lo : -1;
}

// One sequence's cached rows: rows 0 .. cap-1 exist.  (Two registers' worth: the kernels' roles keep
// it across a whole walk.)
struct SeqRows {
    unsigned long long at;  // paged: the address of this sequence's block ids; contiguous: its first row
    int cap;
};

__device__ __forceinline__ SeqRows seq_rows(const ChunkKv &c, int s) {
    SeqRows r;
    if (c.table) {
        r.at = reinterpret_cast<unsigned long long>(c.table + static_cast<size_t>(s) * c.max_blocks);
        r.cap = c.cap;
    } else {
        long long row0 = c.row_off ? __ldg(reinterpret_cast<const long long *>(c.row_off) + s) : 0;
        long long cap = c.caps ? __ldg(c.caps + s) : c.cap;
        // rows exist only inside the arena
        if (row0 < 0 || row0 >= c.rows) {
            row0 = 0;
            cap = 0;
        } else if (cap > c.rows - row0) {
            cap = c.rows - row0;
        }
        if (cap > c.cap) cap = c.cap;  // max_cap bounds every cap_s
        r.at = static_cast<unsigned long long>(row0);
        r.cap = cap < 0 ? 0 : static_cast<int>(cap);
    }
    return r;
}

// The pool (or arena) row of logical row j in [0, cap), or -1 where the block is missing.
__device__ __forceinline__ long long seq_row(const ChunkKv &c, const SeqRows &r, int j) {
    if (!c.table) return static_cast<long long>(r.at) + j;
    const int b = __ldg(reinterpret_cast<const int32_t *>(r.at) + (j >> c.block_shift));
    if (b < 0 || b >= c.pool_blocks) return -1;
    return (static_cast<long long>(b) << c.block_shift) + (j & ((1 << c.block_shift) - 1));
}

// Four consecutive values of a cached row (element 4*i4 of the row), in fp32.
template <typename T>
__device__ __forceinline__ float4 row_ld4(const void *base, long long row, int W, long long row_bytes, int i4) {
    const unsigned char *p = static_cast<const unsigned char *>(base) + row * row_bytes;
    if constexpr (std::is_same<T, Q8>::value) {
        return ld4_q8(p, W, i4);
    } else if constexpr (std::is_same<T, __half>::value) {
        const uint2 u = reinterpret_cast<const uint2 *>(p)[i4];
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
        return make_float4(x.x, x.y, y.x, y.y);
    } else {
        return reinterpret_cast<const float4 *>(p)[i4];
    }
}

// Whether the query at position p sees the cached row j (j < cap is checked apart): causal, and
// with a window of the last `window` positions (0: no limit) or one of the first n_sink rows.
__device__ __forceinline__ bool chunk_sees(long long p, int j, int window, int n_sink) {
    return j <= p && (window == 0 || j > p - window || j < n_sink);
}
// Whether it sees any of the sequence's rows 0 .. cap-1.
__device__ __forceinline__ bool chunk_sees_any(long long p, int cap, int window, int n_sink) {
    const long long last = p < cap - 1 ? p : cap - 1;
    return last >= 0 && (window == 0 || last > p - window || n_sink > 0);
}

}  // namespace minf
