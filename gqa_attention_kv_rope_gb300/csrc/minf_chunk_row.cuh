// minf_chunk_row.cuh -- one output row (a token and a head) of the chunk attention by one warp.
//
// The definition, as directly as a warp can compute it: the visible keys in groups of 32, a key a
// lane, with the running maximum and sum of an online softmax in fp32; then every lane adds the
// group's weighted V rows for its own dimensions, leaving out the hidden ones, so that nothing a
// hidden row holds (infinities, NaN, whatever an unwritten row has) reaches the result.  Weights are
// at most 1 and a row has fewer than 2^31 keys, so with the weights of V taken 2^-32 times no sum of
// finite values passes the range of fp32 (a term below 2^-117 of an output is lost).  Nor does a
// score of finite rows: one that does is summed again from operands 2^-66 times, and maxima and
// differences of scores are taken in 64 bits.
#pragma once

#include "minf_chunk.cuh"

namespace minf {

struct RowJob {
    const float *q;  // hd_kv values
    float *out;      // hd_kv values
    SeqRows rows;
    long long p;     // the query's position
    int hk;          // kv head
};

constexpr float kValueScale = 2.3283064365386963e-10f;  // 2^-32

// q . K[row] of one kv head, both times `f`.
template <typename T, int HD>
__device__ __forceinline__ float attn_dot(const ChunkKv &c, const float *q, long long row, int hk, float f) {
    constexpr int D4 = HD / 4;
    const float4 *q4 = reinterpret_cast<const float4 *>(q);
    float s = 0.0f;
#pragma unroll 4
    for (int d = 0; d < D4; ++d) {
        const float4 k = row_ld4<T>(c.k, row, c.W, c.row_bytes, hk * D4 + d), x = __ldg(q4 + d);
        s = fmaf(x.x * f, k.x * f, s);
        s = fmaf(x.y * f, k.y * f, s);
        s = fmaf(x.z * f, k.z * f, s);
        s = fmaf(x.w * f, k.w * f, s);
    }
    return s;
}

// (The rows of a block that is missing count as zeros; the kernels' producers report it.)
template <typename T, int HD>
__device__ __forceinline__ void attn_row(const ChunkKv &c, const RowJob &job, float scale_log2, int window, int n_sink) {
    constexpr int D4 = HD / 4, PER = HD / 32;  // values a lane owns
    const int lane = threadIdx.x & 31;
    const long long last = job.p < job.rows.cap - 1 ? job.p : job.rows.cap - 1;  // last visible key
    double m = -INFINITY;
    float l = 0.0f, acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.0f;
    // key groups: from 0 while sinks are left, then from the window's first key
    const long long first = window == 0 ? 0 : (job.p - window + 1 > 0 ? job.p - window + 1 : 0);
    for (long long j0 = n_sink > 0 ? 0 : (first & ~31LL); j0 <= last; j0 += 32) {
        if (window && j0 >= n_sink && j0 + 31 < first) j0 = first & ~31LL;
        if (j0 > last) break;
        const int j = static_cast<int>(j0) + lane;
        const bool see = j <= last && chunk_sees(job.p, j, window, n_sink);
        long long row = -1;
        if (see) row = seq_row(c, job.rows, j);
        double s = 0.0;
        if (row >= 0) {
            const float x = attn_dot<T, HD>(c, job.q, row, job.hk, 1.0f);
            s = x;
            if (!(fabsf(x) < INFINITY)) s = static_cast<double>(attn_dot<T, HD>(c, job.q, row, job.hk, 0x1p-66f)) * 0x1p132;
        }
        s = see ? s * scale_log2 : -INFINITY;
        double mx = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double t = __shfl_xor_sync(0xffffffffu, mx, o);
            mx = mx > t || mx != mx ? mx : t;  // a NaN score stays
        }
        const double mn = m > mx || m != m ? m : mx, base = mn == -INFINITY ? 0.0 : mn;
        const float corr = exp2f(static_cast<float>(m - base)), pr = see ? exp2f(static_cast<float>(s - base)) : 0.0f;
        m = mn;
        float sum = pr;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * corr + sum;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] *= corr;
        if (!__any_sync(0xffffffffu, row >= 0)) continue;
        for (int b0 = 0; b0 < 32; b0 += 4) {  // four rows' loads in flight
            float4 v[4];
            float pb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long rb = __shfl_sync(0xffffffffu, row, b0 + i);
                pb[i] = __shfl_sync(0xffffffffu, pr, b0 + i);
                pb[i] = rb < 0 ? 0.0f : pb[i] * kValueScale;  // (a missing block's row counts in l)
                v[i] = rb >= 0 ? row_ld4<T>(c.v, rb, c.W, c.row_bytes, job.hk * D4 + lane * PER / 4) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (PER == 4) {
                    acc[0] = fmaf(pb[i], v[i].x, acc[0]);
                    acc[1] = fmaf(pb[i], v[i].y, acc[1]);
                    acc[2] = fmaf(pb[i], v[i].z, acc[2]);
                    acc[3] = fmaf(pb[i], v[i].w, acc[3]);
                } else {
                    acc[0] = fmaf(pb[i], lane & 1 ? v[i].z : v[i].x, acc[0]);
                    acc[1] = fmaf(pb[i], lane & 1 ? v[i].w : v[i].y, acc[1]);
                }
            }
        }
    }
    // nothing visible: zeros.  Nothing but scores of minus infinity: 0 / 0, as the softmax of such rows is.
    const bool none = !chunk_sees_any(job.p, job.rows.cap, window, n_sink);
    const float inv = 1.0f / (l * kValueScale);
#pragma unroll
    for (int i = 0; i < PER; ++i) job.out[lane * PER + i] = none ? 0.0f : acc[i] * inv;
}

// The rows of an item that are marked in `odd`, a row a warp: q and out are the item's first row's, p0 its position,
// g the rows of a token.  (One call out of line, with the arithmetic of the rows inside: with the rows' loop in the
// kernels, whatever changed in it moved their hot loops' registers and instructions; 1043 us against 1015 over
// ragged binary16 prompts.)
template <typename T, int HD>
__device__ __noinline__ void attn_rows_again(const ChunkKv &c, const int *odd, int rows, int warp, int warps, const float *q,
                                             float *out, int g, int nh, int hd, SeqRows sr, long long p0, int hk,
                                             float scale_log2, int window, int n_sink) {
    for (int r = warp; r < rows; r += warps) {
        if (!odd[r]) continue;
        RowJob job;
        const long long at = static_cast<long long>(r / g) * nh + r % g;
        job.q = q + at * hd;
        job.out = out + at * HD;
        job.rows = sr;
        job.p = p0 + r / g;
        job.hk = hk;
        attn_row<T, HD>(c, job, scale_log2, window, n_sink);
    }
}

}  // namespace minf
