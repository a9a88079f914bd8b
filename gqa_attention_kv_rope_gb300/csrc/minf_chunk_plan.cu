// minf_chunk_plan.cu -- the one-block kernel that cuts a chunk attention into stretches.
#include "minf_chunk_plan.cuh"
#include "minf_sm103.cuh"

namespace minf {

namespace {

constexpr int kPlanThreads = 512;

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
    gdc_launch_dependents();  // the attention kernel sets itself up meanwhile
    __shared__ long long warp_sum[kPlanThreads / 32];
    __shared__ long long s_total;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int bad = 0;
    for (int s = tid; a.sq.off && s <= a.sq.n_seq; s += kPlanThreads) {
        const int o = __ldg(a.sq.off + s);
        if (o < 0 || o > a.sq.nt || (s > 0 && o < __ldg(a.sq.off + s - 1))) bad = 1;
    }
    for (int b = tid; b < a.max_ctas; b += kPlanThreads) a.tickets[b] = 0;
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            flag_error(a.err, MINF_ERRBIT_CHUNK);
            a.head->total = 0;
            a.head->ctas = 0;
        }
        return;
    }
    // a warp a sequence, a lane a token tile: running sums of the tiles' units
    for (int s = warp; s < a.sq.n_seq; s += kPlanThreads / 32) {
        int lo, hi;
        chunk_rows(a.sq.off, a.sq.nt, s, lo, hi);
        const long long past = __ldg(a.sq.n_past + s), base = tile_base(lo, s, a.tt);
        const int cap = seq_rows(a.c, s).cap, n = hi - lo, tiles = n < a.least || n > a.most ? 0 : (n + a.tt - 1) / a.tt;
        long long run = 0;
        int reported = 0;
        for (int t0 = 0; t0 < tiles; t0 += 32) {
            const int t = t0 + lane;
            int u = 0;
            if (t < tiles) {
                const long long p0 = past + static_cast<long long>(t) * a.tt;
                const int cnt = min(a.tt, n - t * a.tt);
                u = item_keys(p0, p0 + cnt - 1, cap, a.window, a.n_sink, a.kt).units;
                if (p0 < 0 || p0 + cnt - 1 >= cap) reported = 1;
            }
            long long x = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (t < tiles) a.tile_units[base + t] = run + x;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (reported) flag_error(a.err, MINF_ERRBIT_ATTN_POS);
        if (lane == 0) a.seq_units[s] = run * a.nk;
    }
    __syncthreads();
    // units before each sequence: a stretch of sequences a thread, then the threads' sums
    const int per = (a.sq.n_seq + kPlanThreads - 1) / kPlanThreads;
    const int s0 = min(tid * per, a.sq.n_seq), s1 = min(s0 + per, a.sq.n_seq);
    long long sum = 0;
    for (int s = s0; s < s1; ++s) sum += a.seq_units[s];
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    long long before = inc - sum;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    for (int s = s0; s < s1; ++s) {
        const long long u = a.seq_units[s];
        a.seq_units[s] = before;
        before += u;
    }
    if (tid == kPlanThreads - 1) {  // (the last thread's running sum is the total)
        a.seq_units[a.sq.n_seq] = before;
        s_total = before;
    }
    __syncthreads();
    const long long total = s_total;
    long long want = (total + a.min_units - 1) / a.min_units;
    const int ctas = static_cast<int>(want < a.max_ctas ? want : a.max_ctas);
    if (tid == 0) {
        a.head->total = total;
        a.head->ctas = ctas;
    }
    for (int b = tid; b < ctas; b += kPlanThreads) {
        const long long x = stretch_start(total, ctas, b);
        int l = 0, r = a.sq.n_seq;  // the last sequence that starts at or before x and has units
        while (r - l > 1) {
            const int mid = (l + r) >> 1;
            if (a.seq_units[mid] <= x)
                l = mid;
            else
                r = mid;
        }
        int lo, hi;
        chunk_rows(a.sq.off, a.sq.nt, l, lo, hi);
        const long long *tu = a.tile_units + tile_base(lo, l, a.tt);
        const int tiles = (hi - lo + a.tt - 1) / a.tt;
        const long long rest = x - a.seq_units[l];
        const long long per_head = tu[tiles - 1], in_head = rest % per_head;
        const int head = static_cast<int>(rest / per_head);
        int tl = -1, tr = tiles - 1;  // the first tile whose running sum passes in_head
        while (tr - tl > 1) {
            const int mid = (tl + tr) >> 1;
            if (tu[mid] > in_head)
                tr = mid;
            else
                tl = mid;
        }
        PlanStart st;
        st.unit = x;
        st.seq = l;
        st.head = head;
        st.tile = tr;
        st.u = static_cast<int>(in_head - (tr > 0 ? tu[tr - 1] : 0));
        a.starts[b] = st;
    }
}

}  // namespace

int launch_chunk_plan(const PlanArgs &a, cudaStream_t s) {
    plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? MINF_OK : MINF_ERR_CUDA;
}

}  // namespace minf
