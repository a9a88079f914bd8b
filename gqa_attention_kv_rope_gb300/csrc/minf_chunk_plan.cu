// minf_chunk_plan.cu -- the kernel that cuts a chunk attention into stretches, a block a plan.
#include "minf_chunk_plan.cuh"
#include "minf_sm103.cuh"

namespace minf {

namespace {

constexpr int kPlanThreads = kPlanMost;
constexpr int kHeld = 1024;     // sequences and token tiles whose sums are also held in shared memory
constexpr int kFewTiles = 4;    // token tiles that a sequence's own thread adds up

// A thread a sequence (its loads are the only ones that wait on memory), a warp for a sequence of many
// token tiles; then a thread a stretch looks its start up in the sums.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ Plans plans) {
    const PlanArgs &a = plans.a[blockIdx.x];
    gdc_launch_dependents();  // the attention kernel sets itself up meanwhile
    __shared__ long long warp_sum[kPlanThreads / 32];
    __shared__ long long held_seq[kHeld + 1], held_tile[kHeld];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t tiles_most = plan_tiles(a.sq.nt, a.sq.n_seq, a.tt);
    long long *seq_units = a.sq.n_seq <= kHeld ? held_seq : a.seq_units;
    long long *tile_units = tiles_most <= kHeld ? held_tile : a.tile_units;
    for (int b = tid; b < a.max_ctas; b += kPlanThreads) a.tickets[b] = 0;
    long long before = 0;  // units of the sequences of earlier passes
    int bad = 0, reported = 0;
    for (int s0 = 0; s0 < a.sq.n_seq; s0 += kPlanThreads) {
        const int s = s0 + tid;
        int lo = s, n = 0, cap = 0, past = 0;
        if (s < a.sq.n_seq) {
            int hi = s + 1;
            if (a.sq.off) {
                lo = __ldg(a.sq.off + s);
                hi = __ldg(a.sq.off + s + 1);
            }
            past = __ldg(a.sq.n_past + s);
            cap = seq_rows(a.c, s).cap;
            if (lo < 0 || hi < lo || hi > a.sq.nt) bad = 1;  // (nondecreasing within [0, nt])
            lo = min(max(lo, 0), a.sq.nt);
            hi = min(max(hi, lo), a.sq.nt);
            n = hi - lo;
        }
        const int tiles = n < a.least || n > a.most ? 0 : (n + a.tt - 1) / a.tt;
        if (tiles > 0 && (past < 0 || static_cast<long long>(past) + n > cap)) reported = 1;
        auto units = [&](int t, int pst, int cnt, int cp) -> long long {
            const long long p0 = static_cast<long long>(pst) + static_cast<long long>(t) * a.tt;
            return item_keys(p0, p0 + min(a.tt, cnt - t * a.tt) - 1, cp, a.window, a.n_sink, a.kt).units;
        };
        long long total = 0;
        if (tiles <= kFewTiles) {
            for (int t = 0; t < tiles; ++t) {
                total += units(t, past, n, cap);
                tile_units[tile_base(lo, s, a.tt) + t] = total;
            }
        }
        for (unsigned many = __ballot_sync(0xffffffffu, tiles > kFewTiles); many; many &= many - 1) {
            const int l = __ffs(many) - 1;
            const int t_n = __shfl_sync(0xffffffffu, tiles, l), t_lo = __shfl_sync(0xffffffffu, lo, l);
            const int t_past = __shfl_sync(0xffffffffu, past, l), t_cnt = __shfl_sync(0xffffffffu, n, l), t_cap = __shfl_sync(0xffffffffu, cap, l);
            const long long base = tile_base(t_lo, s0 + warp * 32 + l, a.tt);
            long long run = 0;
            for (int t0 = 0; t0 < t_n; t0 += 32) {
                const int t = t0 + lane;
                long long x = t < t_n ? units(t, t_past, t_cnt, t_cap) : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (t < t_n) tile_units[base + t] = run + x;
                run += __shfl_sync(0xffffffffu, x, 31);
            }
            if (lane == l) total = run;
        }
        total *= a.nk;
        // units before each sequence
        long long inc = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        long long here = before + inc - total;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const long long y = warp_sum[w];
            if (w < warp) here += y;
            before += y;
        }
        if (s < a.sq.n_seq) seq_units[s] = a.seq_units[s] = here;  // (the walks look it up there)
        __syncthreads();  // warp_sum is free for the next pass
    }
    if (reported) flag_error(a.err, MINF_ERRBIT_ATTN_POS);
    if (__syncthreads_or(bad)) {
        if (tid == 0) {
            flag_error(a.err, MINF_ERRBIT_CHUNK);
            a.head->total = 0;
            a.head->ctas = 0;
        }
        return;
    }
    const long long total = before;
    const long long want = total / a.min_units;
    const int ctas = static_cast<int>(want < 1 ? 1 : (want < a.max_ctas ? want : a.max_ctas));
    if (total == 0) {  // nothing to do (no new token that this plan takes)
        if (tid == 0) {
            a.head->total = 0;
            a.head->ctas = 0;
        }
        return;
    }
    // a thread a stretch: its start, moved to an item's border that is near
    __shared__ long long start[kPlanMost + 1];
    __shared__ int first_hi[kPlanMost + 1];
    __shared__ int kept_warp[kPlanThreads / 32];
    long long x = tid < ctas ? tid * total / ctas : total;
    int l = 0, tile = 0, head = 0, tiles = 0;
    long long in_tile = 0, item = 0;
    const long long *tu = nullptr;
    auto locate = [&]() {  // the item of unit x and its place there
        l = seq_of_unit(seq_units, a.sq.n_seq, x);
        int lo, hi;
        chunk_rows(a.sq.off, a.sq.nt, l, lo, hi);
        tu = tile_units + tile_base(lo, l, a.tt);
        tiles = (hi - lo + a.tt - 1) / a.tt;
        const long long rest = x - seq_units[l], per_head = tu[tiles - 1], in_head = rest % per_head;
        head = static_cast<int>(rest / per_head);
        int tl = -1, tr = tiles - 1;  // the first tile whose running sum passes in_head
        while (tr - tl > 1) {
            const int mid = (tl + tr) >> 1;
            if (tu[mid] > in_head)
                tr = mid;
            else
                tl = mid;
        }
        tile = tr;
        const long long tile0 = tr > 0 ? tu[tr - 1] : 0;
        in_tile = in_head - tile0;
        item = tu[tr] - tile0;
    };
    if (tid < ctas) {
        locate();
        if (in_tile <= a.snap) {
            x -= in_tile;
            in_tile = 0;
        } else if (item - in_tile <= a.snap) {
            x += item - in_tile;
            if (x < total) locate();
        }
    }
    // stretches that start where the one before them does are none
    start[tid] = x;
    __syncthreads();
    const bool keep = tid < ctas && x < total && (tid == 0 || start[tid - 1] != x);
    const unsigned kept = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) kept_warp[warp] = __popc(kept);
    __syncthreads();
    int at = __popc(kept & ((1u << lane) - 1)), n = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const int y = kept_warp[w];
        if (w < warp) at += y;
        n += y;
    }
    if (keep) start[at] = x;
    __syncthreads();
    if (tid == 0) {
        start[n] = total;
        a.head->total = total;
        a.head->ctas = n;
    }
    // the stretches of the item that this one starts inside of
    int lo = at, hi = at;
    if (keep && in_tile > 0) {
        const long long item0 = x - in_tile, item1 = item0 + item;
        while (start[lo] > item0) --lo;
        while (hi + 1 < n && start[hi + 1] < item1) ++hi;
    }
    if (keep) first_hi[at] = hi;
    __syncthreads();
    if (keep) {
        PlanStart st;
        st.unit = x;
        st.end = start[at + 1];
        st.seq = l;
        st.head = head;
        st.tile = tile;
        st.u = static_cast<int>(in_tile);
        st.first_lo = lo;
        st.first_hi = hi;
        st.last_hi = at + 1 < n ? first_hi[at + 1] : at;
        st.pad = 0;
        a.starts[at] = st;
    }
}

}  // namespace

int launch_chunk_plan(const Plans &p, int n, cudaStream_t s) {
    plan_kernel<<<n, kPlanThreads, 0, s>>>(p);
    return cudaPeekAtLastError() == cudaSuccess ? MINF_OK : MINF_ERR_CUDA;
}

}  // namespace minf
