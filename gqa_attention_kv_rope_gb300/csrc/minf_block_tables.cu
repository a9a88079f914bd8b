// minf_block_tables.cu -- the paged cache's block tables, kept on the device: what a step needs before its store and
// attention (offsets, positions, pool rows, blocks from the free list) from the sequences' lengths, and blocks given
// back.
//
// The list of free blocks is a stack: its last id goes out first, and of what comes back the first is its last again.
// With B rows a block, sequence s holds held_s = ceil(past_s / B) blocks and needs ceil((past_s + new_s) / B); the sums
// over the sequences before it say where its tokens (chunk_off) and its new blocks on the list begin.  A few thousand
// sums and 8 bytes a token are latency, not bandwidth: so one launch, and nothing that goes through memory between its
// parts.  Every CTA of one cluster adds all lengths up for itself (shared memory holds the sums of up to 16384
// sequences), then takes its share of the tokens and blocks, each of which finds its sequence by a search in the sums.
// The cluster's barrier says when every CTA has read the free list's length, which may be updated in place.  (A grid
// without a cluster would need a second launch or a counter in a workspace for that.)
#include <cooperative_groups.h>

#include "minf_common.cuh"
#include "minf_kernels.h"

namespace minf {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMostSeqs = 16384;

// Exclusive sums over the block's threads, of K numbers at once; the totals in `total`, all threads' bits in `bits`.
// (`warps` is free for the next call after a barrier.)
template <int K>
struct WarpSums {
    long long x[K][kWarps];
    int bits[kWarps];
};
template <int K>
__device__ __forceinline__ void scan_threads(long long (&x)[K], int &bits, WarpSums<K> &warps, long long (&total)[K]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long inc[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        inc[k] = x[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc[k], o);
            if (lane >= o) inc[k] += y;
        }
        if (lane == 31) warps.x[k][warp] = inc[k];
    }
    const int warp_bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0) warps.bits[warp] = warp_bits;
    __syncthreads();
    bits = __reduce_or_sync(0xffffffffu, warps.bits[lane]);  // (32 warps)
#pragma unroll
    for (int k = 0; k < K; ++k) {
        long long w = warps.x[k][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        total[k] = __shfl_sync(0xffffffffu, w, 31);
        const long long before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
        x[k] = inc[k] - x[k] + (warp ? before : 0);
    }
}

// The last s in [0, n) with sum[s] <= x (sum nondecreasing, sum[0] <= x).
__device__ __forceinline__ int last_not_above(const int *sum, int n, int x) {
    int l = 0, r = n;
    while (r - l > 1) {
        const int mid = (l + r) >> 1;
        if (sum[mid] <= x)
            l = mid;
        else
            r = mid;
    }
    return l;
}

__device__ __forceinline__ int blocks_of(long long rows, int shift) {
    return static_cast<int>((rows + (1LL << shift) - 1) >> shift);
}

__global__ void __launch_bounds__(kThreads) grow_kernel(const BlockGrowArgs a) {
    extern __shared__ int sums[];
    __shared__ WarpSums<2> warps;
    int *off = sums, *take = off + a.n_seq + 1, *past = take + a.n_seq + 1;  // tokens and blocks before s, cached rows
    const int tid = threadIdx.x, at = blockIdx.x * kThreads + tid, step = gridDim.x * kThreads;
    const int n_free = *a.n_free;
    const cg::cluster_group cluster = cg::this_cluster();
    const int per = (a.n_seq + kThreads - 1) / kThreads, s0 = min(tid * per, a.n_seq), s1 = min(s0 + per, a.n_seq);
    const long long cap = static_cast<long long>(a.max_blocks) << a.block_shift;
    long long sum[2] = {0, 0}, totals[2];  // tokens, blocks
    int bad = 0;
    for (int s = s0; s < s1; ++s) {
        const long long p = __ldg(a.n_past + s), n = __ldg(a.n_new + s);
        if (p < 0 || n < 0) {
            bad |= MINF_ERRBIT_CHUNK;
            continue;
        }
        if (p + n > cap) bad |= MINF_ERRBIT_STORE_POS;
        past[s] = static_cast<int>(p);
        off[s] = static_cast<int>(n);
        take[s] = blocks_of(p + n, a.block_shift) - blocks_of(p, a.block_shift);
        sum[0] += n;
        sum[1] += take[s];
    }
    scan_threads(sum, bad, warps, totals);
    const long long toks = totals[0], blks = totals[1];
    long long tok0 = sum[0], blk0 = sum[1];
    if (toks > a.nt) bad |= MINF_ERRBIT_CHUNK;
    if (n_free < 0 || n_free > a.max_free || blks > n_free) bad |= MINF_ERRBIT_BLOCK;
    if (bad) {  // nothing is taken, and the step has no tokens
        for (int s = at; s <= a.n_seq; s += step) a.chunk_off[s] = 0;
        for (int t = at; t < (a.pos || a.slot ? a.nt : 0); t += step) {
            if (a.pos) a.pos[t] = -1;
            if (a.slot) a.slot[t] = -1;
        }
        if (at == 0) flag_error(a.err, bad);
        cluster.sync();
        if (at == 0) *a.n_free_out = n_free;
        return;
    }
    for (int s = s0; s < s1; ++s) {
        const int n = off[s], b = take[s];
        off[s] = static_cast<int>(tok0);
        take[s] = static_cast<int>(blk0);
        tok0 += n;
        blk0 += b;
    }
    if (tid == 0) {
        off[a.n_seq] = static_cast<int>(toks);
        take[a.n_seq] = static_cast<int>(blks);
    }
    __syncthreads();
    const int32_t *ids = a.free_ids + n_free - 1;  // the call's blocks: ids[0], ids[-1], ids[-2] ..
    for (int s = at; s <= a.n_seq; s += step) a.chunk_off[s] = off[s];
    int missing = 0;
    auto outside = [&](int id) { return id < 0 || id >= a.pool_blocks; };
    for (int i = at; i < blks; i += step) {
        const int s = last_not_above(take, a.n_seq, i), id = __ldg(ids - i);
        a.table[static_cast<size_t>(s) * a.max_blocks + blocks_of(past[s], a.block_shift) + (i - take[s])] = id;
        missing |= outside(id);
    }
    const int mask = (1 << a.block_shift) - 1;
    if (!a.pos && !a.slot) {  // (else the tokens look their blocks up)
        for (int s = at; s < a.n_seq; s += step)
            if (off[s + 1] > off[s] && (past[s] & mask))
                missing |= outside(a.table[static_cast<size_t>(s) * a.max_blocks + (past[s] >> a.block_shift)]);
    }
    // positions and pool rows: four tokens a thread
    for (int t0 = 4 * at; t0 < (a.pos || a.slot ? a.nt : 0); t0 += 4 * step) {
        int pos[4], slot[4];
        int s = t0 < toks ? last_not_above(off, a.n_seq, t0) : 0, have = -1, have_s = -1, id = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = t0 + e;
            pos[e] = slot[e] = -1;
            if (t >= toks) continue;
            while (t >= off[s + 1]) ++s;
            const int p = past[s] + (t - off[s]), b = p >> a.block_shift;
            if (b != have || s != have_s) {
                const int held = blocks_of(past[s], a.block_shift);
                id = b < held ? a.table[static_cast<size_t>(s) * a.max_blocks + b] : __ldg(ids - (take[s] + (b - held)));
                have = b;
                have_s = s;
                missing |= outside(id);
            }
            pos[e] = p;
            if (!outside(id)) slot[e] = (id << a.block_shift) | (p & mask);
        }
        const bool whole = t0 + 4 <= a.nt;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            int32_t *to = o ? a.slot : a.pos;
            const int *x = o ? slot : pos;
            if (!to) continue;
            if (whole && a.vec) {
                *reinterpret_cast<int4 *>(to + t0) = make_int4(x[0], x[1], x[2], x[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t0 + e < a.nt) to[t0 + e] = x[e];
            }
        }
    }
    if (missing) flag_error(a.err, MINF_ERRBIT_BLOCK);
    cluster.sync();  // every CTA has read n_free
    if (at == 0) *a.n_free_out = n_free - static_cast<int>(blks);
}

// The entries of all sequences' ranges in a row, cut into equal stretches, one a CTA: counted, the counts exchanged
// across the cluster, then moved.
__global__ void __launch_bounds__(kThreads) release_kernel(const BlockReleaseArgs a) {
    extern __shared__ int sums[];
    __shared__ WarpSums<1> warps[2];  // (in turn)
    __shared__ int count;
    int *before = sums, *first = before + a.n_seq + 1;  // entries of the ranges before s's, its first
    const int tid = threadIdx.x;
    const int n_free = *a.n_free;
    const cg::cluster_group cluster = cg::this_cluster();
    const int per = (a.n_seq + kThreads - 1) / kThreads, s0 = min(tid * per, a.n_seq), s1 = min(s0 + per, a.n_seq);
    const long long cap = static_cast<long long>(a.max_blocks) << a.block_shift;
    long long at0[1] = {0}, totals[1];
    int none = 0;
    for (int s = s0; s < s1; ++s) {
        const long long lo = min(max(static_cast<long long>(__ldg(a.row_lo + s)), 0LL), cap), hi = min(static_cast<long long>(__ldg(a.row_hi + s)), cap);
        const int b0 = blocks_of(lo, a.block_shift), b1 = hi > 0 ? static_cast<int>(hi >> a.block_shift) : 0;
        first[s] = b0;
        before[s] = max(b1 - b0, 0);
        at0[0] += before[s];
    }
    scan_threads(at0, none, warps[0], totals);
    const long long total = totals[0];
    // (n_seq * max_blocks entries at most, below 2^31)
    for (int s = s0; s < s1; ++s) {
        const int n = before[s];
        before[s] = static_cast<int>(at0[0]);
        at0[0] += n;
    }
    if (tid == 0) before[a.n_seq] = static_cast<int>(total);
    __syncthreads();
    const int ctas = gridDim.x, cta = blockIdx.x;
    const int lo = static_cast<int>(total * cta / ctas), hi = static_cast<int>(total * (cta + 1) / ctas);
    auto entry = [&](int i) -> int32_t * {
        const int s = last_not_above(before, a.n_seq, i);
        return a.table + static_cast<size_t>(s) * a.max_blocks + first[s] + (i - before[s]);
    };
    auto held = [&](int id) { return id >= 0 && id < a.pool_blocks; };
    // a thread's first entry and its id stay in registers
    int32_t *mine = nullptr;
    int id = -1;
    long long nth[1] = {0}, here[1];
    for (int i = lo + tid; i < hi; i += kThreads) {
        int32_t *e = entry(i);
        const int x = *e;
        nth[0] += held(x);
        if (!mine) mine = e, id = x;
    }
    scan_threads(nth, none, warps[1], here);
    if (tid == 0) count = static_cast<int>(here[0]);
    cluster.sync();
    const int lane = tid & 31;
    const unsigned theirs = lane < ctas ? *cluster.map_shared_rank(&count, lane) : 0;  // (16 CTAs at most)
    const long long all = __reduce_add_sync(0xffffffffu, theirs);
    long long base = __reduce_add_sync(0xffffffffu, lane < cta ? theirs : 0u);
    cluster.sync();  // the counts are read, and n_free
    if (n_free < 0 || n_free + all > a.max_free) {
        if (cta == 0 && tid == 0) {
            flag_error(a.err, MINF_ERRBIT_BLOCK);
            *a.n_free_out = n_free;
        }
        return;
    }
    int bad = 0;
    int32_t *ids = a.free_ids + n_free + all - 1;  // the last to go back is put on the list first
    auto give = [&](int32_t *e, int x, long long nth) {
        *e = -1;
        bad |= x >= a.pool_blocks;
        if (held(x)) ids[-nth] = x;
    };
    if (hi - lo <= kThreads) {
        if (mine) give(mine, id, base + nth[0]);
    } else {
        for (int i0 = lo, turn = 0; i0 < hi; i0 += kThreads, turn ^= 1) {  // the same for every thread of the CTA
            const int i = i0 + tid;
            int32_t *e = i < hi ? entry(i) : nullptr;
            const int x = e ? *e : -1;
            nth[0] = held(x);
            scan_threads(nth, none, warps[turn], here);
            if (e) give(e, x, base + nth[0]);
            base += here[0];
        }
    }
    if (bad) flag_error(a.err, MINF_ERRBIT_BLOCK);
    if (cta == 0 && tid == 0) *a.n_free_out = n_free + static_cast<int>(all);
}

// CTAs of the cluster: one where that leaves a thread few turns; 16 for the largest calls (9.1 us for 1024 prompts of
// 120,000 tokens, 12.9 with 8).
int ctas_for(long long turns) { return turns <= 4 * kThreads ? 1 : turns <= 16 * kThreads ? 8 : 16; }

template <typename Args>
int launch(void (*kernel)(Args), const Args &a, int arrays, long long turns, cudaStream_t s) {
    const size_t smem = static_cast<size_t>(arrays) * (a.n_seq + 1) * sizeof(int);
    // What a kernel is allowed is state of the whole context: always the same, so that no thread's call lowers it between
    // another's setting and its launch.
    const int most = arrays * (kMostSeqs + 1) * static_cast<int>(sizeof(int));
    // (48 KB without the setting, a kernel's own arrays included)
    constexpr size_t kOwn = 1024;
    static_assert(sizeof(WarpSums<2>) + 64 <= kOwn && 2 * sizeof(WarpSums<1>) + 64 <= kOwn, "the kernels' own arrays");
    if (smem + kOwn > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
        return MINF_ERR_CUDA;
    int ctas = ctas_for(turns);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    for (;; ctas = 8) {
        cfg.gridDim = dim3(ctas);
        attr[0].val.clusterDim.x = ctas;
        int clusters = 0;
        if (ctas <= 8 || (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                          cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0))
            break;
        // (no part of this GPU has 16 SMs side by side: no error, and none for those who ask for the last one)
        (void)cudaGetLastError();
    }
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? MINF_OK : MINF_ERR_CUDA;
}

int set_blocks(int max_blocks, int block_rows, int64_t pool_rows, int n_seq, int *shift, int *pool_blocks) {
    if (max_blocks <= 0 || pool_rows < 0 || n_seq < 0) return MINF_ERR_ARG;
    if (block_rows < 16 || block_rows > 4096 || (block_rows & (block_rows - 1))) return MINF_ERR_UNSUPPORTED;
    constexpr long long kMostRows = 0x7fffffffLL - 4096;  // rows and positions are 32-bit, as for the chunk operators
    if (pool_rows % block_rows || pool_rows > kMostRows || static_cast<long long>(max_blocks) * block_rows > kMostRows ||
        n_seq > kMostSeqs || static_cast<long long>(n_seq) * max_blocks > kMostRows)
        return MINF_ERR_UNSUPPORTED;
    *shift = 0;
    while ((1 << *shift) < block_rows) ++*shift;
    *pool_blocks = static_cast<int>(pool_rows / block_rows);
    return MINF_OK;
}

bool aligned4(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Arrays of int32.  What a call writes lies apart from all else that it is given (a CTA may write while another still
// reads), but for n_free_out, which may be n_free.
struct Ints {
    const void *p;
    long long n;
};
bool apart(const Ints &a, const Ints &b) {
    if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x + 4 * static_cast<uintptr_t>(a.n) <= y || y + 4 * static_cast<uintptr_t>(b.n) <= x;
}
template <int NW, int NR>
bool all_apart(const Ints (&writes)[NW], const Ints (&reads)[NR]) {
    for (int i = 0; i < NW; ++i) {
        for (int j = 0; j < i; ++j)
            if (!apart(writes[i], writes[j])) return false;
        for (int j = 0; j < NR; ++j)
            if (!apart(writes[i], reads[j])) return false;
    }
    return true;
}

}  // namespace

}  // namespace minf

using namespace minf;

extern "C" {

int minf_block_table_grow(int32_t *block_table, int max_blocks, int block_rows, int64_t pool_rows, const int32_t *n_past,
                          const int32_t *n_new, int n_seq, const int32_t *free_ids, int max_free, const int32_t *n_free,
                          int32_t *n_free_out, int32_t *chunk_off, int32_t *pos, int32_t *slot, int nt, int32_t *err,
                          minf_stream_t stream) {
    BlockGrowArgs a = {};
    const int st = set_blocks(max_blocks, block_rows, pool_rows, n_seq, &a.block_shift, &a.pool_blocks);
    if (st != MINF_OK) return st;
    const bool some = n_seq > 0;
    if ((some && (!aligned4(block_table) || !aligned4(n_past) || !aligned4(n_new))) || (max_free > 0 && !aligned4(free_ids)) ||
        max_free < 0 || nt < 0 || !aligned4(n_free) || !aligned4(n_free_out) || !aligned4(chunk_off) ||
        (pos && !aligned4(pos)) || (slot && !aligned4(slot)) || !aligned4(err))
        return MINF_ERR_ARG;
    if (nt > 0x7fffffff - 65536) return MINF_ERR_UNSUPPORTED;  // (the last turn's index stays below 2^31)
    const long long cells = static_cast<long long>(n_seq) * max_blocks;
    const Ints writes[] = {{block_table, cells}, {chunk_off, n_seq + 1LL}, {pos, nt}, {slot, nt}, {err, 1}, {n_free_out, 1}};
    const Ints reads[] = {{n_past, n_seq}, {n_new, n_seq}, {free_ids, max_free}, {n_free == n_free_out ? nullptr : n_free, 1}};
    if (!all_apart(writes, reads)) return MINF_ERR_ARG;
    a.table = block_table;
    a.max_blocks = max_blocks;
    a.n_past = n_past;
    a.n_new = n_new;
    a.n_seq = n_seq;
    a.free_ids = free_ids;
    a.max_free = max_free;
    a.n_free = n_free;
    a.n_free_out = n_free_out;
    a.chunk_off = chunk_off;
    a.pos = pos;
    a.slot = slot;
    a.nt = nt;
    a.vec = (!pos || aligned16(pos)) && (!slot || aligned16(slot));
    a.err = err;
    return launch(grow_kernel, a, 3, (pos || slot ? nt / 4 : 0) + n_seq, reinterpret_cast<cudaStream_t>(stream));
}

int minf_block_table_release(int32_t *block_table, int max_blocks, int block_rows, int64_t pool_rows, const int32_t *row_lo,
                             const int32_t *row_hi, int n_seq, int32_t *free_ids, int max_free, const int32_t *n_free,
                             int32_t *n_free_out, int32_t *err, minf_stream_t stream) {
    BlockReleaseArgs a = {};
    const int st = set_blocks(max_blocks, block_rows, pool_rows, n_seq, &a.block_shift, &a.pool_blocks);
    if (st != MINF_OK) return st;
    if ((n_seq > 0 && (!aligned4(block_table) || !aligned4(row_lo) || !aligned4(row_hi))) || max_free < 0 ||
        (max_free > 0 && !aligned4(free_ids)) || !aligned4(n_free) || !aligned4(n_free_out) || !aligned4(err))
        return MINF_ERR_ARG;
    const Ints writes[] = {{block_table, static_cast<long long>(n_seq) * max_blocks}, {free_ids, max_free}, {err, 1}, {n_free_out, 1}};
    const Ints reads[] = {{row_lo, n_seq}, {row_hi, n_seq}, {n_free == n_free_out ? nullptr : n_free, 1}};
    if (!all_apart(writes, reads)) return MINF_ERR_ARG;
    a.table = block_table;
    a.max_blocks = max_blocks;
    a.row_lo = row_lo;
    a.row_hi = row_hi;
    a.n_seq = n_seq;
    a.free_ids = free_ids;
    a.max_free = max_free;
    a.n_free = n_free;
    a.n_free_out = n_free_out;
    a.err = err;
    return launch(release_kernel, a, 2, static_cast<long long>(n_seq) * max_blocks, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
