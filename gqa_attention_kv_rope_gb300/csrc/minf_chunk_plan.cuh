// minf_chunk_plan.cuh -- how the attention of ragged chunks is spread over the SMs.
//
// Work is counted in units: an item is a tile of `tt` consecutive tokens of one sequence with one
// kv head's query heads, and its units are the key tiles of `kt` rows that any of its tokens sees
// (the sinks' tiles, then the window's).  All units in order (sequence, kv head, token tile, key
// tile) are cut into equal stretches, one a CTA, so every CTA streams the same amount whatever the
// lengths are.  (A cut that would fall within `snap` units of an item's border falls on it, and no
// stretch is shorter than min_units: a part of an item costs about a tile to write and to join.)  An
// item that lies in one stretch is finished by its CTA; one that crosses stretches is joined, in order,
// by the last of its CTAs to finish: two calls with the same inputs add in the same order.
//
// The lengths are device data, so the cut is made on the device, by a kernel of one block a plan ahead of
// the attention kernel (which is launched at once and waits for it).  That kernel also checks
// chunk_off and zeroes the join tickets, so a workspace needs no preparation and carries nothing
// from one call to the next.
#pragma once

#include "minf_chunk.cuh"
#include "minf_sm103.cuh"

namespace minf {

struct ItemKeys {
    int n_sink_tiles;  // tiles 0 .. n_sink_tiles-1, then first_tile ..
    int first_tile;
    int units;         // at least 1: an item without keys still writes its zeros
    int lo, hi, sink;  // rows that some token of the item sees: [lo, hi) and [0, sink)
};

// The key tiles of the item with tokens at positions p0 .. p1 of a sequence of `cap` rows.
__host__ __device__ __forceinline__ ItemKeys item_keys(long long p0, long long p1, int cap, int window, int n_sink,
                                                       int kt) {
    ItemKeys k;
    const long long top = p1 + 1 < cap ? p1 + 1 : cap;
    k.hi = top > 0 ? static_cast<int>(top) : 0;
    const long long lo = window && p0 - window + 1 > 0 ? p0 - window + 1 : 0;
    k.lo = lo < k.hi ? static_cast<int>(lo) : k.hi;
    k.sink = window ? (n_sink < k.hi ? n_sink : k.hi) : 0;
    k.first_tile = k.lo / kt;
    const int end = (k.hi + kt - 1) / kt, sink_end = (k.sink + kt - 1) / kt;
    k.n_sink_tiles = sink_end < k.first_tile ? sink_end : k.first_tile;
    if (k.lo == k.hi) {  // nothing in the window (clamped capacity): the sinks alone
        k.units = sink_end;
        k.n_sink_tiles = sink_end;
    } else {
        k.units = k.n_sink_tiles + (end - k.first_tile);
    }
    if (k.units < 1) k.units = 1;
    return k;
}
__host__ __device__ __forceinline__ int unit_tile(const ItemKeys &k, int u) {
    return u < k.n_sink_tiles ? u : k.first_tile + (u - k.n_sink_tiles);
}

// A stretch: where it starts (an item and a unit of it) and ends, and which stretches share its first
// and its last item.
struct PlanStart {
    long long unit, end;  // of all units
    int seq, head, tile, u;
    int first_lo, first_hi;  // stretches of the first item (where u > 0)
    int last_hi;             // last stretch of the item that the next stretch goes on with
    int pad;
};

struct PlanHead {
    long long total;  // units; 0: chunk_off is bad, nothing is to be done
    int ctas;         // stretches (the rest of the grid has none)
    int pad;
};

constexpr int kPlanMost = 512;  // stretches: a thread of the plan kernel each

struct PlanArgs {
    ChunkKv c;
    ChunkSeqs sq;
    int nk, tt, kt, window, n_sink;
    int max_ctas, min_units, snap;  // stretches at most (kPlanMost at most); see above
    int least, most;          // chunk lengths that this plan takes (the others have no units)
    PlanHead *head;
    PlanStart *starts;        // [max_ctas]
    int *tickets;             // [max_ctas]
    long long *seq_units;     // [n_seq] units of the sequences before s
    long long *tile_units;    // units of a sequence's token tiles up to and with this one, one kv head
    int32_t *err;
};

// Token tiles of sequence s start at this place of tile_units (tiles of earlier sequences never
// reach it: each has at most len/tt + 1).
__device__ __forceinline__ long long tile_base(int chunk_lo, int s, int tt) {
    return static_cast<long long>(chunk_lo / tt) + s;
}
__host__ __device__ inline size_t plan_tiles(int nt, int n_seq, int tt) { return static_cast<size_t>(nt / tt) + n_seq + 1; }

// Workspace offsets: the plan, then `parts` slots of `part_bytes`.
struct PlanLayout {
    size_t head, starts, tickets, seq_units, tile_units, parts, total;
};
inline PlanLayout plan_layout(int nt, int n_seq, int tt, int max_ctas, size_t part_bytes) {
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    PlanLayout l;
    l.head = 0;
    l.starts = 256;
    l.tickets = l.starts + up(static_cast<size_t>(max_ctas) * sizeof(PlanStart));
    l.seq_units = l.tickets + up(static_cast<size_t>(max_ctas) * sizeof(int));
    l.tile_units = l.seq_units + up((static_cast<size_t>(n_seq) + 1) * sizeof(long long));
    l.parts = l.tile_units + up(plan_tiles(nt, n_seq, tt) * sizeof(long long));
    l.total = l.parts + 2 * static_cast<size_t>(max_ctas) * part_bytes;
    return l;
}

// The sequence of unit x (below the total): the last that starts at or before it (those that the plan does not take
// have no units).
__device__ __forceinline__ int seq_of_unit(const long long *seq_units, int n_seq, long long x) {
    int l = 0, r = n_seq;
    while (r - l > 1) {
        const int mid = l + ((r - l) >> 1);
        if (seq_units[mid] <= x)
            l = mid;
        else
            r = mid;
    }
    return l;
}

// The plans of one call: that of the kernel for long chunks and that of the one for few rows, where it runs both.
struct Plans {
    PlanArgs a[2];
};
int launch_chunk_plan(const Plans &p, int n, cudaStream_t s);

// What both attention kernels are launched with.
struct AttnParams {
    ChunkAttnArgs a;
    const PlanHead *head;
    const PlanStart *starts;
    int *tickets;
    const long long *seq_units;  // [n_seq] units of the sequences before s
    float *parts;
    float scale_log2;
    int tt, kt;       // tokens of an item, keys of a tile
    int box_rows;     // rows of a TMA copy
    int least, most;  // chunk lengths this launch takes
};

// Fills the plan's arguments and the kernel's pointers for a workspace laid out as `lay`.
inline void plan_args(PlanArgs &pl, AttnParams &p, const PlanLayout &lay, void *workspace, int max_ctas, int min_units, int snap) {
    char *ws = static_cast<char *>(workspace);
    pl = {};
    pl.c = p.a.c;
    pl.sq = p.a.sq;
    pl.nk = p.a.nk;
    pl.tt = p.tt;
    pl.kt = p.kt;
    pl.window = p.a.window;
    pl.n_sink = p.a.n_sink;
    pl.max_ctas = max_ctas;
    pl.min_units = min_units;
    pl.snap = snap;
    pl.least = p.least;
    pl.most = p.most;
    pl.head = reinterpret_cast<PlanHead *>(ws + lay.head);
    pl.starts = reinterpret_cast<PlanStart *>(ws + lay.starts);
    pl.tickets = reinterpret_cast<int *>(ws + lay.tickets);
    pl.seq_units = reinterpret_cast<long long *>(ws + lay.seq_units);
    pl.tile_units = reinterpret_cast<long long *>(ws + lay.tile_units);
    pl.err = p.a.err;
    p.head = pl.head;
    p.starts = pl.starts;
    p.tickets = pl.tickets;
    p.seq_units = pl.seq_units;
    p.parts = reinterpret_cast<float *>(ws + lay.parts);
}

// A CTA's way through its stretch, segment by segment: a segment is the stretch's part of one item.
// Every role of a CTA walks the same segments on its own.
struct Walk {
    int left;             // units of the stretch from the segment's first on
    int seq, head, tile;  // the item
    int lo, n, past;      // its sequence: first packed row, new tokens, cached rows before them
    SeqRows rows;
    ItemKeys keys;
    int cnt;              // tokens of the item
    int u0, u1;           // the segment's units of the item
};

__device__ __forceinline__ void walk_seq(Walk &w, const AttnParams &p) {
    int hi;
    chunk_rows(p.a.sq.off, p.a.sq.nt, w.seq, w.lo, hi);
    w.n = hi - w.lo;
    w.past = __ldg(p.a.sq.n_past + w.seq);
    w.rows = seq_rows(p.a.c, w.seq);
}
// Position of the item's first token.
__device__ __forceinline__ long long walk_pos(const Walk &w, const AttnParams &p) {
    return static_cast<long long>(w.past) + w.tile * p.tt;
}
// Packed row of the item's first token.
__device__ __forceinline__ int walk_row(const Walk &w, const AttnParams &p) { return w.lo + w.tile * p.tt; }

template <int KT>
__device__ __forceinline__ void walk_item(Walk &w, const AttnParams &p) {
    w.cnt = min(p.tt, w.n - w.tile * p.tt);
    const long long p0 = walk_pos(w, p);
    w.keys = item_keys(p0, p0 + w.cnt - 1, w.rows.cap, p.a.window, p.a.n_sink, KT);
    w.u1 = w.left < w.keys.units - w.u0 ? w.u0 + w.left : w.keys.units;
}
// The first segment; false where the stretch is empty.
template <int KT>
__device__ __forceinline__ bool walk_begin(Walk &w, const AttnParams &p, int ctas) {
    if (static_cast<int>(blockIdx.x) >= ctas) return false;
    const PlanStart st = p.starts[blockIdx.x];
    w.left = static_cast<int>(st.end - st.unit);
    w.seq = st.seq;
    w.head = st.head;
    w.tile = st.tile;
    w.u0 = st.u;
    if (w.left <= 0) return false;
    walk_seq(w, p);
    walk_item<KT>(w, p);
    return true;
}
template <int KT>
__device__ __forceinline__ bool walk_next(Walk &w, const AttnParams &p) {
    w.left -= w.u1 - w.u0;
    if (w.left <= 0) return false;
    w.u0 = 0;  // units are left, so the item was finished
    if ((w.tile + 1) * p.tt < w.n) {
        ++w.tile;
    } else {
        w.tile = 0;
        if (++w.head == p.a.nk) {
            w.head = 0;
            ++w.seq;
            walk_seq(w, p);
            if (w.n < p.least || w.n > p.most) {
                // sequences that another launch takes, or without tokens: however many, they are passed at once
                w.seq = seq_of_unit(p.seq_units, p.a.sq.n_seq, p.starts[blockIdx.x].end - w.left);
                walk_seq(w, p);
            }
        }
    }
    walk_item<KT>(w, p);
    return true;
}

// mbar_wait of the attention kernels.  Rows that are computed again by their definition (attn_row) may take
// far longer than the wait's budget; while they are (abort_flag is kRowsAgain) the clock of everyone who
// waits for that CTA's next step starts anew.  abort_flag is 1 once a wait has run out.
constexpr int kRowsAgain = 2;
__device__ __forceinline__ uint32_t gtimer_lo() {  // nanoseconds, modulo 2^32: one register
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
__device__ __forceinline__ bool chunk_wait(unsigned long long *b, uint32_t parity, volatile int *abort_flag, int32_t *err) {
    if (mbar_try(b, parity)) return true;
    if (*abort_flag == 1) return false;
    uint32_t t0 = gtimer_lo();
    while (true) {
        if (mbar_try(b, parity)) return true;
        const int f = *abort_flag;
        if (f == 1) return false;
        if (f == kRowsAgain) t0 = gtimer_lo();
        if (gtimer_lo() - t0 > static_cast<uint32_t>(kWaitBudgetNs)) {
            *abort_flag = 1;
            flag_error(err, MINF_ERRBIT_TIMEOUT);
            return false;
        }
    }
}
// One thread says so around the rows (it leaves the flag of a wait that has run out as it is).
__device__ __forceinline__ void rows_again(int *abort_flag, bool on) {
    atomicCAS(abort_flag, on ? 0 : kRowsAgain, on ? kRowsAgain : 0);
}

// The stretches that share the segment's item (only of a segment that is not a whole item).
__device__ __forceinline__ void walk_parts(const Walk &w, const AttnParams &p, int &b0, int &b1) {
    const PlanStart *st = p.starts + blockIdx.x;
    b0 = w.u0 > 0 ? st->first_lo : static_cast<int>(blockIdx.x);
    b1 = w.u0 > 0 ? st->first_hi : st->last_hi;
}

// Row j of the sequence is seen by some token of the item; some row of [j, j + n) is.
__device__ __forceinline__ bool item_sees(const ItemKeys &k, int j) { return (j >= k.lo && j < k.hi) || j < k.sink; }
__device__ __forceinline__ bool item_sees_some(const ItemKeys &k, int j, int n) {
    return (j < k.hi && j + n > k.lo && k.lo < k.hi) || j < k.sink;
}

}  // namespace minf
