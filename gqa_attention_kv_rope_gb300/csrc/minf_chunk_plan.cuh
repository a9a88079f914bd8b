// minf_chunk_plan.cuh -- how the attention of ragged chunks is spread over the SMs.
//
// Work is counted in units: an item is a tile of `tt` consecutive tokens of one sequence with one
// kv head's query heads, and its units are the key tiles of `kt` rows that any of its tokens sees
// (the sinks' tiles, then the window's).  All units in order (sequence, kv head, token tile, key
// tile) are cut into equal stretches, one a CTA, so every CTA streams the same amount whatever the
// lengths are.  An item that lies in one stretch is finished by its CTA; one that crosses
// stretches is joined, in order, by the last of its CTAs to finish: two calls with the same
// inputs add in the same order.
//
// The lengths are device data, so the cut is made on the device by a one-block kernel ahead of
// the attention kernel (which is launched at once and waits for it).  That kernel also checks
// chunk_off and zeroes the join tickets, so a workspace needs no preparation and carries nothing
// from one call to the next.
#pragma once

#include "minf_chunk.cuh"

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

// Where a stretch starts: an item and a unit of it.
struct PlanStart {
    long long unit;  // of all units
    int seq, head, tile, u;
};

struct PlanHead {
    long long total;  // units; 0: chunk_off is bad, nothing is to be done
    int ctas;         // stretches (the rest of the grid has none)
    int pad;
};

struct PlanArgs {
    ChunkKv c;
    ChunkSeqs sq;
    int nk, tt, kt, window, n_sink;
    int max_ctas, min_units;  // stretches at most; units a stretch should have at least
    int least, most;          // chunk lengths that this plan takes (the others have no units)
    PlanHead *head;
    PlanStart *starts;        // [max_ctas]
    int *tickets;             // [max_ctas]
    long long *seq_units;     // [n_seq + 1] units of the sequences before s
    long long *tile_units;    // units of a sequence's token tiles up to and with this one, one kv head
    int32_t *err;
};

// Token tiles of sequence s start at this place of tile_units (tiles of earlier sequences never
// reach it: each has at most len/tt + 1).
__device__ __forceinline__ long long tile_base(int chunk_lo, int s, int tt) {
    return static_cast<long long>(chunk_lo / tt) + s;
}
inline size_t plan_tiles(int nt, int n_seq, int tt) { return static_cast<size_t>(nt / tt) + n_seq + 1; }

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

// The first unit of stretch b, and the stretch that holds unit x.
__host__ __device__ __forceinline__ long long stretch_start(long long total, int ctas, long long b) {
    return b * total / ctas;
}
__host__ __device__ __forceinline__ int stretch_of(long long total, int ctas, long long x) {
    return static_cast<int>(((x + 1) * ctas - 1) / total);
}

int launch_chunk_plan(const PlanArgs &a, cudaStream_t s);

}  // namespace minf
