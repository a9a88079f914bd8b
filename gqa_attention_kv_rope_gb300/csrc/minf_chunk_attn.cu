// minf_chunk_attn.cu -- attention of chunks of new tokens over cached sequences: which kernel runs.
#include "minf_chunk_tiles.h"
#include "minf_common.cuh"

namespace minf {

namespace {

// The limits of minf_chunk_tiles.h.  kStreamRows and kStreamRowsF16, query rows (tokens x heads of a kv head) up to
// which the streaming kernel runs alone: measured on 16 query heads over 8 kv heads of 128 dims, 64 sequences of
// 4096 rows, streaming kernel and tiles: binary16 16 rows 195 and 210 us, 32 rows 363 and 212; Q8_0 32 rows 627 and
// 725; fp32 (16 sequences) 238 and 267.  (The 32-row instances keep 128 sums a thread at 128 dims and spill 570 and
// 760 bytes.)  One sequence of 8192 rows, binary16: 8 rows 25 and 56, 32 rows 49 and 54 (there the tiles are taken).
// kStreamRowsQ4 (minf_chunk_q4.cu, whose items are 8 rows of whole tokens: what does not fit one is another pass): the same
// 64 sequences 8 rows 109 us and 256, 16 rows 196 and 256 (24 rows 268 and 265 once); 8 sequences 16 rows 46 and 52, 24
// rows 55 and 53.  14 heads on 2 of 64 dims, 64 sequences: 14 rows 48 and 61, 21 rows 63 and 62; 8 sequences: 14 rows 22 and
// 31, 28 rows 28 and 31.  With 3 or 5 heads a kv head 15 rows are three passes: 24 heads on 8 of 128 dims, 64 sequences 283
// and 257, 8 sequences 56 and 52, one 38 and 42; 12 heads on 4, 64 sequences 158 and 143, one 29 and 52.
// kFewRows, in a call that also has long chunks: there the streaming kernel takes the few tokens of the others, after
// the tiles.  31 single tokens with 3 chunks of 391, Q8_0: 267 us, all in tiles 575; with the streaming kernel laid
// out for 32 rows 533 (it computes as many for every token).  31 times 4 tokens of two heads with chunks of 391, 300
// and 200 and 31 times 5, which go to the tiles: Q8_0 267 and 515 us, fp32 512 and 685, binary16 178 and 193.

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// A call whose chunks all fit the streaming kernel runs that alone; one sequence with a longer chunk
// runs the tiles alone; a batch runs both, each over its own sequences, one after the other.
struct Choice {
    bool stream, tiles;
    int rows, most;  // of the streaming kernel
};
Choice choose(int kv, int n_seq, int g, int max_chunk) {
    const long long rows = static_cast<long long>(g) * max_chunk;
    if (rows <= (kv == kKvF16 ? kStreamRowsF16 : kv == kKvQ4 ? kStreamRowsQ4 : kStreamRows)) return {true, false, static_cast<int>(rows), 0x7fffffff};
    return {n_seq > 1, true, kFewRows, kFewRows / g};
}

}  // namespace

size_t chunk_attn_workspace_bytes(int nt, int n_seq, int nh, int nk, int hd_kv, int max_chunk, bool q4) {
    if (nt <= 0 || n_seq <= 0 || nh <= 0 || nk <= 0 || nh % nk || !decode_supported(nh, nk, hd_kv, hd_kv) || max_chunk <= 0)
        return 0;  // (at most 8 heads a kv head: the layouts divide by them)
    size_t most = 0;  // of the types
    for (const int kv : {kKvF32, kKvF16, kKvQ8, kKvQ4}) {
        if (kv == kKvQ4 && !q4) continue;
        const Choice c = choose(kv, n_seq, nh / nk, max_chunk);
        const size_t need = (c.tiles ? up256(chunk_tiles_workspace(nt, n_seq, nh, nk, hd_kv)) : 0) +
                            (!c.stream        ? 0
                             : kv == kKvQ4 ? chunk_q4_workspace(nt, n_seq, nh, nk, hd_kv, c.rows)
                                           : chunk_stream_workspace(nt, n_seq, nh, nk, hd_kv, c.rows));
        if (need > most) most = need;
    }
    return most;
}

int launch_chunk_attn(const ChunkAttnArgs &a, cudaStream_t s) {
    if (a.sq.nt == 0 || a.sq.n_seq == 0) return MINF_OK;
    const Choice c = choose(a.c.kv, a.sq.n_seq, a.nh / a.nk, a.max_chunk);
    char *ws = static_cast<char *>(a.ws);
    Plans plans = {};
    AttnParams tiles, stream;
    int n = 0;
    if (c.tiles) {
        plan_chunk_tiles(plans.a[n++], tiles, a, ws, c.stream ? c.most + 1 : 1);
        ws += up256(chunk_tiles_workspace(a.sq.nt, a.sq.n_seq, a.nh, a.nk, a.hd_kv));
    }
    const bool q4 = a.c.kv == kKvQ4;
    if (c.stream) (q4 ? plan_chunk_q4 : plan_chunk_stream)(plans.a[n++], stream, a, ws, c.rows, c.most);
    int st = launch_chunk_plan(plans, n, s);
    if (st == MINF_OK && c.tiles) st = launch_chunk_tiles(tiles, s);
    if (st == MINF_OK && c.stream) st = (q4 ? launch_chunk_q4 : launch_chunk_stream)(stream, c.rows, s);
    return st;
}

}  // namespace minf
