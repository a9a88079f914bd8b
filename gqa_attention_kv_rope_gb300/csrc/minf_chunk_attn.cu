// minf_chunk_attn.cu -- attention of chunks of new tokens over cached sequences: which kernel runs.
#include "minf_chunk_tiles.h"
#include "minf_common.cuh"

namespace minf {

namespace {

constexpr int kStreamRows = 32;  // query rows (tokens x heads of a kv head) the streaming kernel takes at once
constexpr int kFewRows = 8;      // and in a call that also has long chunks

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// A call whose chunks all fit the streaming kernel runs that alone; one sequence with a longer chunk
// runs the tiles alone; a batch runs both, each over its own sequences.
struct Choice {
    bool stream, tiles;
    int rows, most;  // of the streaming kernel
};
Choice choose(int n_seq, int g, int max_chunk) {
    const long long rows = static_cast<long long>(g) * max_chunk;
    if (rows <= kStreamRows) return {true, false, static_cast<int>(rows), 0x7fffffff};
    return {n_seq > 1, true, kFewRows, kFewRows / g};
}

}  // namespace

size_t chunk_attn_workspace_bytes(int nt, int n_seq, int nh, int nk, int hd_kv, int max_chunk) {
    if (nt <= 0 || n_seq <= 0 || nh <= 0 || nk <= 0 || nh % nk || (hd_kv != 64 && hd_kv != 128) || max_chunk <= 0) return 0;
    const Choice c = choose(n_seq, nh / nk, max_chunk);
    return (c.tiles ? up256(chunk_tiles_workspace(nt, n_seq, nh, nk, hd_kv)) : 0) +
           (c.stream ? chunk_stream_workspace(nt, n_seq, nh, nk, hd_kv, c.rows) : 0);
}

int launch_chunk_attn(const ChunkAttnArgs &a, cudaStream_t s) {
    if (a.sq.nt == 0 || a.sq.n_seq == 0) return MINF_OK;
    const Choice c = choose(a.sq.n_seq, a.nh / a.nk, a.max_chunk);
    char *ws = static_cast<char *>(a.ws);
    Plans plans = {};
    AttnParams tiles, stream;
    int n = 0;
    if (c.tiles) {
        plan_chunk_tiles(plans.a[n++], tiles, a, ws, c.stream ? c.most + 1 : 1);
        ws += up256(chunk_tiles_workspace(a.sq.nt, a.sq.n_seq, a.nh, a.nk, a.hd_kv));
    }
    if (c.stream) plan_chunk_stream(plans.a[n++], stream, a, ws, c.rows, c.most);
    int st = launch_chunk_plan(plans, n, s);
    if (st == MINF_OK && c.tiles) st = launch_chunk_tiles(tiles, s);
    if (st == MINF_OK && c.stream) st = launch_chunk_stream(stream, c.rows, s);
    return st;
}

}  // namespace minf
