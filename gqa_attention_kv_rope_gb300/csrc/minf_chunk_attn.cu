// minf_chunk_attn.cu -- attention of chunks of new tokens over cached sequences: which kernel runs.
#include "minf_chunk_tiles.h"
#include "minf_common.cuh"

namespace minf {

size_t chunk_attn_workspace_bytes(int nt, int n_seq, int nh, int nk, int hd_kv, int max_chunk) {
    if (nt <= 0 || n_seq <= 0 || nh <= 0 || nk <= 0 || nh % nk || (hd_kv != 64 && hd_kv != 128) || max_chunk <= 0) return 0;
    return chunk_tiles_workspace(nt, n_seq, nh, nk, hd_kv);
}

int launch_chunk_attn(const ChunkAttnArgs &a, cudaStream_t s) {
    if (a.sq.nt == 0 || a.sq.n_seq == 0) return MINF_OK;
    return launch_chunk_tiles(a, s);
}

}  // namespace minf
