// minf_chunk_tiles.h -- the kernels behind launch_chunk_attn.
#pragma once

#include "minf_kernels.h"

namespace minf {

// 128-row tiles on the tensor cores (minf_chunk_tiles.cu).
size_t chunk_tiles_workspace(int nt, int n_seq, int nh, int nk, int hd_kv);
int launch_chunk_tiles(const ChunkAttnArgs &a, cudaStream_t s);

}  // namespace minf
