// minf_chunk_tiles.h -- the two kernels behind launch_chunk_attn (each with its plan; `workspace` holds
// at least the bytes that its function below says).
#pragma once

#include "minf_kernels.h"

namespace minf {

// 128-row tiles on the tensor cores (minf_chunk_tiles.cu), for the sequences with at least `least`
// new tokens.
size_t chunk_tiles_workspace(int nt, int n_seq, int nh, int nk, int hd_kv);
int launch_chunk_tiles(const ChunkAttnArgs &a, void *workspace, int least, cudaStream_t s);

// A stream of the cached rows past up to `rows` query rows at a time (minf_chunk_stream.cu), for the
// sequences with at most `most` new tokens.
size_t chunk_stream_workspace(int nt, int n_seq, int nh, int nk, int hd_kv, int rows);
int launch_chunk_stream(const ChunkAttnArgs &a, void *workspace, int rows, int most, cudaStream_t s);

}  // namespace minf
