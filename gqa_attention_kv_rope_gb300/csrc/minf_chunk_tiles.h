// minf_chunk_tiles.h -- the two kernels behind launch_chunk_attn.  Each has a plan (minf_chunk_plan.cuh): the
// plan_ function fills in the plan's arguments and the kernel's, over a workspace of at least the bytes
// that the third function says; the plan is to be launched ahead of the kernel.
#pragma once

#include "minf_chunk_plan.cuh"

namespace minf {

// Query rows up to which the streaming kernel runs alone, over binary16 rows and over the others, and up to which it
// takes sequences in a batch with longer chunks (minf_chunk_attn.cu says why).  It has instances for 8, 16 and 32
// rows, over binary16 for 8 and 16.
constexpr int kStreamRows = 32, kStreamRowsF16 = 16, kFewRows = 8;
static_assert(kStreamRows <= 32 && kStreamRowsF16 <= 16 && kFewRows <= 16, "instances of the streaming kernel");

// 128-row tiles on the tensor cores (minf_chunk_tiles.cu), for the sequences with at least `least`
// new tokens.
void plan_chunk_tiles(PlanArgs &plan, AttnParams &p, const ChunkAttnArgs &a, void *workspace, int least);
int launch_chunk_tiles(const AttnParams &p, cudaStream_t s);
size_t chunk_tiles_workspace(int nt, int n_seq, int nh, int nk, int hd_kv);

// A stream of the cached rows past up to `rows` query rows at a time (minf_chunk_stream.cu), for the
// sequences with at most `most` new tokens.
void plan_chunk_stream(PlanArgs &plan, AttnParams &p, const ChunkAttnArgs &a, void *workspace, int rows, int most);
int launch_chunk_stream(const AttnParams &p, int rows, cudaStream_t s);
size_t chunk_stream_workspace(int nt, int n_seq, int nh, int nk, int hd_kv, int rows);

}  // namespace minf
