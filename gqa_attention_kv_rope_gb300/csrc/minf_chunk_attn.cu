// minf_chunk_attn.cu -- attention of chunks of new tokens over cached sequences.
#include "minf_chunk_row.cuh"

namespace minf {

namespace {

// One warp a row (token, head).
template <typename T, int HD>
__global__ void __launch_bounds__(128) chunk_row_kernel(const ChunkAttnArgs a, float scale_log2) {
    const long long rows = static_cast<long long>(a.sq.nt) * a.nh;
    int bad = 0;
    for (int s = threadIdx.x; a.sq.off && s <= a.sq.n_seq; s += 128) {
        const int o = __ldg(a.sq.off + s);
        if (o < 0 || o > a.sq.nt || (s > 0 && o < __ldg(a.sq.off + s - 1))) bad = 1;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) flag_error(a.err, MINF_ERRBIT_CHUNK);
        return;
    }
    for (long long r = blockIdx.x * 4LL + (threadIdx.x >> 5); r < rows; r += gridDim.x * 4LL) {
        const int t = static_cast<int>(r / a.nh), h = static_cast<int>(r - static_cast<long long>(t) * a.nh);
        const int s = chunk_seq_of(a.sq.off, a.sq.n_seq, t);
        if (s < 0) continue;
        RowJob job;
        job.rows = seq_rows(a.c, s);
        job.p = static_cast<long long>(__ldg(a.sq.n_past + s)) + (t - (a.sq.off ? __ldg(a.sq.off + s) : s));
        job.hk = h / (a.nh / a.nk);
        job.q = a.q + static_cast<size_t>(r) * a.hd;
        job.out = a.out + static_cast<size_t>(r) * HD;
        const bool missing = attn_row<T, HD>(a.c, job, scale_log2, a.window, a.n_sink);
        if ((threadIdx.x & 31) == 0) {
            if (missing) flag_error(a.err, MINF_ERRBIT_BLOCK);
            if (job.p < 0 || job.p >= job.rows.cap) flag_error(a.err, MINF_ERRBIT_ATTN_POS);
        }
    }
}

template <int HD>
void launch_rows(const ChunkAttnArgs &a, float sl, cudaStream_t s) {
    const long long want = (static_cast<long long>(a.sq.nt) * a.nh + 3) / 4;
    const int grid = static_cast<int>(want < 16LL * sm_count() ? want : 16LL * sm_count());
    if (a.c.kv == kKvQ8)
        chunk_row_kernel<Q8, HD><<<grid, 128, 0, s>>>(a, sl);
    else if (a.c.kv == kKvF16)
        chunk_row_kernel<__half, HD><<<grid, 128, 0, s>>>(a, sl);
    else
        chunk_row_kernel<float, HD><<<grid, 128, 0, s>>>(a, sl);
}

}  // namespace

size_t chunk_attn_workspace_bytes(int nt, int n_seq, int nh, int nk, int hd_kv, int max_chunk) {
    if (nt <= 0 || n_seq <= 0 || nh <= 0 || nk <= 0 || nh % nk || (hd_kv != 64 && hd_kv != 128) || max_chunk <= 0) return 0;
    return 256;
}

int launch_chunk_attn(const ChunkAttnArgs &a, cudaStream_t s) {
    if (a.sq.nt == 0 || a.sq.n_seq == 0) return MINF_OK;
    const float sl = a.scale * kLog2e;
    if (a.hd_kv == 64)
        launch_rows<64>(a, sl, s);
    else
        launch_rows<128>(a, sl, s);
    return cudaPeekAtLastError() == cudaSuccess ? MINF_OK : MINF_ERR_CUDA;
}

}  // namespace minf
