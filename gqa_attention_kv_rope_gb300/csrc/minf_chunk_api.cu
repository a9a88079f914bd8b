// minf_chunk_api.cu -- the C ABI of the chunk operators: argument validation, then the launches.
#include <cmath>

#include "minf_common.cuh"
#include "minf_kernels.h"

using namespace minf;

namespace {

inline cudaStream_t cs(minf_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool ok_f(const void *p) { return p != nullptr && aligned16(p); }

bool ok_axes(int n_axis, const uint8_t *pair_axis, int hd) {
    if (n_axis < 1 || n_axis > 255 || (n_axis > 1 && !pair_axis)) return false;
    if (pair_axis)
        for (int i = 0; i < hd / 2; ++i)
            if (pair_axis[i] >= n_axis) return false;
    return true;
}

int check_geometry(int nh, int nk, int hd, int hd_kv) {
    if (nh <= 0 || nk <= 0 || hd <= 0 || hd_kv <= 0) return MINF_ERR_ARG;
    if (hd < hd_kv || nh % nk != 0) return MINF_ERR_GEOMETRY;
    if ((hd & 1) || (hd_kv & 1)) return MINF_ERR_ARG;
    if (static_cast<long long>(nh) * hd > (1 << 20)) return MINF_ERR_UNSUPPORTED;
    return decode_supported(nh, nk, hd, hd_kv) ? MINF_OK : MINF_ERR_UNSUPPORTED;
}

long long row_bytes_of(int kv, int W) {
    return kv == kKvQ4 ? q4_row_bytes(W) : kv == kKvQ8 ? q8_row_bytes(W) : (kv == kKvF16 ? 2LL : 4LL) * W;
}

// Rows stay below 2^31 (tensor-map coordinates and positions are 32-bit), bytes do not.
constexpr long long kMaxRowsKv = 0x7fffffffLL - 4096;

int set_paged(ChunkKv *c, const void *k, const void *v, int kv, int64_t pool_rows, int W, const int32_t *table,
              int max_blocks, int block_rows, int n_seq) {
    if (!ok_f(k) || !ok_f(v) || (!table && n_seq != 0) || pool_rows <= 0 || max_blocks <= 0) return MINF_ERR_ARG;
    if (block_rows < 16 || block_rows > 4096 || (block_rows & (block_rows - 1))) return MINF_ERR_UNSUPPORTED;
    if (pool_rows % block_rows || static_cast<long long>(max_blocks) * block_rows > kMaxRowsKv || pool_rows > kMaxRowsKv)
        return MINF_ERR_UNSUPPORTED;
    *c = {};
    c->k = k;
    c->v = v;
    c->kv = kv;
    c->W = W;
    c->row_bytes = row_bytes_of(kv, W);
    c->rows = pool_rows;
    c->table = table;
    c->max_blocks = max_blocks;
    while ((1 << c->block_shift) < block_rows) ++c->block_shift;
    c->pool_blocks = static_cast<int>(pool_rows / block_rows);
    c->cap = max_blocks * block_rows;
    return MINF_OK;
}

// Two stretches of `bytes`-byte values share some.  (A query row is read again after parts of out are written.)
bool overlap(const void *a, size_t na, const void *b, size_t nb, size_t bytes = sizeof(float)) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb * bytes && y < x + na * bytes;
}

// Whether the rotated rows can be written while others are read: an output is its input or apart from it (a value
// is turned with its partner half a head away), and apart from everything else.
bool ok_in_place(const float *out, const float *in, size_t n) { return out == in || !overlap(out, n, in, n); }
bool ok_rope_rows(const float *q_out, const float *k_out, const float *q, const float *k, const float *v, size_t nq, size_t nk) {
    return ok_in_place(q_out, q, nq) && !overlap(q_out, nq, k, nk) && !overlap(q_out, nq, v, nk) &&
           (!k_out || (ok_in_place(k_out, k, nk) && !overlap(k_out, nk, q, nq) && !overlap(k_out, nk, v, nk) &&
                       !overlap(k_out, nk, q_out, nq)));
}

bool ok_seqs(const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq) {
    return (n_past || n_seq == 0) && nt >= 0 && n_seq >= 0 && (chunk_off || nt == n_seq);
}

// Arrays of nt rows: of no rows they may be null, as empty tensors are.
bool ok_rows(const void *p, int nt) { return p ? aligned16(p) : nt == 0; }

int rope_store(float *q_out, float *k_out, const float *q, const float *k, const float *v, const int32_t *rope_pos,
               int n_axis, const uint8_t *pair_axis, const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq,
               int nh, int nk, int hd, int hd_kv, float theta, float freq_scale, int style, void *k_pool, void *v_pool,
               int kv, int64_t pool_rows, const int32_t *table, int max_blocks, int block_rows, int32_t *err,
               minf_stream_t stream) {
    int st = check_geometry(nh, nk, hd, hd_kv);
    if (st != MINF_OK) return st;
    if (hd % 8) return MINF_ERR_UNSUPPORTED;
    ChunkStoreArgs a = {};
    st = set_paged(&a.c, k_pool, v_pool, kv, pool_rows, nk * hd_kv, table, max_blocks, block_rows, n_seq);
    if (st != MINF_OK) return st;
    if (!ok_rows(q_out, nt) || (k_out && !ok_f(k_out)) || !ok_rows(q, nt) || !ok_rows(k, nt) || !ok_rows(v, nt) || !err ||
        !ok_seqs(chunk_off, n_past, nt, n_seq) || (style != 0 && style != 1) || !ok_axes(n_axis, pair_axis, hd))
        return MINF_ERR_ARG;
    if (nt == 0 || n_seq == 0) return MINF_OK;
    if (!ok_rope_rows(q_out, k_out, q, k, v, static_cast<size_t>(nt) * nh * hd, static_cast<size_t>(nt) * nk * hd_kv))
        return MINF_ERR_ARG;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q = q;
    a.k = k;
    a.v = v;
    a.rope_pos = rope_pos;
    a.n_axis = n_axis;
    a.sq = {chunk_off, n_past, nt, n_seq};
    a.nh = nh;
    a.nk = nk;
    a.hd = hd;
    a.hd_kv = hd_kv;
    a.style = style;
    a.err = err;
    return launch_chunk_store(a, theta, freq_scale, pair_axis, cs(stream));
}

int read_rows(void *k_rows, void *v_rows, int rows_f16, const void *k_pool, const void *v_pool, int kv,
              int64_t pool_rows, int row_width, const int32_t *table, int max_blocks, int block_rows,
              const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq, int32_t *err, minf_stream_t stream) {
    if (row_width <= 0 || row_width > (1 << 20) || row_width % (kv == kKvQ8 || kv == kKvQ4 ? 32 : kv == kKvF16 ? 8 : 4)) return MINF_ERR_ARG;
    if (rows_f16 && row_width % 8) return MINF_ERR_ARG;
    ChunkReadArgs a = {};
    const int st = set_paged(&a.c, k_pool, v_pool, kv, pool_rows, row_width, table, max_blocks, block_rows, n_seq);
    if (st != MINF_OK) return st;
    if (!ok_rows(k_rows, nt) || !ok_rows(v_rows, nt) || !err || !ok_seqs(chunk_off, n_past, nt, n_seq)) return MINF_ERR_ARG;
    if (nt == 0 || n_seq == 0) return MINF_OK;
    const size_t n = static_cast<size_t>(nt) * row_width;
    if (overlap(k_rows, n, v_rows, n, rows_f16 ? 2 : 4)) return MINF_ERR_ARG;
    a.k_rows = k_rows;
    a.v_rows = v_rows;
    a.f16 = rows_f16 != 0;
    a.sq = {chunk_off, n_past, nt, n_seq};
    a.err = err;
    return launch_chunk_read(a, cs(stream));
}

int attention(ChunkAttnArgs &a, float *out, const float *q, const int32_t *chunk_off, const int32_t *n_past, int nt,
              int n_seq, int max_chunk, int nh, int nk, int hd, int hd_kv, float scale, int window, int n_sink, void *ws,
              size_t ws_bytes, int32_t *err, minf_stream_t stream) {
    if (!ok_rows(out, nt) || !ok_rows(q, nt) || !err || !ok_seqs(chunk_off, n_past, nt, n_seq) || max_chunk <= 0 || window < 0 ||
        n_sink < 0)
        return MINF_ERR_ARG;
    if (nt == 0 || n_seq == 0) return MINF_OK;
    const size_t need = chunk_attn_workspace_bytes(nt, n_seq, nh, nk, hd_kv, max_chunk, a.c.kv == kKvQ4);
    if (!ws || !aligned16(ws) || ws_bytes < need) return MINF_ERR_WORKSPACE;
    if (overlap(out, static_cast<size_t>(nt) * nh * hd_kv, q, static_cast<size_t>(nt) * nh * hd)) return MINF_ERR_ARG;
    a.out = out;
    a.q = q;
    a.sq = {chunk_off, n_past, nt, n_seq};
    a.max_chunk = max_chunk;
    a.nh = nh;
    a.nk = nk;
    a.hd = hd;
    a.hd_kv = hd_kv;
    a.scale = scale;
    a.window = window;
    a.n_sink = window ? n_sink : 0;  // without a window every row is visible anyway
    a.err = err;
    a.ws = ws;
    a.ws_bytes = ws_bytes;
    return launch_chunk_attn(a, cs(stream));
}

int attn_paged(float *out, const float *q, const void *k_pool, const void *v_pool, int kv, int64_t pool_rows,
               const int32_t *table, int max_blocks, int block_rows, const int32_t *chunk_off, const int32_t *n_past,
               int nt, int n_seq, int max_chunk, int nh, int nk, int hd, int hd_kv, float scale, int window, int n_sink,
               void *ws, size_t ws_bytes, int32_t *err, minf_stream_t stream) {
    int st = check_geometry(nh, nk, hd, hd_kv);
    if (st != MINF_OK) return st;
    ChunkAttnArgs a = {};
    st = set_paged(&a.c, k_pool, v_pool, kv, pool_rows, nk * hd_kv, table, max_blocks, block_rows, n_seq);
    if (st != MINF_OK) return st;
    return attention(a, out, q, chunk_off, n_past, nt, n_seq, max_chunk, nh, nk, hd, hd_kv, scale, window, n_sink, ws,
                     ws_bytes, err, stream);
}

int attn_window(float *out, const float *q, const void *k_reg, const void *v_reg, int kv, const int64_t *row_off,
                const int32_t *caps, int max_cap, int64_t arena_rows, const int32_t *chunk_off, const int32_t *n_past,
                int nt, int n_seq, int max_chunk, int nh, int nk, int hd, int hd_kv, float scale, int window, int n_sink,
                void *ws, size_t ws_bytes, int32_t *err, minf_stream_t stream) {
    const int st = check_geometry(nh, nk, hd, hd_kv);
    if (st != MINF_OK) return st;
    if (!ok_f(k_reg) || !ok_f(v_reg) || max_cap <= 0 || (row_off && arena_rows <= 0)) return MINF_ERR_ARG;
    if (!row_off && n_seq > 1) return MINF_ERR_ARG;  // one set of regions holds one sequence
    const long long rows = row_off ? arena_rows : max_cap;
    if (rows > kMaxRowsKv || max_cap > kMaxRowsKv) return MINF_ERR_UNSUPPORTED;
    ChunkAttnArgs a = {};
    a.c.k = k_reg;
    a.c.v = v_reg;
    a.c.kv = kv;
    a.c.W = nk * hd_kv;
    a.c.row_bytes = row_bytes_of(kv, a.c.W);
    a.c.rows = rows;
    a.c.row_off = row_off;
    a.c.caps = caps;
    a.c.cap = max_cap;
    return attention(a, out, q, chunk_off, n_past, nt, n_seq, max_chunk, nh, nk, hd, hd_kv, scale, window, n_sink, ws,
                     ws_bytes, err, stream);
}

int layer_step(float *xn, const float *h, const float *gain, float eps, int n_embd, float *q, float *k, const float *v,
               const int32_t *rope_pos, int n_axis, const uint8_t *pair_axis, const int32_t *chunk_off,
               const int32_t *n_past, int nt, int n_seq, int max_chunk, void *k_pool, void *v_pool, int kv,
               int64_t pool_rows, const int32_t *table, int max_blocks, int block_rows, int nh, int nk, int hd, int hd_kv,
               float theta, float freq_scale, int style, int window, int n_sink, float *out, void *ws, size_t ws_bytes,
               int32_t *err, minf_stream_t stream) {
    int st = check_geometry(nh, nk, hd, hd_kv);
    if (st != MINF_OK) return st;
    // everything is checked before the first launch
    ChunkKv c;
    st = set_paged(&c, k_pool, v_pool, kv, pool_rows, nk * hd_kv, table, max_blocks, block_rows, n_seq);
    if (st != MINF_OK) return st;
    if (hd % 8) return MINF_ERR_UNSUPPORTED;
    if (((!xn || !h) && nt != 0) || n_embd <= 0 || !ok_rows(q, nt) || !ok_rows(k, nt) || !ok_rows(v, nt) ||
        !ok_rows(out, nt) || !err ||
        !ok_seqs(chunk_off, n_past, nt, n_seq) || max_chunk <= 0 || window < 0 || n_sink < 0 ||
        (style != 0 && style != 1) || !ok_axes(n_axis, pair_axis, hd))
        return MINF_ERR_ARG;
    if (nt == 0 || n_seq == 0) return MINF_OK;
    if (!ws || !aligned16(ws) || ws_bytes < chunk_attn_workspace_bytes(nt, n_seq, nh, nk, hd_kv, max_chunk, kv == kKvQ4))
        return MINF_ERR_WORKSPACE;
    if (overlap(out, static_cast<size_t>(nt) * nh * hd_kv, q, static_cast<size_t>(nt) * nh * hd) ||
        !ok_rope_rows(q, k, q, k, v, static_cast<size_t>(nt) * nh * hd, static_cast<size_t>(nt) * nk * hd_kv))
        return MINF_ERR_ARG;
    st = launch_rms_norm(xn, h, gain, nt, n_embd, eps, cs(stream));
    if (st != MINF_OK) return st;
    st = rope_store(q, k, q, k, v, rope_pos, n_axis, pair_axis, chunk_off, n_past, nt, n_seq, nh, nk, hd, hd_kv, theta,
                    freq_scale, style, k_pool, v_pool, kv, pool_rows, table, max_blocks, block_rows, err, stream);
    if (st != MINF_OK) return st;
    return attn_paged(out, q, k_pool, v_pool, kv, pool_rows, table, max_blocks, block_rows, chunk_off, n_past, nt, n_seq,
                      max_chunk, nh, nk, hd, hd_kv, 1.0f / sqrtf(static_cast<float>(hd)), window, n_sink, ws, ws_bytes,
                      err, stream);
}

}  // namespace

extern "C" {

int minf_rope_axes(float *y, const float *x, const int32_t *pos, int nt, int n_axis, const uint8_t *pair_axis,
                   int n_head, int hd, float theta, float freq_scale, int style, int32_t *err, minf_stream_t stream) {
    if (((!y || !x || !pos) && nt != 0) || !err || nt < 0 || n_head <= 0 || hd <= 0 || (hd & 1) || hd > 2 * kMaxHalf) return MINF_ERR_ARG;
    if ((style != 0 && style != 1) || !ok_axes(n_axis, pair_axis, hd)) return MINF_ERR_ARG;
    if (static_cast<long long>(n_head) * hd > (1 << 20)) return MINF_ERR_UNSUPPORTED;
    if (nt > 0 && !ok_in_place(y, x, static_cast<size_t>(nt) * n_head * hd)) return MINF_ERR_ARG;
    RopeAxesArgs a = {y, x, pos, err, nt, n_axis, n_head, hd, style};
    return launch_rope_axes(a, theta, freq_scale, pair_axis, cs(stream));
}

size_t minf_attn_chunk_workspace_bytes(int nt, int n_seq, int n_head, int n_kv_head, int hd_kv, int max_chunk) {
    return chunk_attn_workspace_bytes(nt, n_seq, n_head, n_kv_head, hd_kv, max_chunk);
}

int minf_rope_kv_append_chunk_paged(float *q_out, float *k_out, const float *q, const float *k, const float *v,
                                    const int32_t *rope_pos, int n_axis, const uint8_t *pair_axis,
                                    const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq, int n_head,
                                    int n_kv_head, int hd, int hd_kv, float theta, float freq_scale, int style,
                                    float *k_pool, float *v_pool, int64_t pool_rows, const int32_t *block_table,
                                    int max_blocks, int block_rows, int32_t *err, minf_stream_t stream) {
    return rope_store(q_out, k_out, q, k, v, rope_pos, n_axis, pair_axis, chunk_off, n_past, nt, n_seq, n_head, n_kv_head,
                      hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, kKvF32, pool_rows, block_table, max_blocks,
                      block_rows, err, stream);
}

int minf_kv_read_chunk_paged(void *k_rows, void *v_rows, int rows_f16, const float *k_pool, const float *v_pool,
                             int64_t pool_rows, int row_width, const int32_t *block_table, int max_blocks,
                             int block_rows, const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq,
                             int32_t *err, minf_stream_t stream) {
    return read_rows(k_rows, v_rows, rows_f16, k_pool, v_pool, kKvF32, pool_rows, row_width, block_table, max_blocks,
                     block_rows, chunk_off, n_past, nt, n_seq, err, stream);
}

int minf_gqa_attn_chunk_paged(float *out, const float *q, const float *k_pool, const float *v_pool, int64_t pool_rows,
                              const int32_t *block_table, int max_blocks, int block_rows, const int32_t *chunk_off,
                              const int32_t *n_past, int nt, int n_seq, int max_chunk, int n_head, int n_kv_head, int hd,
                              int hd_kv, float scale, int window, int n_sink, void *ws, size_t ws_bytes, int32_t *err,
                              minf_stream_t stream) {
    return attn_paged(out, q, k_pool, v_pool, kKvF32, pool_rows, block_table, max_blocks, block_rows, chunk_off, n_past, nt,
                      n_seq, max_chunk, n_head, n_kv_head, hd, hd_kv, scale, window, n_sink, ws, ws_bytes, err, stream);
}

int minf_gqa_attn_window(float *out, const float *q, const float *k_reg, const float *v_reg, const int64_t *seq_row_off,
                         const int32_t *seq_cap, int max_cap, int64_t arena_rows, const int32_t *chunk_off,
                         const int32_t *n_past, int nt, int n_seq, int max_chunk, int n_head, int n_kv_head, int hd,
                         int hd_kv, float scale, int window, int n_sink, void *ws, size_t ws_bytes, int32_t *err,
                         minf_stream_t stream) {
    return attn_window(out, q, k_reg, v_reg, kKvF32, seq_row_off, seq_cap, max_cap, arena_rows, chunk_off, n_past, nt, n_seq,
                       max_chunk, n_head, n_kv_head, hd, hd_kv, scale, window, n_sink, ws, ws_bytes, err, stream);
}

int minf_layer_attn_step_chunk_paged(float *xn, const float *h, const float *gain, float eps, int n_embd, float *q,
                                     float *k, const float *v, const int32_t *rope_pos, int n_axis,
                                     const uint8_t *pair_axis, const int32_t *chunk_off, const int32_t *n_past, int nt,
                                     int n_seq, int max_chunk, float *k_pool, float *v_pool, int64_t pool_rows,
                                     const int32_t *block_table, int max_blocks, int block_rows, int n_head,
                                     int n_kv_head, int hd, int hd_kv, float theta, float freq_scale, int style,
                                     int window, int n_sink, float *out, void *ws, size_t ws_bytes, int32_t *err,
                                     minf_stream_t stream) {
    return layer_step(xn, h, gain, eps, n_embd, q, k, v, rope_pos, n_axis, pair_axis, chunk_off, n_past, nt, n_seq,
                      max_chunk, k_pool, v_pool, kKvF32, pool_rows, block_table, max_blocks, block_rows, n_head, n_kv_head,
                      hd, hd_kv, theta, freq_scale, style, window, n_sink, out, ws, ws_bytes, err, stream);
}

int minf_rope_kv_append_chunk_paged_f16(float *q_out, float *k_out, const float *q, const float *k, const float *v,
                                    const int32_t *rope_pos, int n_axis, const uint8_t *pair_axis,
                                    const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq, int n_head,
                                    int n_kv_head, int hd, int hd_kv, float theta, float freq_scale, int style,
                                    uint16_t *k_pool, uint16_t *v_pool, int64_t pool_rows, const int32_t *block_table,
                                    int max_blocks, int block_rows, int32_t *err, minf_stream_t stream) {
    return rope_store(q_out, k_out, q, k, v, rope_pos, n_axis, pair_axis, chunk_off, n_past, nt, n_seq, n_head, n_kv_head,
                      hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, kKvF16, pool_rows, block_table, max_blocks,
                      block_rows, err, stream);
}

int minf_kv_read_chunk_paged_f16(void *k_rows, void *v_rows, int rows_f16, const uint16_t *k_pool, const uint16_t *v_pool,
                             int64_t pool_rows, int row_width, const int32_t *block_table, int max_blocks,
                             int block_rows, const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq,
                             int32_t *err, minf_stream_t stream) {
    return read_rows(k_rows, v_rows, rows_f16, k_pool, v_pool, kKvF16, pool_rows, row_width, block_table, max_blocks,
                     block_rows, chunk_off, n_past, nt, n_seq, err, stream);
}

int minf_gqa_attn_chunk_paged_f16(float *out, const float *q, const uint16_t *k_pool, const uint16_t *v_pool, int64_t pool_rows,
                              const int32_t *block_table, int max_blocks, int block_rows, const int32_t *chunk_off,
                              const int32_t *n_past, int nt, int n_seq, int max_chunk, int n_head, int n_kv_head, int hd,
                              int hd_kv, float scale, int window, int n_sink, void *ws, size_t ws_bytes, int32_t *err,
                              minf_stream_t stream) {
    return attn_paged(out, q, k_pool, v_pool, kKvF16, pool_rows, block_table, max_blocks, block_rows, chunk_off, n_past, nt,
                      n_seq, max_chunk, n_head, n_kv_head, hd, hd_kv, scale, window, n_sink, ws, ws_bytes, err, stream);
}

int minf_gqa_attn_window_f16(float *out, const float *q, const uint16_t *k_reg, const uint16_t *v_reg, const int64_t *seq_row_off,
                         const int32_t *seq_cap, int max_cap, int64_t arena_rows, const int32_t *chunk_off,
                         const int32_t *n_past, int nt, int n_seq, int max_chunk, int n_head, int n_kv_head, int hd,
                         int hd_kv, float scale, int window, int n_sink, void *ws, size_t ws_bytes, int32_t *err,
                         minf_stream_t stream) {
    return attn_window(out, q, k_reg, v_reg, kKvF16, seq_row_off, seq_cap, max_cap, arena_rows, chunk_off, n_past, nt, n_seq,
                       max_chunk, n_head, n_kv_head, hd, hd_kv, scale, window, n_sink, ws, ws_bytes, err, stream);
}

int minf_layer_attn_step_chunk_paged_f16(float *xn, const float *h, const float *gain, float eps, int n_embd, float *q,
                                     float *k, const float *v, const int32_t *rope_pos, int n_axis,
                                     const uint8_t *pair_axis, const int32_t *chunk_off, const int32_t *n_past, int nt,
                                     int n_seq, int max_chunk, uint16_t *k_pool, uint16_t *v_pool, int64_t pool_rows,
                                     const int32_t *block_table, int max_blocks, int block_rows, int n_head,
                                     int n_kv_head, int hd, int hd_kv, float theta, float freq_scale, int style,
                                     int window, int n_sink, float *out, void *ws, size_t ws_bytes, int32_t *err,
                                     minf_stream_t stream) {
    return layer_step(xn, h, gain, eps, n_embd, q, k, v, rope_pos, n_axis, pair_axis, chunk_off, n_past, nt, n_seq,
                      max_chunk, k_pool, v_pool, kKvF16, pool_rows, block_table, max_blocks, block_rows, n_head, n_kv_head,
                      hd, hd_kv, theta, freq_scale, style, window, n_sink, out, ws, ws_bytes, err, stream);
}

int minf_rope_kv_append_chunk_paged_q8(float *q_out, float *k_out, const float *q, const float *k, const float *v,
                                    const int32_t *rope_pos, int n_axis, const uint8_t *pair_axis,
                                    const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq, int n_head,
                                    int n_kv_head, int hd, int hd_kv, float theta, float freq_scale, int style,
                                    uint8_t *k_pool, uint8_t *v_pool, int64_t pool_rows, const int32_t *block_table,
                                    int max_blocks, int block_rows, int32_t *err, minf_stream_t stream) {
    return rope_store(q_out, k_out, q, k, v, rope_pos, n_axis, pair_axis, chunk_off, n_past, nt, n_seq, n_head, n_kv_head,
                      hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, kKvQ8, pool_rows, block_table, max_blocks,
                      block_rows, err, stream);
}

int minf_kv_read_chunk_paged_q8(void *k_rows, void *v_rows, int rows_f16, const uint8_t *k_pool, const uint8_t *v_pool,
                             int64_t pool_rows, int row_width, const int32_t *block_table, int max_blocks,
                             int block_rows, const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq,
                             int32_t *err, minf_stream_t stream) {
    return read_rows(k_rows, v_rows, rows_f16, k_pool, v_pool, kKvQ8, pool_rows, row_width, block_table, max_blocks,
                     block_rows, chunk_off, n_past, nt, n_seq, err, stream);
}

int minf_gqa_attn_chunk_paged_q8(float *out, const float *q, const uint8_t *k_pool, const uint8_t *v_pool, int64_t pool_rows,
                              const int32_t *block_table, int max_blocks, int block_rows, const int32_t *chunk_off,
                              const int32_t *n_past, int nt, int n_seq, int max_chunk, int n_head, int n_kv_head, int hd,
                              int hd_kv, float scale, int window, int n_sink, void *ws, size_t ws_bytes, int32_t *err,
                              minf_stream_t stream) {
    return attn_paged(out, q, k_pool, v_pool, kKvQ8, pool_rows, block_table, max_blocks, block_rows, chunk_off, n_past, nt,
                      n_seq, max_chunk, n_head, n_kv_head, hd, hd_kv, scale, window, n_sink, ws, ws_bytes, err, stream);
}

int minf_gqa_attn_window_q8(float *out, const float *q, const uint8_t *k_reg, const uint8_t *v_reg, const int64_t *seq_row_off,
                         const int32_t *seq_cap, int max_cap, int64_t arena_rows, const int32_t *chunk_off,
                         const int32_t *n_past, int nt, int n_seq, int max_chunk, int n_head, int n_kv_head, int hd,
                         int hd_kv, float scale, int window, int n_sink, void *ws, size_t ws_bytes, int32_t *err,
                         minf_stream_t stream) {
    return attn_window(out, q, k_reg, v_reg, kKvQ8, seq_row_off, seq_cap, max_cap, arena_rows, chunk_off, n_past, nt, n_seq,
                       max_chunk, n_head, n_kv_head, hd, hd_kv, scale, window, n_sink, ws, ws_bytes, err, stream);
}

int minf_layer_attn_step_chunk_paged_q8(float *xn, const float *h, const float *gain, float eps, int n_embd, float *q,
                                     float *k, const float *v, const int32_t *rope_pos, int n_axis,
                                     const uint8_t *pair_axis, const int32_t *chunk_off, const int32_t *n_past, int nt,
                                     int n_seq, int max_chunk, uint8_t *k_pool, uint8_t *v_pool, int64_t pool_rows,
                                     const int32_t *block_table, int max_blocks, int block_rows, int n_head,
                                     int n_kv_head, int hd, int hd_kv, float theta, float freq_scale, int style,
                                     int window, int n_sink, float *out, void *ws, size_t ws_bytes, int32_t *err,
                                     minf_stream_t stream) {
    return layer_step(xn, h, gain, eps, n_embd, q, k, v, rope_pos, n_axis, pair_axis, chunk_off, n_past, nt, n_seq,
                      max_chunk, k_pool, v_pool, kKvQ8, pool_rows, block_table, max_blocks, block_rows, n_head, n_kv_head,
                      hd, hd_kv, theta, freq_scale, style, window, n_sink, out, ws, ws_bytes, err, stream);
}

int minf_rope_kv_append_chunk_paged_q4(float *q_out, float *k_out, const float *q, const float *k, const float *v,
                                    const int32_t *rope_pos, int n_axis, const uint8_t *pair_axis,
                                    const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq, int n_head,
                                    int n_kv_head, int hd, int hd_kv, float theta, float freq_scale, int style,
                                    uint8_t *k_pool, uint8_t *v_pool, int64_t pool_rows, const int32_t *block_table,
                                    int max_blocks, int block_rows, int32_t *err, minf_stream_t stream) {
    return rope_store(q_out, k_out, q, k, v, rope_pos, n_axis, pair_axis, chunk_off, n_past, nt, n_seq, n_head, n_kv_head,
                      hd, hd_kv, theta, freq_scale, style, k_pool, v_pool, kKvQ4, pool_rows, block_table, max_blocks,
                      block_rows, err, stream);
}

int minf_kv_read_chunk_paged_q4(void *k_rows, void *v_rows, int rows_f16, const uint8_t *k_pool, const uint8_t *v_pool,
                             int64_t pool_rows, int row_width, const int32_t *block_table, int max_blocks,
                             int block_rows, const int32_t *chunk_off, const int32_t *n_past, int nt, int n_seq,
                             int32_t *err, minf_stream_t stream) {
    return read_rows(k_rows, v_rows, rows_f16, k_pool, v_pool, kKvQ4, pool_rows, row_width, block_table, max_blocks,
                     block_rows, chunk_off, n_past, nt, n_seq, err, stream);
}

int minf_gqa_attn_chunk_paged_q4(float *out, const float *q, const uint8_t *k_pool, const uint8_t *v_pool, int64_t pool_rows,
                              const int32_t *block_table, int max_blocks, int block_rows, const int32_t *chunk_off,
                              const int32_t *n_past, int nt, int n_seq, int max_chunk, int n_head, int n_kv_head, int hd,
                              int hd_kv, float scale, int window, int n_sink, void *ws, size_t ws_bytes, int32_t *err,
                              minf_stream_t stream) {
    return attn_paged(out, q, k_pool, v_pool, kKvQ4, pool_rows, block_table, max_blocks, block_rows, chunk_off, n_past, nt,
                      n_seq, max_chunk, n_head, n_kv_head, hd, hd_kv, scale, window, n_sink, ws, ws_bytes, err, stream);
}

int minf_gqa_attn_window_q4(float *out, const float *q, const uint8_t *k_reg, const uint8_t *v_reg, const int64_t *seq_row_off,
                         const int32_t *seq_cap, int max_cap, int64_t arena_rows, const int32_t *chunk_off,
                         const int32_t *n_past, int nt, int n_seq, int max_chunk, int n_head, int n_kv_head, int hd,
                         int hd_kv, float scale, int window, int n_sink, void *ws, size_t ws_bytes, int32_t *err,
                         minf_stream_t stream) {
    return attn_window(out, q, k_reg, v_reg, kKvQ4, seq_row_off, seq_cap, max_cap, arena_rows, chunk_off, n_past, nt, n_seq,
                       max_chunk, n_head, n_kv_head, hd, hd_kv, scale, window, n_sink, ws, ws_bytes, err, stream);
}

int minf_layer_attn_step_chunk_paged_q4(float *xn, const float *h, const float *gain, float eps, int n_embd, float *q,
                                     float *k, const float *v, const int32_t *rope_pos, int n_axis,
                                     const uint8_t *pair_axis, const int32_t *chunk_off, const int32_t *n_past, int nt,
                                     int n_seq, int max_chunk, uint8_t *k_pool, uint8_t *v_pool, int64_t pool_rows,
                                     const int32_t *block_table, int max_blocks, int block_rows, int n_head,
                                     int n_kv_head, int hd, int hd_kv, float theta, float freq_scale, int style,
                                     int window, int n_sink, float *out, void *ws, size_t ws_bytes, int32_t *err,
                                     minf_stream_t stream) {
    return layer_step(xn, h, gain, eps, n_embd, q, k, v, rope_pos, n_axis, pair_axis, chunk_off, n_past, nt, n_seq,
                      max_chunk, k_pool, v_pool, kKvQ4, pool_rows, block_table, max_blocks, block_rows, n_head, n_kv_head,
                      hd, hd_kv, theta, freq_scale, style, window, n_sink, out, ws, ws_bytes, err, stream);
}

}  // extern "C"
