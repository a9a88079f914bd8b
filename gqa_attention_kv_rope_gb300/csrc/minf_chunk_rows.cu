// minf_chunk_rows.cu -- the row work of chunks of new tokens: several-axis RoPE, RoPE + store
// into paged K/V (converted or quantised as it is written), and the read back.
//
// Rotation ("11 . Attention, vec ops, and the KV cache", §2.3 and §3.2.2, with a position per
// axis): pair i of token t turns by pos[axis(i)][t] * f_i, f_i = freq_scale / theta^(2i/hd).
// The angle is taken in turns: f_i / 2 pi as a 64-bit fraction F, and pos * F in 64-bit integers,
// whose overflow drops exactly the whole turns.  F is off by at most 2^-53 of itself, so the
// angle of position 2^31 is still good to 2^-22 turns x f_i; a product in fp32 is off by 2^-24 of
// pos * f_i radians, 2.4e-3 at position 40960.  The integer product costs three multiplies.
//
// All of it is bounded by memory: each value is read once and written once, in float4s.  A block
// takes a few tokens: it resolves their rows and the sines and cosines of their angles once into
// shared memory (every head of a token shares them), then sweeps the tokens' heads.
#include <cmath>

#include "minf_chunk.cuh"

namespace minf {

void axis_table(AxisTable *t, int hd, float theta, float freq_scale, const unsigned char *pair_axis) {
    const double two_pi = 6.283185307179586476925286766559;
    for (int i = 0; i < kMaxHalf; ++i) {
        t->turn[i] = 0;
        t->axis[i] = 0;
        if (i >= hd / 2) continue;
        const double e = static_cast<double>(2 * i) / static_cast<double>(hd);
        const double f = static_cast<double>(freq_scale) / std::pow(static_cast<double>(theta), e) / two_pi;
        const double frac = f - std::floor(f);  // whole turns a position drop out
        if (frac < 1.0)                         // (NaN for a theta that is not positive: angle 0)
            t->turn[i] = static_cast<unsigned long long>(std::ldexp(frac, 64));  // at most 2^64 - 2^11
        if (pair_axis) t->axis[i] = pair_axis[i];
    }
}

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 4;  // tokens of a block

// Cosine and sine of pos * F turns: the product's top 32 bits are the angle in [-1/2, 1/2) turns.
__device__ __forceinline__ float2 turn_sincos(int pos, unsigned long long F) {
    const unsigned long long ph = static_cast<unsigned long long>(static_cast<unsigned>(pos)) * F;
    const float half_turns = static_cast<float>(static_cast<int>(ph >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float2 cs;
    sincospif(half_turns, &cs.y, &cs.x);
    return cs;
}

__device__ __forceinline__ void turn_pair(float &a, float &b, float2 cs) {
    const float x = a, y = b;
    a = x * cs.x - y * cs.y;
    b = x * cs.y + y * cs.x;
}

// Unit u of a head row (8 values): four pairs, as two float4.  style 0: values 4u.. and
// 4u + hd/2..; style 1: values 8u.. and 8u + 4...
__device__ __forceinline__ void unit_at(int u, int hd, int style, int &i0, int &i1) {
    i0 = style == 0 ? u : 2 * u;
    i1 = style == 0 ? u + (hd >> 3) : 2 * u + 1;
}
__device__ __forceinline__ void turn_unit(float4 &a, float4 &b, int style, const float2 *cs) {
    if (style == 0) {
        turn_pair(a.x, b.x, cs[0]);
        turn_pair(a.y, b.y, cs[1]);
        turn_pair(a.z, b.z, cs[2]);
        turn_pair(a.w, b.w, cs[3]);
    } else {
        turn_pair(a.x, a.y, cs[0]);
        turn_pair(a.z, a.w, cs[1]);
        turn_pair(b.x, b.y, cs[2]);
        turn_pair(b.z, b.w, cs[3]);
    }
}

// kVec: hd a multiple of 8 (rows of float4 units); otherwise pair by pair.
template <bool kVec>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const RopeAxesArgs a, const __grid_constant__ AxisTable tab,
                                                             int tok) {
    __shared__ float2 cs[kMaxTok][kMaxHalf];
    __shared__ int bad[kMaxTok];
    const int half = a.hd >> 1, t0 = blockIdx.x * tok;
    const int n = min(tok, a.nt - t0);
    if (threadIdx.x < kMaxTok) bad[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        const int pos = __ldg(a.pos + static_cast<size_t>(tab.axis[p]) * a.nt + t0 + t);
        if (pos < 0) bad[t] = 1;
        cs[t][p] = turn_sincos(pos, tab.turn[p]);
    }
    __syncthreads();
    if (threadIdx.x < n && bad[threadIdx.x] && blockIdx.y == 0) flag_error(a.err, MINF_ERRBIT_ROPE_POS);
    const int per = kVec ? a.hd >> 3 : half;  // units of a head row
    const int total = n * a.nh * per;
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < total; i += gridDim.y * kThreads) {
        const int row = i / per, u = i - row * per, t = row / a.nh;
        const size_t at = (static_cast<size_t>(t0) * a.nh + row) * a.hd;
        const float2 *c = cs[t];
        if constexpr (kVec) {
            int i0, i1;
            unit_at(u, a.hd, a.style, i0, i1);
            const float4 *x = reinterpret_cast<const float4 *>(a.x + at);
            float4 *y = reinterpret_cast<float4 *>(a.y + at);
            float4 v0 = x[i0], v1 = x[i1];
            if (!bad[t]) turn_unit(v0, v1, a.style, c + 4 * u);
            y[i0] = v0;
            y[i1] = v1;
        } else {
            const int i0 = a.style == 0 ? u : 2 * u, i1 = a.style == 0 ? u + half : 2 * u + 1;
            float v0 = a.x[at + i0], v1 = a.x[at + i1];
            if (!bad[t]) turn_pair(v0, v1, c[u]);
            a.y[at + i0] = v0;
            a.y[at + i1] = v1;
        }
    }
}

// Tokens a block: kMaxTok where that still leaves every SM several blocks, else one, with the
// token's heads spread over up to `split` blocks.
void row_grid(int nt, long long units_tok, int &tok, dim3 &grid) {
    const int sms = sm_count();
    tok = nt >= kMaxTok * 4 * sms ? kMaxTok : 1;
    long long split = 1;
    if (nt < 4 * sms) {
        split = (units_tok + kThreads - 1) / kThreads;
        const long long room = (4LL * sms + nt - 1) / nt;
        if (split > room) split = room;
        if (split > 64) split = 64;
    }
    grid = dim3(static_cast<unsigned>((static_cast<long long>(nt) + tok - 1) / tok), static_cast<unsigned>(split));
}

}  // namespace

int launch_rope_axes(const RopeAxesArgs &a, float theta, float freq_scale, const unsigned char *pair_axis,
                     cudaStream_t s) {
    if (a.nt == 0) return MINF_OK;
    AxisTable tab;
    axis_table(&tab, a.hd, theta, freq_scale, pair_axis);
    const bool vec = a.hd % 8 == 0 && aligned16(a.x) && aligned16(a.y);
    int tok;
    dim3 grid;
    row_grid(a.nt, static_cast<long long>(a.nh) * (vec ? a.hd / 8 : a.hd / 2), tok, grid);
    if (vec)
        rope_axes_kernel<true><<<grid, kThreads, 0, s>>>(a, tab, tok);
    else
        rope_axes_kernel<false><<<grid, kThreads, 0, s>>>(a, tab, tok);
    return cudaPeekAtLastError() == cudaSuccess ? MINF_OK : MINF_ERR_CUDA;
}

// ----------------------------------------------------------------------------- RoPE + store
namespace {

__device__ __forceinline__ void put_row4(float *row, int i4, float4 v) { reinterpret_cast<float4 *>(row)[i4] = v; }
__device__ __forceinline__ void put_row4(__half *row, int i4, float4 v) {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    reinterpret_cast<uint2 *>(row)[i4] =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// The quants of four values with 1/d given (halves away from zero, as the other Q8_0 stores).
__device__ __forceinline__ uint32_t q8_pack(float4 x, float id) {
    const int a = static_cast<int>(roundf(__fmul_rn(x.x, id))), b = static_cast<int>(roundf(__fmul_rn(x.y, id)));
    const int c = static_cast<int>(roundf(__fmul_rn(x.z, id))), e = static_cast<int>(roundf(__fmul_rn(x.w, id)));
    return (static_cast<uint32_t>(a) & 0xffu) | ((static_cast<uint32_t>(b) & 0xffu) << 8) |
           ((static_cast<uint32_t>(c) & 0xffu) << 16) | ((static_cast<uint32_t>(e) & 0xffu) << 24);
}
__device__ __forceinline__ float amax4(float4 x) {
    return fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
}

// A Q8_0 row's zero padding after its scales (up to 14 bytes).
__device__ __forceinline__ void q8_pad(unsigned char *row, int W, long long rb) {
    for (long long b = W + W / 16; b < rb; b += 2) *reinterpret_cast<uint16_t *>(row + b) = 0;
}

// Blocks take `tok` tokens (blockIdx.x) and every gridDim.y-th stretch of their units.  The units
// of a token, in order: q heads, k heads (8 values a unit) and v (4 values a unit).  Each count
// is a multiple of 8 units (hd_kv 64 or 128; q's is rounded up), so the eight (or four) lanes that
// share a Q8_0 block are always active together.
template <typename T>
__global__ void __launch_bounds__(kThreads) chunk_store_kernel(const ChunkStoreArgs a,
                                                               const __grid_constant__ AxisTable tq,
                                                               const __grid_constant__ AxisTable tk, int tok) {
    __shared__ float2 cq[kMaxTok][kMaxHalf], ck[kMaxTok][kMaxHalf];
    __shared__ long long dst[kMaxTok];  // pool row of the token, -1: not stored
    __shared__ int pos0[kMaxTok];       // cache position
    __shared__ int state[kMaxTok];      // 0 a token, 1 left unrotated, 2 padding: nothing is written
    const int hq = a.hd >> 1, hk = a.hd_kv >> 1, t0 = blockIdx.x * tok;
    const int n = min(tok, a.sq.nt - t0);
    const bool first = blockIdx.y == 0;
    if (blockIdx.x == 0 && first && a.sq.off) {  // chunk_off: nondecreasing within [0, nt]
        for (int s = threadIdx.x; s <= a.sq.n_seq; s += kThreads) {
            const int o = __ldg(a.sq.off + s);
            if (o < 0 || o > a.sq.nt || (s > 0 && o < __ldg(a.sq.off + s - 1))) flag_error(a.err, MINF_ERRBIT_CHUNK);
        }
    }
    if (threadIdx.x < n) {
        const int t = t0 + threadIdx.x, s = chunk_seq_of(a.sq.off, a.sq.n_seq, t);
        long long row = -1;
        int st = 2, pos = 0;
        if (s >= 0) {
            const SeqRows r = seq_rows(a.c, s);
            const long long p = static_cast<long long>(__ldg(a.sq.n_past + s)) + (t - (a.sq.off ? __ldg(a.sq.off + s) : s));
            st = 0;
            pos = p < 0 ? -1 : (p > 0x7fffffffLL ? 0x7fffffff : static_cast<int>(p));
            if (p < 0 || p >= r.cap) {
                if (first) flag_error(a.err, MINF_ERRBIT_STORE_POS);
            } else {
                row = seq_row(a.c, r, static_cast<int>(p));
                if (row < 0 && first) flag_error(a.err, MINF_ERRBIT_BLOCK);
            }
        }
        dst[threadIdx.x] = row;
        pos0[threadIdx.x] = pos;
        state[threadIdx.x] = st;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * hq; i += kThreads) {
        const int t = i / hq, p = i - t * hq;
        const int pos = a.rope_pos ? __ldg(a.rope_pos + static_cast<size_t>(tq.axis[p]) * a.sq.nt + t0 + t) : pos0[t];
        if (pos < 0 && state[t] == 0) state[t] = 1;
        cq[t][p] = turn_sincos(pos, tq.turn[p]);
        if (p < hk) ck[t][p] = a.hd == a.hd_kv ? cq[t][p] : turn_sincos(pos, tk.turn[p]);
    }
    __syncthreads();
    if (threadIdx.x < n && state[threadIdx.x] == 1 && first) flag_error(a.err, MINF_ERRBIT_ROPE_POS);
    const int nq = a.nh * (a.hd >> 3), uq = (nq + 7) & ~7, uk = a.nk * (a.hd_kv >> 3), uv = a.c.W >> 2;
    const int per = uq + uk + uv, total = n * per;
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < total; i += gridDim.y * kThreads) {
        const int t = i / per;
        int u = i - t * per;
        if (state[t] == 2) continue;
        const bool turn = state[t] == 0;
        const long long row = dst[t];
        const unsigned mask = 0xffu << (threadIdx.x & 24u);
        if (u < uq) {
            if (u >= nq) continue;
            const int per_h = a.hd >> 3, h = u / per_h;
            u -= h * per_h;
            const size_t at = (static_cast<size_t>(t0 + t) * a.nh + h) * a.hd;
            int i0, i1;
            unit_at(u, a.hd, a.style, i0, i1);
            float4 x0 = reinterpret_cast<const float4 *>(a.q + at)[i0], x1 = reinterpret_cast<const float4 *>(a.q + at)[i1];
            if (turn) turn_unit(x0, x1, a.style, cq[t] + 4 * u);
            reinterpret_cast<float4 *>(a.q_out + at)[i0] = x0;
            reinterpret_cast<float4 *>(a.q_out + at)[i1] = x1;
            continue;
        }
        u -= uq;
        if (u < uk) {
            const int per_h = a.hd_kv >> 3, h = u / per_h;
            u -= h * per_h;
            const size_t at = (static_cast<size_t>(t0 + t) * a.nk + h) * a.hd_kv;
            int i0, i1;
            unit_at(u, a.hd_kv, a.style, i0, i1);
            float4 x0 = reinterpret_cast<const float4 *>(a.k + at)[i0], x1 = reinterpret_cast<const float4 *>(a.k + at)[i1];
            if (turn) turn_unit(x0, x1, a.style, ck[t] + 4 * u);
            if (a.k_out) {
                reinterpret_cast<float4 *>(a.k_out + at)[i0] = x0;
                reinterpret_cast<float4 *>(a.k_out + at)[i1] = x1;
            }
            if constexpr (std::is_same<T, Q8>::value) {
                // style 0: x0 (and x1) of eight consecutive lanes are one 32-value block each;
                // style 1: x0 and x1 of four consecutive lanes are one block
                float m0 = amax4(x0), m1 = amax4(x1);
                if (a.style == 1) m0 = m1 = fmaxf(m0, m1);
                m0 = fmaxf(m0, __shfl_xor_sync(mask, m0, 1));
                m1 = fmaxf(m1, __shfl_xor_sync(mask, m1, 1));
                m0 = fmaxf(m0, __shfl_xor_sync(mask, m0, 2));
                m1 = fmaxf(m1, __shfl_xor_sync(mask, m1, 2));
                if (a.style == 0) {
                    m0 = fmaxf(m0, __shfl_xor_sync(mask, m0, 4));
                    m1 = fmaxf(m1, __shfl_xor_sync(mask, m1, 4));
                }
                if (row >= 0) {
                    unsigned char *rowp = static_cast<unsigned char *>(const_cast<void *>(a.c.k)) + row * a.c.row_bytes;
                    const float d0 = __fdiv_rn(m0, 127.0f), d1 = __fdiv_rn(m1, 127.0f);
                    const float r0 = d0 != 0.0f ? __fdiv_rn(1.0f, d0) : 0.0f, r1 = d1 != 0.0f ? __fdiv_rn(1.0f, d1) : 0.0f;
                    uint32_t *qp = reinterpret_cast<uint32_t *>(rowp + h * a.hd_kv);
                    qp[i0] = q8_pack(x0, r0);
                    qp[i1] = q8_pack(x1, r1);
                    __half *sp = reinterpret_cast<__half *>(rowp + a.c.W) + h * (a.hd_kv >> 5);
                    if ((i0 & 7) == 0) sp[i0 >> 3] = __float2half_rn(d0);
                    if ((i1 & 7) == 0) sp[i1 >> 3] = __float2half_rn(d1);
                    if (h == 0 && u == 0) q8_pad(rowp, a.c.W, a.c.row_bytes);
                }
            } else if (row >= 0) {
                T *rowp = static_cast<T *>(const_cast<void *>(a.c.k)) + static_cast<size_t>(row) * a.c.W + h * a.hd_kv;
                put_row4(rowp, i0, x0);
                put_row4(rowp, i1, x1);
            }
            continue;
        }
        u -= uk;
        const float4 x = reinterpret_cast<const float4 *>(a.v)[static_cast<size_t>(t0 + t) * uv + u];
        if constexpr (std::is_same<T, Q8>::value) {
            float d;
            const uint32_t q = quant4(x, mask, d);
            if (row >= 0) {
                unsigned char *rowp = static_cast<unsigned char *>(const_cast<void *>(a.c.v)) + row * a.c.row_bytes;
                reinterpret_cast<uint32_t *>(rowp)[u] = q;
                if ((u & 7) == 0) reinterpret_cast<__half *>(rowp + a.c.W)[u >> 3] = __float2half_rn(d);
                if (u == 0) q8_pad(rowp, a.c.W, a.c.row_bytes);
            }
        } else if (row >= 0) {
            put_row4(static_cast<T *>(const_cast<void *>(a.c.v)) + static_cast<size_t>(row) * a.c.W, u, x);
        }
    }
}

// ----------------------------------------------------------------------------- read back
// Row t of the outputs is the cached row of the chunk's token t, converted to fp32 or binary16.
template <typename T, bool kF16>
__global__ void __launch_bounds__(kThreads) chunk_read_kernel(const ChunkReadArgs a, int tok) {
    __shared__ long long src[kMaxTok];
    const int t0 = blockIdx.x * tok, n = min(tok, a.sq.nt - t0);
    const bool first = blockIdx.y == 0;
    if (blockIdx.x == 0 && first && a.sq.off) {
        for (int s = threadIdx.x; s <= a.sq.n_seq; s += kThreads) {
            const int o = __ldg(a.sq.off + s);
            if (o < 0 || o > a.sq.nt || (s > 0 && o < __ldg(a.sq.off + s - 1))) flag_error(a.err, MINF_ERRBIT_CHUNK);
        }
    }
    if (threadIdx.x < n) {
        const int t = t0 + threadIdx.x, s = chunk_seq_of(a.sq.off, a.sq.n_seq, t);
        long long row = -2;  // padding: the output row is left as it was
        if (s >= 0) {
            const SeqRows r = seq_rows(a.c, s);
            const long long p = static_cast<long long>(__ldg(a.sq.n_past + s)) + (t - (a.sq.off ? __ldg(a.sq.off + s) : s));
            row = -1;  // no such row: zeros
            if (p < 0 || p >= r.cap) {
                if (first) flag_error(a.err, MINF_ERRBIT_STORE_POS);
            } else {
                row = seq_row(a.c, r, static_cast<int>(p));
                if (row < 0 && first) flag_error(a.err, MINF_ERRBIT_BLOCK);
            }
        }
        src[threadIdx.x] = row;
    }
    __syncthreads();
    const int w4 = a.c.W >> 2, total = n * 2 * w4;
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < total; i += gridDim.y * kThreads) {
        const int t = i / (2 * w4), u = i - t * 2 * w4;
        const bool v = u >= w4;
        const int c = v ? u - w4 : u;
        const long long row = src[t];
        if (row == -2) continue;
        const float4 x = row < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                 : row_ld4<T>(v ? a.c.v : a.c.k, row, a.c.W, a.c.row_bytes, c);
        const size_t at = static_cast<size_t>(t0 + t) * a.c.W;
        if constexpr (kF16)
            put_row4(static_cast<__half *>(v ? a.v_rows : a.k_rows) + at, c, x);
        else
            put_row4(static_cast<float *>(v ? a.v_rows : a.k_rows) + at, c, x);
    }
}

}  // namespace

int launch_chunk_store(const ChunkStoreArgs &a, float theta, float freq_scale, const unsigned char *pair_axis,
                       cudaStream_t s) {
    if (a.sq.nt == 0) return MINF_OK;
    AxisTable tq, tk = {};
    axis_table(&tq, a.hd, theta, freq_scale, pair_axis);
    if (a.hd_kv != a.hd) axis_table(&tk, a.hd_kv, theta, freq_scale, pair_axis);  // (else k turns as q does)
    int tok;
    dim3 grid;
    row_grid(a.sq.nt, static_cast<long long>(a.nh) * (a.hd / 8) + a.nk * (a.hd_kv / 8) + a.c.W / 4, tok, grid);
    if (a.c.kv == kKvQ8)
        chunk_store_kernel<Q8><<<grid, kThreads, 0, s>>>(a, tq, tk, tok);
    else if (a.c.kv == kKvF16)
        chunk_store_kernel<__half><<<grid, kThreads, 0, s>>>(a, tq, tk, tok);
    else
        chunk_store_kernel<float><<<grid, kThreads, 0, s>>>(a, tq, tk, tok);
    return cudaPeekAtLastError() == cudaSuccess ? MINF_OK : MINF_ERR_CUDA;
}

int launch_chunk_read(const ChunkReadArgs &a, cudaStream_t s) {
    if (a.sq.nt == 0) return MINF_OK;
    int tok;
    dim3 grid;
    row_grid(a.sq.nt, a.c.W / 2, tok, grid);
    if (a.c.kv == kKvQ8) {
        if (a.f16)
            chunk_read_kernel<Q8, true><<<grid, kThreads, 0, s>>>(a, tok);
        else
            chunk_read_kernel<Q8, false><<<grid, kThreads, 0, s>>>(a, tok);
    } else if (a.c.kv == kKvF16) {
        if (a.f16)
            chunk_read_kernel<__half, true><<<grid, kThreads, 0, s>>>(a, tok);
        else
            chunk_read_kernel<__half, false><<<grid, kThreads, 0, s>>>(a, tok);
    } else {
        if (a.f16)
            chunk_read_kernel<float, true><<<grid, kThreads, 0, s>>>(a, tok);
        else
            chunk_read_kernel<float, false><<<grid, kThreads, 0, s>>>(a, tok);
    }
    return cudaPeekAtLastError() == cudaSuccess ? MINF_OK : MINF_ERR_CUDA;
}

}  // namespace minf
