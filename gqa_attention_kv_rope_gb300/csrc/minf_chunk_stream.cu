// minf_chunk_stream.cu -- chunk attention for few query rows a sequence (single tokens, drafted
// tokens): a stream of the cached rows at memory speed.
//
// An item is up to 8*NT query rows (tokens x the g heads of one kv head).  One CTA an SM walks its
// stretch of units (minf_chunk_plan.cuh), 64 keys a unit: producer warps keep a ring of K and V
// tiles full with TMA copies of the rows as they are stored; groups of four warps compute, a group a
// tile and a warp 16 of its keys, each with its own running maximum, sum and output; they are joined once
// an item.
//
// The work per byte is small (8*NT rows), so what matters is that the products cost little and need
// no barrier between warps: warp-level m16n8k16 products with the keys as the 16 rows and the
// queries as the 8 columns (mma.sync; a tcgen05 tile would compute 128 rows for the few there are).
//   S^T = K Q^T    16 keys x 8 queries
//   O^T += V^T P^T  16 dims x 8 queries, with P^T the transposed S^T (movmatrix)
// Precision: binary16 K and V are exact operands, Q and P are split into binary16 halves hi + lo
// (two products).  Q8_0 quants are exact binary16 integers: block scales are applied to the 32-dim
// partial scores, and to P before it weighs a block of V (P_b = p * scale_b; each key's exponent
// goes into the softmax as in minf_chunk_tiles.cu, so that P_b stays in binary16's range).  fp32 rows
// are split into three bfloat16 terms (24 bits, fp32's range), six products.
//
// The order of a contraction is free as long as both operands agree, so Q8_0 and fp32 rows are read
// from shared memory in the words a lane can take at once, and Q is laid out to match.
#include <cuda_bf16.h>

#include <cmath>

#include "minf_chunk_plan.cuh"
#include "minf_chunk_row.cuh"
#include "minf_chunk_tiles.h"
#include "minf_sm103.cuh"

namespace minf {

namespace {

constexpr int KT = 64;              // keys of a tile
// P is at most 2^(shift + slack) = 2^15; outputs are rescaled when a row's scores have grown by 2^slack.  The
// halves keep P to 2^-25: n keys that all lose as much are off by n 2^-25 of a sum of at least 2^shift.
constexpr float kShift = 12.0f, kSlack = 3.0f;

// A tile's products into the sums, in rounded fp32: the tensor cores' own accumulation cuts the low bits off,
// always towards zero (2e-5 after the 65536 keys of one stretch, now below 2e-6).
__device__ __forceinline__ void sum4(float *acc, const float *d) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += d[e];
}

template <int HD, typename T, int NT>
struct Cfg {
    static constexpr bool F32 = std::is_same<T, float>::value, Q = std::is_same<T, Q8>::value;
    static constexpr int R = 8 * NT;
    static constexpr int EB = F32 ? 4 : (Q ? 1 : 2);
    static constexpr int SLABS = HD * EB > 128 ? HD * EB / 128 : 1;  // 128-byte-wide pieces of a row
    static constexpr int kRow = HD * EB / SLABS;                     // bytes of a row in a slab
    static constexpr bool SW = kRow == 128;                          // 128-byte swizzle
    static constexpr int kTile = KT * HD * EB;                       // K or V of a stage
    static constexpr int kScale = HD / 32 * 2;                       // Q8_0: bytes of a row's scales
    static constexpr int kScales = Q ? KT * kScale : 0;
    static constexpr int kStage = (2 * (kTile + kScales) + 1023) / 1024 * 1024;
    // Groups of four computing warps, a group a tile.  The last warp group are the producers; registers move
    // from it to the computing warps (256 * 208 + 128 * 88 = 384 * 168, the launch's).
    static constexpr int G = 2;
    static constexpr int kWarps = 4 * G, kComputeThreads = 32 * kWarps, kThreads = kComputeThreads + 128;
    static constexpr int kComputeRegs = 208, kOtherRegs = 88;
    static constexpr int TERMS = F32 ? 3 : 2;                        // of Q
    static constexpr int kQRow = HD * 2 + 16;                        // bytes of a Q row (spread over the banks)
    static constexpr int kQ = TERMS * R * kQRow;
    static constexpr int kRegs = NT * (HD / 16) * 4;                 // fp32 outputs a lane
    static constexpr int kJoin = kWarps * (HD / 16) * 4 * 32 * 4;    // every warp's outputs of 8 rows
    static constexpr int kRoom = 227 * 1024 - 1024 - kQ - kJoin - 6 * 1024;
    // a multiple of the groups, so that a stage is always the same group's: its warps then wait on every
    // phase of its barrier
    static constexpr int NS = kRoom / kStage > 8 ? 8 : kRoom / kStage / G * G;
    // producer warps: a stage is always the same producer's too, for the same reason
    static constexpr int kProducers = NS % 4 == 0 ? 4 : 2;
    static constexpr int kOffQ = NS * kStage, kOffJoin = kOffQ + kQ, kOffMeta = kOffJoin + kJoin;
    static_assert(NS >= 2 && NS % G == 0 && NS % kProducers == 0 && kStage % 1024 == 0 && kQ % 16 == 0, "ring");
};

struct Meta {
    unsigned long long full[8], empty[8];
    float q_fac[32];
    int4 lim[32];                       // a row's window: hi, lo, sink
    float m[8][32], l[8][32];
    int odd[32];
    int abort_flag, last;
};

// ----------------------------------------------------------------------------- warp-level wrappers
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// The power of two that brings `amax` to [2^14, 2^15), as an exponent (0 for zero).
__device__ __forceinline__ int row_shift(float amax) {
    const int ex = static_cast<int>((__float_as_uint(amax) >> 23) & 0xff) - 127;
    const int sh = amax > 0.0f ? 14 - ex : 0;
    return sh > 126 ? 126 : (sh < -126 ? -126 : sh);
}
// binary16 halves: hi = round(x), lo = round(x - hi).
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
// Three bfloat16 terms of two values (low half: x).
__device__ __forceinline__ uint32_t bf2(float x, float y) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}
__device__ __forceinline__ void split3(float x, float y, uint32_t &a, uint32_t &b, uint32_t &c) {
    a = bf2(x, y);
    x -= __uint_as_float(a << 16), y -= __uint_as_float(a & 0xffff0000u);
    b = bf2(x, y);
    x -= __uint_as_float(b << 16), y -= __uint_as_float(b & 0xffff0000u);
    c = bf2(x, y);
}
// Bytes 0, 1 (or 2, 3) of u = q ^ 0x80 per byte as two binary16 integers q: 0x6400 | u is 1024 + u.
__device__ __forceinline__ uint32_t q_pair(uint32_t u, uint32_t sel) {
    const uint32_t x = __byte_perm(u, 0x64646464u, sel);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&x), __floats2half2_rn(1152.0f, 1152.0f));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Byte offset of 16-byte chunk c of row r in a slab.
template <typename C>
__device__ __forceinline__ uint32_t at16(int r, int c) {
    return static_cast<uint32_t>(r) * C::kRow + (static_cast<uint32_t>(C::SW ? c ^ (r & 7) : c) << 4);
}

// ----------------------------------------------------------------------------- the producer
struct Maps {
    CUtensorMap k, v;
};

// Producer warp `pw` takes every kProducers-th tile (one warp's instructions for a tile take longer than
// the tile's bytes).  A lane looks up two of the tile's rows (their block ids one of its
// tiles ahead, so that no load is waited for), and issues one of its TMA copies; Q8_0's scales come
// beside them, a few bytes a row, by cp.async (as TMA boxes they would cost as many requests as the
// quants).
template <int HD, typename T, int NT>
__device__ __forceinline__ void produce(unsigned char *ring, Meta &mt, const Maps &maps, const AttnParams &p, int pw,
                                        int ctas) {
    using C = Cfg<HD, T, NT>;
    const int lane = threadIdx.x & 31;
    const ChunkKv &c = p.a.c;
    const int pieces = KT / p.box_rows, copies = 2 * C::SLABS * pieces;  // at most 2 * 4 slabs * 4 pieces
    const int is_v = lane / (C::SLABS * pieces), rest = lane % (C::SLABS * pieces), piece = rest / C::SLABS, part = rest % C::SLABS;
    volatile int *abort_flag = &mt.abort_flag;
    Walk w;  // of the tile ahead
    bool more = walk_begin<KT>(w, p, ctas);
    int u = more ? w.u0 : 0;
    // `by` tiles on in the stretch
    auto step = [&](int by) {
        while (more && by > 0) {
            const int left = w.u1 - u;
            if (by < left) {
                u += by;
                return;
            }
            by -= left;
            more = walk_next<KT>(w, p);
            u = w.u0;
        }
    };
    const int box_mask = -p.box_rows;  // (a power of two)
    int id[2], jj = 0, head = 0;       // the tile ahead: block ids (or the first row), -2: hidden
    auto look_up = [&]() {
        const int j0 = unit_tile(w.keys, u) * KT;
        jj = j0 + lane;
        head = w.head;
        // a row is copied where a visible one lies in its box; rows past the capacity have no block
        const bool inside = j0 >= w.keys.lo && j0 + KT <= w.keys.hi;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = jj + 32 * i;
            id[i] = -2;
            if (inside || (item_sees_some(w.keys, j & box_mask, p.box_rows) && (j < w.rows.cap || !c.table)))
                id[i] = c.table ? __ldg(reinterpret_cast<const int32_t *>(w.rows.at) + (j >> c.block_shift)) : static_cast<int>(w.rows.at);
        }
        step(C::kProducers);
    };
    step(pw);
    if (!more) return;
    look_up();
    for (int n = pw, on = 1; on; n += C::kProducers) {
        const int st = n % C::NS, hd = head;
        int row[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = jj + 32 * i;
            row[i] = static_cast<int>(c.rows);  // past the map's end: zeros
            if (id[i] == -2) continue;
            if (!c.table)
                row[i] = static_cast<int>(min(static_cast<long long>(id[i]) + j, c.rows));
            else if (id[i] >= 0 && id[i] < c.pool_blocks)
                row[i] = (id[i] << c.block_shift) + (j & ((1 << c.block_shift) - 1));
            else
                flag_error(p.a.err, MINF_ERRBIT_BLOCK);
        }
        on = more;
        if (more) look_up();
        const int key = piece * p.box_rows;
        const int r0 = __shfl_sync(0xffffffffu, row[0], key & 31), r1 = __shfl_sync(0xffffffffu, row[1], key & 31);
        if (n >= C::NS && !__all_sync(0xffffffffu, chunk_wait(&mt.empty[st], ((n / C::NS) - 1) & 1, abort_flag, p.a.err))) return;
        if (lane == 0) mbar_expect_tx(&mt.full[st], 2 * C::kTile);
        __syncwarp();
        unsigned char *stage = ring + st * C::kStage;
        if (lane < copies) {
            unsigned char *dst = stage + is_v * C::kTile + part * (KT * C::kRow) + key * C::kRow;
            tma_load_2d_stream(dst, is_v ? &maps.v : &maps.k, hd * HD + part * (C::kRow / C::EB), key < 32 ? r0 : r1, &mt.full[st]);
        }
        if constexpr (C::Q) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = row[i & 1];
                const bool there = r < c.rows;
                const unsigned char *src = static_cast<const unsigned char *>(i < 2 ? c.k : c.v) +
                                           (there ? r * c.row_bytes + c.W + hd * C::kScale : 0);
                const uint32_t dst = su32(stage + 2 * C::kTile + (i < 2 ? 0 : C::kScales) + (lane + 32 * (i & 1)) * C::kScale);
                // (a size of zero writes zeros)
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(C::kScale),
                             "r"(there ? C::kScale : 0)
                             : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(su32(&mt.full[st])) : "memory");
        }
        __syncwarp();
    }
}

// ----------------------------------------------------------------------------- the computing warps
template <int HD, typename T, int NT>
__device__ __forceinline__ void compute(unsigned char *smem, Meta &mt, const AttnParams &p, int ctas) {
    using C = Cfg<HD, T, NT>;
    constexpr int R = C::R, MT = HD / 16, NB = HD / 32, kWarps = C::kWarps;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n8 = lane >> 2, c4 = lane & 3;
    const int grp = warp >> 2, key0 = (warp & 3) * 16;
    const int g = p.a.nh / p.a.nk;
    unsigned char *qs = smem + C::kOffQ;
    float *join = reinterpret_cast<float *>(smem + C::kOffJoin);
    volatile int *abort_flag = &mt.abort_flag;
    constexpr size_t kPart = static_cast<size_t>(R) * (HD + 2);
    int n = 0;
    Walk w;
    for (bool more = walk_begin<KT>(w, p, ctas); more; more = walk_next<KT>(w, p)) {
        const int rows = w.cnt * g, tiles = w.u1 - w.u0;
        // Q: a warp a row
        for (int r = warp; r < R; r += kWarps) {
            constexpr int V = HD / 32;  // values a lane: 4 or 2
            float x[V];
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = 0.0f;
            if (r < rows) {
                const long long t = walk_row(w, p) + r / g;
                const float *src = p.a.q + (t * p.a.nh + w.head * g + r % g) * p.a.hd + lane * V;
                if constexpr (V == 4) {
                    const float4 y = __ldg(reinterpret_cast<const float4 *>(src));
                    x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
                } else {
                    const float2 y = __ldg(reinterpret_cast<const float2 *>(src));
                    x[0] = y.x, x[1] = y.y;
                }
            }
            unsigned char *dst = qs + r * C::kQRow + lane * V * 2;
            if constexpr (C::F32) {
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    uint32_t a, b, c;
                    split3(x[e], x[e + 1], a, b, c);
                    *reinterpret_cast<uint32_t *>(dst + e * 2) = a;
                    *reinterpret_cast<uint32_t *>(dst + R * C::kQRow + e * 2) = b;
                    *reinterpret_cast<uint32_t *>(dst + 2 * R * C::kQRow + e * 2) = c;
                }
                if (lane == 0) mt.q_fac[r] = 1.0f;
            } else {
                float am = 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) am = fmaxf(am, fabsf(x[e]));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
                const int sh = row_shift(am);
                const float f = pow2i(sh);
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    uint32_t hi, lo;
                    split2(x[e] * f, x[e + 1] * f, hi, lo);
                    *reinterpret_cast<uint32_t *>(dst + e * 2) = hi;
                    *reinterpret_cast<uint32_t *>(dst + R * C::kQRow + e * 2) = lo;
                }
                if (lane == 0) mt.q_fac[r] = pow2i(-sh);
            }
            if (lane == 0) {
                const long long pos = walk_pos(w, p) + r / g;
                int4 lim = make_int4(0, 0, 0, 0);
                if (r < rows && pos >= 0) {
                    lim.x = pos + 1 < w.rows.cap ? static_cast<int>(pos + 1) : w.rows.cap;
                    if (p.a.window) {
                        const long long lo = pos - p.a.window + 1;
                        lim.y = lo <= 0 ? 0 : (lo < lim.x ? static_cast<int>(lo) : lim.x);
                        lim.z = min(p.a.n_sink, lim.x);
                    }
                }
                mt.lim[r] = lim;
                mt.odd[r] = 0;
            }
        }
        named_sync(1, C::kComputeThreads);
        float c[NT][2], m[NT][2], l[NT][2];
        float acc[C::kRegs];  // [NT][MT][4]
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                c[t][e] = p.scale_log2 * mt.q_fac[t * 8 + 2 * c4 + e];
                m[t][e] = -INFINITY;
                l[t][e] = 0.0f;
            }
#pragma unroll
        for (int r = 0; r < C::kRegs; ++r) acc[r] = 0.0f;
        // keys seen by every row: no mask
        const long long first = walk_pos(w, p), last = first + w.cnt - 1;
        const long long all_hi = first + 1 < w.rows.cap ? first + 1 : w.rows.cap;
        const long long all_lo = p.a.window && last - p.a.window + 1 > 0 ? last - p.a.window + 1 : 0;
        for (int i = 0; i < tiles; ++i) {
            const int q = n + i;
            if (q % C::G != grp) continue;
            const int st = q % C::NS, j0 = unit_tile(w.keys, w.u0 + i) * KT + key0;
            unsigned char *kst = smem + st * C::kStage, *vst = kst + C::kTile;
            chunk_wait(&mt.full[st], (q / C::NS) & 1, abort_flag, p.a.err);
            if (item_sees_some(w.keys, j0, 16)) {
                const bool edge = j0 < w.keys.lo || j0 + 16 > w.keys.hi;
                if (!C::Q && edge) {
                    // rows that no token sees must hold zeros in V (their weight is zero, but 0 * inf is not)
#pragma unroll 1
                    for (int k = 0; k < 16; ++k) {
                        if (item_sees(w.keys, j0 + k)) continue;
#pragma unroll
                        for (int s = 0; s < C::SLABS; ++s)
                            if (lane < C::kRow / 16)
                                *reinterpret_cast<uint4 *>(vst + s * (KT * C::kRow) + (key0 + k) * C::kRow + lane * 16) = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                    fence_async_smem();
                }
                // ---- scores
                float s[NT][4];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[t][e] = 0.0f;
                float ve[2] = {0.0f, 0.0f}, vw[2] = {1.0f, 1.0f}, vr[2][NB];  // Q8_0: V's exponents, 2^-e, relative scales
                if constexpr (C::Q) {
                    const unsigned char *ksc = kst + 2 * C::kTile, *vsc = ksc + C::kScales;
                    float kf[2][NB];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = key0 + n8 + 8 * h;
                        float mx = 0.0f;
#pragma unroll
                        for (int b = 0; b < NB; b += 2) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(ksc + key * C::kScale + b * 2));
                            kf[h][b] = f.x, kf[h][b + 1] = f.y;
                            float2 v = __half22float2(*reinterpret_cast<const __half2 *>(vsc + key * C::kScale + b * 2));
                            if (edge && !item_sees(w.keys, j0 + n8 + 8 * h)) v = make_float2(0.0f, 0.0f);
                            vr[h][b] = v.x, vr[h][b + 1] = v.y;
                            mx = fmaxf(mx, fmaxf(fabsf(v.x), fabsf(v.y)));
                        }
                        int ex = static_cast<int>((__float_as_uint(mx) >> 23) & 0xff) - 126;  // scales are at most 2^ex
                        ex = ex < -24 ? -24 : (ex > 16 ? 16 : ex);  // (binary16's range; zero: -24)
                        ve[h] = static_cast<float>(ex);
                        vw[h] = pow2i(-ex);
#pragma unroll
                        for (int b = 0; b < NB; ++b) vr[h][b] *= vw[h];
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint32_t a[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint2 x = *reinterpret_cast<const uint2 *>(kst + at16<C>(key0 + n8 + 8 * h, 2 * b + (c4 >> 1)) + (c4 & 1) * 8);
                            const uint32_t u0 = x.x ^ 0x80808080u, u1 = x.y ^ 0x80808080u;
                            a[0][h] = q_pair(u0, 0x4140), a[0][2 + h] = q_pair(u0, 0x4342);
                            a[1][h] = q_pair(u1, 0x4140), a[1][2 + h] = q_pair(u1, 0x4342);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const unsigned char *qr = qs + (t * 8 + n8) * C::kQRow + (b * 32 + c4 * 8) * 2;
                            const uint4 qh = *reinterpret_cast<const uint4 *>(qr), ql = *reinterpret_cast<const uint4 *>(qr + R * C::kQRow);
                            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_f16(d, a[0], qh.x, qh.y);
                            mma_f16(d, a[1], qh.z, qh.w);
                            mma_f16(d, a[0], ql.x, ql.y);
                            mma_f16(d, a[1], ql.z, ql.w);
                            s[t][0] = fmaf(d[0], kf[0][b], s[t][0]);
                            s[t][1] = fmaf(d[1], kf[0][b], s[t][1]);
                            s[t][2] = fmaf(d[2], kf[1][b], s[t][2]);
                            s[t][3] = fmaf(d[3], kf[1][b], s[t][3]);
                        }
                    }
                } else if constexpr (C::F32) {
#pragma unroll
                    for (int kk = 0; kk < MT; ++kk) {
                        uint32_t a1[4], a2[4], a3[4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float4 x = *reinterpret_cast<const float4 *>(kst + (kk >> 1) * (KT * 128) + at16<C>(key0 + n8 + 8 * h, (kk & 1) * 4 + c4));
                            split3(x.x, x.y, a1[h], a2[h], a3[h]);
                            split3(x.z, x.w, a1[2 + h], a2[2 + h], a3[2 + h]);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const unsigned char *qr = qs + (t * 8 + n8) * C::kQRow + (kk * 16 + c4 * 4) * 2;
                            const uint2 q1 = *reinterpret_cast<const uint2 *>(qr), q2 = *reinterpret_cast<const uint2 *>(qr + R * C::kQRow);
                            const uint2 q3 = *reinterpret_cast<const uint2 *>(qr + 2 * R * C::kQRow);
                            mma_bf16(s[t], a1, q1.x, q1.y);
                            mma_bf16(s[t], a1, q2.x, q2.y);
                            mma_bf16(s[t], a2, q1.x, q1.y);
                            mma_bf16(s[t], a1, q3.x, q3.y);
                            mma_bf16(s[t], a2, q2.x, q2.y);
                            mma_bf16(s[t], a3, q1.x, q1.y);
                        }
                    }
                } else {
#pragma unroll
                    for (int k2 = 0; k2 < MT; k2 += 2) {
                        uint32_t a[2][4];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            ldsm4(su32(kst + ((k2 + k) >> 2) * (KT * 128) + at16<C>(key0 + (lane & 15), ((k2 + k) & 3) * 2 + (lane >> 4))), a[k]);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int term = 0; term < 2; ++term) {
                                uint32_t b[4];
                                ldsm4(su32(qs + (term * R + t * 8 + (lane & 7)) * C::kQRow + k2 * 32 + (lane >> 3) * 16), b);
                                mma_f16(s[t], a[0], b[0], b[1]);
                                mma_f16(s[t], a[1], b[2], b[3]);
                            }
                    }
                }
                // ---- softmax of 16 keys (lanes of one c4 share two rows; their keys are n8 and n8 + 8)
                const bool mask = !(j0 >= all_lo && j0 + 16 <= all_hi) && !(j0 + 16 <= p.a.n_sink && j0 + 16 <= all_hi);
                uint32_t b_hi[NT][C::Q ? NB : 1][2], b_lo[NT][C::Q ? NB : 1][2], b_3[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = fmaf(s[t][e], c[t][e & 1], C::Q ? ve[e >> 1] : 0.0f);
                    if (mask) {
                        const int4 l0 = mt.lim[t * 8 + 2 * c4], l1 = mt.lim[t * 8 + 2 * c4 + 1];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = j0 + n8 + 8 * (e >> 1);
                            const int4 lim = (e & 1) ? l1 : l0;
                            const bool see = (j < lim.x) & ((j >= lim.y) | (j < lim.z));
                            x[e] = see ? x[e] : -INFINITY;
                        }
                    }
                    float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
                        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
                    }
                    float corr[2] = {1.0f, 1.0f};
                    bool grow = false;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (mx[e] > m[t][e] + kSlack || (m[t][e] == -INFINITY && mx[e] > m[t][e])) {
                            corr[e] = ex2_approx(m[t][e] - mx[e]);
                            m[t][e] = mx[e];
                            l[t][e] *= corr[e];
                            grow = true;
                        }
                    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                        for (int r = 0; r < MT * 4; ++r) acc[t * MT * 4 + r] *= corr[r & 1];
                    }
                    const float b0 = m[t][0] == -INFINITY ? 0.0f : m[t][0] - kShift, b1 = m[t][1] == -INFINITY ? 0.0f : m[t][1] - kShift;
                    float pr[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) pr[e] = ex2_approx(x[e] - ((e & 1) ? b1 : b0));
                    if constexpr (C::Q) {
                        l[t][0] = fmaf(pr[0], vw[0], fmaf(pr[2], vw[1], l[t][0]));
                        l[t][1] = fmaf(pr[1], vw[0], fmaf(pr[3], vw[1], l[t][1]));
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t hi, lo;
                                split2(pr[2 * h] * vr[h][b], pr[2 * h + 1] * vr[h][b], hi, lo);
                                b_hi[t][b][h] = transpose8(hi);
                                b_lo[t][b][h] = transpose8(lo);
                            }
                    } else {
                        l[t][0] += pr[0] + pr[2];
                        l[t][1] += pr[1] + pr[3];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t hi, lo;
                            if constexpr (C::F32) {
                                uint32_t x3;
                                split3(pr[2 * h], pr[2 * h + 1], hi, lo, x3);
                                b_3[t][h] = transpose8(x3);
                            } else {
                                split2(pr[2 * h], pr[2 * h + 1], hi, lo);
                            }
                            b_hi[t][0][h] = transpose8(hi);
                            b_lo[t][0][h] = transpose8(lo);
                        }
                    }
                }
                // ---- outputs
                if constexpr (C::Q) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint32_t wd[4];  // dims 32b + 4 n8 .. + 3 of keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int key = key0 + 2 * c4 + (k & 1) + 8 * (k >> 1);
                            wd[k] = *reinterpret_cast<const uint32_t *>(vst + at16<C>(key, 2 * b + (n8 >> 2)) + (n8 & 3) * 4) ^ 0x80808080u;
                        }
                        const uint32_t t0 = __byte_perm(wd[0], wd[1], 0x5140), t1 = __byte_perm(wd[0], wd[1], 0x7362);
                        const uint32_t t2 = __byte_perm(wd[2], wd[3], 0x5140), t3 = __byte_perm(wd[2], wd[3], 0x7362);
                        const uint32_t a0[4] = {q_pair(t0, 0x4140), q_pair(t0, 0x4342), q_pair(t2, 0x4140), q_pair(t2, 0x4342)};
                        const uint32_t a1[4] = {q_pair(t1, 0x4140), q_pair(t1, 0x4342), q_pair(t3, 0x4140), q_pair(t3, 0x4342)};
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float d0[4] = {}, d1[4] = {};
                            mma_f16(d0, a0, b_lo[t][b][0], b_lo[t][b][1]);
                            mma_f16(d1, a1, b_lo[t][b][0], b_lo[t][b][1]);
                            mma_f16(d0, a0, b_hi[t][b][0], b_hi[t][b][1]);
                            mma_f16(d1, a1, b_hi[t][b][0], b_hi[t][b][1]);
                            sum4(&acc[(t * MT + 2 * b) * 4], d0);
                            sum4(&acc[(t * MT + 2 * b + 1) * 4], d1);
                        }
                    }
                } else if constexpr (C::F32) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float4 x[4];  // dims 32b + 4 n8 .. + 3 of the lane's four keys
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x[k] = *reinterpret_cast<const float4 *>(vst + b * (KT * 128) + at16<C>(key0 + 2 * c4 + (k & 1) + 8 * (k >> 1), n8));
#pragma unroll
                        for (int i2 = 0; i2 < 2; ++i2) {
                            uint32_t a1[4], a2[4], a3[4];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float4 u = x[2 * h], v = x[2 * h + 1];
                                split3(i2 ? u.z : u.x, i2 ? v.z : v.x, a1[2 * h], a2[2 * h], a3[2 * h]);
                                split3(i2 ? u.w : u.y, i2 ? v.w : v.y, a1[2 * h + 1], a2[2 * h + 1], a3[2 * h + 1]);
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                float d[4] = {};
                                mma_bf16(d, a3, b_hi[t][0][0], b_hi[t][0][1]);
                                mma_bf16(d, a2, b_lo[t][0][0], b_lo[t][0][1]);
                                mma_bf16(d, a1, b_3[t][0], b_3[t][1]);
                                mma_bf16(d, a2, b_hi[t][0][0], b_hi[t][0][1]);
                                mma_bf16(d, a1, b_lo[t][0][0], b_lo[t][0][1]);
                                mma_bf16(d, a1, b_hi[t][0][0], b_hi[t][0][1]);
                                sum4(&acc[(t * MT + 2 * b + i2) * 4], d);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < MT; ++k) {
                        uint32_t a[4];
                        ldsm4t(su32(vst + (k >> 2) * (KT * 128) + at16<C>(key0 + (lane >> 4) * 8 + (lane & 7), (k & 3) * 2 + ((lane >> 3) & 1))), a);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float d[4] = {};
                            mma_f16(d, a, b_lo[t][0][0], b_lo[t][0][1]);
                            mma_f16(d, a, b_hi[t][0][0], b_hi[t][0][1]);
                            sum4(&acc[(t * MT + k) * 4], d);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&mt.empty[st]);
        }
        n += tiles;
        // ---- join the warps: row by row their maxima and sums, then, 16 dims a warp, their outputs in order
        float M[NT][2], L[NT][2], res[NT][4];
        auto join_all = [&]() {
            if (n8 == 0) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mt.m[warp][t * 8 + 2 * c4 + e] = m[t][e];
                        mt.l[warp][t * 8 + 2 * c4 + e] = l[t][e];
                    }
            }
            named_sync(1, C::kComputeThreads);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = t * 8 + 2 * c4 + e;
                    float mm = -INFINITY, ll = 0.0f;
#pragma unroll
                    for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, mt.m[k][r]);
#pragma unroll
                    for (int k = 0; k < kWarps; ++k) {
                        const float mk = mt.m[k][r], lk = mt.l[k][r];
                        if (mk != -INFINITY || lk != 0.0f) ll = fmaf(lk, ex2_approx(mk - mm), ll);
                    }
                    M[t][e] = mm;
                    L[t][e] = ll;
                    // a warp that saw nothing adds nothing, whatever it holds
                    f[e] = m[t][e] == -INFINITY && l[t][e] == 0.0f ? 0.0f : ex2_approx(m[t][e] - mm);
                }
                if (t > 0) named_sync(1, C::kComputeThreads);
#pragma unroll
                for (int r = 0; r < MT * 4; ++r)
                    join[(warp * MT * 4 + r) * 32 + lane] = f[r & 1] == 0.0f ? 0.0f : acc[t * MT * 4 + r] * f[r & 1];
                named_sync(1, C::kComputeThreads);
                if (warp < MT) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float y = 0.0f;
#pragma unroll
                        for (int k = 0; k < kWarps; ++k) y += join[(k * MT * 4 + warp * 4 + e) * 32 + lane];
                        res[t][e] = y;
                    }
                }
            }
        };
        int b0, b1;
        const bool whole = w.u0 == 0 && w.u1 == w.keys.units;
        if (!whole) walk_parts(w, p, b0, b1);  // (in flight meanwhile)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], o);
        join_all();
        bool finish = whole;
        if (!whole) {
            auto part_of = [&](int b) { return p.parts + (2 * static_cast<size_t>(b) + (b == b0 ? 1 : 0)) * kPart; };
            float *part = p.parts + (2 * static_cast<size_t>(blockIdx.x) + (w.u0 == 0 ? 1 : 0)) * kPart;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (warp < MT) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) part[((t * MT + warp) * 4 + e) * 32 + lane] = res[t][e];
                }
                if (warp == 0 && n8 == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        part[R * HD + t * 8 + 2 * c4 + e] = M[t][e];
                        part[R * HD + R + t * 8 + 2 * c4 + e] = L[t][e];
                    }
                }
            }
            named_sync(1, C::kComputeThreads);
            if (tid == 0) {
                __threadfence();  // (the whole CTA's part: the barrier ordered it before this)
                mt.last = atomicAdd(p.tickets + b0, 1) == b1 - b0;
                __threadfence();
            }
            named_sync(1, C::kComputeThreads);
            finish = mt.last != 0;
            if (finish) {  // join the stretches' parts, dealt out to the warps in order, then the warps
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        m[t][e] = -INFINITY;
                        l[t][e] = 0.0f;
                    }
#pragma unroll
                for (int r = 0; r < C::kRegs; ++r) acc[r] = 0.0f;
#pragma unroll 1
                for (int b = b0 + warp; b <= b1; b += kWarps) {
                    const float *q = part_of(b);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float y[MT * 4], fo[2], fn[2];
#pragma unroll
                        for (int r = 0; r < MT * 4; ++r) y[r] = __ldcg(q + (t * MT * 4 + r) * 32 + lane);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float mb = __ldcg(q + R * HD + t * 8 + 2 * c4 + e), lb = __ldcg(q + R * HD + R + t * 8 + 2 * c4 + e);
                            const bool none = mb == -INFINITY && lb == 0.0f, first = m[t][e] == -INFINITY && l[t][e] == 0.0f;
                            const float mn = fmaxf(m[t][e], mb);
                            fo[e] = first ? 0.0f : ex2_approx(m[t][e] - mn);
                            fn[e] = none ? 0.0f : ex2_approx(mb - mn);
                            l[t][e] = (first ? 0.0f : l[t][e] * fo[e]) + (none ? 0.0f : lb * fn[e]);
                            m[t][e] = mn;
                        }
#pragma unroll
                        for (int r = 0; r < MT * 4; ++r) {
                            float &a = acc[t * MT * 4 + r];
                            a = a * fo[r & 1] + (fn[r & 1] == 0.0f ? 0.0f : y[r] * fn[r & 1]);
                        }
                    }
                }
                join_all();
            }
        }
        bool again = false;
        if (finish) {
            bool odd = false;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = t * 8 + 2 * c4 + e;
                    if (warp >= MT || r >= rows) continue;
                    // (a sum of zero, where it sees nothing or nothing but scores of minus infinity, gives NaN here)
                    const float inv = 1.0f / L[t][e];
                    float *out = p.a.out + (static_cast<long long>(walk_row(w, p) + r / g) * p.a.nh + w.head * g + r % g) * HD;
                    bool bad = false;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float y = res[t][2 * h + e] * inv;
                        const int d = C::Q || C::F32 ? (warp >> 1) * 32 + 4 * n8 + 2 * (warp & 1) + h : warp * 16 + n8 + 8 * h;
                        out[d] = y;
                        bad |= !(fabsf(y) < INFINITY);
                    }
                    if (bad) mt.odd[r] = 1;
                    odd |= bad;
                }
            // rows that are not finite: by the definition, a row a warp
            again = !named_all(1, C::kComputeThreads, !odd);
            if (again) {
                if (tid == 0) rows_again(&mt.abort_flag, true);
                const long long at = static_cast<long long>(walk_row(w, p)) * p.a.nh + w.head * g;
                attn_rows_again<T, HD>(p.a.c, mt.odd, rows, warp, kWarps, p.a.q + at * p.a.hd, p.a.out + at * HD, g, p.a.nh,
                                       p.a.hd, w.rows, walk_pos(w, p), w.head, p.scale_log2, p.a.window, p.a.n_sink);
            }
        }
        named_sync(1, C::kComputeThreads);  // Q, limits and the join buffer are free
        if (again && tid == 0) rows_again(&mt.abort_flag, false);
    }
}

template <int HD, typename T, int NT>
__global__ void __launch_bounds__(Cfg<HD, T, NT>::kThreads, 1)
    chunk_stream_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnParams p) {
    using C = Cfg<HD, T, NT>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Meta &mt = *reinterpret_cast<Meta *>(smem + C::kOffMeta);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&mt.full[i], C::Q ? 33 : 1);  // the copies' bytes, and each lane's scales
            mbar_init(&mt.empty[i], 4);             // the warps of the group that takes the tile
        }
        mt.abort_flag = 0;
        mbar_init_fence();
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    __syncthreads();
    gdc_wait();  // the plan, and everything before it
    const int ctas = p.head->ctas;
    if (warp < C::kWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kComputeRegs));
        compute<HD, T, NT>(smem, mt, p, ctas);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        if (warp < C::kWarps + C::kProducers) produce<HD, T, NT>(smem, mt, maps, p, warp - C::kWarps, ctas);
    }
    if (*static_cast<volatile int *>(&mt.abort_flag) == 1) {
        // a wait ran out: let copies in flight land before shared memory goes away
        const unsigned long long t0 = gtimer();
        while (gtimer() - t0 < kWaitBudgetNs / 4) {
        }
    }
}

template <int HD, typename T, int NT>
int launch(const AttnParams &p, int grid, cudaStream_t s) {
    using C = Cfg<HD, T, NT>;
    const ChunkKv &c = p.a.c;
    Maps maps;
    const CUtensorMapDataType dt = C::F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                          : (C::Q ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
    const uint64_t cols = static_cast<uint64_t>(c.row_bytes / C::EB), rows = static_cast<uint64_t>(c.rows);
    if (!make_tensor_map_2d(&maps.k, c.k, dt, C::EB, cols, rows, C::kRow / C::EB, p.box_rows, C::SW) ||
        !make_tensor_map_2d(&maps.v, c.v, dt, C::EB, cols, rows, C::kRow / C::EB, p.box_rows, C::SW))
        return MINF_ERR_CUDA;
    constexpr int kSmem = C::kOffMeta + static_cast<int>(sizeof(Meta)) + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    auto kernel = chunk_stream_kernel<HD, T, NT>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return MINF_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p) == cudaSuccess ? MINF_OK : MINF_ERR_CUDA;
}

template <int HD, int NT>
int launch_kind(const AttnParams &p, int grid, cudaStream_t s) {
    if (p.a.c.kv == kKvF16) {
        if constexpr (NT <= 2)
            return launch<HD, __half, NT>(p, grid, s);
        else
            return MINF_ERR_UNSUPPORTED;  // (such calls go to the tiles)
    }
    return p.a.c.kv == kKvQ8 ? launch<HD, Q8, NT>(p, grid, s) : launch<HD, float, NT>(p, grid, s);
}

int row_tiles(int rows) { return rows <= 8 ? 1 : (rows <= 16 ? 2 : 4); }

PlanLayout stream_layout(int nt, int n_seq, int g, int hd_kv, int n8) {
    return plan_layout(nt, n_seq, 8 * n8 / g, sm_count(), static_cast<size_t>(8 * n8) * (hd_kv + 2) * sizeof(float));
}

}  // namespace

size_t chunk_stream_workspace(int nt, int n_seq, int nh, int nk, int hd_kv, int rows) {
    return stream_layout(nt, n_seq, nh / nk, hd_kv, row_tiles(rows)).total;
}

void plan_chunk_stream(PlanArgs &plan, AttnParams &p, const ChunkAttnArgs &a, void *workspace, int rows, int most) {
    const int sms = sm_count(), g = a.nh / a.nk, n8 = row_tiles(rows);
    p = {};
    p.a = a;
    p.tt = 8 * n8 / g;
    p.kt = KT;
    p.least = 1;
    p.most = most;
    p.scale_log2 = a.scale * kLog2e;
    p.box_rows = a.c.table && (1 << a.c.block_shift) < KT ? 1 << a.c.block_shift : KT;
    plan_args(plan, p, stream_layout(a.sq.nt, a.sq.n_seq, g, a.hd_kv, n8), workspace, sms < kPlanMost ? sms : kPlanMost, 2, 1);
}

int launch_chunk_stream(const AttnParams &p, int rows, cudaStream_t s) {
    const int sms = sm_count(), n8 = row_tiles(rows);
    if (p.a.hd_kv == 64)
        return n8 == 1 ? launch_kind<64, 1>(p, sms, s) : n8 == 2 ? launch_kind<64, 2>(p, sms, s) : launch_kind<64, 4>(p, sms, s);
    return n8 == 1 ? launch_kind<128, 1>(p, sms, s) : n8 == 2 ? launch_kind<128, 2>(p, sms, s) : launch_kind<128, 4>(p, sms, s);
}

}  // namespace minf
