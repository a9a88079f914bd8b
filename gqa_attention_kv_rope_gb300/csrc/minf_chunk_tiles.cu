// minf_chunk_tiles.cu -- chunk attention on the 5th-generation tensor cores: the kernel for chunks
// of many rows.
//
// An item is 128 query rows: up to 128 / g consecutive tokens of one sequence with the g query
// heads of one kv head (row = token * g + head), so that a K/V tile is read once for the whole
// group.  A CTA walks its stretch of units (minf_chunk_plan.cuh); per tile of 128 keys:
//   S = Q K^T   tcgen05.mma kind::f16, M = N = 128, Q from TMEM, into one of two TMEM buffers
//   P = 2^(s - m)   two threads a row (64 keys each): read S, mask, share the row's maximum,
//                   and write P as binary16 halves hi + lo over the S they came from
//   O += P V    tcgen05.mma kind::f16 with P from TMEM, V as it lies in memory (keys x dims, the
//               transposed operand), into TMEM
// Q and P come from TMEM because an operand pair from shared memory (8 KB a 128x128x16 step) takes
// 97 clocks of its bandwidth, against 64 of tensor work with one of them in TMEM.
// S of the next tile runs while the row threads work on this one; the tile after next goes into the
// buffer that P V has just finished with.  O is rescaled only when a row's maximum has grown by
// more than 2^8 since the last time (P is then at most 2^15, still a binary16 value, and the rescale
// is a rare pass over O instead of one a tile).
//
// Precision: fp32 results from binary16 products.  Every operand that is not exactly binary16 is
// split into hi + lo halves (22 bits), scaled by a power of two that keeps both normal; a product
// is hi*hi + hi*lo + lo*hi.  A binary16 cache is exact as it is, so its products take two MMAs
// (Q and P are split); Q8_0 values (18 bits) and fp32 values take three.  Query rows and K rows are
// scaled row by row (the factor comes back in with the score).  V rows are scaled row by row too:
// V_j = V'_j 2^e_j, and the softmax runs on t_j = s_j + e_j, so P'_j = 2^(t_j - M) weighs V'_j and
// P'_j 2^-e_j is the term of the sum: a large row cannot push the others out of binary16's range for
// the rows that do not see it.  (Rows below 2^-46 keep the scale 2^60: what they lose is below 2^-70.)
//
// Roles of a CTA (one an SM): warps 0-7 rows, warp 8 issues the MMAs, warp 11 copies the next
// item's Q rows in, then the producers: for binary16 warps 9 and 10 issue TMA copies of K and V
// (straight into the swizzled layout the tensor cores read; a block or a stretch of rows a copy);
// otherwise warps 12-15 load, split and write K, and warps 16-19 V.
//
// Values in rows that no token of the item sees are zeroed in V (P is zero there, but 0 * inf is
// not); rows that only some tokens see can still carry infinities or NaN into the sums of those that
// do not: a row whose result is not finite is computed again by its definition (attn_row), which
// leaves hidden rows out.
#include <cmath>

#include "minf_chunk_plan.cuh"
#include "minf_chunk_row.cuh"
#include "minf_chunk_tiles.h"
#include "minf_sm103.cuh"

namespace minf {

namespace {

constexpr int BM = 128, KT = 128;
constexpr int kRowThreads = 256;  // warps 0-7: two threads a query row
constexpr int kMmaWarp = 8;
constexpr float kShift = 7.0f, kSlack = 8.0f;  // P is at most 2^(shift + slack) = 2^15
// TMEM columns: the S buffers (P over them: hi, then lo, two keys a column), O, Q (hi, then lo, two dims a
// column)
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384, kTmemCols = 512;

template <int HD, typename T>
struct Cfg {
    static constexpr bool HL = !std::is_same<T, __half>::value;  // K and V as hi + lo halves
    static constexpr int SLABS = HD / 64;                        // 128-byte-wide slabs of a tile
    static constexpr int TERMS = HL ? 2 : 1;
    static constexpr int NS = HL ? (HD == 64 ? 2 : 1) : (HD == 64 ? 4 : 2);  // K and V stages
    // Warp groups: rows (0, 1), then MMA and TMA warps (2), then the splitting producers (3, 4).  The
    // rows' threads hold 64 scores and their halves, so registers move to them from the other groups;
    // the shares add up to no more than the launch's: 256 * 208 + 128 * 88 = 384 * 168, and
    // 256 * 144 + 384 * 64 = 640 * 96.
    static constexpr int kThreads = HL ? 640 : 384;
    static constexpr int kRowRegs = HL ? 144 : 208, kOtherRegs = HL ? 64 : 88;
    static constexpr int kQRow = HD * 4 + 16;  // bytes of a staged Q row (spread over the banks)
};

template <int HD, typename T>
struct Smem {
    using C = Cfg<HD, T>;
    unsigned char k[C::NS][C::TERMS][C::SLABS][KT * 128];
    unsigned char v[C::NS][C::TERMS][C::SLABS][KT * 128];
    unsigned char q[BM * C::kQRow];                    // the item's Q rows, fp32
    unsigned long long q_in, q_free, q_full, p_ready[2], o_done[2], s_full[2], k_full[C::NS], k_empty[C::NS], v_full[C::NS], v_empty[C::NS];
    unsigned long long k_stat[4], v_stat[4];           // hi + lo kinds: factors of a tile written
    float mx[2][2][BM], sum[2][BM];
    int odd[BM];                                       // rows whose result is not finite
    alignas(16) float k_fac[C::HL ? 4 : 1][KT];        // K row factors, V row exponents and 2^-e
    alignas(16) float v_exp[C::HL ? 4 : 1][KT], v_inv[C::HL ? 4 : 1][KT];
    uint32_t tmem_base;
    int abort_flag, last;
};

struct TileParams {
    ChunkAttnArgs a;
    const PlanHead *head;
    const PlanStart *starts;
    int *tickets;
    float *parts;
    float scale_log2;
    int tt;        // tokens of a tile
    int box_rows;  // rows of a TMA copy
    int least;     // sequences with shorter chunks are not this kernel's (see launch_chunk_attn)
};

// ----------------------------------------------------------------------------- tensor-core wrappers
// Descriptor of a 128-byte-swizzled operand in shared memory (rows of 128 bytes, atoms of 8 rows).
// K-major (Q, K): the next 8 rows along M/N are 1024 bytes on.  MN-major (V: rows are keys): the next
// 8 keys are 1024 bytes on (stride offset), the next 64 dims one slab on (leading offset).
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t leading_bytes) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((leading_bytes >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
// kind::f16, binary16 operands, fp32 accumulators; B transposed (MN-major) on request.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
                 : "memory");
}
__device__ __forceinline__ void commit(unsigned long long *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(bar)) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this warp's lanes.
__device__ __forceinline__ void tm_ld32(uint32_t t, uint32_t *u) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t t, uint32_t *u) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t *u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Byte offset of the 16-byte chunk c of a row in a 128-byte-swizzled slab.
__device__ __forceinline__ uint32_t sw16(int row, int c) {
    return static_cast<uint32_t>(row) * 128u + ((static_cast<uint32_t>(c) ^ static_cast<uint32_t>(row & 7)) << 4);
}

// The power of two that brings a row's largest magnitude to [2^14, 2^15), as 2^sh; 1 for a row of
// zeros.  Larger sh than `most` are cut to it.
__device__ __forceinline__ int row_shift(float amax, int most) {
    const int ex = static_cast<int>((__float_as_uint(amax) >> 23) & 0xff) - 127;
    const int sh = amax > 0.0f ? 14 - ex : most < 0 ? 0 : (most < 126 ? most : 0);
    return sh > most ? most : (sh < -126 ? -126 : sh);
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ float2 bits2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

// Two values as binary16 halves: hi = round(x), lo = round(x - hi).
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const float2 r = fma2(f, make_float2(-1.0f, -1.0f), make_float2(x, y));
    const __half2 l = __floats2half2_rn(r.x, r.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// ----------------------------------------------------------------------------- the walk over segments
// A segment is a stretch's part of one item.  Every role walks the same segments.
struct Walk {
    long long unit, end;  // of all units
    int seq, head, tile, u;
    int lo, hi;           // packed rows of the sequence
    long long past;
    SeqRows rows;
    // the segment
    ItemKeys keys;
    int t0, cnt;          // tokens of the item: first (in the chunk) and count
    int u0, u1;           // its units in this stretch
};

__device__ __forceinline__ void walk_seq(Walk &w, const TileParams &p) {
    chunk_rows(p.a.sq.off, p.a.sq.nt, w.seq, w.lo, w.hi);
    w.past = __ldg(p.a.sq.n_past + w.seq);
    w.rows = seq_rows(p.a.c, w.seq);
}
__device__ __forceinline__ void walk_item(Walk &w, const TileParams &p) {
    w.t0 = w.tile * p.tt;
    w.cnt = min(p.tt, w.hi - w.lo - w.t0);
    const long long p0 = w.past + w.t0;
    w.keys = item_keys(p0, p0 + w.cnt - 1, w.rows.cap, p.a.window, p.a.n_sink, KT);
    w.u0 = w.u;
    const long long left = w.end - w.unit;
    w.u1 = left < w.keys.units - w.u0 ? w.u0 + static_cast<int>(left) : w.keys.units;
}
// The first segment; false where the stretch is empty.
__device__ __forceinline__ bool walk_begin(Walk &w, const TileParams &p, long long total, int ctas) {
    if (static_cast<int>(blockIdx.x) >= ctas) return false;
    const PlanStart st = p.starts[blockIdx.x];
    w.unit = st.unit;
    w.end = stretch_start(total, ctas, blockIdx.x + 1LL);
    w.seq = st.seq;
    w.head = st.head;
    w.tile = st.tile;
    w.u = st.u;
    if (w.unit >= w.end) return false;
    walk_seq(w, p);
    walk_item(w, p);
    return true;
}
__device__ __forceinline__ bool walk_next(Walk &w, const TileParams &p) {
    w.unit += w.u1 - w.u0;
    if (w.unit >= w.end) return false;
    w.u = 0;  // units are left, so the item was finished
    if ((w.tile + 1) * p.tt < w.hi - w.lo) {
        ++w.tile;
    } else {
        w.tile = 0;
        if (++w.head == p.a.nk) {
            w.head = 0;
            do {
                ++w.seq;
                walk_seq(w, p);
            } while (w.hi - w.lo < p.least);
        }
    }
    walk_item(w, p);
    return true;
}

// Row j of the sequence is seen by some token of the item.
__device__ __forceinline__ bool item_sees(const ItemKeys &k, int j) {
    return (j >= k.lo && j < k.hi) || j < k.sink;
}

// ----------------------------------------------------------------------------- producers
// One warp: TMA copies of the stretch's K (or V) tiles, a lane a copy.  A copy that no visible row
// lies in, or whose block is missing, reads past the map's end: zeros.
template <int HD, typename T, bool kV>
__device__ __forceinline__ void copy_tiles(Smem<HD, T> &sm, const CUtensorMap &map, const TileParams &p, long long total,
                                           int ctas) {
    using C = Cfg<HD, T>;
    const int lane = threadIdx.x & 31;
    constexpr uint32_t kTileBytes = KT * HD * 2;
    const int pieces = KT / p.box_rows, copies = pieces * C::SLABS;
    volatile int *abort_flag = &sm.abort_flag;
    Walk w;
    int n = 0;
    for (bool more = walk_begin(w, p, total, ctas); more; more = walk_next(w, p)) {
        for (int u = w.u0; u < w.u1; ++u, ++n) {
            const int st = n % C::NS, j0 = unit_tile(w.keys, u) * KT;
            unsigned long long *full = kV ? &sm.v_full[st] : &sm.k_full[st], *empty = kV ? &sm.v_empty[st] : &sm.k_empty[st];
            long long row = 0;
            const int piece = lane / C::SLABS, slab = lane % C::SLABS;
            const int j = j0 + piece * p.box_rows;
            if (lane < copies) {  // (at most 8 pieces of 16 rows x 2 slabs)
                // any visible row in [j, j + box)?
                const bool need = (j < w.keys.hi && j + p.box_rows > w.keys.lo && w.keys.lo < w.keys.hi) || j < w.keys.sink;
                row = need ? seq_row(w.rows, j) : p.a.c.rows;
                if (row < 0) {
                    if (!kV) flag_error(p.a.err, MINF_ERRBIT_BLOCK);
                    row = p.a.c.rows;
                }
            }
            if (n >= C::NS && !__all_sync(0xffffffffu, mbar_wait(empty, ((n / C::NS) - 1) & 1, abort_flag, p.a.err))) return;
            if (lane == 0) mbar_expect_tx(full, kTileBytes);
            __syncwarp();
            if (lane < copies)
                tma_load_2d((kV ? sm.v[st][0][slab] : sm.k[st][0][slab]) + piece * p.box_rows * 128, &map,
                            w.head * HD + slab * 64, static_cast<int>(row), full);
            __syncwarp();
        }
    }
}

// One warp: the next item's Q rows into the stage as soon as the row threads have taken the last ones.
template <int HD, typename T>
__device__ __forceinline__ void copy_q(Smem<HD, T> &sm, const TileParams &p, long long total, int ctas) {
    using C = Cfg<HD, T>;
    const int lane = threadIdx.x & 31, g = p.a.nh / p.a.nk;
    volatile int *abort_flag = &sm.abort_flag;
    Walk w;
    int seg = 0;
    for (bool more = walk_begin(w, p, total, ctas); more; more = walk_next(w, p), ++seg) {
        if (seg > 0 && !__all_sync(0xffffffffu, mbar_wait(&sm.q_free, (seg - 1) & 1, abort_flag, p.a.err))) return;
        const int rows = w.cnt * g;
        if (lane == 0) mbar_expect_tx(&sm.q_in, static_cast<uint32_t>(rows) * HD * 4);
        __syncwarp();
        for (int r = lane; r < rows; r += 32) {
            const long long t = w.lo + w.t0 + r / g;
            bulk_load(sm.q + r * C::kQRow, p.a.q + (t * p.a.nh + w.head * g + r % g) * p.a.hd, HD * 4, &sm.q_in);
        }
        __syncwarp();
    }
}

// Eight values of a cached row (8 * i8 ..), for the splitting producers.
template <typename T>
__device__ __forceinline__ void ld8(const unsigned char *row, int W, int i8, float (&x)[8]) {
    float4 a, b;
    if constexpr (std::is_same<T, Q8>::value) {
        const uint2 q = reinterpret_cast<const uint2 *>(row)[i8];
        const float s = __half2float(reinterpret_cast<const __half *>(row + W)[i8 >> 2]);
        a = deq4(q.x, s);
        b = deq4(q.y, s);
    } else {
        a = reinterpret_cast<const float4 *>(row)[2 * i8];
        b = reinterpret_cast<const float4 *>(row)[2 * i8 + 1];
    }
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ float amax8(const float (&x)[8]) {
    return fmaxf(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))),
                 fmaxf(fmaxf(fabsf(x[4]), fabsf(x[5])), fmaxf(fabsf(x[6]), fabsf(x[7]))));
}

// Four warps: the stretch's K (or V) tiles as scaled hi + lo halves; a warp takes 32 of a tile's rows.
// Lane r resolves row r (its block, and an L2 prefetch) one tile ahead; the values are loaded by eight
// lanes a row, eight values of each slab a lane, four rows at a time and several such steps in flight.
// V's row exponents also go out one tile ahead of its values: the row threads need them with S, while
// the V stage may still be in use.
template <int HD, typename T, bool kV>
__device__ __forceinline__ void split_tiles(Smem<HD, T> &sm, const TileParams &p, int warp, long long total, int ctas) {
    using C = Cfg<HD, T>;
    constexpr bool Q = std::is_same<T, Q8>::value;
    constexpr int STEP = Q ? 4 : 2;  // four-row steps in flight
    const int lane = threadIdx.x & 31, l8 = lane & 7, sub = lane >> 3;
    volatile int *abort_flag = &sm.abort_flag;
    const unsigned char *base = static_cast<const unsigned char *>(kV ? p.a.c.v : p.a.c.k);
    Walk w;  // of the tile ahead
    int u = 0, ahead = 0;
    bool more = walk_begin(w, p, total, ctas);
    if (more) u = w.u0;
    // the tile ahead: this lane's row (null: hidden or missing), its head, and V's row exponents
    const unsigned char *nxt = nullptr;
    int nxt_head = 0;
    auto look_ahead = [&]() {
        nxt = nullptr;
        nxt_head = w.head;
        const int j = unit_tile(w.keys, u) * KT + warp * 32 + lane;
        if (item_sees(w.keys, j)) {
            const long long row = seq_row(w.rows, j);
            if (row >= 0)
                nxt = base + row * p.a.c.row_bytes;
            else if (!kV)
                flag_error(p.a.err, MINF_ERRBIT_BLOCK);
        }
        if (nxt) {
            const unsigned char *v = nxt + w.head * (HD * (Q ? 1 : 4));
#pragma unroll
            for (int b = 0; b < HD * (Q ? 1 : 4); b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(v + b));
        }
        if constexpr (kV) {
            const int r = warp * 32 + lane;
            if constexpr (Q) {  // no value is above 127 scales
                float am = 0.0f;
                if (nxt) {
                    const __half *sc = reinterpret_cast<const __half *>(nxt + p.a.c.W) + w.head * (HD / 32);
#pragma unroll
                    for (int b = 0; b < HD / 32; ++b) am = fmaxf(am, 127.0f * fabsf(__half2float(sc[b])));
                }
                const int sh = row_shift(am, 60);
                sm.v_exp[ahead & 3][r] = static_cast<float>(-sh);
                sm.v_inv[ahead & 3][r] = pow2i(sh);
            } else {
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += 8) {
                    float am[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const unsigned char *ptr = reinterpret_cast<const unsigned char *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(nxt), r0 + 4 * i + sub));
                        if (!ptr) continue;
#pragma unroll
                        for (int s = 0; s < C::SLABS; ++s) {
                            float x[8];
                            ld8<T>(ptr, p.a.c.W, w.head * (HD / 8) + s * 8 + l8, x);
                            am[i] = fmaxf(am[i], amax8(x));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) am[i] = fmaxf(am[i], __shfl_xor_sync(0xffffffffu, am[i], o));
                        if (l8 == 0) {
                            const int sh = row_shift(am[i], 60), rr = warp * 32 + r0 + 4 * i + sub;
                            sm.v_exp[ahead & 3][rr] = static_cast<float>(-sh);
                            sm.v_inv[ahead & 3][rr] = pow2i(sh);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.v_stat[ahead & 3]);
        }
        ++ahead;
        if (++u == w.u1) {
            more = walk_next(w, p);
            u = w.u0;
        }
    };
    if (!more) return;
    look_ahead();
    for (int n = 0; n < ahead; ++n) {
        const int st = n % C::NS, head = nxt_head;
        const unsigned char *cur = nxt;
        if (more) look_ahead();
        bool ready = n < C::NS;
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += 4 * STEP) {
            uint2 raw[Q ? STEP : 1][C::SLABS];  // quants, and their blocks' scales
            float sc[Q ? STEP : 1][C::SLABS];
            float x[Q ? 1 : STEP][C::SLABS][8];
#pragma unroll
            for (int i = 0; i < STEP; ++i) {
                const unsigned char *ptr = reinterpret_cast<const unsigned char *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(cur), r0 + 4 * i + sub));
#pragma unroll
                for (int s = 0; s < C::SLABS; ++s) {
                    const int i8 = head * (HD / 8) + s * 8 + l8;
                    if constexpr (Q) {
                        raw[i][s] = make_uint2(0, 0);
                        sc[i][s] = 0.0f;
                        if (ptr) {
                            raw[i][s] = __ldg(reinterpret_cast<const uint2 *>(ptr) + i8);
                            sc[i][s] = __half2float(reinterpret_cast<const __half *>(ptr + p.a.c.W)[i8 >> 2]);
                        }
                    } else if (ptr) {
                        ld8<T>(ptr, p.a.c.W, i8, x[i][s]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[i][s][e] = 0.0f;
                    }
                }
            }
            if (!ready) {  // (the first rows' loads are in flight)
                if (!__all_sync(0xffffffffu, mbar_wait(kV ? &sm.v_empty[st] : &sm.k_empty[st], ((n / C::NS) - 1) & 1,
                                                       abort_flag, p.a.err)))
                    return;
                ready = true;
            }
#pragma unroll
            for (int i = 0; i < STEP; ++i) {
                const int r = warp * 32 + r0 + 4 * i + sub;
                float f;
                if constexpr (kV) {
                    f = sm.v_inv[n & 3][r];
                } else {
                    float am;
                    if constexpr (Q) {
                        am = fabsf(sc[i][0]);
                        if constexpr (C::SLABS == 2) am = fmaxf(am, fabsf(sc[i][1]));
                        am *= 127.0f;  // no value is above 127 scales
                        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 4));  // (four lanes share a block)
                    } else {
                        am = amax8(x[i][0]);
                        if constexpr (C::SLABS == 2) am = fmaxf(am, amax8(x[i][1]));
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
                    }
                    const int sh = row_shift(am, 126);
                    f = pow2i(sh);
                    if (l8 == 0) sm.k_fac[n & 3][r] = pow2i(-sh);
                }
#pragma unroll
                for (int s = 0; s < C::SLABS; ++s) {
                    float y[8];
                    if constexpr (Q) {
                        const float4 a = deq4(raw[i][s].x, sc[i][s] * f), b = deq4(raw[i][s].y, sc[i][s] * f);
                        y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w, y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = x[i][s][e] * f;
                    }
                    uint4 hi, lo;
                    split2(y[0], y[1], hi.x, lo.x);
                    split2(y[2], y[3], hi.y, lo.y);
                    split2(y[4], y[5], hi.z, lo.z);
                    split2(y[6], y[7], hi.w, lo.w);
                    unsigned char *h = kV ? sm.v[st][0][s] : sm.k[st][0][s], *l = kV ? sm.v[st][C::TERMS - 1][s] : sm.k[st][C::TERMS - 1][s];
                    *reinterpret_cast<uint4 *>(h + sw16(r, l8)) = hi;
                    *reinterpret_cast<uint4 *>(l + sw16(r, l8)) = lo;
                }
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (!kV) mbar_arrive(&sm.k_stat[n & 3]);
            mbar_arrive(kV ? &sm.v_full[st] : &sm.k_full[st]);
        }
    }
}

// ----------------------------------------------------------------------------- the MMAs
template <int HD, typename T>
__device__ __forceinline__ void issue_mmas(Smem<HD, T> &sm, const TileParams &p, uint32_t tmem, long long total, int ctas) {
    using C = Cfg<HD, T>;
    volatile int *abort_flag = &sm.abort_flag;
    constexpr uint32_t kIdS = idesc_f16(BM, KT, false), kIdO = idesc_f16(BM, HD, true);
    constexpr uint32_t kSlab = KT * 128;
    const uint64_t dk = desc128(su32(sm.k), 16), dv = desc128(su32(sm.v), kSlab);
    constexpr uint64_t kStage = static_cast<uint64_t>(C::TERMS) * C::SLABS * kSlab >> 4;  // in descriptor units
    constexpr uint64_t kTerm = static_cast<uint64_t>(C::SLABS) * kSlab >> 4;
    const uint32_t qh = tmem + kColQ, ql = qh + HD / 2;
    int n = 0, seg = 0;
    Walk w;
    for (bool more = walk_begin(w, p, total, ctas); more; more = walk_next(w, p), ++seg) {
        const int tiles = w.u1 - w.u0;
        if (!mbar_wait(&sm.q_full, seg & 1, abort_flag, p.a.err)) return;
        auto scores = [&](int i) -> bool {
            const int st = (n + i) % C::NS;
            if (!mbar_wait(&sm.k_full[st], ((n + i) / C::NS) & 1, abort_flag, p.a.err)) return false;
            tc_after();
            const uint32_t d = tmem + kColS + static_cast<uint32_t>((n + i) & 1) * KT;
            const uint64_t k0 = dk + st * kStage;
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const uint64_t o = static_cast<uint64_t>(kk >> 2) * (kSlab >> 4) + 2 * (kk & 3);
                mma_ts(d, qh + kk * 8, k0 + o, kIdS, kk > 0);
                mma_ts(d, ql + kk * 8, k0 + o, kIdS, true);
                if constexpr (C::HL) mma_ts(d, qh + kk * 8, k0 + kTerm + o, kIdS, true);
            }
            commit(&sm.s_full[(n + i) & 1]);
            commit(&sm.k_empty[st]);
            return true;
        };
        if (!scores(0)) return;
        if (tiles > 1 && !scores(1)) return;
        for (int i = 0; i < tiles; ++i) {
            const int st = (n + i) % C::NS;
            if (!mbar_wait(&sm.v_full[st], ((n + i) / C::NS) & 1, abort_flag, p.a.err)) return;
            if (!mbar_wait(&sm.p_ready[(n + i) & 1], ((n + i) >> 1) & 1, abort_flag, p.a.err)) return;
            tc_after();
            const uint32_t p0 = tmem + kColS + static_cast<uint32_t>((n + i) & 1) * KT;
            const uint64_t v0 = dv + st * kStage;
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk) {
                const uint64_t o = static_cast<uint64_t>(kk) * (16 * 128 >> 4);
                const uint32_t ph = p0 + kk * 8, pl = ph + 64;
                mma_ts(tmem + kColO, ph, v0 + o, kIdO, i > 0 || kk > 0);
                mma_ts(tmem + kColO, pl, v0 + o, kIdO, true);
                if constexpr (C::HL) mma_ts(tmem + kColO, ph, v0 + kTerm + o, kIdO, true);
            }
            commit(&sm.o_done[(n + i) & 1]);
            commit(&sm.v_empty[st]);
            if (i + 2 < tiles) {  // over P of this tile: once its product is done
                if (!mbar_wait(&sm.o_done[(n + i) & 1], ((n + i) >> 1) & 1, abort_flag, p.a.err)) return;
                if (!scores(i + 2)) return;
            }
        }
        n += tiles;
    }
}

// ----------------------------------------------------------------------------- the rows
template <int HD, typename T>
__device__ __forceinline__ void do_rows(Smem<HD, T> &sm, const TileParams &p, uint32_t tmem, long long total, int ctas) {
    using C = Cfg<HD, T>;
    constexpr int HALF = HD / 2;  // dims of O a thread owns
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int half = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    const int g = p.a.nh / p.a.nk;
    volatile int *abort_flag = &sm.abort_flag;
    int32_t *err = p.a.err;
    int n = 0, seg = 0;
    Walk w;
    for (bool more = walk_begin(w, p, total, ctas); more; more = walk_next(w, p), ++seg) {
        const int rows = w.cnt * g, tiles = w.u1 - w.u0;
        // this half row of Q, scaled, as hi + lo halves into TMEM (all MMAs that read the last ones are done)
        float c;
        {
            mbar_wait(&sm.q_in, seg & 1, abort_flag, err);
            float4 x[HALF / 4];
            float am = 0.0f;
#pragma unroll
            for (int d = 0; d < HALF / 4; ++d) {
                x[d] = row < rows ? *reinterpret_cast<const float4 *>(sm.q + row * C::kQRow + (half * (HALF / 4) + d) * 16)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                am = fmaxf(am, fmaxf(fmaxf(fabsf(x[d].x), fabsf(x[d].y)), fmaxf(fabsf(x[d].z), fabsf(x[d].w))));
            }
            sm.sum[half][row] = am;
            if (half == 0) sm.odd[row] = 0;
            named_sync(1, kRowThreads);
            if (tid == 0) mbar_arrive(&sm.q_free);  // (every thread has read its part)
            const int sh = row_shift(fmaxf(sm.sum[0][row], sm.sum[1][row]), 126);
            const float f = pow2i(sh);
            c = p.scale_log2 * pow2i(-sh);
#pragma unroll
            for (int d0 = 0; d0 < HALF / 4; d0 += 8) {  // 32 dims: 16 columns
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    split2(x[d0 + d].x * f, x[d0 + d].y * f, hi[2 * d], lo[2 * d]);
                    split2(x[d0 + d].z * f, x[d0 + d].w * f, hi[2 * d + 1], lo[2 * d + 1]);
                }
                tm_st16(lanes + kColQ + half * (HALF / 2) + d0 * 2, hi);
                tm_st16(lanes + kColQ + HD / 2 + half * (HALF / 2) + d0 * 2, lo);
            }
            tm_wait_st();
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_full);
        }
        const bool warp_live = (row & ~31) < rows, live = row < rows;
        // this row's window: keys [r_lo, r_hi) and [0, r_sink)
        const long long pos = w.past + w.t0 + row / g;
        int r_hi = 0, r_lo = 0, r_sink = 0;
        if (live && pos >= 0) {
            r_hi = pos + 1 < w.rows.cap ? static_cast<int>(pos + 1) : w.rows.cap;
            if (p.a.window) {
                const long long lo = pos - p.a.window + 1;
                r_lo = lo <= 0 ? 0 : (lo < r_hi ? static_cast<int>(lo) : r_hi);
                r_sink = min(p.a.n_sink, r_hi);
            }
        }
        // tiles in [all_lo, all_hi) (rows) are seen whole by every row: no mask
        const long long first = w.past + w.t0, last = first + w.cnt - 1;
        const long long all_hi = first + 1 < w.rows.cap ? first + 1 : w.rows.cap;
        const long long all_lo = p.a.window && last - p.a.window + 1 > 0 ? last - p.a.window + 1 : 0;
        float m = -INFINITY, l = 0.0f;
        for (int i = 0; i < tiles; ++i) {
            const int j0 = unit_tile(w.keys, w.u0 + i) * KT, q = n + i;
            mbar_wait(&sm.s_full[q & 1], (q >> 1) & 1, abort_flag, err);
            tc_after();
            if (!C::HL && (j0 < w.keys.lo || j0 + KT > w.keys.hi)) {
                // rows of this tile that no token sees: V must hold zeros there
                mbar_wait(&sm.v_full[q % C::NS], (q / C::NS) & 1, abort_flag, err);
                if (half == 0 && !item_sees(w.keys, j0 + row)) {
#pragma unroll
                    for (int s = 0; s < C::SLABS; ++s)
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch)
                            *reinterpret_cast<uint4 *>(sm.v[q % C::NS][0][s] + row * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
            }
            if (!warp_live) {
                named_sync(1, kRowThreads);
            } else {
                uint32_t x[64];  // scores, as bits
                tm_ld32(lanes + kColS + (q & 1) * KT + half * 64, x);
                tm_ld32(lanes + kColS + (q & 1) * KT + half * 64 + 32, x + 32);
                if constexpr (C::HL) {
                    mbar_wait(&sm.k_stat[q & 3], (q >> 2) & 1, abort_flag, err);
                    mbar_wait(&sm.v_stat[q & 3], (q >> 2) & 1, abort_flag, err);
                }
                tm_wait_ld();
                const bool mask = !(j0 >= all_lo && j0 + KT <= all_hi) && !(j0 + KT <= p.a.n_sink && j0 + KT <= all_hi);
                const float2 cc = make_float2(c, c);
#pragma unroll
                for (int e = 0; e < 64; e += 4) {
                    float2 a = mul2(bits2(x[e], x[e + 1]), cc), b = mul2(bits2(x[e + 2], x[e + 3]), cc);
                    if constexpr (C::HL) {
                        const float4 kf = *reinterpret_cast<const float4 *>(&sm.k_fac[q & 3][half * 64 + e]);
                        const float4 ve = *reinterpret_cast<const float4 *>(&sm.v_exp[q & 3][half * 64 + e]);
                        a = fma2(a, lo2(kf), lo2(ve));
                        b = fma2(b, hi2(kf), hi2(ve));
                    }
                    x[e] = __float_as_uint(a.x), x[e + 1] = __float_as_uint(a.y);
                    x[e + 2] = __float_as_uint(b.x), x[e + 3] = __float_as_uint(b.y);
                }
                if (mask) {
                    const int jb = j0 + half * 64, e_hi = r_hi - jb, e_lo = r_lo - jb, e_sink = r_sink - jb;
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        const bool see = (e < e_hi) & ((e >= e_lo) | (e < e_sink));
                        x[e] = see ? x[e] : 0xff800000u;  // -infinity
                    }
                }
                float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 64; e += 8)
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        mt[f] = fmaxf(fmaxf(mt[f], __uint_as_float(x[e + f])), __uint_as_float(x[e + 4 + f]));
                sm.mx[q & 1][half][row] = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
                tc_before();
                named_sync(1, kRowThreads);  // both threads of a row have read S: P may go over it
                tc_after();
                const float mn = fmaxf(sm.mx[q & 1][0][row], sm.mx[q & 1][1][row]);
                const bool grow = mn > m + kSlack || (m == -INFINITY && mn > m);
                float corr = 1.0f;
                if (grow) {
                    corr = ex2_approx(m - mn);
                    m = mn;
                }
                if (i > 0 && __any_sync(0xffffffffu, grow)) {
                    mbar_wait(&sm.o_done[(q - 1) & 1], ((q - 1) >> 1) & 1, abort_flag, err);
                    tc_after();
#pragma unroll 1
                    for (int d = 0; d < HALF; d += 16) {
                        uint32_t o[16];
                        tm_ld16(lanes + kColO + half * HALF + d, o);
                        tm_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                        tm_st16(lanes + kColO + half * HALF + d, o);
                    }
                }
                const float base = m == -INFINITY ? 0.0f : m - kShift;
                const float2 nb = make_float2(-base, -base);
                float2 s2 = make_float2(0.0f, 0.0f), s3 = s2;
#pragma unroll
                for (int e0 = 0; e0 < 64; e0 += 32) {
                    uint32_t ph[16], pl[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float2 a = add2(bits2(x[e0 + e], x[e0 + e + 1]), nb), b = add2(bits2(x[e0 + e + 2], x[e0 + e + 3]), nb);
                        a = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                        b = make_float2(ex2_approx(b.x), ex2_approx(b.y));
                        if constexpr (C::HL) {
                            const float4 vi = *reinterpret_cast<const float4 *>(&sm.v_inv[q & 3][half * 64 + e0 + e]);
                            s2 = fma2(a, lo2(vi), s2);
                            s3 = fma2(b, hi2(vi), s3);
                        } else {
                            s2 = add2(s2, a);
                            s3 = add2(s3, b);
                        }
                        split2(a.x, a.y, ph[e >> 1], pl[e >> 1]);
                        split2(b.x, b.y, ph[(e >> 1) + 1], pl[(e >> 1) + 1]);
                    }
                    tm_st16(lanes + kColS + (q & 1) * KT + half * 32 + (e0 >> 1), ph);
                    tm_st16(lanes + kColS + (q & 1) * KT + 64 + half * 32 + (e0 >> 1), pl);
                }
                l = l * corr + ((s2.x + s2.y) + (s3.x + s3.y));
                tm_wait_st();
            }
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_ready[q & 1]);
        }
        n += tiles;
        mbar_wait(&sm.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag, err);
        tc_after();
        sm.sum[half][row] = l;
        named_sync(1, kRowThreads);
        l = sm.sum[0][row] + sm.sum[1][row];
        const long long item0 = w.unit - w.u0;  // the item's first unit
        const bool whole = w.u0 == 0 && w.u1 == w.keys.units;
        float *out = p.a.out + (static_cast<long long>(w.lo + w.t0 + row / g) * p.a.nh + w.head * g + row % g) * HD + half * HALF;
        bool finish = whole, odd = false;
        if (whole) {
            if (warp_live) {
                const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
                for (int d = 0; d < HALF; d += 32) {
                    uint32_t o[32];
                    tm_ld32(lanes + kColO + half * HALF + d, o);
                    tm_wait_ld();
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            float4 y;
                            y.x = l == 0.0f ? 0.0f : __uint_as_float(o[e]) * inv;
                            y.y = l == 0.0f ? 0.0f : __uint_as_float(o[e + 1]) * inv;
                            y.z = l == 0.0f ? 0.0f : __uint_as_float(o[e + 2]) * inv;
                            y.w = l == 0.0f ? 0.0f : __uint_as_float(o[e + 3]) * inv;
                            odd |= !(fabsf(y.x) < INFINITY && fabsf(y.y) < INFINITY && fabsf(y.z) < INFINITY && fabsf(y.w) < INFINITY);
                            reinterpret_cast<float4 *>(out)[(d + e) >> 2] = y;
                        }
                    }
                }
            }
        } else {
            // this stretch's part: O as [dims / 4][rows] float4, then the rows' maxima and sums
            constexpr size_t kPart = static_cast<size_t>(BM) * (HD + 2);
            float *part = p.parts + (2 * static_cast<size_t>(blockIdx.x) + (w.u0 == 0 ? 1 : 0)) * kPart;
            if (warp_live) {
#pragma unroll
                for (int d = 0; d < HALF; d += 32) {
                    uint32_t o[32];
                    tm_ld32(lanes + kColO + half * HALF + d, o);
                    tm_wait_ld();
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            reinterpret_cast<float4 *>(part)[((half * HALF + d + e) >> 2) * BM + row] =
                                make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                    }
                }
                if (live && half == 0) {
                    part[BM * HD + row] = m;
                    part[BM * (HD + 1) + row] = l;
                }
            }
            __threadfence();
            named_sync(1, kRowThreads);
            const int b0 = stretch_of(total, ctas, item0), b1 = stretch_of(total, ctas, item0 + w.keys.units - 1);
            if (tid == 0) sm.last = atomicAdd(p.tickets + b0, 1) == b1 - b0;
            named_sync(1, kRowThreads);
            finish = sm.last != 0;
            if (finish && live) {
                __threadfence();
                // join the parts in the order of their keys
                float M = -INFINITY;
#pragma unroll 4
                for (int b = b0; b <= b1; ++b) {
                    const float *q = p.parts + (2 * static_cast<size_t>(b) + (b == b0 ? 1 : 0)) * kPart;
                    M = fmaxf(M, __ldcg(q + BM * HD + row));
                }
#pragma unroll 1
                for (int d0 = 0; d0 < HALF / 4; d0 += 8) {  // 32 dims at a time
                    float L = 0.0f;
                    float4 acc[8];
#pragma unroll
                    for (int d = 0; d < 8; ++d) acc[d] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                    for (int b = b0; b <= b1; ++b) {
                        const float *q = p.parts + (2 * static_cast<size_t>(b) + (b == b0 ? 1 : 0)) * kPart;
                        const float mb = __ldcg(q + BM * HD + row), lb = __ldcg(q + BM * (HD + 1) + row);
                        float4 y[8];
#pragma unroll
                        for (int d = 0; d < 8; ++d) y[d] = __ldcg(reinterpret_cast<const float4 *>(q) + (half * (HALF / 4) + d0 + d) * BM + row);
                        if (mb == -INFINITY && lb == 0.0f) continue;  // saw nothing
                        const float f = ex2_approx(mb - M);
                        L = fmaf(lb, f, L);
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            acc[d].x = fmaf(y[d].x, f, acc[d].x);
                            acc[d].y = fmaf(y[d].y, f, acc[d].y);
                            acc[d].z = fmaf(y[d].z, f, acc[d].z);
                            acc[d].w = fmaf(y[d].w, f, acc[d].w);
                        }
                    }
                    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (L != 0.0f) y = make_float4(acc[d].x * inv, acc[d].y * inv, acc[d].z * inv, acc[d].w * inv);
                        odd |= !(fabsf(y.x) < INFINITY && fabsf(y.y) < INFINITY && fabsf(y.z) < INFINITY && fabsf(y.w) < INFINITY);
                        reinterpret_cast<float4 *>(out)[d0 + d] = y;
                    }
                }
            }
        }
        if (finish) {
            if (odd) sm.odd[row] = 1;
            named_sync(1, kRowThreads);
            // rows that are not finite: by the definition, a row a warp
            for (int r = warp; r < rows; r += kRowThreads / 32) {
                if (!sm.odd[r]) continue;
                RowJob job;
                const long long t = w.lo + w.t0 + r / g;
                job.q = p.a.q + (t * p.a.nh + w.head * g + r % g) * p.a.hd;
                job.out = p.a.out + (t * p.a.nh + w.head * g + r % g) * HD;
                job.rows = w.rows;
                job.p = w.past + w.t0 + r / g;
                job.hk = w.head;
                attn_row<T, HD>(p.a.c, job, p.scale_log2, p.a.window, p.a.n_sink);
            }
        }
        tc_before();
        named_sync(1, kRowThreads);  // sm.odd and sm.sum are free for the next segment
    }
}

template <int HD, typename T>
__global__ void __launch_bounds__(Cfg<HD, T>::kThreads, 1)
    chunk_tiles_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ TileParams p) {
    using C = Cfg<HD, T>;
    extern __shared__ unsigned char smem_raw[];
    Smem<HD, T> &sm = *reinterpret_cast<Smem<HD, T> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(&sm.q_in, 1);
        mbar_init(&sm.q_free, 1);
        mbar_init(&sm.q_full, kRowThreads / 32);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.p_ready[i], kRowThreads / 32);
            mbar_init(&sm.o_done[i], 1);
            mbar_init(&sm.s_full[i], 1);
        }
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&sm.k_full[i], C::HL ? 4 : 1);
            mbar_init(&sm.v_full[i], C::HL ? 4 : 1);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm.k_stat[i], 4);
            mbar_init(&sm.v_stat[i], 4);
        }
        sm.abort_flag = 0;
        mbar_init_fence();
        if (!C::HL) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&sm.tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = sm.tmem_base;
    gdc_wait();  // the plan, and everything before it
    const long long total = p.head->total;
    const int ctas = p.head->ctas;
    if (warp < kRowThreads / 32) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRowRegs));
        do_rows<HD, T>(sm, p, tmem, total, ctas);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        if (warp == kMmaWarp) {
            if (lane == 0) issue_mmas<HD, T>(sm, p, tmem, total, ctas);
            __syncwarp();
        } else if (warp == kMmaWarp + 3) {
            copy_q<HD, T>(sm, p, total, ctas);
        } else if constexpr (C::HL) {
            if (warp >= 16)
                split_tiles<HD, T, true>(sm, p, warp - 16, total, ctas);
            else if (warp >= 12)
                split_tiles<HD, T, false>(sm, p, warp - 12, total, ctas);
        } else {
            if (warp == kMmaWarp + 1)
                copy_tiles<HD, T, false>(sm, tm_k, p, total, ctas);
            else if (warp == kMmaWarp + 2)
                copy_tiles<HD, T, true>(sm, tm_v, p, total, ctas);
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == kMmaWarp) {
        if (*static_cast<volatile int *>(&sm.abort_flag)) {
            // a wait ran out: let copies and MMAs in flight finish before TMEM and shared memory go away
            const unsigned long long t0 = gtimer();
            while (gtimer() - t0 < kWaitBudgetNs / 4) {
            }
        }
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int HD, typename T>
int launch(const TileParams &p, int grid, cudaStream_t s) {
    using C = Cfg<HD, T>;
    CUtensorMap tk = {}, tv = {};
    if constexpr (!C::HL) {
        const ChunkKv &c = p.a.c;
        if (!make_tensor_map_2d(&tk, c.k, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, c.W, static_cast<uint64_t>(c.rows), 64,
                                p.box_rows, true) ||
            !make_tensor_map_2d(&tv, c.v, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, c.W, static_cast<uint64_t>(c.rows), 64,
                                p.box_rows, true))
            return MINF_ERR_CUDA;
    }
    constexpr int kSmem = static_cast<int>(sizeof(Smem<HD, T>)) + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    auto kernel = chunk_tiles_kernel<HD, T>;
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
    return cudaLaunchKernelEx(&cfg, kernel, tk, tv, p) == cudaSuccess ? MINF_OK : MINF_ERR_CUDA;
}

PlanLayout tiles_layout(int nt, int n_seq, int nh, int nk, int hd_kv) {
    return plan_layout(nt, n_seq, BM / (nh / nk), sm_count(), static_cast<size_t>(BM) * (hd_kv + 2) * sizeof(float));
}

}  // namespace

size_t chunk_tiles_workspace(int nt, int n_seq, int nh, int nk, int hd_kv) {
    return tiles_layout(nt, n_seq, nh, nk, hd_kv).total;
}

int launch_chunk_tiles(const ChunkAttnArgs &a, void *workspace, int least, cudaStream_t s) {
    const int sms = sm_count();
    const PlanLayout lay = tiles_layout(a.sq.nt, a.sq.n_seq, a.nh, a.nk, a.hd_kv);
    char *ws = static_cast<char *>(workspace);
    TileParams p = {};
    p.a = a;
    p.tt = BM / (a.nh / a.nk);
    p.least = least;
    p.head = reinterpret_cast<const PlanHead *>(ws + lay.head);
    p.starts = reinterpret_cast<const PlanStart *>(ws + lay.starts);
    p.tickets = reinterpret_cast<int *>(ws + lay.tickets);
    p.parts = reinterpret_cast<float *>(ws + lay.parts);
    p.scale_log2 = a.scale * kLog2e;
    p.box_rows = a.c.table && (1 << a.c.block_shift) < KT ? 1 << a.c.block_shift : KT;
    PlanArgs pl = {};
    pl.c = a.c;
    pl.sq = a.sq;
    pl.nk = a.nk;
    pl.tt = p.tt;
    pl.kt = KT;
    pl.window = a.window;
    pl.n_sink = a.n_sink;
    pl.max_ctas = sms;
    pl.min_units = 1;
    pl.least = least;
    pl.most = 0x7fffffff;
    pl.head = const_cast<PlanHead *>(p.head);
    pl.starts = const_cast<PlanStart *>(p.starts);
    pl.tickets = p.tickets;
    pl.seq_units = reinterpret_cast<long long *>(ws + lay.seq_units);
    pl.tile_units = reinterpret_cast<long long *>(ws + lay.tile_units);
    pl.err = a.err;
    const int st = launch_chunk_plan(pl, s);
    if (st != MINF_OK) return st;
    if (a.hd_kv == 64)
        return a.c.kv == kKvQ8    ? launch<64, Q8>(p, sms, s)
               : a.c.kv == kKvF16 ? launch<64, __half>(p, sms, s)
                                  : launch<64, float>(p, sms, s);
    return a.c.kv == kKvQ8    ? launch<128, Q8>(p, sms, s)
           : a.c.kv == kKvF16 ? launch<128, __half>(p, sms, s)
                              : launch<128, float>(p, sms, s);
}

}  // namespace minf
