// minf_chunk_tiles.cu -- chunk attention on the 5th-generation tensor cores: the kernel for chunks
// of many rows.
//
// An item is 128 query rows: up to 128 / g consecutive tokens of one sequence with the g query
// heads of one kv head (row = token * g + head), so that a K/V tile is read once for the whole
// group.  A CTA walks its stretch of units (minf_chunk_plan.cuh); per tile of 128 keys:
//   S = Q K^T   tcgen05.mma kind::f16, M = N = 128, Q from TMEM, into one of two TMEM buffers
//   P = 2^(s - m)   two threads a row (64 keys each): read S, mask, share the row's maximum,
//                   and write P as binary16 halves hi + lo over the scores they came from
//   O = P V     tcgen05.mma kind::f16 with P from TMEM, V as it lies in memory (keys x dims, the
//               transposed operand), into TMEM; the row threads add the tile's O to their sums in
//               registers (sum = sum 2^(m_old - m) + O) while S and P of the next tile are under way
// Q and P come from TMEM because an operand pair from shared memory (8 KB a 128x128x16 step) takes
// 97 clocks of its bandwidth, against 64 of tensor work with one of them in TMEM.
// S of the next tile runs while the row threads work on this one; the tile after next goes into the
// buffer that P V has just finished with.
// The sums over the tiles are not left to the tensor cores: their accumulation cuts the low bits off, always
// towards zero, so that an output over 12000 keys was 2e-5 off 64 bits.  Added tile by tile in rounded fp32
// it is 8e-7 off (a plain fp32 evaluation: 1.7e-6), for 2% of the time.
//
// Precision: fp32 results from binary16 products.  Every operand that is not exactly binary16 is
// split into hi + lo halves (22 bits), scaled by a power of two that keeps both normal; a product
// is hi*hi + hi*lo + lo*hi.  A binary16 cache is exact as it is, so its products take two MMAs
// (Q and P are split); Q8_0 values (18 bits) and fp32 values take three.  Query rows and K rows are
// scaled row by row (the factor comes back in with the score).  V rows are scaled row by row too:
// V_j = V'_j 2^e_j, and the softmax runs on t_j = s_j + e_j, so P'_j = 2^(t_j - M) weighs V'_j and
// P'_j 2^-e_j is the term of the sum: a large row cannot push the others out of binary16's range for
// the rows that do not see it.  (Rows below 2^-46 keep the scale 2^60: what they lose is below 2^-70.)
// A term of the sum goes through P'_j, which is lost below 2^-126: where the exponents of the tiles that a row goes
// over are more than kSpan apart (fp32 rows alone can be) the row is computed again by its definition.  Within
// kSpan what is lost scores at least 126 - kSpan below the row's best key: a weight below 2^-46.
// Where a tile's rows are within 2^16 of its largest, as they nearly always are, one factor serves the
// whole tile (its small rows still have all their 22 bits) and the row threads need no factor a key:
// those would take half of the shared-memory bandwidth.
//
// Roles of a CTA (one an SM): warps 0-7 rows, warp 8 issues S, warp 10 issues P V (two warps, so that
// neither's waits hold up the other's products: one warp for both measured 1180 us against 1142 on the
// batch below); then the producers: for binary16 warps 9 (K) and 11 (V and the next item's Q rows) issue TMA
// copies straight into the swizzled layout that the tensor cores read, a block or a stretch of rows a
// copy; otherwise warp 9 resolves the tiles' rows ahead, warp 11 copies Q rows, and warps 12-19 load,
// split and write K and V in turn.
//
// What bounds it, on a batch of six ragged prompts of up to 2048 tokens over up to 12000 cached binary16 rows
// (16 query heads on 8 of 128 dims; 684 GFLOP): 1.12 ms, 612 TFLOP/s, twice that on the tensor cores, whose
// measured rate of 1.88 PFLOP/s allows 0.73 ms.  A CTA takes 1.74 million clocks for its 552 tiles and 7 to 8
// items (at 1.69 GHz, under the power limit): 3150 a tile with the items' edges.  Within a tile S and P V take
// 2600 clocks, 81 to 88 a 128x128x16 step, where the tensor cores' rate is 64 and a library product of 8192^3 takes
// 68, and the row threads 2500.  S cut into two halves of 64 keys, so that the first could start earlier,
// measured 1260 us.  Under a window of 8 tiles (6000 tokens, 1024 rows: 163 us) a tile takes 5800 clocks with the
// items' edges.  At 128 dims (2048 tokens over 8192 rows: 592 and 1007 us) Q8_0 tiles take 8700 clocks and fp32 ones
// 13500, against 3100 of tensor work in three products: the splitting warps write 128 KB of halves a tile, there is
// one stage of them beside the staged Q rows (66 KB, in use once an item), and the warps of a CTA wait on one
// another; of fp32 rows V is read a second time for its maxima.  Tried there and not kept: K split a tile ahead of V (265 us against 264 on 34 sequences, 31 of them single
// tokens), the tiles' factors found by the warp that resolves the rows (277 us).
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
constexpr int kSplitWarps = 8, kSplitRows = KT / kSplitWarps;  // rows of K and of V of a tile a warp takes
// The warps after the row threads': S, K copies (or rows resolved), P V, V copies (or Q rows)
constexpr int kScoreWarp = 0, kKeyWarp = 1, kValueWarp = 2, kQueryWarp = 3;
// P is at most 2^kShift, and lo keeps it to 2^-25: n keys that all lose as much are off by n 2^-25 of a sum of
// at least 2^kShift (2^-23 for 2^17 of them).
constexpr float kShift = 15.0f;
constexpr int kSpan = 80;
// TMEM columns: the S buffers (P over them: of each 32 keys hi, then lo, two keys a column), O of a tile, Q (hi,
// then lo, two dims a column)
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384, kTmemCols = 512;

template <int HD, typename T>
struct Cfg {
    static constexpr bool HL = !std::is_same<T, __half>::value;  // K and V as hi + lo halves
    static constexpr int SLABS = HD / 64;                        // 128-byte-wide slabs of a tile
    static constexpr int TERMS = HL ? 2 : 1;
    static constexpr int NS = HL ? (HD == 64 ? 2 : 1) : (HD == 64 ? 4 : 2);  // K and V stages
    // Row threads: two threads a row, each with half of a tile's keys and of the row's dims.  (Four,
    // which hide one another's waits better but meet at a wider barrier: 1155 us against 1102 over binary16.)
    static constexpr int PARTS = 2, COLS = KT / PARTS, DIMS = HD / PARTS;
    static constexpr int kRowThreads = 128 * PARTS, kRowWarps = kRowThreads / 32;
    // Warp groups: rows (0, 1), the issuing and copying warps (2), the splitting producers (3, 4).  The rows'
    // threads hold scores and 64 output sums, so registers move to them; the shares add up to the
    // launch's: 256 * 208 + 128 * 88 = 384 * 168, and 256 * 152 + 128 * 48 + 256 * 64 = 640 * 96.
    static constexpr int kThreads = HL ? 640 : 384;
    static constexpr int kRowRegs = HL ? 152 : 208, kIssueRegs = HL ? 48 : 88;
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
    unsigned long long row_full[4], row_free[4];       // and its rows resolved, taken
    alignas(16) float out[BM][36];                     // 32 dims of the output rows on their way out
    float mx[2][C::PARTS][BM], sum[C::PARTS][BM];
    int odd[BM];                                       // rows whose result is not finite
    int token[BM];                                     // of each row (a division otherwise)
    // the row threads' walk (here, not in every thread's registers): segment n in walk[n % 2]
    Walk walk[2];
    int more[2];
    int2 all;                                          // keys that every row of the item sees
    // hi + lo kinds, tile n in slot n % 4: K row factors, V row exponents and 2^-e; the smallest and the
    // largest shifts of each splitting warp's rows (K, V); what the row threads go by
    alignas(16) float k_fac[C::HL ? 4 : 1][KT];
    alignas(16) float v_exp[C::HL ? 4 : 1][KT], v_inv[C::HL ? 4 : 1][KT];
    int rows[C::HL ? 4 : 1][KT];                       // rows of the pool (-1: zeros)
    int row_head[C::HL ? 4 : 1];                       // their kv head (-1: no more tiles)
    int2 shifts[2][C::HL ? 4 : 1][kSplitWarps];
    struct TileFactors {
        float exp, fac;  // the tile's: V's e and 2^-e; K's factor in fac
        int by_row;      // its rows have their own
    } k_tile[C::HL ? 4 : 1], v_tile[C::HL ? 4 : 1];
    int2 v_span[C::HL ? 4 : 1], span;  // V's smallest and largest exponents: of a tile, of the segment
    uint32_t tmem_base;
    int abort_flag, last;
    // the row threads lead the two issuing warps (which would need registers to walk on their own): tiles of
    // the segment whose Q is ready (0: no more), and whether the tile whose P is ready is the last of all
    int seg_tiles, p_last[2];
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
// The whole warp comes here with the same operands and its leader issues: operands that the compiler knows
// to be the warp's own stay in uniform registers (from one lane's registers each one is moved there first).
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{\n .reg .pred p, l;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 l, %5, 0;\n @l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(leader)
                 : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, unsigned long long *bar) {
    asm volatile("{\n .reg .pred l;\n setp.ne.b32 l, %1, 0;\n @l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(su32(bar)),
                 "r"(leader)
                 : "memory");
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
__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t *u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t t, const uint32_t *u) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(u[0]), "r"(u[1]),
                 "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}
template <int N>
__device__ __forceinline__ void tm_st(uint32_t t, const uint32_t *u) {
    if constexpr (N == 8)
        tm_st8(t, u);
    else
        tm_st16(t, u);
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_shared(uint32_t addr, const uint32_t (&u)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
}

// Floats of a part: O, the rows' maxima and sums, V's exponents.
__host__ __device__ constexpr size_t part_floats(int hd) { return static_cast<size_t>(BM) * (hd + 2) + 4; }

// Byte offset of the 16-byte chunk c of a row in a 128-byte-swizzled slab.
__device__ __forceinline__ uint32_t sw16(int row, int c) {
    return static_cast<uint32_t>(row) * 128u + ((static_cast<uint32_t>(c) ^ static_cast<uint32_t>(row & 7)) << 4);
}

// The power of two that brings a row's largest magnitude to [2^14, 2^15), as 2^sh within -126 .. most; 1 for a
// row of zeros.
__device__ __forceinline__ int row_shift(float amax, int most) {
    const int ex = static_cast<int>((__float_as_uint(amax) >> 23) & 0xff) - 127;
    return amax > 0.0f ? max(min(14 - ex, most), -126) : 0;
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

// ----------------------------------------------------------------------------- producers
// One warp: an item's Q rows into the stage.
template <int HD, typename T>
__device__ __forceinline__ void copy_q_rows(Smem<HD, T> &sm, const AttnParams &p, const Walk &w) {
    using C = Cfg<HD, T>;
    const int lane = threadIdx.x & 31, g = p.a.nh / p.a.nk, rows = w.cnt * g;
    if (lane == 0) mbar_expect_tx(&sm.q_in, static_cast<uint32_t>(rows) * HD * 4);
    __syncwarp();
    for (int r = lane; r < rows; r += 32) {
        const long long t = walk_row(w, p) + r / g;
        bulk_load(sm.q + r * C::kQRow, p.a.q + (t * p.a.nh + w.head * g + r % g) * p.a.hd, HD * 4, &sm.q_in);
    }
    __syncwarp();
}

// One warp: TMA copies of the stretch's K (or V) tiles, a lane a copy.  A copy that no visible row
// lies in, or whose block is missing, reads past the map's end: zeros.
template <int HD, typename T, bool kV>
__device__ __forceinline__ void copy_tiles(Smem<HD, T> &sm, const CUtensorMap &map, const AttnParams &p, int ctas) {
    using C = Cfg<HD, T>;
    const int lane = threadIdx.x & 31;
    constexpr uint32_t kTileBytes = KT * HD * 2;
    const int pieces = KT / p.box_rows, copies = pieces * C::SLABS;
    volatile int *abort_flag = &sm.abort_flag;
    Walk w;
    int n = 0, seg = 0;
    for (bool more = walk_begin<KT>(w, p, ctas); more; more = walk_next<KT>(w, p), ++seg) {
        if constexpr (kV) {
            // (the last item's rows were taken when it began, tiles ago)
            if (seg > 0 && !__all_sync(0xffffffffu, chunk_wait(&sm.q_free, (seg - 1) & 1, abort_flag, p.a.err))) return;
            copy_q_rows<HD, T>(sm, p, w);
        }
        for (int u = w.u0; u < w.u1; ++u, ++n) {
            const int st = n % C::NS, j0 = unit_tile(w.keys, u) * KT;
            unsigned long long *full = kV ? &sm.v_full[st] : &sm.k_full[st], *empty = kV ? &sm.v_empty[st] : &sm.k_empty[st];
            long long row = 0;
            const int piece = lane / C::SLABS, slab = lane % C::SLABS;
            const int j = j0 + piece * p.box_rows;
            if (lane < copies) {  // (at most 8 pieces of 16 rows x 2 slabs)
                // any visible row in [j, j + box)?
                row = item_sees_some(w.keys, j, p.box_rows) ? seq_row(p.a.c, w.rows, j) : p.a.c.rows;
                if (row < 0) {
                    if (!kV) flag_error(p.a.err, MINF_ERRBIT_BLOCK);
                    row = p.a.c.rows;
                }
            }
            if (n >= C::NS && !__all_sync(0xffffffffu, chunk_wait(empty, ((n / C::NS) - 1) & 1, abort_flag, p.a.err))) return;
            if (lane == 0) mbar_expect_tx(full, kTileBytes);
            __syncwarp();
            if (lane < copies)
                tma_load_2d((kV ? sm.v[st][0][slab] : sm.k[st][0][slab]) + piece * p.box_rows * 128, &map,
                            w.head * HD + slab * 64, static_cast<int>(row), full);
            __syncwarp();
        }
    }
}

// One warp: all items' Q rows, each as soon as the row threads have taken the last one's.
template <int HD, typename T>
__device__ __forceinline__ void copy_q(Smem<HD, T> &sm, const AttnParams &p, int ctas) {
    volatile int *abort_flag = &sm.abort_flag;
    Walk w;
    int seg = 0;
    for (bool more = walk_begin<KT>(w, p, ctas); more; more = walk_next<KT>(w, p), ++seg) {
        if (seg > 0 && !__all_sync(0xffffffffu, chunk_wait(&sm.q_free, (seg - 1) & 1, abort_flag, p.a.err))) return;
        copy_q_rows<HD, T>(sm, p, w);
    }
}

// What a splitting warp (split_tiles) holds of its 16 rows of a tile: eight lanes load, split and write a row, four
// rows a step.
//
// Q8_0: VPL consecutive values a lane, all 16 rows held as they are stored, loaded as soon as the last tile's have
// been written.
template <int HD>
struct SplitQ8 {
    static constexpr int VPL = HD / 8, CH = VPL / 8;  // values and 16-byte chunks of halves a lane
    static constexpr int STEPS = kSplitRows / 4;
    uint2 raw[STEPS][CH];
    // Values of hidden rows are whatever row 0 holds times a scale of zero.
    static __device__ __forceinline__ uint2 load_scales(const void *base, const ChunkKv &c, int row, int head) {
        uint2 d = make_uint2(0, 0);
        if (row < 0) return d;
        const unsigned char *q = static_cast<const unsigned char *>(base) + row * c.row_bytes + c.W + head * (HD / 16);
        if constexpr (HD == 128)
            d = __ldg(reinterpret_cast<const uint2 *>(q));
        else
            d.x = __ldg(reinterpret_cast<const uint32_t *>(q));
        return d;
    }
    static __device__ __forceinline__ float most(uint2 d) {  // no value is above 127 scales
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&d.x)), b = __half22float2(*reinterpret_cast<const __half2 *>(&d.y));
        return 127.0f * fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y)));
    }
    // scale * 2^sh is a binary16 value (2^sh is exact; what a far smaller block's scale loses is below
    // 2^-33 of the row's largest value).
    static __device__ __forceinline__ uint32_t times(uint32_t d, float f) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&d));
        const __half2 y = __floats2half2_rn(a.x * f, a.y * f);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
    __device__ __forceinline__ void load(const void *pool, const ChunkKv &c, int row, int head, int sub, int l8) {
        const unsigned char *base = static_cast<const unsigned char *>(pool) + head * HD + l8 * VPL;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int r = max(__shfl_sync(0xffffffffu, row, 4 * i + sub), 0);
            const unsigned char *q = base + r * c.row_bytes;
            if constexpr (CH == 2) {
                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(q));
                raw[i][0] = make_uint2(x.x, x.y);
                raw[i][1] = make_uint2(x.z, x.w);
            } else {
                raw[i][0] = __ldg(reinterpret_cast<const uint2 *>(q));
            }
        }
    }
    // hi is the rounded product of a scaled scale and a quant, two binary16 values; the rest, at most 7 bits,
    // comes exactly out of a fused multiply-add.
    // d: the scaled scales, of row r in lane lane0 + r.
    __device__ __forceinline__ void put(uint32_t hi0, uint32_t lo0, uint2 d, int lane0, int warp, int sub, int l8) {
        // where the lane's chunks go in even and odd steps (four rows on, the swizzle differs in one bit)
        uint32_t at[2][CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int chunk = l8 * CH + (CH == 2 ? (c ^ (l8 >> 2)) : 0);  // of the row; eight a slab
            at[0][c] = hi0 + (chunk >> 3) * (KT * 128) + sw16(warp * kSplitRows + sub, chunk & 7);
            at[1][c] = at[0][c] ^ 64u;
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            uint32_t dd = __shfl_sync(0xffffffffu, d.x, lane0 + 4 * i + sub);
            int b = l8 * VPL / 32;  // the lane's block of the row
            if constexpr (HD == 128) {
                const uint32_t dy = __shfl_sync(0xffffffffu, d.y, lane0 + 4 * i + sub);
                dd = b & 2 ? dy : dd;
            }
            dd = __byte_perm(dd, dd, b & 1 ? 0x3232 : 0x1010);
            const __half2 s = *reinterpret_cast<const __half2 *>(&dd);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                // lanes 4-7 (the second slab) take their chunks in the other order: no bank twice
                const int cc = CH == 2 ? (c ^ (l8 >> 2)) : 0;
                const uint2 q2 = CH == 2 ? (cc ? raw[i][CH - 1] : raw[i][0]) : raw[i][0];
                const uint32_t u[2] = {q2.x ^ 0x80808080u, q2.y ^ 0x80808080u};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w = __byte_perm(u[e >> 1], 0x64646464u, (e & 1) ? 0x4342 : 0x4140);
                    const __half2 q = __hsub2(*reinterpret_cast<const __half2 *>(&w), __floats2half2_rn(1152.0f, 1152.0f));
                    const __half2 h = __hmul2_rn(q, s), l = __hfma2(q, s, __hneg2(h));
                    hi[e] = *reinterpret_cast<const uint32_t *>(&h);
                    lo[e] = *reinterpret_cast<const uint32_t *>(&l);
                }
                st_shared(at[i & 1][c] + i * 512, hi);
                st_shared(at[i & 1][c] + i * 512 + (lo0 - hi0), lo);
            }
            asm volatile("" ::: "memory");  // a step at a time: more in flight would go through local memory
        }
    }
};

// fp32 rows: eight values of each slab a lane, eight rows in flight.
template <int HD>
struct SplitF32 {
    static constexpr int SLABS = HD / 64, STEP = 2;  // (two four-row steps)
    float x[STEP][SLABS][8];

    __device__ __forceinline__ void load(const void *base, const ChunkKv &c, int row, int head, int r0, int sub, int l8) {
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
            const int r = __shfl_sync(0xffffffffu, row, r0 + 4 * i + sub);
            const float4 *q = reinterpret_cast<const float4 *>(static_cast<const unsigned char *>(base) + max(r, 0) * c.row_bytes) + head * (HD / 4) + 2 * l8;
#pragma unroll
            for (int s = 0; s < SLABS; ++s) {
                float4 a = __ldg(q + s * 16), b = __ldg(q + s * 16 + 1);
                if (r < 0) a = b = make_float4(0.f, 0.f, 0.f, 0.f);
                x[i][s][0] = a.x, x[i][s][1] = a.y, x[i][s][2] = a.z, x[i][s][3] = a.w;
                x[i][s][4] = b.x, x[i][s][5] = b.y, x[i][s][6] = b.z, x[i][s][7] = b.w;
            }
        }
    }
    __device__ __forceinline__ float amax(int i) const {  // of step i's row, in all of its lanes
        float m = 0.0f;
#pragma unroll
        for (int s = 0; s < SLABS; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[i][s][e]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
    }
    __device__ __forceinline__ void put(uint32_t hi0, uint32_t lo0, int i, int r, int l8, float f) {
        const float2 ff = make_float2(f, f);
#pragma unroll
        for (int s = 0; s < SLABS; ++s) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 y = mul2(make_float2(x[i][s][2 * e], x[i][s][2 * e + 1]), ff);
                split2(y.x, y.y, hi[e], lo[e]);
            }
            const uint32_t at = s * (KT * 128) + sw16(r, l8);
            st_shared(hi0 + at, hi);
            st_shared(lo0 + at, lo);
        }
    }
};

// Warp 9: the rows of every tile of the stretch, up to four tiles ahead.
template <int HD, typename T>
__device__ __forceinline__ void resolve_rows(Smem<HD, T> &sm, const AttnParams &p, int ctas) {
    const int lane = threadIdx.x & 31;
    const ChunkKv &c = p.a.c;
    volatile int *abort_flag = &sm.abort_flag;
    int n = 0;
    Walk w;
    bool more = walk_begin<KT>(w, p, ctas);
    int u = more ? w.u0 : 0;
    for (bool on = more; on; ++n) {
        const int slot = n & 3;
        if (n >= 4 && !__all_sync(0xffffffffu, chunk_wait(&sm.row_free[slot], ((n >> 2) - 1) & 1, abort_flag, p.a.err))) return;
        on = more;
        if (on) {
            const int j0 = unit_tile(w.keys, u) * KT + lane;
            long long row[KT / 32];
#pragma unroll
            for (int i = 0; i < KT / 32; ++i) row[i] = item_sees(w.keys, j0 + 32 * i) ? seq_row(c, w.rows, j0 + 32 * i) : -2;
#pragma unroll
            for (int i = 0; i < KT / 32; ++i) {
                if (row[i] == -1) flag_error(p.a.err, MINF_ERRBIT_BLOCK);
                sm.rows[slot][32 * i + lane] = row[i] < 0 ? -1 : static_cast<int>(row[i]);
            }
            if (lane == 0) sm.row_head[slot] = w.head;
            if (++u == w.u1) {
                more = walk_next<KT>(w, p);
                u = w.u0;
            }
        } else if (lane == 0) {
            sm.row_head[slot] = -1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.row_full[slot]);
    }
}

// The stretch's K and V tiles as scaled hi + lo halves.  (The rows come resolved from warp 9: a walk of their own
// would take the registers that the splitting warps hold rows in.)  V's exponents go out a tile ahead: the row
// threads need them with S, while the V stage may still be in use.  fp32 rows are prefetched into L2.
// The splitting warps take K and V of a tile in turn, 16 rows each: K of the next tile while P V runs, V while
// S does.  (Four warps for K and four for V took twice as long over a product's operand, with the tensor cores
// waiting for it.)  Lanes 0-15 hold what belongs to the warp's K rows, lanes 16-31 to its V rows.
template <int HD, typename T>
__device__ __forceinline__ void split_tiles(Smem<HD, T> &sm, const AttnParams &p, int warp) {
    using C = Cfg<HD, T>;
    constexpr bool Q = std::is_same<T, Q8>::value;
    const int lane = threadIdx.x & 31, l8 = lane & 7, sub = lane >> 3, kv = lane >> 4;
    const int my_row = warp * kSplitRows + (lane & 15);
    const ChunkKv &c = p.a.c;
    const void *pool = kv ? c.v : c.k;
    volatile int *abort_flag = &sm.abort_flag;
    std::conditional_t<Q, SplitQ8<HD>, SplitF32<HD>> sk, sv;
    uint2 scales = make_uint2(0, 0);
    int row = -1, head = -1;  // the rows taken last
    // The rows of tile n; false once a wait has run out.
    auto take_rows = [&](int n) -> bool {
        const int slot = n & 3;
        const bool ok = chunk_wait(&sm.row_full[slot], (n >> 2) & 1, abort_flag, p.a.err);
        head = ok ? sm.row_head[slot] : -1;
        row = head < 0 ? -1 : sm.rows[slot][my_row];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.row_free[slot]);
        if constexpr (Q) {
            scales = sk.load_scales(pool, c, row, max(head, 0));
        } else if (row >= 0) {
            const unsigned char *q = static_cast<const unsigned char *>(pool) + row * c.row_bytes + head * (HD * 4);
#pragma unroll
            for (int b = 0; b < HD * 4; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + b));
        }
        return ok;
    };
    // This lane's row's shift in tile n, whose rows were taken last, agreed on by the warps: the tile's where
    // its rows are within 2^16 of its largest, else the row's own (fp32 K rows: always their own, elsewhere).
    // False, in all of the warps, once a wait has run out in one of them: they leave together.
    int sh = 0, by_row = 0;
    auto agree = [&](int n, bool ok) -> bool {
        const int slot = n & 3;
        float am = 0.0f;
        if constexpr (Q) {
            am = sk.most(scales);
        } else {
#pragma unroll 1
            for (int r0 = 0; r0 < kSplitRows; r0 += 8) {
                sv.load(c.v, c, row, max(head, 0), r0, sub, l8);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float y = __shfl_sync(0xffffffffu, sv.amax(i), (lane & 3) * 8);  // to the row's lanes
                    if (((lane & 15) >> 2) == (r0 >> 2) + i) am = y;
                }
            }
        }
        sh = row_shift(am, kv ? 60 : 126);
        const int none = 1 << 20;  // rows of zeros go by whatever the others do
        int least = am > 0.0f ? sh : none, most = am > 0.0f ? sh : -none;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        }
        if ((lane & 15) == 0) sm.shifts[kv][slot][warp] = make_int2(least, most);
        if (!named_all(2, kSplitWarps * 32, ok)) return false;
#pragma unroll
        for (int k = 0; k < kSplitWarps; ++k) {
            const int2 o = sm.shifts[kv][slot][k];
            least = min(least, o.x);
            most = max(most, o.y);
        }
        by_row = most - least > 16;  // (no row at all: not row by row)
        // (a row of zeros goes by the largest row's: any will do for its values, and its weight stays)
        if (!by_row || !(am > 0.0f)) sh = least == none ? 0 : least;
        if (head < 0) return true;
        // V's exponents out
        if (kv) {
            if (by_row) sm.v_exp[slot][my_row] = static_cast<float>(-sh);
            if (by_row || !Q) sm.v_inv[slot][my_row] = pow2i(sh);
            if (warp == 0 && lane == 16) {
                sm.v_tile[slot] = {by_row ? 0.0f : static_cast<float>(-sh), by_row ? 1.0f : pow2i(sh), by_row};
                sm.v_span[slot] = by_row ? make_int2(-most, -least) : make_int2(-sh, -sh);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.v_stat[slot]);
        return true;
    };
    bool ok = take_rows(0);
    if constexpr (Q) {
        sk.load(c.k, c, row, max(head, 0), sub, l8);
        sv.load(c.v, c, row, max(head, 0), sub, l8);
    }
    if (!agree(0, ok)) return;
    for (int n = 0; head >= 0; ++n) {
        const int st = n % C::NS, slot = n & 3, cur = row, cur_head = head, phase = ((n / C::NS) - 1) & 1;
        const uint32_t k_hi = su32(sm.k[st][0][0]), v_hi = su32(sm.v[st][0][0]), to_lo = C::SLABS * KT * 128;
        uint2 d = make_uint2(0, 0);  // Q8_0: the scaled scales
        if constexpr (Q) d = make_uint2(sk.times(scales.x, pow2i(sh)), sk.times(scales.y, pow2i(sh)));
        // K
        ok = true;
        if constexpr (Q) {
            if (n >= C::NS) ok = chunk_wait(&sm.k_empty[st], phase, abort_flag, p.a.err);
            __syncwarp();
            if (!kv && by_row) sm.k_fac[slot][my_row] = pow2i(-sh);
            if (warp == 0 && lane == 0) sm.k_tile[slot] = {0.0f, by_row ? 1.0f : pow2i(-sh), by_row};
            sk.put(k_hi, k_hi + to_lo, d, 0, warp, sub, l8);
        } else {
#pragma unroll 1
            for (int r0 = 0; r0 < kSplitRows; r0 += 8) {
                sk.load(c.k, c, cur, cur_head, r0, sub, l8);
                if (r0 == 0) {
                    if (n >= C::NS) ok = chunk_wait(&sm.k_empty[st], phase, abort_flag, p.a.err);
                    __syncwarp();
                    if (warp == 0 && lane == 0) sm.k_tile[slot] = {0.0f, 1.0f, 1};
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = warp * kSplitRows + r0 + 4 * i + sub, s = row_shift(sk.amax(i), 126);
                    if (l8 == 0) sm.k_fac[slot][r] = pow2i(-s);
                    sk.put(k_hi, k_hi + to_lo, i, r, l8, pow2i(s));
                }
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&sm.k_stat[slot]);
            mbar_arrive(&sm.k_full[st]);
        }
        ok = take_rows(n + 1) && ok;
        if constexpr (Q) sk.load(c.k, c, row, max(head, 0), sub, l8);
        // V
        if constexpr (Q) {
            if (n >= C::NS) ok = chunk_wait(&sm.v_empty[st], phase, abort_flag, p.a.err) && ok;
            __syncwarp();
            sv.put(v_hi, v_hi + to_lo, d, 16, warp, sub, l8);
        } else {
#pragma unroll 1
            for (int r0 = 0; r0 < kSplitRows; r0 += 8) {
                sv.load(c.v, c, cur, cur_head, r0, sub, l8);
                if (r0 == 0) {
                    if (n >= C::NS) ok = chunk_wait(&sm.v_empty[st], phase, abort_flag, p.a.err) && ok;
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = warp * kSplitRows + r0 + 4 * i + sub;
                    sv.put(v_hi, v_hi + to_lo, i, r, l8, sm.v_inv[slot][r]);
                }
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.v_full[st]);
        if constexpr (Q) sv.load(c.v, c, row, max(head, 0), sub, l8);
        if (!agree(n + 1, ok)) return;
    }
}

// ----------------------------------------------------------------------------- the MMAs
// In descriptor units: the halves of a tile, and a stage.
template <int HD, typename T>
struct Desc {
    using C = Cfg<HD, T>;
    static constexpr uint32_t kSlab = KT * 128;
    static constexpr uint64_t kTerm = static_cast<uint64_t>(C::SLABS) * kSlab >> 4;
    static constexpr uint64_t kStage = C::TERMS * kTerm;
};

// chunk_wait by a warp, whose lanes go on or leave together.
__device__ __forceinline__ bool all_wait(unsigned long long *b, uint32_t parity, volatile int *abort_flag, int32_t *err) {
    return __all_sync(0xffffffffu, chunk_wait(b, parity, abort_flag, err));
}

template <int HD, typename T>
__device__ __forceinline__ void issue_scores(Smem<HD, T> &sm, uint32_t tmem, int32_t *err) {
    using C = Cfg<HD, T>;
    using D = Desc<HD, T>;
    volatile int *abort_flag = &sm.abort_flag;
    constexpr uint32_t kId = idesc_f16(BM, KT, false);
    const uint64_t dk = desc128(su32(sm.k), 16);
    const uint32_t qh = tmem + kColQ, ql = qh + HD / 2;
    const uint32_t leader = (threadIdx.x & 31) == 0;
    for (int n = 0, seg = 0;; ++seg) {
        if (!all_wait(&sm.q_full, seg & 1, abort_flag, err)) return;
        const int tiles = __shfl_sync(0xffffffffu, *static_cast<volatile int *>(&sm.seg_tiles), 0);
        if (tiles == 0) return;
        for (int i = 0; i < tiles; ++i, ++n) {
            const int st = n % C::NS;
            if (!all_wait(&sm.k_full[st], (n / C::NS) & 1, abort_flag, err)) return;
            // this buffer's last P: its product must be done (the item's first two tiles: with the last item)
            if (i >= 2 && !all_wait(&sm.o_done[n & 1], ((n - 2) >> 1) & 1, abort_flag, err)) return;
            tc_after();
            const uint32_t d = tmem + kColS + static_cast<uint32_t>(n & 1) * KT;
            const uint64_t k0 = dk + st * D::kStage;
            // (a slab at a time: all descriptors at once would go through local memory)
#pragma unroll 1
            for (int s = 0; s < C::SLABS; ++s) {
                const uint64_t ks = k0 + s * (D::kSlab >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_ts(leader, d, qh + s * 32 + kk * 8, ks + 2 * kk, kId, s > 0 || kk > 0);
                    mma_ts(leader, d, ql + s * 32 + kk * 8, ks + 2 * kk, kId, true);
                    if constexpr (C::HL) mma_ts(leader, d, qh + s * 32 + kk * 8, ks + D::kTerm + 2 * kk, kId, true);
                }
            }
            commit(leader, &sm.s_full[n & 1]);
            commit(leader, &sm.k_empty[st]);
        }
    }
}

template <int HD, typename T>
__device__ __forceinline__ void issue_values(Smem<HD, T> &sm, uint32_t tmem, int32_t *err) {
    using C = Cfg<HD, T>;
    using D = Desc<HD, T>;
    volatile int *abort_flag = &sm.abort_flag;
    constexpr uint32_t kId = idesc_f16(BM, HD, true);
    const uint64_t dv = desc128(su32(sm.v), D::kSlab);
    const uint32_t leader = (threadIdx.x & 31) == 0;
    for (int n = 0;; ++n) {
        const int st = n % C::NS;
        if (!all_wait(&sm.p_ready[n & 1], (n >> 1) & 1, abort_flag, err)) return;
        const int last = __shfl_sync(0xffffffffu, *static_cast<volatile int *>(&sm.p_last[n & 1]), 0);
        if (!all_wait(&sm.v_full[st], (n / C::NS) & 1, abort_flag, err)) return;
        tc_after();
        const uint64_t v0 = dv + st * D::kStage;
        const uint32_t p0 = tmem + kColS + static_cast<uint32_t>(n & 1) * KT;
#pragma unroll 4
        for (int kk = 0; kk < KT / 16; ++kk) {
            const uint64_t o = static_cast<uint64_t>(kk) * (16 * 128 >> 4);
            const uint32_t ph = p0 + (kk >> 1) * 32 + (kk & 1) * 8;  // 32 keys' hi halves, then their lo halves
            mma_ts(leader, tmem + kColO, ph, v0 + o, kId, kk > 0);
            mma_ts(leader, tmem + kColO, ph + 16, v0 + o, kId, true);
            if constexpr (C::HL) mma_ts(leader, tmem + kColO, ph, v0 + D::kTerm + o, kId, true);
        }
        commit(leader, &sm.o_done[n & 1]);
        commit(leader, &sm.v_empty[st]);
        if (last) return;
    }
}

// ----------------------------------------------------------------------------- the rows
template <int HD, typename T>
__device__ __forceinline__ void do_rows(Smem<HD, T> &sm, const AttnParams &p, uint32_t tmem, int ctas) {
    using C = Cfg<HD, T>;
    constexpr int PARTS = C::PARTS, COLS = C::COLS, DIMS = C::DIMS;  // keys and dims of a thread
    constexpr int OD = 32 / PARTS;                                    // dims of a part in an output pass
    constexpr bool F32 = std::is_same<T, float>::value;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int part = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    const int g = p.a.nh / p.a.nk;
    volatile int *abort_flag = &sm.abort_flag;
    int32_t *err = p.a.err;
    if (part == 0) sm.token[row] = row / g;
    if (tid == 0) sm.more[0] = walk_begin<KT>(sm.walk[0], p, ctas);
    named_sync(1, C::kRowThreads);
    int n = 0;
    for (int seg = 0; sm.more[seg & 1]; ++seg) {
        const Walk &w = sm.walk[seg & 1];
        const int rows = w.cnt * g, tiles = w.u1 - w.u0;
        // this part of the Q row, scaled, as hi + lo halves into TMEM (all MMAs that read the last ones are done)
        float c;
        {
            chunk_wait(&sm.q_in, seg & 1, abort_flag, err);
            float4 x[DIMS / 4];
            float am = 0.0f;
#pragma unroll
            for (int d = 0; d < DIMS / 4; ++d) {
                x[d] = row < rows ? *reinterpret_cast<const float4 *>(sm.q + row * C::kQRow + (part * (DIMS / 4) + d) * 16)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                am = fmaxf(am, fmaxf(fmaxf(fabsf(x[d].x), fabsf(x[d].y)), fmaxf(fabsf(x[d].z), fabsf(x[d].w))));
            }
            sm.sum[part][row] = am;
            if (part == 0) sm.odd[row] = 0;
            named_sync(1, C::kRowThreads);
            if (tid == 0) mbar_arrive(&sm.q_free);  // (every thread has read its part)
            am = sm.sum[0][row];
#pragma unroll
            for (int k = 1; k < PARTS; ++k) am = fmaxf(am, sm.sum[k][row]);
            const int sh = row_shift(am, 126);
            const float f = p.scale_log2 < 0.0f ? -pow2i(sh) : p.scale_log2 == 0.0f ? 0.0f : pow2i(sh);
            // S * c is the score in powers of two, c > 0: a row's largest S is its largest score (the sign of
            // the caller's scale is Q's, and so is a scale of zero: times an infinite key it is not a number; c is
            // then the smallest one, so that hidden keys' -infinity stays)
            c = fabsf(p.scale_log2) * pow2i(-sh);
            if (c == 0.0f) c = __uint_as_float(1u);
            constexpr int QD = DIMS < 32 ? DIMS : 32;  // dims of a store: half as many columns
#pragma unroll
            for (int d0 = 0; d0 < DIMS / 4; d0 += QD / 4) {
                uint32_t hi[QD / 2], lo[QD / 2];
#pragma unroll
                for (int d = 0; d < QD / 4; ++d) {
                    split2(x[d0 + d].x * f, x[d0 + d].y * f, hi[2 * d], lo[2 * d]);
                    split2(x[d0 + d].z * f, x[d0 + d].w * f, hi[2 * d + 1], lo[2 * d + 1]);
                }
                tm_st<QD / 2>(lanes + kColQ + part * (DIMS / 2) + d0 * 2, hi);
                tm_st<QD / 2>(lanes + kColQ + HD / 2 + part * (DIMS / 2) + d0 * 2, lo);
            }
            tm_wait_st();
            tc_before();
            if (tid == 0) sm.seg_tiles = tiles;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_full);
        }
        const bool warp_live = (row & ~31) < rows, live = row < rows;
        if (tid == 0) {
            // keys in [x, y) are seen by every row: their tiles need no mask
            const long long first = walk_pos(w, p), last = first + w.cnt - 1;
            const long long lo = p.a.window && last - p.a.window + 1 > 0 ? last - p.a.window + 1 : 0;
            const long long hi = first + 1 < w.rows.cap ? first + 1 : w.rows.cap;
            sm.all = make_int2(lo < 0x7fffffff ? static_cast<int>(lo) : 0x7fffffff, hi > 0 ? static_cast<int>(hi) : 0);
            // the next segment
            Walk next = w;
            sm.more[(seg + 1) & 1] = walk_next<KT>(next, p);
            sm.walk[(seg + 1) & 1] = next;
        }
        named_sync(1, C::kRowThreads);
        float m = -INFINITY, l = 0.0f, last_corr = 1.0f;
        int span_lo = 0x7fff, span_hi = -0x7fff;  // of V's exponents
        float2 acc[DIMS / 2];
#pragma unroll
        for (int d = 0; d < DIMS / 2; ++d) acc[d] = make_float2(0.0f, 0.0f);
        // O of tile q, which stands at that tile's maximum, into the sums, which stand at the one before
        auto fold = [&](int q) {
            chunk_wait(&sm.o_done[q & 1], (q >> 1) & 1, abort_flag, err);
            tc_after();
            const float2 f = make_float2(last_corr, last_corr);
#pragma unroll
            for (int d = 0; d < DIMS; d += 32) {
                uint32_t o[32];
                tm_ld32(lanes + kColO + part * DIMS + d, o);
                tm_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 2) acc[(d + e) >> 1] = fma2(acc[(d + e) >> 1], f, bits2(o[e], o[e + 1]));
            }
        };
        for (int i = 0; i < tiles; ++i) {
            const int j0 = unit_tile(w.keys, w.u0 + i) * KT, q = n + i;
            chunk_wait(&sm.s_full[q & 1], (q >> 1) & 1, abort_flag, err);
            tc_after();
            if (!warp_live) {
                named_sync(1, C::kRowThreads);
            } else {
                float cc = c, ve = 0.0f, vi = 1.0f;
                bool k_rows = false, v_rows = false;
                if constexpr (C::HL) {
                    chunk_wait(&sm.k_stat[q & 3], (q >> 2) & 1, abort_flag, err);
                    chunk_wait(&sm.v_stat[q & 3], (q >> 2) & 1, abort_flag, err);
                    const auto fk = sm.k_tile[q & 3], fv = sm.v_tile[q & 3];
                    if (F32) {
                        const int2 o = sm.v_span[q & 3];
                        span_lo = min(span_lo, o.x), span_hi = max(span_hi, o.y);
                    }
                    k_rows = fk.by_row, v_rows = fv.by_row;
                    cc = c * fk.fac;  // (1, 0 and 1 where they are row by row)
                    ve = fv.exp;
                    vi = fv.fac;
                }
                const float tile_c = cc;
                // key by key factors (all fp32 tiles have them for K, Q8_0 tiles rarely): t = S c k + e as the scores are
                // read, else one multiply-add below takes S to its exponential
                const bool by_key = C::HL && (k_rows || v_rows);
                if (by_key) cc = 1.0f;
                const int2 all = sm.all;
                const bool mask = j0 + KT > all.y || (j0 < all.x && j0 + KT > p.a.n_sink);
                int r_hi = 0, r_lo = 0, r_sink = 0;  // this row's window: keys [r_lo, r_hi) and [0, r_sink)
                if (mask && live) {
                    const long long pos = walk_pos(w, p) + sm.token[row];
                    r_hi = static_cast<int>(pos + 1 < w.rows.cap ? (pos + 1 > 0 ? pos + 1 : 0) : w.rows.cap);
                    if (p.a.window) {
                        const long long lo = pos - p.a.window + 1;
                        r_lo = lo > 0 ? static_cast<int>(lo < 0x7fffffff ? lo : 0x7fffffff) : 0;
                        r_sink = min(p.a.n_sink, r_hi);
                    }
                }
                const uint32_t s_col = lanes + kColS + (q & 1) * KT + part * COLS;
                // 32 of the thread's scores, hidden ones as -infinity
                auto scores = [&](int h, uint32_t *x) {
                    tm_ld32(s_col + h, x);
                    tm_wait_ld();
                    if (by_key) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            float4 kf = make_float4(tile_c, tile_c, tile_c, tile_c), vv = make_float4(ve, ve, ve, ve);
                            if (k_rows) {
                                const float4 f = *reinterpret_cast<const float4 *>(&sm.k_fac[q & 3][part * COLS + h + e]);
                                kf = make_float4(f.x * tile_c, f.y * tile_c, f.z * tile_c, f.w * tile_c);
                            }
                            if (v_rows) vv = *reinterpret_cast<const float4 *>(&sm.v_exp[q & 3][part * COLS + h + e]);
                            const float2 a = fma2(bits2(x[e], x[e + 1]), lo2(kf), lo2(vv)), b = fma2(bits2(x[e + 2], x[e + 3]), hi2(kf), hi2(vv));
                            x[e] = __float_as_uint(a.x), x[e + 1] = __float_as_uint(a.y);
                            x[e + 2] = __float_as_uint(b.x), x[e + 3] = __float_as_uint(b.y);
                        }
                    }
                    if (mask) {
                        const int jb = j0 + part * COLS + h, e_hi = r_hi - jb, e_lo = r_lo - jb, e_sink = r_sink - jb;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const bool see = (e < e_hi) & ((e >= e_lo) | (e < e_sink));
                            x[e] = see ? x[e] : 0xff800000u;  // -infinity
                        }
                    }
                };
                constexpr bool kHold = !C::HL;  // (registers for all of the scores; else they are read again)
                uint32_t xs[kHold ? COLS : 32];
                float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int h = 0; h < COLS; h += 32) {
                    uint32_t *x = xs + (kHold ? h : 0);
                    scores(h, x);
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            mt[f] = fmaxf(fmaxf(mt[f], __uint_as_float(x[e + f])), __uint_as_float(x[e + 4 + f]));
                }
                sm.mx[q & 1][part][row] = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
                named_sync(1, C::kRowThreads);
                float mn = sm.mx[q & 1][0][row];
#pragma unroll
                for (int k = 1; k < PARTS; ++k) mn = fmaxf(mn, sm.mx[q & 1][k][row]);
                const float te = by_key ? 0.0f : ve;
                mn = fmaxf(m, mn * cc + te);
                const float corr = mn == -INFINITY ? 1.0f : ex2_approx(m - mn);
                m = mn;
                const float base = m == -INFINITY ? 0.0f : m - kShift;
                const float2 c2 = make_float2(cc, cc), nb = make_float2(te - base, te - base);
                float2 s2 = make_float2(0.0f, 0.0f), s3 = s2;
#pragma unroll
                for (int h = 0; h < COLS; h += 32) {
                    uint32_t *x = xs + (kHold ? h : 0), ph[16], pl[16];
                    if (!kHold) scores(h, x);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float2 a = fma2(bits2(x[e], x[e + 1]), c2, nb), b = fma2(bits2(x[e + 2], x[e + 3]), c2, nb);
                        a = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                        b = make_float2(ex2_approx(b.x), ex2_approx(b.y));
                        if (C::HL && v_rows) {  // each key's own 2^-e
                            const float4 f = *reinterpret_cast<const float4 *>(&sm.v_inv[q & 3][part * COLS + h + e]);
                            s2 = fma2(a, lo2(f), s2);
                            s3 = fma2(b, hi2(f), s3);
                        } else {
                            s2 = add2(s2, a);
                            s3 = add2(s3, b);
                        }
                        split2(a.x, a.y, ph[e >> 1], pl[e >> 1]);
                        split2(b.x, b.y, ph[(e >> 1) + 1], pl[(e >> 1) + 1]);
                    }
                    // over the scores they came from: 32 keys' hi halves, then their lo halves
                    tm_st16(s_col + h, ph);
                    tm_st16(s_col + h + 16, pl);
                }
                const float sum = (s2.x + s2.y) + (s3.x + s3.y);
                l = l * corr + (C::HL ? sum * vi : sum);
                if (i > 0) fold(q - 1);  // (P V of this tile goes over it)
                last_corr = corr;
                tm_wait_st();
            }
            if (!C::HL && (j0 < w.keys.lo || j0 + KT > w.keys.hi)) {
                // rows of this tile that no token sees: V must hold zeros there
                chunk_wait(&sm.v_full[q % C::NS], (q / C::NS) & 1, abort_flag, err);
                if (part == 0 && !item_sees(w.keys, j0 + row)) {
#pragma unroll
                    for (int s = 0; s < C::SLABS; ++s)
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch)
                            *reinterpret_cast<uint4 *>(sm.v[q % C::NS][0][s] + row * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
            }
            tc_before();
            if (tid == 0) sm.p_last[q & 1] = i + 1 == tiles && tiles == w.left;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_ready[q & 1]);
        }
        n += tiles;
        if (F32 && tid == 0) sm.span = make_int2(span_lo, span_hi);
        if (warp_live) fold(n - 1);
        sm.sum[part][row] = l;
        named_sync(1, C::kRowThreads);
        l = sm.sum[0][row];
#pragma unroll
        for (int k = 1; k < PARTS; ++k) l += sm.sum[k][row];
        const bool whole = w.u0 == 0 && w.u1 == w.keys.units;
        // 32 dims of a row (OD of each part's) at a time through shared memory, so that they go out together (a
        // thread's own 16 bytes a row at a time cost 32 transactions an instruction)
        float *item_out = p.a.out + (static_cast<long long>(walk_row(w, p)) * p.a.nh + w.head * g) * HD;
        auto put = [&](const float *y, int d) {
#pragma unroll
            for (int e = 0; e < OD; e += 4)
                *reinterpret_cast<float4 *>(&sm.out[row][part * OD + e]) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            named_sync(1, C::kRowThreads);
#pragma unroll
            for (int k = 0; k < 128 * 8 / C::kRowThreads; ++k) {
                const int r = k * (C::kRowThreads / 8) + (tid >> 3), q = (tid & 7) * 4;  // eight lanes a row
                if (r < rows) {
                    const int t = sm.token[r];
                    *reinterpret_cast<float4 *>(item_out + (t * p.a.nh + r - t * g) * HD + q / OD * DIMS + q % OD + d) =
                        *reinterpret_cast<const float4 *>(&sm.out[r][q]);
                }
            }
            named_sync(1, C::kRowThreads);
        };
        bool finish = whole, odd = false, again = false;
        if (whole) {
            if (F32) odd = sm.span.y - sm.span.x > kSpan;
            const float inv = 1.0f / l;  // (l zero, where a row sees nothing or nothing but scores of minus infinity: NaN)
#pragma unroll
            for (int d = 0; d < DIMS; d += 16) {
                float y[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 o = acc[(d + e) >> 1];
                    y[e] = (e & 1 ? o.y : o.x) * inv;
                    odd |= !(fabsf(y[e]) < INFINITY);
                }
#pragma unroll
                for (int e = 0; e < 16; e += OD) put(y + e, d + e);
            }
        } else {
            // this stretch's part: O as [dims / 4][rows] float4, then the rows' maxima and sums and V's exponents
            constexpr size_t kPart = part_floats(HD);
            float *mine = p.parts + (2 * static_cast<size_t>(blockIdx.x) + (w.u0 == 0 ? 1 : 0)) * kPart;
            if (live) {
#pragma unroll
                for (int d = 0; d < DIMS; d += 4)
                    reinterpret_cast<float4 *>(mine)[((part * DIMS + d) >> 2) * BM + row] =
                        make_float4(acc[d >> 1].x, acc[d >> 1].y, acc[(d >> 1) + 1].x, acc[(d >> 1) + 1].y);
                if (part == 0) {
                    mine[BM * HD + row] = m;
                    mine[BM * (HD + 1) + row] = l;
                }
            }
            if (F32 && tid == 0) *reinterpret_cast<int2 *>(mine + BM * (HD + 2)) = sm.span;
            int b0, b1;
            walk_parts(w, p, b0, b1);
            named_sync(1, C::kRowThreads);
            if (tid == 0) {
                __threadfence();  // (the whole CTA's part: the barrier ordered it before this)
                sm.last = atomicAdd(p.tickets + b0, 1) == b1 - b0;
                __threadfence();
            }
            named_sync(1, C::kRowThreads);
            finish = sm.last != 0;
            if (finish) {
                // join the parts in the order of their keys (dead rows read what is there and are not put); two
                // parts' loads are in flight at a time
                constexpr int JD = C::HL ? 32 : DIMS;  // dims of a pass
                int2 span = sm.span;
#pragma unroll 1
                for (int d0 = 0; d0 < DIMS; d0 += JD) {
                    float M = -INFINITY, L = 0.0f;
                    float y[JD];
#pragma unroll
                    for (int d = 0; d < JD; ++d) y[d] = 0.0f;
#pragma unroll(C::HL ? 1 : 2)
                    for (int b = b0; b <= b1; ++b) {
                        const float *q = p.parts + (2 * static_cast<size_t>(b) + (b == b0 ? 1 : 0)) * kPart;
                        const float mb = __ldcg(q + BM * HD + row), lb = __ldcg(q + BM * (HD + 1) + row);
                        float4 x[JD / 4];
#pragma unroll
                        for (int d = 0; d < JD / 4; ++d) x[d] = __ldcg(reinterpret_cast<const float4 *>(q) + ((part * DIMS + d0) / 4 + d) * BM + row);
                        if (F32) {
                            const int2 o = __ldcg(reinterpret_cast<const int2 *>(q + BM * (HD + 2)));
                            span = make_int2(min(span.x, o.x), max(span.y, o.y));
                        }
                        if (mb == -INFINITY && lb == 0.0f) continue;  // saw nothing, whatever it holds
                        const float mn = fmaxf(M, mb), fo = ex2_approx(M - mn), fn = ex2_approx(mb - mn);
                        M = mn;
                        L = L * fo + lb * fn;
#pragma unroll
                        for (int d = 0; d < JD / 4; ++d) {
                            y[4 * d] = y[4 * d] * fo + x[d].x * fn;
                            y[4 * d + 1] = y[4 * d + 1] * fo + x[d].y * fn;
                            y[4 * d + 2] = y[4 * d + 2] * fo + x[d].z * fn;
                            y[4 * d + 3] = y[4 * d + 3] * fo + x[d].w * fn;
                        }
                    }
                    const float inv = 1.0f / L;
#pragma unroll
                    for (int d = 0; d < JD; ++d) {
                        y[d] *= inv;
                        odd |= !(fabsf(y[d]) < INFINITY);
                    }
                    if (F32) odd |= span.y - span.x > kSpan;
#pragma unroll
                    for (int d = 0; d < JD; d += OD) put(y + d, d0 + d);
                }
            }
        }
        if (finish) {
            odd = odd && live;
            if (odd) sm.odd[row] = 1;
            // rows that are not finite: by the definition, a row a warp
            again = !named_all(1, C::kRowThreads, !odd);
            if (again) {
                if (tid == 0) rows_again(&sm.abort_flag, true);
                const long long at = static_cast<long long>(walk_row(w, p)) * p.a.nh + w.head * g;
                attn_rows_again<T, HD>(p.a.c, sm.odd, rows, warp, C::kRowWarps, p.a.q + at * p.a.hd, p.a.out + at * HD, g,
                                       p.a.nh, p.a.hd, w.rows, walk_pos(w, p), w.head, p.scale_log2, p.a.window, p.a.n_sink);
            }
        }
        tc_before();
        named_sync(1, C::kRowThreads);  // sm.odd and sm.sum are free for the next segment
        if (again && tid == 0) rows_again(&sm.abort_flag, false);
    }
    if (tid == 0) sm.seg_tiles = 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full);
}

template <int HD, typename T>
__global__ void __launch_bounds__(Cfg<HD, T>::kThreads, 1)
    chunk_tiles_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ AttnParams p) {
    using C = Cfg<HD, T>;
    extern __shared__ unsigned char smem_raw[];
    Smem<HD, T> &sm = *reinterpret_cast<Smem<HD, T> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(&sm.q_in, 1);
        mbar_init(&sm.q_free, 1);
        mbar_init(&sm.q_full, C::kRowWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.p_ready[i], C::kRowWarps);
            mbar_init(&sm.o_done[i], 1);
            mbar_init(&sm.s_full[i], 1);
        }
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&sm.k_full[i], C::HL ? kSplitWarps : 1);
            mbar_init(&sm.v_full[i], C::HL ? kSplitWarps : 1);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sm.k_stat[i], kSplitWarps);
            mbar_init(&sm.v_stat[i], kSplitWarps);
            mbar_init(&sm.row_full[i], 1);
            mbar_init(&sm.row_free[i], kSplitWarps);
        }
        sm.abort_flag = 0;
        mbar_init_fence();
        if (!C::HL) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }
    }
    if (warp == C::kRowWarps + kScoreWarp) {
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
    const int ctas = p.head->ctas;
    const int role = warp - C::kRowWarps;
    const bool idle = static_cast<int>(blockIdx.x) >= ctas;  // no stretch
    if (warp < C::kRowWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRowRegs));
        if (!idle) do_rows<HD, T>(sm, p, tmem, ctas);
    } else if (!C::HL || warp < C::kRowWarps + 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssueRegs));
        if (warp == C::kRowWarps + kScoreWarp) {
            if (!idle) issue_scores<HD, T>(sm, __shfl_sync(0xffffffffu, tmem, 0), p.a.err);
        } else if (role == kValueWarp) {
            if (!idle) issue_values<HD, T>(sm, __shfl_sync(0xffffffffu, tmem, 0), p.a.err);
        } else if constexpr (C::HL) {
            if (role == kQueryWarp)
                copy_q<HD, T>(sm, p, ctas);
            else
                resolve_rows<HD, T>(sm, p, ctas);
        } else if (role == kKeyWarp) {
            copy_tiles<HD, T, false>(sm, tm_k, p, ctas);
        } else {
            copy_tiles<HD, T, true>(sm, tm_v, p, ctas);
        }
    } else if constexpr (C::HL) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(64));
        if (!idle) split_tiles<HD, T>(sm, p, role - 4);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == C::kRowWarps + kScoreWarp) {
        if (*static_cast<volatile int *>(&sm.abort_flag) == 1) {
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
int launch(const AttnParams &p, int grid, cudaStream_t s) {
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
    return plan_layout(nt, n_seq, BM / (nh / nk), sm_count(), part_floats(hd_kv) * sizeof(float));
}

}  // namespace

size_t chunk_tiles_workspace(int nt, int n_seq, int nh, int nk, int hd_kv) {
    return tiles_layout(nt, n_seq, nh, nk, hd_kv).total;
}

void plan_chunk_tiles(PlanArgs &plan, AttnParams &p, const ChunkAttnArgs &a, void *workspace, int least) {
    const int sms = sm_count();
    p = {};
    p.a = a;
    p.tt = BM / (a.nh / a.nk);
    p.kt = KT;
    p.least = least;
    p.most = 0x7fffffff;
    p.scale_log2 = a.scale * kLog2e;
    p.box_rows = a.c.table && (1 << a.c.block_shift) < KT ? 1 << a.c.block_shift : KT;
    plan_args(plan, p, tiles_layout(a.sq.nt, a.sq.n_seq, a.nh, a.nk, a.hd_kv), workspace, sms < kPlanMost ? sms : kPlanMost, 1, 0);
}

int launch_chunk_tiles(const AttnParams &p, cudaStream_t s) {
    const int sms = sm_count(), kv = p.a.c.kv;
    if (p.a.hd_kv == 64)
        return kv == kKvQ8 ? launch<64, Q8>(p, sms, s) : kv == kKvF16 ? launch<64, __half>(p, sms, s) : launch<64, float>(p, sms, s);
    return kv == kKvQ8 ? launch<128, Q8>(p, sms, s) : kv == kKvF16 ? launch<128, __half>(p, sms, s) : launch<128, float>(p, sms, s);
}

}  // namespace minf
