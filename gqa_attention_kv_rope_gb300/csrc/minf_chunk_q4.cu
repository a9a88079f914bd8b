// minf_chunk_q4.cu -- chunk attention over Q4 rows for few query rows a sequence (single tokens, drafted tokens): a
// stream of whole cached rows, all kv heads at once.
//
// A Q4 row is short: 64 bytes of codes and 8 of scales a head of 128 values.  A stream a head, as minf_chunk_stream.cu
// makes it, would fetch a sector of scales for 8 bytes of them, and put a row's 576 bytes together from requests far
// apart.  Here an item is a token tile with a group of up to eight kv heads (all of them, where there are no more):
// producer warps keep a ring of tiles of whole rows full with TMA copies, and each computing warp takes one head's part of
// them (and one of kp equal parts of the keys, where there are fewer than eight heads), so that no two warps of a tile
// have to meet: with its own maxima, sums and outputs a warp only waits for the ring.
//
// Products are warp-level m16n8k16 with the keys as the 16 rows and the queries as the 8 columns.
//   S^T = K Q^T     the codes themselves are the operand: a nibble in bits 2 to 5 of a half is the subnormal binary16
//                   number 4 u 2^-24 (64 u 2^-24 in bits 6 to 9: Q has 1/16 there), exact in the tensor cores.
//                   Per 32-value block S_b = sum q u 2^-22 - 8 sum q 2^-22 (what the sums start from), s = sum_b d_b S_b:
//                   a mask a pair of codes and a shift a word, where u - 8 as a binary16 number would take another
//                   instruction a pair.  The tensor cores line a product up by the exponents of its operands, 2^-14 for
//                   every subnormal one, and cut off what is below some 24 bits; codes left in bits 0 to 3 lose two bits
//                   more there (outputs of 2 queries a key: 9.7e-7 off relative to their norm, not 3.1e-7; 112 us for 64
//                   sequences of up to 8192 rows instead of 114), codes all brought to bits 4 to 7 gain little over
//                   this (3.0e-7) for 116 us.
//   O^T += V^T P^T  the values d (u - 8), exact binary16 numbers.  (An offset taken out of the sums afterwards would not
//                   do here: over n keys the sums shrink by sqrt(n) against it.)
// Q and P are split into binary16 halves hi + lo.  Where an item has at most four query rows the halves stand side by
// side in the eight columns (PACK): one product does both, and the columns are added at the end; with more rows
// the halves take a product each: 64 sequences of 4096 rows with two query rows a key 95 us, 109 in the variant of 8.  The
// sums over Q's halves are kept apart there too: in one sum the offset of the codes pushes lo's bits out where queries have
// a large common part (of ten times their spread: outputs 1.6e-5 off, not 7e-7; 107 us, not 109).
//
// What bounds it, on 64 sequences of up to 8192 rows (16 query heads on 8 of 128 dims, 382 MB of rows, once from memory):
// 114 us, 3.35 TB/s.  The producers alone would need 66 us, the computing warps 112 with the rows already there: some 650
// instructions a warp for 32 keys of a head (a tile takes 2210 clocks; 2460, of which scores 950, softmax 420 and values
// 1020, before the offset moved into the products), for every half of codes a mask and a share of a shift, for every pair
// of values a mask, an exponent and two half2 steps.  Issue slots are half full, the pipes 39 (integer), 36 (fp32 and half)
// and 18 per cent (tensor): eight warps of 208 registers, two a scheduler, do not cover each other's latencies, and more do
// not fit (twelve 147 us, sixteen with half the keys each 200 with spills; as pairs, one warp for scores and one for
// values, 115; scores of the next tile under the values of this one 121).  Short calls are latency: one token over 128
// rows 9.5 us in a graph with the plan's launch.
#include <cmath>

#include "minf_chunk_plan.cuh"
#include "minf_chunk_row.cuh"
#include "minf_chunk_tiles.h"
#include "minf_sm103.cuh"
#include "minf_warp_mma.cuh"

namespace minf {

namespace {

constexpr int kWarps = 8, kProducers = 2, kThreads = 32 * (kWarps + 4);  // (registers move between groups of four)
constexpr int kComputeRegs = 208, kOtherRegs = 88;  // 256 * 208 + 128 * 88 = 384 * 168, the launch's
constexpr int kSteps = 2, kKeys = 16 * kSteps;       // of a tile, a warp
// P is at most 2^(shift + slack) = 2^15, as in minf_chunk_stream.cu.
constexpr float kShift = 12.0f, kSlack = 3.0f;
constexpr int kMostStages = 8;
// The join of a part takes a warp 740 clocks, a tile 2210.  One sequence of 40,000 rows, 8 heads of 128 dims: 100 us in
// 152 stretches, 76 in the 64 that follow from this (79 with half of it, 72 with twice; 71 now, the plan being shorter); of 16,000 rows 93 and 50 (58,
// 52); of 4096 rows 46 and 34.  (The parts' loads two and three at a time, without more of them in a lane: 99 and 98; a
// row after the other, its values across the lanes: 71, but 75 us against 66 for 32 drafts, whose joins are short.)
constexpr float kJoin = 0.3f;

// How a call's rows lie in the ring: a stage is K and V of a tile, each the rows' codes (with their scales, where an item has
// all kv heads) and then, else, 16-byte pieces with the group's scales.
struct Geo {
    int hg, kp, kt;       // kv heads of an item, parts of the keys, keys of a tile (32 kp)
    int whole;            // an item has all kv heads: rows are copied whole
    int codes;            // bytes of a row's codes in an item
    int pitch;            // bytes from row to row
    int scale_pitch, scale_at;  // the same of scales, bytes to the first row's (whole: in the rows)
    int side, stage, stages;    // bytes of K (or V), of a stage; stages
};

struct Params {
    CUtensorMap k, v, k_scales, v_scales;  // (scales: where rows are not copied whole)
    AttnParams p;
    Geo g;
};

struct Meta {
    unsigned long long full[kMostStages], empty[kMostStages];
    alignas(8) float m[kWarps][8];
    alignas(8) float l[kWarps][8];
    int odd[8][8], last[8];             // a head's
    int abort_flag, again;              // 1 once a wait has run out; warps that compute rows again
};

// Up to 16 tries in three instructions each: what waits must not take the issue slots of what computes.
__device__ __forceinline__ bool mbar_try16(unsigned long long *b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .u32 i;\n mov.u32 i, 0;\n"
        "TRY:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra DONE;\n"
        " add.u32 i, i, 1;\n setp.lt.u32 q, i, 16;\n @q bra TRY;\n"
        "DONE:\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(su32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
// chunk_wait, with any number of warps at rows that are computed again.
__device__ __forceinline__ bool ring_wait_long(unsigned long long *b, uint32_t parity, Meta &mt, int32_t *err) {
    volatile int *abort_flag = &mt.abort_flag, *again = &mt.again;
    uint32_t t0 = gtimer_lo();
    while (true) {
        if (*abort_flag) return false;
        if (mbar_try16(b, parity)) return true;
        if (*again) t0 = gtimer_lo();
        if (gtimer_lo() - t0 > static_cast<uint32_t>(kWaitBudgetNs)) {
            *abort_flag = 1;
            flag_error(err, MINF_ERRBIT_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ bool ring_wait(unsigned long long *b, uint32_t parity, Meta &mt, int32_t *err) {
    return mbar_try16(b, parity) || ring_wait_long(b, parity, mt, err);
}

// Loads from the ring are plain ones and the products pure functions of their operands (no `volatile`), so that the
// compiler is free to run the loads and conversions of one block under the products of another.
__device__ __forceinline__ uint32_t ld32(const unsigned char *a) { return *reinterpret_cast<const uint32_t *>(a); }
template <int N>  // halves of a head's scales, in N/2 words
__device__ __forceinline__ void ld_scales(const unsigned char *a, uint32_t (&x)[N / 2]) {
    if constexpr (N == 4) {
        const uint2 y = *reinterpret_cast<const uint2 *>(a);
        x[0] = y.x, x[1] = y.y;
    } else {
        x[0] = ld32(a);
    }
}
// Two pairs of a product's four results, whose rows are n8 (lo) and n8 + 8 (hi).
struct Frag {
    float2 lo, hi;
};
__device__ __forceinline__ void mma(Frag &d, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d.lo.x), "+f"(d.lo.y), "+f"(d.hi.x), "+f"(d.hi.y)
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from a value a column.
__device__ __forceinline__ void mma_from(Frag &d, float2 c, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
        : "=f"(d.lo.x), "=f"(d.lo.y), "=f"(d.hi.x), "=f"(d.hi.y)
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y));
}
// The same from zero.
__device__ __forceinline__ void mma0(Frag &d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d.lo.x), "=f"(d.lo.y), "=f"(d.hi.x), "=f"(d.hi.y)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // (transpose8 of minf_warp_mma.cuh, free to move)
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
    const __half2 y = __hmul2_rn(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&y);
}
__device__ __forceinline__ float2 h2f(uint32_t a) { return __half22float2(*reinterpret_cast<const __half2 *>(&a)); }

// ----------------------------------------------------------------------------- the producers
// Producer warp pw takes every kProducers-th tile (and, the stages being a multiple of that, always the same stages), a
// lane a box of rows of K or V.  The boxes are wider than the rows by 16 bytes where that spreads the rows over
// the banks.  Boxes that no visible row lies in, or whose block is missing, are read past the map's end: zeros.  (Bulk
// copies of single rows, 64 a tile, took as many instructions as half of a tile's products: each is issued by itself.)
__device__ __forceinline__ void produce(unsigned char *ring, Meta &mt, const Params &P, int pw, int ctas) {
    const AttnParams &p = P.p;
    const Geo &g = P.g;
    const ChunkKv &c = p.a.c;
    const int lane = threadIdx.x & 31, boxes = g.kt / p.box_rows;  // at most 16
    const int is_v = lane >= boxes, box = is_v ? lane - boxes : lane;
    int n = 0, use = 0, mine = pw;  // tiles so far, uses of this warp's stages, its next tile
    Walk w;
    for (bool more = walk_begin<0>(w, p, ctas); more; more = walk_next<0>(w, p)) {
        const int scale0 = (c.W >> 1) + w.head * g.hg * (p.a.hd_kv >> 4);  // bytes to the group's scales
        for (; mine < n + (w.u1 - w.u0); mine += kProducers) {
            const int j = unit_tile(w.keys, w.u0 + mine - n) * g.kt + box * p.box_rows, st = mine % g.stages;
            long long row = c.rows;
            if (lane < 2 * boxes && item_sees_some(w.keys, j, p.box_rows)) {
                row = seq_row(c, w.rows, j);
                if (row < 0) {
                    if (!is_v) flag_error(p.a.err, MINF_ERRBIT_BLOCK);
                    row = c.rows;
                }
            }
            if (use >= g.stages / kProducers) {
                const int turn = mine / g.stages - 1;
                if (!__all_sync(0xffffffffu, ring_wait(&mt.empty[st], turn & 1, mt, p.a.err))) return;
            }
            ++use;
            if (lane == 0) mbar_expect_tx(&mt.full[st], 2 * g.side);
            __syncwarp();
            unsigned char *dst = ring + st * g.stage + is_v * g.side;
            if (lane < 2 * boxes) {
                tma_load_2d_stream(dst + box * p.box_rows * g.pitch, is_v ? &P.v : &P.k, g.whole ? 0 : w.head * (g.codes >> 3),
                                   static_cast<int>(row), &mt.full[st]);
                if (!g.whole)
                    tma_load_2d_stream(dst + g.scale_at + box * p.box_rows * g.scale_pitch, is_v ? &P.v_scales : &P.k_scales,
                                       (scale0 & ~15) >> 3, static_cast<int>(row), &mt.full[st]);
            }
            __syncwarp();
        }
        n += w.u1 - w.u0;
    }
}

// ----------------------------------------------------------------------------- the computing warps
template <int HD, bool PACK>
__device__ __forceinline__ void compute(const unsigned char *ring, float *join, Meta &mt, const Params &P, int ctas) {
    constexpr int NB = HD / 32, MT = HD / 16, NR = MT * 4;  // blocks, 16-dim tiles, outputs a lane
    constexpr int R = PACK ? 4 : 8;                         // query rows
    const AttnParams &p = P.p;
    const Geo &G = P.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n8 = lane >> 2, c4 = lane & 3;
    const int hl = warp % G.hg, part = warp / G.hg;  // head of the group, part of the keys
    const bool active = part < G.kp;
    const int g = p.a.nh / p.a.nk;
    const uint32_t sel = (n8 & 1) ? 0x7632u : 0x5410u;  // a lane's halves of V's words
    const size_t kPart = static_cast<size_t>(G.hg) * (8 * HD + 16);
    int st = 0, phase = 0;
    Walk w;
    for (bool more = walk_begin<0>(w, p, ctas); more; more = walk_next<0>(w, p)) {
        const int rows = w.cnt * g, tiles = w.u1 - w.u0, head = w.head * G.hg + hl;
        // Q: the lane's dims 32 b + 8 c4 .. + 7 of query n8 (of query n8 & 3, PACK), hi and lo
        constexpr int TERMS = PACK ? 1 : 2;
        uint32_t q[TERMS][NB][4];
        float2 off[TERMS][NB];  // - 8 sum q 2^-22 of a block, of queries 2 c4, 2 c4 + 1: what its products start from
        float cf[2];
        const long long at = static_cast<long long>(walk_row(w, p)) * p.a.nh + head * g;  // row of token 0, query head 0
        {
            const int r = n8 & (R - 1);
            const bool live = active && r < rows;
            const float *src = p.a.q + (at + static_cast<long long>(r / g) * p.a.nh + r % g) * p.a.hd + c4 * 8;
            float4 x[NB][2];
            float am = 0.0f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    x[b][h] = live ? __ldg(reinterpret_cast<const float4 *>(src + 32 * b) + h) : make_float4(0.f, 0.f, 0.f, 0.f);
                    am = fmaxf(am, fmaxf(fmaxf(fabsf(x[b][h].x), fabsf(x[b][h].y)), fmaxf(fabsf(x[b][h].z), fabsf(x[b][h].w))));
                }
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
            const int sh = row_shift(am);
            const float f = pow2i(sh);
            float sum[TERMS][NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int t = 0; t < TERMS; ++t) sum[t][b] = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 y = x[b][k >> 1];
                    uint32_t hi, lo;
                    split2(((k & 1) ? y.z : y.x) * f, ((k & 1) ? y.w : y.y) * f, hi, lo);
                    if (PACK && n8 >= 4) hi = lo;
                    const float2 a = h2f(hi);
                    sum[0][b] += a.x + a.y;
                    if constexpr (!PACK) {
                        const float2 e = h2f(lo);
                        sum[1][b] += e.x + e.y;
                    }
                    // codes four bits up count sixteen times
                    const uint32_t sixteenth = 0x2c002c00u;
                    q[0][b][k] = (k & 1) ? h2mul(hi, sixteenth) : hi;
                    if constexpr (!PACK) q[1][b][k] = (k & 1) ? h2mul(lo, sixteenth) : lo;
                }
#pragma unroll
                for (int t = 0; t < TERMS; ++t) {
                    sum[t][b] += __shfl_xor_sync(0xffffffffu, sum[t][b], 1);
                    sum[t][b] += __shfl_xor_sync(0xffffffffu, sum[t][b], 2);
                }
            }
            const float back = p.scale_log2 * pow2i(-sh);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int from = (2 * c4 + e) * 4;
                cf[e] = __shfl_sync(0xffffffffu, back, from) * 0x1p22f;
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
#pragma unroll
                    for (int b = 0; b < NB; ++b) (e ? off[t][b].y : off[t][b].x) = __shfl_sync(0xffffffffu, sum[t][b], from) * -0x1p-19f;
            }
        }
        float m[2] = {-INFINITY, -INFINITY};
        float2 l = make_float2(0.0f, 0.0f), acc[NR / 2];
#pragma unroll
        for (int r = 0; r < NR / 2; ++r) acc[r] = make_float2(0.0f, 0.0f);
        // Units [plain0, plain1): every row sees all of the warp's keys there (sinks' tiles apart).
        const long long first = walk_pos(w, p);
        int plain0, plain1;
        {
            const long long last = first + w.cnt - 1, all_hi = (first + 1 < w.rows.cap ? first + 1 : w.rows.cap) - part * kKeys;
            const long long all_lo = (p.a.window && last - p.a.window + 1 > 0 ? last - p.a.window + 1 : 0) - part * kKeys;
            const int from = w.keys.n_sink_tiles - w.keys.first_tile;  // a tile's unit
            plain0 = max(all_lo > 0 ? static_cast<int>((all_lo + G.kt - 1) / G.kt) : 0, w.keys.first_tile) + from;
            plain1 = (all_hi >= kKeys ? static_cast<int>((all_hi - kKeys) / G.kt) + 1 : 0) + from;
        }
        const int codes = hl * (HD / 2);
        const int scales = G.scale_at + (G.whole ? 0 : ((p.a.c.W >> 1) + w.head * G.hg * (HD / 16)) & 15) + hl * (HD / 16);
        const float2 c2 = make_float2(cf[0], cf[1]);
        for (int i = 0; i < tiles; ++i) {
            ring_wait(&mt.full[st], phase, mt, p.a.err);
            const bool plain = w.u0 + i >= plain0 && w.u0 + i < plain1;
            const int j0 = plain ? 0 : unit_tile(w.keys, w.u0 + i) * G.kt + part * kKeys;
            if (active && (plain || item_sees_some(w.keys, j0, kKeys))) {
                const unsigned char *kst = ring + st * G.stage, *vst = kst + G.side;
                const unsigned char *krow = kst + (part * kKeys + n8) * G.pitch + codes, *vrow = vst + (part * kKeys + 2 * c4) * G.pitch + codes;
                const unsigned char *ksc = kst + (part * kKeys + n8) * G.scale_pitch + scales, *vsc = vst + (part * kKeys + 2 * c4) * G.scale_pitch + scales;
                // ---- scales
                uint32_t ks[kSteps][2][NB / 2], vs[kSteps][4][NB / 2];  // of keys 16 s + n8 + 8 h; 16 s + 2 c4 (+ 1, + 8, + 9)
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) ld_scales<NB>(ksc + (16 * s + 8 * h) * G.scale_pitch, ks[s][h]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) ld_scales<NB>(vsc + (16 * s + (k & 1) + 8 * (k >> 1)) * G.scale_pitch, vs[s][k]);
                }
                if (!plain) {
                    asm volatile("" ::: "memory");  // (a branch: as predicated instructions this would run in every tile)
                    // V of rows that nobody sees: their weight is zero, but zero times what is not a number is not
                    auto dead = [&](int key) { return !item_sees(w.keys, j0 + key); };
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int b = 0; b < NB / 2; ++b) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) vs[s][k][b] = dead(16 * s + 2 * c4 + (k & 1) + 8 * (k >> 1)) ? 0 : vs[s][k][b];
                        }
                }
                // ---- scores
                // (in this order: every load, then every first product, every second one and the sums, so that each has
                // the others' time to arrive; lo's before hi's, in sums of their own)
                Frag x[kSteps], d[kSteps][NB];
                uint32_t y[kSteps][NB][2];
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int b = 0; b < NB; ++b) y[s][b][h] = ld32(krow + (16 * s + 8 * h) * G.pitch + b * 16 + c4 * 4);
#pragma unroll
                for (int t = TERMS - 1; t >= 0; --t) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int s = 0; s < kSteps; ++s)
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                const uint32_t y0 = h ? y[s][b][0] >> 6 : y[s][b][0] << 2, y1 = h ? y[s][b][1] >> 6 : y[s][b][1] << 2;
                                const uint32_t a[4] = {y0 & 0x003c003cu, y1 & 0x003c003cu, y0 & 0x03c003c0u, y1 & 0x03c003c0u};
                                if (h == 0)
                                    mma_from(d[s][b], off[t][b], a, q[t][b][0], q[t][b][1]);
                                else
                                    mma(d[s][b], a, q[t][b][2], q[t][b][3]);
                            }
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const float2 f0 = h2f(ks[s][0][b >> 1]), f1 = h2f(ks[s][1][b >> 1]);
                            const float s0 = (b & 1) ? f0.y : f0.x, s1 = (b & 1) ? f1.y : f1.x;
                            const bool first = t == TERMS - 1 && b == 0;
                            x[s].lo = first ? mul2(d[s][b].lo, both(s0)) : make_float2(fmaf(d[s][b].lo.x, s0, x[s].lo.x), fmaf(d[s][b].lo.y, s0, x[s].lo.y));
                            x[s].hi = first ? mul2(d[s][b].hi, both(s1)) : make_float2(fmaf(d[s][b].hi.x, s1, x[s].hi.x), fmaf(d[s][b].hi.y, s1, x[s].hi.y));
                        }
                }
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    if constexpr (PACK) {
                        x[s].lo = add2(x[s].lo, make_float2(__shfl_xor_sync(0xffffffffu, x[s].lo.x, 2), __shfl_xor_sync(0xffffffffu, x[s].lo.y, 2)));
                        x[s].hi = add2(x[s].hi, make_float2(__shfl_xor_sync(0xffffffffu, x[s].hi.x, 2), __shfl_xor_sync(0xffffffffu, x[s].hi.y, 2)));
                    }
                    x[s].lo = mul2(x[s].lo, c2);
                    x[s].hi = mul2(x[s].hi, c2);
                }
                // ---- softmax of the keys (lanes of one c4 share two rows)
                if (!plain) {
                    asm volatile("" ::: "memory");
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = (2 * c4 + e) & (R - 1);
                        const long long pos = first + r / g;
                        const long long hi = r < rows ? (pos + 1 < w.rows.cap ? pos + 1 : w.rows.cap) : 0;
                        const long long lo = p.a.window ? pos - p.a.window + 1 : 0;
                        auto hide = [&](float &y, int j) { y = j < hi && (j >= lo || j < p.a.n_sink) ? y : -INFINITY; };
#pragma unroll
                        for (int s = 0; s < kSteps; ++s) {
                            hide(e ? x[s].lo.y : x[s].lo.x, j0 + 16 * s + n8);
                            hide(e ? x[s].hi.y : x[s].hi.x, j0 + 16 * s + n8 + 8);
                        }
                    }
                }
                float mx[2] = {fmaxf(x[0].lo.x, x[0].hi.x), fmaxf(x[0].lo.y, x[0].hi.y)};
#pragma unroll
                for (int s = 1; s < kSteps; ++s) {
                    mx[0] = fmaxf(mx[0], fmaxf(x[s].lo.x, x[s].hi.x));
                    mx[1] = fmaxf(mx[1], fmaxf(x[s].lo.y, x[s].hi.y));
                }
                // The rows' maxima are needed across the lanes only where some score has grown past the slack, which is rare.
                // (m + slack is -infinity at first: any number is above it)
                if (__any_sync(0xffffffffu, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
                        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], o));
                    }
                    float2 corr = both(1.0f);
                    if (mx[0] > m[0] + kSlack) corr.x = ex2_approx(m[0] - mx[0]), m[0] = mx[0];
                    if (mx[1] > m[1] + kSlack) corr.y = ex2_approx(m[1] - mx[1]), m[1] = mx[1];
                    l = mul2(l, corr);
                    // (PACK: the lo halves of queries 2 c4, 2 c4 + 1 are in the lanes c4 ^ 2, which do the same)
#pragma unroll
                    for (int r = 0; r < NR / 2; ++r) acc[r] = mul2(acc[r], corr);
                }
                const float2 base = make_float2(m[0] == -INFINITY ? 0.0f : kShift - m[0], m[1] == -INFINITY ? 0.0f : kShift - m[1]);
                uint32_t ph[kSteps][2], pl[kSteps][2];
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float2 y = add2(h ? x[s].hi : x[s].lo, base);
                        y = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                        l = add2(l, y);
                        uint32_t hi, lo;
                        split2(y.x, y.y, hi, lo);
                        if constexpr (PACK) {
                            ph[s][h] = transposed(c4 >= 2 ? lo : hi);
                        } else {
                            ph[s][h] = transposed(hi);
                            pl[s][h] = transposed(lo);
                        }
                    }
                // ---- outputs
                uint32_t z[kSteps][NB][2];
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const unsigned char *from = vrow + (16 * s + 8 * k) * G.pitch + b * 16 + (n8 >> 1) * 4;
                            z[s][b][k] = __byte_perm(ld32(from), ld32(from + G.pitch), sel);
                        }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    Frag d0, d1;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        uint32_t a0[4], a1[4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t f = __byte_perm(vs[s][2 * k][b >> 1], vs[s][2 * k + 1][b >> 1], (b & 1) ? 0x7632u : 0x5410u);
                            uint32_t y[4];
                            q4_values(z[s][b][k], f, y);
                            a0[2 * k] = y[0], a0[2 * k + 1] = y[1];
                            a1[2 * k] = y[2], a1[2 * k + 1] = y[3];
                        }
                        const uint32_t(&p1)[2] = PACK ? ph[s] : pl[s];
                        if (s == 0) {
                            mma0(d0, a0[0], a0[1], a0[2], a0[3], p1[0], p1[1]);
                            mma0(d1, a1[0], a1[1], a1[2], a1[3], p1[0], p1[1]);
                        } else {
                            mma(d0, a0, p1[0], p1[1]);
                            mma(d1, a1, p1[0], p1[1]);
                        }
                        if constexpr (!PACK) {
                            mma(d0, a0, ph[s][0], ph[s][1]);
                            mma(d1, a1, ph[s][0], ph[s][1]);
                        }
                    }
                    // (added in rounded fp32: the tensor cores' own sums cut low bits off)
                    acc[4 * b] = add2(acc[4 * b], d0.lo);
                    acc[4 * b + 1] = add2(acc[4 * b + 1], d0.hi);
                    acc[4 * b + 2] = add2(acc[4 * b + 2], d1.lo);
                    acc[4 * b + 3] = add2(acc[4 * b + 3], d1.hi);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&mt.empty[st]);
            if (++st == G.stages) {
                st = 0;
                phase ^= 1;
            }
        }
        if (!active) continue;
        // ---- join: the head's warps, then the stretches
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l.x += __shfl_xor_sync(0xffffffffu, l.x, o);
            l.y += __shfl_xor_sync(0xffffffffu, l.y, o);
        }
        if constexpr (PACK) {
#pragma unroll
            for (int r = 0; r < NR / 2; ++r)
                acc[r] = add2(acc[r], make_float2(__shfl_xor_sync(0xffffffffu, acc[r].x, 2), __shfl_xor_sync(0xffffffffu, acc[r].y, 2)));
        }
        const int bar = 1 + hl, bar_threads = 32 * G.kp;
        if (part == 0 && lane < 8) mt.odd[hl][lane] = 0;
        __syncwarp();
        float *out = p.a.out + at * HD;
        bool odd = false;
        // pair r of a lane: dims 32 b + 8 (n8 / 2) + 2 i + n8 % 2, r = 4 b + i, of the queries 2 c4 and 2 c4 + 1
        float *row0 = nullptr, *row1 = nullptr;
        {
            const int r0 = 2 * c4, r1 = r0 + 1, d = 8 * (n8 >> 1) + (n8 & 1);
            if (r0 < R && r0 < rows) row0 = out + (static_cast<long long>(r0 / g) * p.a.nh + r0 % g) * HD + d;
            if (r1 < R && r1 < rows) row1 = out + (static_cast<long long>(r1 / g) * p.a.nh + r1 % g) * HD + d;
        }
        auto put = [&](int r, float2 y) {
            const int d = 32 * (r >> 2) + 2 * (r & 3);
            if (row0) row0[d] = y.x;
            if (row1) row1[d] = y.y;
            odd |= (row0 && !(fabsf(y.x) < INFINITY)) || (row1 && !(fabsf(y.y) < INFINITY));
            if (row0 && !(fabsf(y.x) < INFINITY)) mt.odd[hl][2 * c4] = 1;
            if (row1 && !(fabsf(y.y) < INFINITY)) mt.odd[hl][2 * c4 + 1] = 1;
        };
        // Every warp of the head calls to(r, pair) for its share of the pairs, over all of them; their m and l are the head's
        // by then (ready is called in between).
        auto join_warps = [&](auto &&to, auto &&ready) {
            if (G.kp == 1) {
                ready();
#pragma unroll
                for (int r = 0; r < NR / 2; ++r) to(r, acc[r]);
                return;
            }
            float2 *buf = reinterpret_cast<float2 *>(join) + lane;
            if (n8 == 0) {
                *reinterpret_cast<float2 *>(&mt.m[warp][2 * c4]) = make_float2(m[0], m[1]);
                *reinterpret_cast<float2 *>(&mt.l[warp][2 * c4]) = l;
            }
#pragma unroll
            for (int r = 0; r < NR / 2; ++r) buf[(warp * (NR / 2) + r) * 32] = acc[r];
            named_sync(bar, bar_threads);
            float2 f[kWarps];
            float M[2] = {-INFINITY, -INFINITY};
            for (int k = 0; k < G.kp; ++k) {
                const float2 mk = *reinterpret_cast<const float2 *>(&mt.m[hl + k * G.hg][2 * c4]);
                M[0] = fmaxf(M[0], mk.x);
                M[1] = fmaxf(M[1], mk.y);
            }
            l = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                f[k] = make_float2(0.0f, 0.0f);
                if (k >= G.kp) continue;
                const float2 mk = *reinterpret_cast<const float2 *>(&mt.m[hl + k * G.hg][2 * c4]), lk = *reinterpret_cast<const float2 *>(&mt.l[hl + k * G.hg][2 * c4]);
                // (a warp that saw nothing adds nothing, whatever it holds)
                if (mk.x != -INFINITY || lk.x != 0.0f) f[k].x = ex2_approx(mk.x - M[0]), l.x = fmaf(lk.x, f[k].x, l.x);
                if (mk.y != -INFINITY || lk.y != 0.0f) f[k].y = ex2_approx(mk.y - M[1]), l.y = fmaf(lk.y, f[k].y, l.y);
            }
            m[0] = M[0], m[1] = M[1];
            ready();
            for (int r = part; r < NR / 2; r += G.kp) {
                float2 y = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    if (k >= G.kp) continue;
                    const float2 x = buf[((hl + k * G.hg) * (NR / 2) + r) * 32];
                    y.x = f[k].x == 0.0f ? y.x : fmaf(x.x, f[k].x, y.x);
                    y.y = f[k].y == 0.0f ? y.y : fmaf(x.y, f[k].y, y.y);
                }
                to(r, y);
            }
        };
        // (a sum of zero, where a row sees nothing or nothing but scores of minus infinity, gives NaN here)
        auto finish = [&] {
            float2 inv;
            join_warps([&](int r, float2 y) { put(r, mul2(y, inv)); }, [&] { inv = make_float2(1.0f / l.x, 1.0f / l.y); });
        };
        if (w.u0 == 0 && w.u1 == w.keys.units) {
            finish();
        } else {
            // this stretch's part of the head: the outputs, then the rows' maxima and sums
            int b0, b1;
            walk_parts(w, p, b0, b1);
            const size_t head_part = static_cast<size_t>(hl) * (8 * HD + 16);
            auto part_of = [&](int b, bool starts) { return p.parts + (2 * static_cast<size_t>(b) + (starts ? 1 : 0)) * kPart + head_part; };
            float *mine = part_of(blockIdx.x, w.u0 == 0);
            join_warps([&](int r, float2 y) { reinterpret_cast<float2 *>(mine)[r * 32 + lane] = y; }, [] {});
            if (part == 0 && n8 == 0) {
                reinterpret_cast<float2 *>(mine + 8 * HD)[c4] = make_float2(m[0], m[1]);
                reinterpret_cast<float2 *>(mine + 8 * HD + 8)[c4] = l;
            }
            named_sync(bar, bar_threads);
            if (part == 0 && lane == 0) {
                __threadfence();  // (the head's whole part: the barrier ordered it before this)
                mt.last[hl] = atomicAdd(p.tickets + b0 * G.hg + hl, 1) == b1 - b0;
                __threadfence();
            }
            named_sync(bar, bar_threads);
            if (mt.last[hl]) {
                // the stretches' parts, dealt out to the head's warps in the order of their keys; a part's loads all in flight
                m[0] = m[1] = -INFINITY;
                l = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int r = 0; r < NR / 2; ++r) acc[r] = make_float2(0.0f, 0.0f);
#pragma unroll 1
                for (int b = b0 + part; b <= b1; b += G.kp) {
                    const float *from = part_of(b, b == b0);
                    const float2 mb = __ldcg(reinterpret_cast<const float2 *>(from + 8 * HD) + c4), lb = __ldcg(reinterpret_cast<const float2 *>(from + 8 * HD + 8) + c4);
                    float2 x[NR / 2];
#pragma unroll
                    for (int r = 0; r < NR / 2; ++r) x[r] = __ldcg(reinterpret_cast<const float2 *>(from) + r * 32 + lane);
                    float2 fo, fn;
                    auto factors = [](float &mo, float &lo, float mn, float ln, float &o, float &n) {
                        const bool none = mn == -INFINITY && ln == 0.0f, first = mo == -INFINITY && lo == 0.0f;
                        const float top = fmaxf(mo, mn);
                        o = first ? 0.0f : ex2_approx(mo - top);
                        n = none ? 0.0f : ex2_approx(mn - top);
                        lo = (first ? 0.0f : lo * o) + (none ? 0.0f : ln * n);
                        mo = top;
                    };
                    factors(m[0], l.x, mb.x, lb.x, fo.x, fn.x);
                    factors(m[1], l.y, mb.y, lb.y, fo.y, fn.y);
#pragma unroll
                    for (int r = 0; r < NR / 2; ++r) {
                        acc[r].x = acc[r].x * fo.x + (fn.x == 0.0f ? 0.0f : x[r].x * fn.x);
                        acc[r].y = acc[r].y * fo.y + (fn.y == 0.0f ? 0.0f : x[r].y * fn.y);
                    }
                }
                named_sync(bar, bar_threads);  // (the first join's buffer has been read)
                finish();
            }
        }
        // rows that are not finite: by the definition, a row a warp of the head
        const bool again = !named_all(bar, bar_threads, !odd);
        if (again) {
            if (lane == 0) atomicAdd(&mt.again, 1);
            attn_rows_again<Q4, HD>(p.a.c, mt.odd[hl], rows, part, G.kp, p.a.q + at * p.a.hd, out, g, p.a.nh, p.a.hd, w.rows,
                                    walk_pos(w, p), head, p.scale_log2, p.a.window, p.a.n_sink);
            __syncwarp();
            if (lane == 0) atomicSub(&mt.again, 1);
        }
        named_sync(bar, bar_threads);  // the join buffer is free
    }
}

template <int HD, bool PACK>
__global__ void __launch_bounds__(kThreads, 1) chunk_q4_kernel(const __grid_constant__ Params P) {
    extern __shared__ unsigned char smem_raw[];
    // the ring, the join buffer, the rest (all 128-byte pieces)
    const uint32_t base = (su32(smem_raw) + 127) & ~127u;
    unsigned char *smem = smem_raw + (base - su32(smem_raw));
    const int ring_bytes = P.g.stage * P.g.stages;
    float *join = reinterpret_cast<float *>(smem + ring_bytes);
    Meta &mt = *reinterpret_cast<Meta *>(smem + ring_bytes + kWarps * 8 * HD * 4);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < P.g.stages; ++i) {
            mbar_init(&mt.full[i], 1);
            mbar_init(&mt.empty[i], kWarps);
        }
        mt.abort_flag = 0;
        mt.again = 0;
        mbar_init_fence();
        prefetch_tensormap(&P.k);
        prefetch_tensormap(&P.v);
        if (!P.g.whole) {
            prefetch_tensormap(&P.k_scales);
            prefetch_tensormap(&P.v_scales);
        }
    }
    __syncthreads();
    gdc_wait();  // the plan, and everything before it
    const int ctas = P.p.head->ctas;
    if (warp < kWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
        compute<HD, PACK>(smem, join, mt, P, ctas);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp < kWarps + kProducers) produce(smem, mt, P, warp - kWarps, ctas);
    }
    if (*static_cast<volatile int *>(&mt.abort_flag)) {
        // a wait ran out: let copies in flight land before shared memory goes away
        const unsigned long long t0 = gtimer();
        while (gtimer() - t0 < kWaitBudgetNs / 4) {
        }
    }
}

// kv heads of an item: all, up to eight; else the largest divisor that keeps the most warps busy.
int group_heads(int nk) {
    if (nk <= kWarps) return nk;
    int best = 1;
    for (int h = 1; h <= kWarps; ++h)
        if (nk % h == 0 && h * (kWarps / h) >= best * (kWarps / best)) best = h;
    return best;
}

int meta_room(int hd_kv) { return kWarps * 8 * hd_kv * 4 + static_cast<int>(sizeof(Meta)) + 128; }

Geo geometry(const ChunkKv &c, int nk, int hd_kv) {
    Geo g = {};
    g.hg = group_heads(nk);
    g.kp = kWarps / g.hg;  // (8, 4, 2, 2, 1 ..: powers of two, so that tiles are whole blocks of a table, or blocks whole tiles)
    g.kt = kKeys * g.kp;
    g.whole = g.hg == nk;
    g.codes = g.hg * hd_kv / 2;
    // Rows an odd number of 16-byte pieces apart: lanes of eight neighbouring rows meet in no bank.
    const int row = g.whole ? static_cast<int>(c.row_bytes) : g.codes;
    g.pitch = row % 32 == 0 ? row + 16 : row;
    // (a group's scales start up to 12 bytes into a piece)
    g.scale_pitch = g.whole ? g.pitch : (g.hg * hd_kv / 16 + 12 + 15) / 16 * 16;
    g.scale_at = g.whole ? c.W / 2 : g.kt * g.pitch;
    g.side = g.kt * (g.whole ? g.pitch : g.pitch + g.scale_pitch);  // (a multiple of 512)
    g.stage = 2 * g.side;
    g.stages = (227 * 1024 - meta_room(hd_kv)) / g.stage;
    g.stages = g.stages >= kMostStages ? kMostStages : g.stages / kProducers * kProducers;
    return g;
}

template <int HD, bool PACK>
int launch(const Params &P, cudaStream_t s) {
    const int smem = P.g.stage * P.g.stages + meta_room(HD);
    if (P.g.stages < kProducers || smem > 227 * 1024) return MINF_ERR_UNSUPPORTED;  // (no geometry that the calls take)
    auto kernel = chunk_q4_kernel<HD, PACK>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess) return MINF_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sm_count());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? MINF_OK : MINF_ERR_CUDA;
}

int item_rows(int rows) { return rows <= 4 ? 4 : 8; }

PlanLayout q4_layout(int nt, int n_seq, int g, int hg, int hd_kv, int rows) {
    return plan_layout(nt, n_seq, item_rows(rows) / g, sm_count(), static_cast<size_t>(hg) * (8 * hd_kv + 16) * sizeof(float), hg);
}

}  // namespace

size_t chunk_q4_workspace(int nt, int n_seq, int nh, int nk, int hd_kv, int rows) {
    return q4_layout(nt, n_seq, nh / nk, group_heads(nk), hd_kv, rows).total;
}

void plan_chunk_q4(PlanArgs &plan, AttnParams &p, const ChunkAttnArgs &a, void *workspace, int rows, int most) {
    const int sms = sm_count(), g = a.nh / a.nk, hg = group_heads(a.nk);
    p = {};
    p.a = a;
    p.tt = item_rows(rows) / g;
    p.kt = kKeys * (kWarps / hg);
    p.heads = a.nk / hg;
    p.least = 1;
    p.most = most;
    p.scale_log2 = a.scale * kLog2e;
    p.box_rows = a.c.table && (1 << a.c.block_shift) < p.kt ? 1 << a.c.block_shift : p.kt;
    plan_args(plan, p, q4_layout(a.sq.nt, a.sq.n_seq, g, hg, a.hd_kv, rows), workspace, sms < kPlanMost ? sms : kPlanMost, 2, 1);
    plan.n_tickets = plan.max_ctas * hg;
    plan.join = kJoin * hg / kWarps;
}

int launch_chunk_q4(const AttnParams &p, int rows, cudaStream_t s) {
    Params P = {};
    P.p = p;
    P.g = geometry(p.a.c, p.a.nk, p.a.hd_kv);
    const bool pack = item_rows(rows) == 4;
    const ChunkKv &c = p.a.c;
    auto map = [&](CUtensorMap *m, const void *base, int box_bytes) {
        return make_tensor_map_2d(m, base, CU_TENSOR_MAP_DATA_TYPE_INT64, 8, static_cast<uint64_t>(c.row_bytes / 8),
                                  static_cast<uint64_t>(c.rows), static_cast<uint32_t>(box_bytes / 8), p.box_rows, false);
    };
    if (!map(&P.k, c.k, P.g.pitch) || !map(&P.v, c.v, P.g.pitch)) return MINF_ERR_CUDA;
    if (!P.g.whole && (!map(&P.k_scales, c.k, P.g.scale_pitch) || !map(&P.v_scales, c.v, P.g.scale_pitch))) return MINF_ERR_CUDA;
    if (p.a.hd_kv == 64) return pack ? launch<64, true>(P, s) : launch<64, false>(P, s);
    return pack ? launch<128, true>(P, s) : launch<128, false>(P, s);
}

}  // namespace minf
