// mq_attention_paged.cu -- attention of a serving step over many sequences at
// once: packed prompts (keys and values in the batch itself) and new tokens
// over a paged KV cache (BF16 in and out, FP32 softmax and accumulation).
//
//   o[t, h, :] = sum_{j <= pos(t)} softmax_j( q[t,h,:] . k[j,g,:] / sqrt(D) ) v[j,g,:],
//   g = h / (H / Hkv), j over the positions of t's own sequence.
//
// Rows of a tile.  The H / Hkv = G query heads of a KV head read the same keys,
// so a 128-row tile holds R = 128 / G tokens times G heads (one TMA box takes
// them out of the batch in that order): the keys cross shared memory once for
// all of them, and a causal tile wastes at most R + 127 positions.
//
// One persistent CTA per SM with two slots, each a 128-row tile with its own
// S / P (128 columns of tensor memory; P in BF16 over S) and O (128 columns):
// while one slot's softmax runs, the tensor cores work for the other.  An item
// of work is 2 R tokens of a sequence and a KV head: slot 0 takes the first R
// tokens, slot 1 the others, both over the same K / V tiles.  An item of at
// most R tokens (single tokens, draft tokens, the rest of a chunk) gives both
// slots the same queries and every other K / V tile; their two results are
// merged in the epilogue, so a decode step keeps two tiles in flight too.
//
// A slot takes a K / V tile as two halves of 64 keys with an S buffer each:
// P V of a half, then S of the next tile's same half over it, while the softmax
// is at the other half (8192-token prompt, in one run: 537 us; tiles of 128 keys
// at a time, where P, P V and the next S are one chain, 697 us; the halves cost
// the tensor cores 392 instead of 256 cycles for each S, as Q crosses shared
// memory twice).
//
// Warps: 0-3 / 4-7 softmax of slot 0 / 1 (a thread per row), 8-11 epilogue,
// 12 / 13 MMA issue of slot 0 / 1, 14 work list and TMA, 15 cleans V tiles.
//
// Roundings: P to BF16 for its product, o to BF16; scores, weights (2^x within
// 2^-22), maxima, sums and o's accumulation are FP32.  The sum that divides is of
// the unrounded weights: P's rounding then moves o by at most 2^-8 a, a = the
// weighted |v|, and o's own by 2^-8 |o|.  (Summed from the rounded ones, as the
// one-sequence attention does, a row with one dominant key is closer and the
// bound 2^-8 |o| wider; it took 567 to 583 instead of 545 to 550 us for the
// 8192-token prompt.)  The running maximum is raised for growths beyond 2^8
// only, which keeps weights below 2^8 and costs nothing in precision, as they are
// floating point.
//
// Cleaning: P is 0 at a masked key, but 0 x NaN is NaN, and what lies behind a
// sequence's last key (unwritten cache rows, another sequence, padding) may be
// anything.  V rows past the item's last key are zeroed in shared memory; a
// non-finite value of a new token (visible to some rows of the tile, masked
// for others) is zeroed too and added again, row by row, in the epilogue.
//
// Work.  Packed prompts: items sorted by length, heaviest first over all heads,
// taken from a counter (one head after the other ended with its long items:
// 617 against 573 us for 8192 tokens of 8 KV heads when that was tried, and no
// better where the keys of all heads are larger than L2).  Paged: the K / V
// tiles of all items in a row, cut into one range of equal cost per CTA; an
// item cut by a border leaves (max, sum, unnormalised o) of its parts, merged
// by a second kernel, so one long sequence fills the GPU as well as many do
// (merged by the CTA that ends last instead: 462 against 374 us for four chunks
// beside 60 single tokens when that was tried, its one SM reads the parts of up to
// 256 rows).
//
// What bounds it (rates of long runs, at 1000 W and 1.46 to 1.63 GHz; a few calls
// after a pause take 10 to 17% less).  Prompts and chunks: the hand-overs between
// softmax and products.  A half takes its softmax warp 1450 cycles among the
// others and 300 of waiting for S, the two slots' products 1300, so the tensor
// pipe does its products in half of the cycles (8192 tokens, 32 / 8 heads: 563
// us, 0.98 PFLOP/s; 16384 tokens over 49152: 16.7 ms, 0.92).  The power limit
// holds for any form and is not the reason by itself: what counts is this form's
// energy and cycles per tile (32768 tokens: 8.4 ms at 1.56 GHz, 8.2 without the
// exponentials, 7.0 for the products alone, without any softmax, at 1.63 GHz).
// Short prompts: 2.3 us from an item's last P to the next one's first S
// and its epilogue of 2 us a slot (16 prompts of 64 to 4096 tokens, 64 / 8
// heads: 464 us, 0.71 PFLOP/s).  Single tokens: the cache's bytes (64 of 512 to
// 8192 positions, 667 MB: 143 us, 4.7 TB/s, of which the list kernel and the
// merge take 11; one of 32768 39 us, 3.4 TB/s; one of 8192 23 us, of which the
// two other kernels take 8).
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "mq_internal.h"
#include "mq_ptx.cuh"

namespace mq {

namespace {

constexpr int kD = 128;
constexpr int kRows = 128;                          // rows of a slot's tile
constexpr int kKeys = 128;                          // keys of a K / V tile
constexpr uint32_t kTileBytes = 128 * kD * 2;       // 32 KB: a Q, K or V tile
constexpr int kRing = 5;                            // K / V tiles in flight or in use
constexpr int kWork = 4;                            // items known ahead
constexpr uint32_t kQOff = 0;                       // a Q tile per slot
constexpr uint32_t kRingOff = 2 * kTileBytes;
constexpr uint32_t kStatOff = kRingOff + kRing * kTileBytes;     // [2 slots][max, sum][128] floats
constexpr uint32_t kWorkOff = kStatOff + 2 * 2 * kRows * 4;      // [kWork] items
constexpr uint32_t kBarOff = kWorkOff + kWork * 64;
constexpr uint32_t kSmemBytes = kBarOff + 592;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512;                 // S0, S1, O0, O1
constexpr uint32_t kOCol = 256;
// log2(e) / sqrt(128): scores in the base-2 exponent domain
constexpr float kScaleLog2 = 0.12751743082459868f;
constexpr float kRescaleThreshold = 8.0f;           // raise the running max past 2^8 growth only

// Barriers, 8 bytes each.  A wait names the parity of a phase, so the phase
// before must be known to be complete and the one after must not complete
// until the wait is over.  The
// slots do not read the same K / V tiles (a dual item's take turns, a slot may
// need one tile less), so a stage has a barrier for the tiles that both read
// and one for those of either alone (sets 0, 1, 2).
enum : uint32_t {
    kBarWorkFull = 0,                       // [kWork]
    kBarWorkEmpty = kBarWorkFull + kWork,   // [kWork]
    kBarQFull = kBarWorkEmpty + kWork,      // [2]
    kBarQEmpty = kBarQFull + 2,             // [2]
    kBarKFull = kBarQEmpty + 2,             // [3][kRing] a K tile has landed
    kBarVFull = kBarKFull + 3 * kRing,      // [kRing] a V tile has (seen by the cleaner)
    kBarKvEmpty = kBarVFull + kRing,        // [kRing]
    kBarClean = kBarKvEmpty + kRing,        // [3][kRing] the V tile may be read
    kBarSFull = kBarClean + 3 * kRing,      // [2 slots][2 halves]
    kBarPFull = kBarSFull + 4,              // [2][2]
    kBarPvDone = kBarPFull + 4,             // [2] every P V product but an item's last
    kBarOFull = kBarPvDone + 2,             // [2] an item's last one
    kBarOEmpty = kBarOFull + 2,             // [2]
    kBarStatFull = kBarOEmpty + 2,          // [2]
    kBarStatEmpty = kBarStatFull + 2,       // [2]
    kBarDrain = kBarStatEmpty + 2,          // [2]
    kBarCount = kBarDrain + 2
};
static_assert(kBarCount * 8 + 16 <= 592, "barriers, TMEM address and abort flag");

// One entry of the work list: up to 2 R tokens of a sequence.
struct Entry {
    int row0;      // batch row of the first token
    int ntok;
    int pos0;      // its position
    int kv;        // packed: batch row of position 0; paged: row of the block table
};

struct alignas(16) Item {
    Entry e;
    int g, t0, t1;       // KV head; K / V tiles [t0, t1) of it
    int kv_len;          // keys from here on do not exist for this item
    int c[2];            // tiles of each slot
    int dual;            // both slots have the same queries and take turns at the tiles
    int part;            // < 0: the whole item, write o; else the partial result's place
    int last;            // no item: end of work
    int bad;             // set by the cleaner: a new token's V is not finite
};
static_assert(sizeof(Item) <= 64, "work ring entry");

// A CTA's range of the paged work: its first item, and the item that begins in
// the range and goes on past it (what the second kernel merges).
struct alignas(16) Range {
    Entry first;
    int e, g, t0;        // entry, KV head and first tile of the first item
    int end_e, end_g, end_t;     // where the range ends (before that tile)
    Entry cut;
    int cut_g, cut_to;   // its KV head and the CTA that ends it (0: no such item)
};

struct Header {          // start of the workspace
    int n_ent;
    int counter;         // packed: next item
};

struct Params {
    PagedAttnArgs a;
    int R, G;            // tokens and heads of a tile
    int max_ent;
    Header *head;
    Entry *ent;
    int64_t *prefix;     // [n_ent + 1] tiles before each entry (paged, work list kernel only)
    Range *ranges;       // [grid] (paged)
    int grid;            // CTAs of the attention
    int self;            // the CTAs find their work themselves (few sequences, see launch_kind)
    float *part;         // [2 grid][part_rows](max, sum) then [part_rows][128]
    int part_rows;
    int wide;            // o's rows are aligned to 32 bytes
    unsigned *err;
};

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

// the three-input maximum that keeps a NaN
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// 2^x of a pair on the FMA and integer pipes: x = n + f with n the nearest
// integer (read from the low bits of x + 1.5 2^23), 2^f by the quintic 1 + f (...)
// of least relative error on [-0.5, 0.5] (9.1e-8, fitted here by Lawson
// iteration; 2^-22 with the roundings, as the transcendental unit's), n added to
// the exponent.  From -127 down (masked scores): exactly 0, as 2^0 is exactly 1;
// between -127 and -126 something below 2^-126.  x < 128.
__device__ __forceinline__ void exp2_pair_fma(uint64_t x, float &y0, float &y1) {
    float x0, x1;
    unpack2(x, x0, x1);
    x = pack2(fmaxf(x0, -127.0f), fmaxf(x1, -127.0f));
    const uint64_t t = fadd2(x, pack2(12582912.0f, 12582912.0f));
    const uint64_t n = fadd2(t, pack2(-12582912.0f, -12582912.0f));
    const uint64_t f = ffma2(n, pack2(-1.0f, -1.0f), x);
    auto twice = [](float c) { return pack2(c, c); };
    uint64_t p = ffma2(f, twice(0.001326472731307149f), twice(0.009671512991189957f));
    p = ffma2(p, f, twice(0.05550733581185341f));
    p = ffma2(p, f, twice(0.24022242426872253f));
    p = ffma2(p, f, twice(0.6931470036506653f));
    p = ffma2(p, f, twice(1.0f));
    float t0, t1, p0, p1;
    unpack2(t, t0, t1);
    unpack2(p, p0, p1);
    y0 = __uint_as_float((__float_as_uint(t0) << 23) + __float_as_uint(p0));
    y1 = __uint_as_float((__float_as_uint(t1) << 23) + __float_as_uint(p1));
}

// Weights of 32 scores to the base 2^-nm as BF16 pairs, their sum (of the
// unrounded weights) added to lp.  Of each 16 pairs kExpFma take the FMA pipes:
// the transcendental unit (16 a clock per SM) needs as long for a tile's
// exponentials as the tensor cores for its products.  Measured with 0 / 2 / 3 /
// 4 / 5 of 16, back to back and in turns: 8192-token prompt 581 / 562 / 559 /
// 549 / 553 us, ragged prompts 454 / 449 / 450 / 451 / 463 us, chunks beside
// single tokens 396 / 386 / 386 / 391 / 405 us, 64 single tokens 129 / 129 / 131
// / 130 / 134 us (2% is within the spread: some gain, its share does not matter
// much).
constexpr int kExpFma = 4;
__device__ __forceinline__ void weights32(const float *s, float nm, uint32_t (&pk)[16], uint64_t (&lp)[2]) {
    const uint64_t sc2 = pack2(kScaleLog2, kScaleLog2), nm2 = pack2(nm, nm);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const uint64_t x = ffma2(pack2(s[2 * k], s[2 * k + 1]), sc2, nm2);
        float y0, y1;
        if ((k + 1) * kExpFma / 16 > k * kExpFma / 16) {
            exp2_pair_fma(x, y0, y1);
        } else {
            unpack2(x, y0, y1);
            y0 = ex2_approx(y0);
            y1 = ex2_approx(y1);
        }
        lp[k & 1] = fadd2(lp[k & 1], pack2(y0, y1));
        const __nv_bfloat162 pb = __floats2bfloat162_rn(y0, y1);
        pk[k] = *reinterpret_cast<const uint32_t *>(&pb);
    }
}

// Bounded wait on a barrier's phase.  The first polls look at no clock: each
// try_wait already suspends the warp for a while, and reading %globaltimer
// after one failed poll cost more than the handover itself (with no product
// and no softmax at all, the barriers alone took 1700 cycles a tile).
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int *abort, unsigned *err) {
    unsigned long long t0 = 0;
#pragma unroll 1
    for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i) {
        if ((i & 127u) != 127u) continue;
        if (*abort) return false;
        const unsigned long long t = global_timer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitLimitNs) {
            atomicOr(err, kDevErrTimeout);
            *abort = 1;
            return false;
        }
    }
    return true;
}
// (draining after the error is latched already)
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > kWaitLimitNs) return false;
    return true;
}
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 32 lanes x 16 consecutive 32-bit columns into registers
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// box {64 columns, G heads, tokens, 1} of the queries
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// 32 bytes in one store where the rows are aligned to that: a warp writes a
// piece of 32 rows at a time, a line each, whatever a piece's size
__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8], int wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// 128-byte-swizzled operand descriptor (see mq_ptx.cuh) with both byte offsets
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
           static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1u) << 46 |
           static_cast<uint64_t>(2u) << 61;
}

// Eight chained BF16 MMAs (K = 16 each) issued by one elected lane of a
// converged warp: kept warp-wide so that the operands stay in uniform
// registers (from a single-lane branch the same eight took ~1100 cycles).
// D (+)= A B^T with A, B K-major; kHalfB: 16-byte units between B's column halves
template <uint32_t kHalfB>
__device__ __forceinline__ void warp_mma8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t"
        ".reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n\t"
        "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\tadd.s64 a4, %1, 1024;\n\t"
        "add.s64 a5, %1, 1026;\n\tadd.s64 a6, %1, 1028;\n\tadd.s64 a7, %1, 1030;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\tadd.s64 b4, %2, %4;\n\t"
        "add.s64 b5, %2, %5;\n\tadd.s64 b6, %2, %6;\n\tadd.s64 b7, %2, %7;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, t;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "n"(kHalfB), "n"(kHalfB + 2), "n"(kHalfB + 4), "n"(kHalfB + 6)
        : "memory");
}
// Four of them, D (+)= A B with A in tensor memory (8 columns a step), B
// MN-major; kStep: 16-byte units between B's 16-row steps
template <uint32_t kStep>
__device__ __forceinline__ void warp_mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t"
        ".reg .b32 a1, a2, a3;\n\t"
        ".reg .b64 b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
        "add.s64 b1, %2, %5;\n\tadd.s64 b2, %2, %6;\n\tadd.s64 b3, %2, %7;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(kStep), "n"(2 * kStep), "n"(3 * kStep)
        : "memory");
}
__device__ __forceinline__ void warp_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// Where a K / V tile's rows lie in shared memory: 8-row groups of 1 KB per
// 64-column half.  Packed (one box of 128 rows per half): the groups of a half
// lie together.  Paged (a box per page, [group][half][8 rows]): the halves of
// a group lie together, so a page of any size lands in the same tile layout.
template <bool kPaged>
struct Layout {
    static constexpr uint32_t kGroup = kPaged ? 2048 : 1024;
    static constexpr uint32_t kHalf = kPaged ? 1024 : 16384;
    // byte offset of 16-byte chunk c (0..15) of row k (128-byte swizzle)
    __device__ static __forceinline__ uint32_t chunk(int k, int c) {
        return (k >> 3) * kGroup + (c >> 3) * kHalf + (k & 7) * 128 + (((c & 7) ^ (k & 7)) << 4);
    }
};

__device__ __forceinline__ int64_t range_begin(int64_t W, int c, int n) { return W * c / n; }

// K / V tiles of an entry, one at least (an entry has a token, and a table row a
// page); cap: positions that a table row has pages for.
__device__ __forceinline__ int entry_tiles(const Entry &e, int64_t cap) {
    return static_cast<int>((min(static_cast<int64_t>(e.pos0) + e.ntok, cap) + kKeys - 1) / kKeys);
}

// Cost of one of an entry's tiles, and of an item besides its tiles, in eighths
// of a tile that one slot takes while the other takes the next.  Measured over
// the CTAs of four chunks beside 60 single tokens: 2.1 us a tile with queries in
// both slots, 1.3 us a tile that they share, 2 and 2.8 us an item (its first
// loads and its epilogue).  These are times of the CTA's work on a tile, whatever
// the heads and pages: such a step takes, with these costs / with 2 : 1, 7 : 4 and
// 1 : 1 for the tiles alone, 376 / 429 / 412 / 454 us (32 / 8 heads, pages of 16),
// 235 / 257 / 249 / 294 (8 / 8 heads), 1376 / 1593 / 1470 / 1450 (64 / 8 heads,
// pages of 64), 441 / 499 / 470 / 437 (32 / 8 heads, pages of 8: more boxes a
// tile); two small chunks beside 98 tokens 106 / 120 / 116 / 112; 64 single
// tokens 144 / 148 / 148 / 147.
constexpr int kCostTwo = 13, kCostOne = 8, kCostItemTwo = 12, kCostItemOne = 18;
__device__ __forceinline__ int tile_cost(const Entry &e, int R) { return e.ntok > R ? kCostTwo : kCostOne; }
__device__ __forceinline__ int item_cost(const Entry &e, int R) { return e.ntok > R ? kCostItemTwo : kCostItemOne; }

// V of a new token i of the entry (for the rows that a cleaned value belongs to)
template <bool kPaged>
__device__ const __nv_bfloat16 *new_value_row(const Params &p, const Item &w, int pos) {
    if (!kPaged)
        return p.a.qkv + static_cast<int64_t>(w.e.kv + pos) * p.a.ldqkv + (p.a.H + p.a.Hkv + w.g) * kD;
    const int id = p.a.table[static_cast<int64_t>(w.e.kv) * p.a.max_pages + (pos >> p.a.ps_shift)];
    if (id < 0 || id >= p.a.n_pages) return nullptr;
    return p.a.v_pages +
           (((static_cast<int64_t>(id) * p.a.Hkv + w.g) << p.a.ps_shift) + (pos & ((1 << p.a.ps_shift) - 1))) * kD;
}

// The new tokens' K and V rows to their slots, one warp per token and KV head
// at a time (16 lanes for K, 16 for V): rows w, w + n, .. of `total`, kAppend of
// them in flight a call.
constexpr int kAppend = 4;
__device__ __forceinline__ int64_t append_total(const PagedAttnArgs &a) {
    return static_cast<int64_t>(max(min(a.T, a.cu[a.B]), 0)) * a.Hkv;
}
__device__ __forceinline__ void append_rows(const PagedAttnArgs &a, int64_t w, int64_t n, int64_t total, int lane) {
    const int64_t n_slots = a.n_pages << a.ps_shift;
    uint4 v[kAppend];
    int64_t dst[kAppend];
#pragma unroll
    for (int u = 0; u < kAppend; ++u) {
        dst[u] = -1;
        const int64_t x = w + u * n;                // (< 2^32)
        if (x >= total) continue;
        const unsigned t = static_cast<unsigned>(x) / a.Hkv, g = static_cast<unsigned>(x) % a.Hkv;
        const int64_t slot = a.slots[t];
        if (slot < 0 || slot >= n_slots) continue;
        dst[u] = ((((slot >> a.ps_shift) * a.Hkv + g) << a.ps_shift) + (slot & ((1 << a.ps_shift) - 1))) * kD;
        v[u] = reinterpret_cast<const uint4 *>(a.qkv + t * a.ldqkv + (a.H + g) * kD +
                                               (lane < 16 ? 0 : a.Hkv * kD))[lane & 15];
    }
#pragma unroll
    for (int u = 0; u < kAppend; ++u)
        if (dst[u] >= 0)
            reinterpret_cast<uint4 *>((lane < 16 ? a.k_pages : a.v_pages) + dst[u])[lane & 15] = v[u];
}

// ---- the work list -----------------------------------------------------------------

constexpr int kMaxCtas = 160;       // the launch uses no more: ranges and partial results have this many places
constexpr int kPrepThreads = 1024;
constexpr int kBins = 4096;
constexpr int kFewSums = 1024;

// Exclusive prefix sum over the block; *total gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *red, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t s = red[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += y;
        }
        red[lane] = s;
    }
    __syncthreads();
    *total = red[31];
    const int64_t r = x - v + (warp ? red[warp - 1] : 0);
    __syncthreads();
    return r;
}

// Block 0 makes the work list; with a paged cache the other blocks meanwhile
// write the new tokens' rows to it (packed prompts: the attention kernel does,
// as nothing there reads the cache).  A few KB of lengths in one block's scans
// and searches: latency, 4 us for one sequence to 8 us for 64; the rows are
// copied in the same time (3349 tokens of 8 KV heads, 27 MB: 12 us cold).
template <bool kPaged>
__global__ void __launch_bounds__(kPrepThreads) paged_prep_kernel(const Params p) {
    extern __shared__ int offs[];                  // [B + 1] entries before each sequence; packed: then kBins bins
    __shared__ int64_t red[32];
    const int tid = threadIdx.x, lane = tid & 31;
    const PagedAttnArgs &a = p.a;
    griddep_wait();
    griddep_launch_dependents();
    if (kPaged && blockIdx.x > 0) {
        const int64_t n = static_cast<int64_t>(gridDim.x - 1) * (kPrepThreads / 32), total = append_total(a);
        for (int64_t w = static_cast<int64_t>(blockIdx.x - 1) * (kPrepThreads / 32) + (tid >> 5); w < total; w += kAppend * n)
            append_rows(a, w, n, total, lane);
        return;
    }
    const int TB = 2 * p.R;
    auto tokens = [&](int b) {                     // rows of sequence b, whatever cu holds
        const int lo = min(max(a.cu[b], 0), a.T), hi = min(max(a.cu[b + 1], 0), a.T);
        return min(max(hi - lo, 0), a.max_new);
    };
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPrepThreads) {
        const int b = b0 + tid;
        int64_t total;
        const int64_t at = block_scan(b < a.B ? (tokens(b) + TB - 1) / TB : 0, red, &total);
        if (b < a.B) offs[b] = static_cast<int>(min(base + at, static_cast<int64_t>(p.max_ent)));
        base += total;
    }
    const int n_ent = static_cast<int>(min(base, static_cast<int64_t>(p.max_ent)));
    if (tid == 0) {
        offs[a.B] = n_ent;
        p.head->n_ent = n_ent;
        p.head->counter = 0;
        if (a.o_amax) *a.o_amax = 0.0f;
    }
    __syncthreads();
    const int64_t cap = kPaged ? static_cast<int64_t>(a.max_pages) << a.ps_shift : INT32_MAX;
    auto entry = [&](int e, int &tiles) {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (offs[mid] <= e) lo = mid; else hi = mid;
        }
        const int first = (e - offs[lo]) * TB;
        const int start = min(max(a.cu[lo], 0), a.T);
        const int ctx = kPaged ? min(max(a.ctx[lo], 0), 1 << 30) : 0;
        Entry r;
        r.row0 = start + first;
        r.ntok = min(tokens(lo) - first, TB);
        r.pos0 = ctx + first;
        r.kv = kPaged ? lo : start;
        tiles = entry_tiles(r, cap);
        return r;
    };
    if (kPaged) {
        // (the search for the borders reads few sums from shared memory)
        __shared__ int64_t few[kFewSums];
        int64_t *const pre = n_ent < kFewSums ? few : p.prefix;
        int64_t at0 = 0;
        for (int e0 = 0; e0 < n_ent; e0 += kPrepThreads) {
            const int e = e0 + tid;
            int tiles = 0, cost = 0;
            if (e < n_ent) {
                const Entry r = entry(e, tiles);
                p.ent[e] = r;
                cost = item_cost(r, p.R) + tiles * tile_cost(r, p.R);
            }
            int64_t total;
            const int64_t at = block_scan(cost, red, &total);
            if (e < n_ent) pre[e] = at0 + at;
            at0 += total;
        }
        if (tid == 0) pre[n_ent] = at0;
        __syncthreads();
        // the ranges: equal shares of the cost of all entries and heads; a border
        // inside an entry falls on its next whole tile
        const int64_t W = at0 * a.Hkv;
        // (a share holds one whole tile at least, so no range inside an item is
        // empty; one between items may be)
        const int64_t most = min(W, max(W / (a.max_new > p.R ? kCostTwo : kCostOne), static_cast<int64_t>(1)));
        const int n = static_cast<int>(min(most, static_cast<int64_t>(p.grid)));
        struct Place {
            int e, g, t;                         // the tile that a border falls on
        };
        auto locate = [&](int c) {
            const int64_t w = range_begin(W, c, n);
            Place r;
            r.g = static_cast<int>(w / at0);
            const int64_t y = w - r.g * at0;
            int lo = 0, hi = n_ent;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (pre[mid] <= y) lo = mid; else hi = mid;
            }
            r.e = lo;
            const Entry en = p.ent[lo];
            const int u = tile_cost(en, p.R);
            r.t = static_cast<int>(max((y - pre[lo] - item_cost(en, p.R) + u - 1) / u, static_cast<int64_t>(0)));
            if (r.t >= entry_tiles(en, cap)) {   // the entry's end: the next one
                r.t = 0;
                if (++r.e == n_ent) {
                    r.e = 0;
                    ++r.g;
                }
            }
            return r;
        };
        __shared__ Place border[kMaxCtas + 1];
        for (int c = tid; c <= n; c += kPrepThreads) border[c] = c < n ? locate(c) : Place{0, a.Hkv, 0};
        __syncthreads();
        for (int c = tid; c < p.grid; c += kPrepThreads) {
            Range r = {};
            if (c < n) {
                const Place lo = border[c], hi = border[c + 1];
                r.e = lo.e;
                r.g = lo.g;
                r.t0 = lo.t;
                if (lo.g < a.Hkv) r.first = p.ent[lo.e];
                r.end_e = hi.e;
                r.end_g = hi.g;
                r.end_t = hi.t;
                // an item cut by the far border that begins in this range
                if (hi.t > 0 && (hi.g != lo.g || hi.e != lo.e || lo.t == 0)) {
                    r.cut = p.ent[hi.e];
                    r.cut_g = hi.g;
                    // the first border past its last tile's start, less one
                    const int u = tile_cost(r.cut, p.R);
                    const int64_t x = hi.g * at0 + pre[hi.e] + item_cost(r.cut, p.R) +
                                      static_cast<int64_t>(entry_tiles(r.cut, cap) - 1) * u + 1;
                    r.cut_to = static_cast<int>(min((x * n + W - 1) / W, static_cast<int64_t>(n))) - 1;
                }
            } else {
                r.g = r.end_g = a.Hkv;
            }
            p.ranges[c] = r;
        }
    } else {
        // counting sort by tiles, most first (the order within a bin does not
        // matter: every item's result is its own)
        int *bins = offs + a.B + 1;
        for (int i = tid; i < kBins; i += kPrepThreads) bins[i] = 0;
        __syncthreads();
        int shift = 0;
        while (((a.T + kKeys - 1) / kKeys >> shift) >= kBins) ++shift;
        for (int e = tid; e < n_ent; e += kPrepThreads) {
            int tiles;
            entry(e, tiles);
            atomicAdd(&bins[kBins - 1 - (tiles >> shift)], 1);
        }
        __syncthreads();
        constexpr int kPer = kBins / kPrepThreads;
        int64_t sum = 0, total;
        for (int i = 0; i < kPer; ++i) sum += bins[tid * kPer + i];
        int64_t at = block_scan(sum, red, &total);
        for (int i = 0; i < kPer; ++i) {
            const int n = bins[tid * kPer + i];
            bins[tid * kPer + i] = static_cast<int>(at);
            at += n;
        }
        __syncthreads();
        for (int e = tid; e < n_ent; e += kPrepThreads) {
            int tiles;
            const Entry r = entry(e, tiles);
            p.ent[atomicAdd(&bins[kBins - 1 - (tiles >> shift)], 1)] = r;
        }
    }
}

// ---- the attention ---------------------------------------------------------------------

// The work of a packed call with at most 32 sequences and at most one item a
// CTA, found by the loading warp of each CTA itself (a lane holds a sequence);
// spares the list kernel.
struct SelfPlan {
    int row0, ntok, pre, size;       // size: blocks of 2 R tokens; pre: of the sequences before

    // returns the blocks of all sequences
    __device__ __forceinline__ int take(const Params &p, int lane) {
        const PagedAttnArgs &a = p.a;
        row0 = ntok = size = 0;
        if (lane < a.B) {
            row0 = min(max(a.cu[lane], 0), a.T);
            ntok = max(min(max(a.cu[lane + 1], 0), a.T) - row0, 0);
            size = (ntok + 2 * p.R - 1) / (2 * p.R);
        }
        int x = size;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        pre = x - size;
        return __shfl_sync(0xFFFFFFFFu, x, 31);
    }
    __device__ __forceinline__ Entry block(int i, int tokens) const {
        const int b = 31 - __clz(__ballot_sync(0xFFFFFFFFu, size > 0 && pre <= i) | 1u);
        const int first = (i - __shfl_sync(0xFFFFFFFFu, pre, b)) * tokens, start = __shfl_sync(0xFFFFFFFFu, row0, b);
        return Entry{start + first, min(__shfl_sync(0xFFFFFFFFu, ntok, b) - first, tokens), first, start};
    }
};

// (bounds, rates and the roles of the warps: at the top of the file)
template <bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = Layout<kPaged>;
    const uint32_t s0 = smem_u32(smem);
    const uint32_t bar = s0 + kBarOff;
    auto B = [&](uint32_t i) { return bar + 8 * i; };
    Item *items = reinterpret_cast<Item *>(smem + kWorkOff);
    float *stat = reinterpret_cast<float *>(smem + kStatOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kBarOff + kBarCount * 8);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + kBarOff + kBarCount * 8 + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.G, R = p.R;
    unsigned *err = p.err;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kWork; ++i) {
            mbar_init(B(kBarWorkFull + i), 1);
            mbar_init(B(kBarWorkEmpty + i), 8 + 4 + 2 + 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(B(kBarVFull + i), 1);
            mbar_init(B(kBarKvEmpty + i), 2);
        }
        for (int i = 0; i < 3 * kRing; ++i) {
            mbar_init(B(kBarKFull + i), 1);
            mbar_init(B(kBarClean + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(B(kBarQFull + i), 1);
            mbar_init(B(kBarQEmpty + i), 1);
            mbar_init(B(kBarPvDone + i), 1);
            mbar_init(B(kBarOFull + i), 1);
            for (int x = 0; x < 2; ++x) {
                mbar_init(B(kBarSFull + 2 * i + x), 1);
                mbar_init(B(kBarPFull + 2 * i + x), 4);
            }
            mbar_init(B(kBarOEmpty + i), 4);
            mbar_init(B(kBarStatFull + i), 4);
            mbar_init(B(kBarStatEmpty + i), 4);
            mbar_init(B(kBarDrain + i), 1);
        }
        fence_barrier_init();
        *abort = (s0 & 1023u) != 0;          // the tiles' swizzle needs 1 KB alignment
        if (s0 & 1023u) atomicOr(err, kDevErrTimeout);
        prefetch_tmap(&tmap_q);
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    if (warp == 12) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch_dependents();
    const bool dead = *abort != 0;

    auto wait = [&](uint32_t b, uint32_t parity) { return wait_phase(b, parity, abort, err); };

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        const int s = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t tS = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + s * 128u;
        const uint32_t tO = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kOCol + s * 128u;
        const int tok_r = r / G;
        uint32_t n_f[2] = {0, 0};               // phases seen of the two S buffers
        uint32_t n_pv = 0, n_o = 0;             // products and items with tiles before this item
        bool ok = !dead;
        for (uint32_t it = 0; ok; ++it) {
            const uint32_t wi = it % kWork;
            ok = __all_sync(0xFFFFFFFFu, wait(B(kBarWorkFull + wi), (it / kWork) & 1));
            if (!ok || items[wi].last) break;
            const Item &w = items[wi];
            const int dual = w.dual, c = w.c[s], t0 = w.t0;
            const int first = dual ? 0 : s * R;                  // the slot's first token
            const int mine = first + tok_r;
            const bool valid = r < R * G && mine < w.e.ntok;
            const int lim = min(w.e.pos0 + mine, w.kv_len - 1);  // the last key of this row
            const int free_to = min(w.e.pos0 + first, w.kv_len - 1);   // every row of the slot sees keys up to here
            const bool busy = __any_sync(0xFFFFFFFFu, valid);
            float m = -INFINITY, l = 0.0f;
            for (int u = 0; u < 2 * c; ++u) {
                // half x of the slot's tile i: 64 keys, its own S and P
                const int i = u >> 1, x = u & 1, j = dual ? t0 + s + 2 * i : t0 + i;
                const uint32_t tX = tS + 64u * x;
                ok = __all_sync(0xFFFFFFFFu, wait(B(kBarSFull + 2 * s + x), n_f[x]++ & 1));
                if (!ok) break;
                if (!busy) {                    // no row of this warp is in the item: P may be anything
                    if (lane == 0) mbar_arrive(B(kBarPFull + 2 * s + x));
                    continue;
                }
                tc_fence_after();
                uint32_t sr[64];
#pragma unroll
                for (int q = 0; q < 2; ++q) tmem_ld32(tX + 32u * q, *reinterpret_cast<uint32_t (*)[32]>(&sr[32 * q]));
                tmem_ld_wait();
                float *sf = reinterpret_cast<float *>(sr);
                const int key0 = j * kKeys + 64 * x;
                if (key0 + 63 > free_to) {
                    const int last = lim - key0;
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (k > last) sf[k] = -INFINITY;
                }
                float mp[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) mp[e] = fmax3_nan(sf[e], sf[8 + e], sf[16 + e]);
#pragma unroll
                for (int k = 24; k < 56; k += 16)
#pragma unroll
                    for (int e = 0; e < 8; ++e) mp[e] = fmax3_nan(mp[e], sf[k + e], sf[k + 8 + e]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mp[e] = fmax3_nan(mp[e], mp[e + 4], sf[56 + e]);
                const float mx = fmax3_nan(fmax3_nan(mp[0], mp[1], mp[2]), fmax3_nan(mp[3], sf[60], sf[61]),
                                           fmax3_nan(sf[62], sf[63], sf[63])) *
                                 kScaleLog2;
                // The base is raised for a growth beyond 2^8 only (weights stay
                // below 2^8, o and the sum share the base); a NaN or infinite
                // score makes the row NaN, as its softmax is.
                const bool need = valid && mx > m + kRescaleThreshold && mx < INFINITY;
                if (__any_sync(0xFFFFFFFFu, valid && !(mx <= m + kRescaleThreshold))) {
                    if (valid && !(mx < INFINITY)) l = __int_as_float(0x7FFFFFFF);
                    const float f = need ? exp2f(m - mx) : 1.0f;
                    if (u > 0) {
                        // the product of the half before is complete (S of this
                        // half came behind the one before that)
                        ok = __all_sync(0xFFFFFFFFu, wait(B(kBarPvDone + s), (n_pv + u - 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            uint32_t ov[16];
                            tmem_ld16(tO + 16u * q, ov);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
                            tmem_st16(tO + 16u * q, ov);
                        }
                    }
                    l *= f;
                    if (need) m = mx;
                }
                const float nm = m == -INFINITY ? 0.0f : -m;     // no key seen yet: every weight is 2^-inf = 0
                uint64_t lp[2] = {0, 0};
                uint32_t pk[16];
                weights32(sf, nm, pk, lp);
                tmem_st16(tX, pk);
                weights32(sf + 32, nm, pk, lp);
                tmem_st16(tX + 16u, pk);
                float a0, a1;
                unpack2(fadd2(lp[0], lp[1]), a0, a1);
                l += a0 + a1;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(B(kBarPFull + 2 * s + x));
            }
            if (!ok) break;
            if (c) n_pv += 2 * c - 1;
            if (c) {
                ok = __all_sync(0xFFFFFFFFu, wait(B(kBarOFull + s), n_o++ & 1));
                if (!ok) break;
                tc_fence_after();
            }
            if (!ok) break;
            ok = __all_sync(0xFFFFFFFFu, it == 0 || wait(B(kBarStatEmpty + s), (it - 1) & 1));
            if (!ok) break;
            stat[s * 256 + r] = m;
            stat[s * 256 + 128 + r] = l;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(B(kBarStatFull + s));
                mbar_arrive(B(kBarWorkEmpty + wi));
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t tO = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kOCol;
        // Packed prompts: the cache rows are written while an item's result is
        // awaited (all of them at the start held up the first items of each CTA
        // by 100 us in a batch of 14681 tokens of 8 KV heads), the rest at the end.
        int64_t app = static_cast<int64_t>(blockIdx.x) * 4 + quarter;
        const int64_t app_n = static_cast<int64_t>(gridDim.x) * 4;
        const int64_t app_total = !kPaged && p.a.slots && !dead ? append_total(p.a) : 0;
        auto append = [&]() {
            append_rows(p.a, app, app_n, app_total, lane);
            app += kAppend * app_n;
        };
        __nv_bfloat162 amax2 = __floats2bfloat162_rn(0.0f, 0.0f);
        bool ok = !dead;
        for (uint32_t it = 0; ok; ++it) {
            const uint32_t wi = it % kWork;
            ok = __all_sync(0xFFFFFFFFu, wait(B(kBarWorkFull + wi), (it / kWork) & 1));
            if (!ok || items[wi].last) break;
            const Item &w = items[wi];
            for (int s = 0; s < 2 && ok; ++s) {
                // both slots of a dual item are finished in one turn
                const bool both = w.dual != 0;
                if (both && s == 1) break;
                for (int q = s; q < (both ? 2 : s + 1) && ok; ++q) {
                    if (!kPaged)
                        while (app < app_total && !__all_sync(0xFFFFFFFFu, mbar_test_wait(B(kBarStatFull + q), it & 1))) append();
                    ok = __all_sync(0xFFFFFFFFu, wait(B(kBarStatFull + q), it & 1));
                }
                if (!ok) break;
                tc_fence_after();
                const int tok = (both ? 0 : s * R) + r / G;
                const bool valid = r < R * G && tok < w.e.ntok;
                const int pos = w.e.pos0 + tok;
                float m = stat[s * 256 + r], l = stat[s * 256 + 128 + r];
                float f0 = 1.0f, f1 = 0.0f;
                if (both) {
                    const float m1 = stat[256 + r], l1 = stat[256 + 128 + r];
                    const float mm = fmaxf(m, m1);
                    if (mm > -INFINITY) {
                        f0 = m > -INFINITY ? exp2f(m - mm) : 0.0f;
                        f1 = m1 > -INFINITY ? exp2f(m1 - mm) : 0.0f;
                    }
                    // (a NaN sum stays one)
                    l = l * f0 + l1 * f1;
                    m = mm;
                }
                const bool two = both && w.c[1] > 0;
                const bool one = w.c[s] > 0;
                // (a row sees one key at least; sum 0: every score is -inf, and o is 0 x inf = NaN)
                const float inv = w.part >= 0 ? 1.0f : 1.0f / l;
                const int prow = (both ? 0 : s * kRows) + r;
                float *pm = nullptr, *po = nullptr;
                if (w.part >= 0) {
                    float *base = p.part + static_cast<int64_t>(w.part) * p.part_rows * (2 + kD);
                    pm = base + prow * 2;
                    po = base + p.part_rows * 2 + static_cast<int64_t>(prow) * kD;
                    if (valid) {
                        pm[0] = m;
                        pm[1] = l;
                    }
                }
                __nv_bfloat16 *orow = p.a.o + static_cast<int64_t>(w.e.row0 + tok) * p.a.ldo + (w.g * G + r % G) * kD;
                const int bad = w.bad;
                const bool any = __any_sync(0xFFFFFFFFu, valid);
                const uint64_t scale0 = pack2(f0 * inv, f0 * inv), scale1 = pack2(f1 * inv, f1 * inv);
                const bool plain = one && !two && !bad && w.part < 0;
                if (any && plain) {
                    // the usual case: the next 16 columns are on their way while
                    // these are rounded and stored
                    uint32_t ov[16];
                    tmem_ld16(tO + s * 128u, ov);
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        tmem_ld_wait();
                        uint64_t f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = fmul2(pair_of(ov[2 * e], ov[2 * e + 1]), scale0);
                        if (c < 7) tmem_ld16(tO + s * 128u + 16u * (c + 1), ov);
                        uint32_t pk[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float y0, y1;
                            unpack2(f[e], y0, y1);
                            const __nv_bfloat162 b = __floats2bfloat162_rn(y0, y1);
                            pk[e] = *reinterpret_cast<const uint32_t *>(&b);
                        }
                        if (p.a.o_amax && valid) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                amax2 = __hmax2(amax2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&pk[e])));
                        }
                        if (valid) store32(orow + 16 * c, pk, p.wide);
                        __syncwarp();
                    }
                }
#pragma unroll 1
                for (int c = 0; any && !plain && c < 8; ++c) {
                    uint32_t o0[16], o1[16];
                    if (one) tmem_ld16(tO + s * 128u + 16u * c, o0);
                    if (two) tmem_ld16(tO + 128u + 16u * c, o1);
                    tmem_ld_wait();
                    uint64_t f[8];              // pairs of o, scaled
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = one ? fmul2(pair_of(o0[2 * e], o0[2 * e + 1]), scale0) : 0;
                    if (two) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = ffma2(pair_of(o1[2 * e], o1[2 * e + 1]), scale1, f[e]);
                    }
                    if (bad && valid) {
                        // cleaned values of the keys this row does see
                        for (int k = max(w.e.pos0 + 1, w.t0 * kKeys); k <= min(min(pos, w.kv_len - 1), w.t1 * kKeys - 1); ++k) {
                            const __nv_bfloat16 *v = new_value_row<kPaged>(p, w, k);
                            if (!v) continue;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float y0 = __bfloat162float(v[16 * c + 2 * e]), y1 = __bfloat162float(v[16 * c + 2 * e + 1]);
                                f[e] = fadd2(f[e], pack2(isfinite(y0) ? 0.0f : y0, isfinite(y1) ? 0.0f : y1));
                            }
                        }
                    }
                    if (valid && w.part >= 0) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<ulonglong2 *>(po + 16 * c)[e] = make_ulonglong2(f[2 * e], f[2 * e + 1]);
                    } else if (valid) {
                        uint32_t pk[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float y0, y1;
                            unpack2(f[e], y0, y1);
                            const __nv_bfloat162 b = __floats2bfloat162_rn(y0, y1);
                            if (p.a.o_amax) amax2 = __hmax2(amax2, __habs2(b));
                            pk[e] = *reinterpret_cast<const uint32_t *>(&b);
                        }
                        store32(orow + 16 * c, pk, p.wide);
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    for (int q = s; q < (both ? 2 : s + 1); ++q) {
                        mbar_arrive(B(kBarStatEmpty + q));
                        if (w.c[q]) mbar_arrive(B(kBarOEmpty + q));
                    }
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(B(kBarWorkEmpty + wi));
        }
        if (!kPaged)
            while (ok && app < app_total) append();
        if (p.a.o_amax) {
            const float amax = fmaxf(__bfloat162float(amax2.x), __bfloat162float(amax2.y));
            const unsigned u = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax));
            if (lane == 0 && u) atomicMax(reinterpret_cast<unsigned *>(p.a.o_amax), u);
        }
    } else {
        if (warp < 14) {
            // -------------------------------------------------------- MMA issue of one slot
            const int s = warp - 12;
            const uint32_t tS = tmem + s * 128u, tO = tmem + kOCol + s * 128u;
            constexpr uint32_t idesc_s = idesc_bf16(128, 64, 0, 0);
            constexpr uint32_t idesc_o = idesc_bf16(128, 128, 0, 1);   // V MN-major
            const uint64_t qd = sdesc_sw128(s0 + kQOff + s * kTileBytes, 16, 1024);
            auto wwait = [&](uint32_t b, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(b, parity)) != 0; };
            uint32_t stage = 0;             // of this item's first K tile
            uint32_t n_s = 0, n_q = 0;      // tiles and items of this slot
            uint32_t k_par = 0, v_par = 0;  // parity of each barrier's next phase
            bool ok = !dead;
            for (uint32_t it = 0; ok; ++it) {
                const uint32_t wi = it % kWork;
                ok = wwait(B(kBarWorkFull + wi), (it / kWork) & 1);
                if (!ok || items[wi].last) break;
                const int n = items[wi].t1 - items[wi].t0, c = items[wi].c[s], other = items[wi].c[s ^ 1];
                const int dual = items[wi].dual;
                __syncwarp();
                if (lane == 0) mbar_arrive(B(kBarWorkEmpty + wi));
                if (c) {
                    ok = wwait(B(kBarQFull + s), n_q & 1);
                    // this slot's first K stage; its next one is 2 (4: dual) stages on
                    uint32_t ks = (stage + (dual && s ? 2 : 0)) % kRing;
                    // a tile that only this slot reads is released by it alone
                    auto alone = [&](int i) { return dual || i >= other; };
                    auto set_of = [&](int i) { return alone(i) ? static_cast<uint32_t>((1 + s) * kRing) : 0u; };
                    // S = Q K^T of half x of the K tile (P of this buffer was read
                    // by an earlier product of this thread: in order)
                    auto issue_s = [&](int x) {
                        const uint64_t kd = sdesc_sw128(s0 + kRingOff + ks * kTileBytes + x * 8 * L::kGroup, 16, L::kGroup);
                        warp_mma8_ss<(L::kHalf >> 4)>(tS + 64 * x, qd, kd, idesc_s);
                        warp_commit(B(kBarSFull + 2 * s + x));
                    };
                    auto k_done = [&](int i) {      // behind the second half of S of tile i
                        warp_commit(B(kBarKvEmpty + ks));
                        if (alone(i)) warp_commit(B(kBarKvEmpty + ks));
                        if (i == c - 1) warp_commit(B(kBarQEmpty + s));
                    };
                    uint32_t kb = set_of(0) + ks;
                    ok = ok && wwait(B(kBarKFull + kb), (k_par >> kb) & 1);
                    if (!ok) break;
                    k_par ^= 1u << kb;
                    tc_fence_after();
                    issue_s(0);
                    issue_s(1);
                    k_done(0);
                    for (int i = 0; i < c && ok; ++i, ++n_s) {
                        const uint32_t vs = ks + 1 == kRing ? 0 : ks + 1;
                        const uint32_t vb = set_of(i) + vs;
                        ok = wwait(B(kBarClean + vb), (v_par >> vb) & 1);
                        v_par ^= 1u << vb;
                        if (i == 0 && n_q > 0) ok = ok && wwait(B(kBarOEmpty + s), (n_q - 1) & 1);
                        constexpr uint32_t kStep = 2 * L::kGroup >> 4;
                        const uint64_t vd = sdesc_sw128(s0 + kRingOff + vs * kTileBytes, L::kHalf, L::kGroup);
                        ks += dual ? 4 : 2;
                        if (ks >= kRing) ks -= kRing;
                        const bool more = i + 1 < c;
                        kb = set_of(i + 1) + ks;
                        // Per half: P V, then S of the next tile's half over it.
                        // Where the next K tile is still on its way (a long cache
                        // streams at the memory's rate) both P V go first, so that
                        // the V tile makes room for the next load.
                        const uint32_t kpar = (k_par >> kb) & 1;
                        auto k_here = [&]() { return __all_sync(0xFFFFFFFFu, mbar_test_wait(B(kBarKFull + kb), kpar)) != 0; };
                        bool early = more && k_here();
                        ok = ok && wwait(B(kBarPFull + 2 * s), n_s & 1);
                        if (!ok) break;
                        tc_fence_after();
                        warp_mma4_ts<kStep>(tO, tS, vd, idesc_o, i > 0);
                        warp_commit(B(kBarPvDone + s));
                        if (more && !early) early = k_here();
                        if (early) issue_s(0);
                        ok = wwait(B(kBarPFull + 2 * s + 1), n_s & 1);
                        if (!ok) break;
                        tc_fence_after();
                        warp_mma4_ts<kStep>(tO, tS + 64, vd + 4 * kStep, idesc_o, 1);
                        warp_commit(B(more ? kBarPvDone + s : kBarOFull + s));     // (an item's last: OFull alone)
                        warp_commit(B(kBarKvEmpty + vs));
                        if (alone(i)) warp_commit(B(kBarKvEmpty + vs));
                        if (more) {
                            if (!early) {
                                ok = wwait(B(kBarKFull + kb), kpar);
                                if (!ok) break;
                                tc_fence_after();
                                issue_s(0);
                            }
                            issue_s(1);
                            k_done(i + 1);
                        }
                        k_par ^= more ? 1u << kb : 0u;
                    }
                    ++n_q;
                }
                stage = (stage + 2u * static_cast<uint32_t>(n)) % kRing;
            }
            // every MMA issued completes before tensor memory is freed
            warp_commit(B(kBarDrain + s));
            wait_drain(B(kBarDrain + s), 0);
            __syncwarp();
        } else if (warp == 14) {
            // -------------------------------------------------------- work list and loads
            const PagedAttnArgs &a = p.a;
            const int64_t cap = kPaged ? static_cast<int64_t>(a.max_pages) << a.ps_shift : INT32_MAX;
            Range range = {};
            int n_ent;
            SelfPlan plan;
            if (!kPaged && p.self) {
                n_ent = plan.take(p, lane);
            } else {
                n_ent = p.head->n_ent;
                if (kPaged) range = p.ranges[blockIdx.x];
            }
            int e = range.e, g = range.g;
            const int page_rows = min(1 << a.ps_shift, kKeys);
            const int n_groups = page_rows / 8;                        // 8-row groups of a box
            const int boxes = kPaged ? kKeys / page_rows : 1;          // boxes of a tile
            const int oob = static_cast<int>((a.n_pages * a.Hkv) << a.ps_shift >> 3);   // behind the last group
            const int q_tok = min(R, a.max_new);
            uint32_t n_kv = 0, n_q[2] = {0, 0};
            uint32_t used = 0, par = 0;          // full barriers (K sets, then V) and the parity of their last phase
            bool ok = !dead;
            for (uint32_t it = 0; ok; ++it) {
                const uint32_t wi = it % kWork;
                // the next item
                Item w = {};
                w.last = 1;
                if (kPaged) {
                    const int from = it == 0 ? range.t0 : 0;
                    if (g < range.end_g || (g == range.end_g && e < range.end_e) ||
                        (g == range.end_g && e == range.end_e && from < range.end_t)) {
                        w.e = it == 0 ? range.first : p.ent[e];
                        const int full = entry_tiles(w.e, cap);
                        w.g = g;
                        w.last = 0;
                        w.t0 = from;
                        w.t1 = g == range.end_g && e == range.end_e ? range.end_t : full;
                        const int place = 2 * static_cast<int>(blockIdx.x);
                        w.part = w.t0 > 0 ? place : (w.t1 < full ? place + 1 : -1);
                        if (++e == n_ent) {
                            e = 0;
                            ++g;
                        }
                    }
                } else {
                    int idx = blockIdx.x;
                    if (p.self) {                // one item a CTA
                        if (it > 0) idx = INT32_MAX;
                    } else {
                        if (lane == 0) idx = atomicAdd(&p.head->counter, 1);
                        idx = __shfl_sync(0xFFFFFFFFu, idx, 0);
                    }
                    if (n_ent > 0 && idx < static_cast<int64_t>(n_ent) * a.Hkv) {
                        w.e = p.self ? plan.block(idx / a.Hkv, 2 * R) : p.ent[idx / a.Hkv];
                        w.g = idx % a.Hkv;
                        w.last = 0;
                        w.t1 = (w.e.pos0 + w.e.ntok + kKeys - 1) / kKeys;
                        w.part = -1;
                    }
                }
                if (!w.last) {
                    w.kv_len = static_cast<int>(min(static_cast<int64_t>(w.e.pos0) + w.e.ntok, cap));
                    w.dual = w.e.ntok <= R;
                    const int n = w.t1 - w.t0;
                    if (w.dual) {
                        w.c[0] = (n + 1) / 2;
                        w.c[1] = n / 2;
                    } else {
                        const int e0 = (min(w.e.pos0 + R, w.kv_len) + kKeys - 1) / kKeys;
                        w.c[0] = max(min(e0, w.t1) - w.t0, 0);
                        w.c[1] = n;
                    }
                }
                ok = __all_sync(0xFFFFFFFFu, it < kWork || wait(B(kBarWorkEmpty + wi), ((it / kWork) - 1) & 1));
                if (!ok) break;
                if (lane == 0) {
                    items[wi] = w;
                    mbar_arrive(B(kBarWorkFull + wi));
                }
                if (w.last) break;
                // its loads: the first K / V pair, the queries, the other pairs
                const int n = w.t1 - w.t0;
                const int *trow = kPaged ? a.table + static_cast<int64_t>(w.e.kv) * a.max_pages : nullptr;
                auto page_of = [&](int j) {         // coordinate of this lane's box of tile j, or -1: nothing to load
                    if (!kPaged) return 0;
                    const int64_t pos = static_cast<int64_t>(j) * kKeys + lane * page_rows;
                    if (lane >= boxes || pos >= w.kv_len) return -1;
                    const int id = trow[pos >> a.ps_shift];
                    if (id < 0 || id >= a.n_pages) return oob;
                    return static_cast<int>((static_cast<int64_t>(id) * a.Hkv + w.g) << a.ps_shift >> 3) +
                           (static_cast<int>(pos & ((1 << a.ps_shift) - 1)) >> 3);
                };
                int coord = page_of(w.t0);
                for (int jj = 0; jj < n && ok; ++jj) {
                    const int next = jj + 1 < n ? page_of(w.t0 + jj + 1) : -1;
                    const uint32_t n_box = kPaged ? __popc(__ballot_sync(0xFFFFFFFFu, coord >= 0)) : 1;
                    const uint32_t bytes = kPaged ? n_box * n_groups * 2048u : kTileBytes;
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t idx = 2 * (n_kv + jj) + kv, st = idx % kRing;
                        ok = __all_sync(0xFFFFFFFFu, idx < kRing || wait(B(kBarKvEmpty + st), ((idx / kRing) - 1) & 1));
                        if (!ok) break;
                        const uint32_t set = w.dual ? 1 + (jj & 1) : (jj < w.c[0] ? 0 : 2);
                        const uint32_t fb = kv ? 3 * kRing + st : set * kRing + st;
                        const uint32_t dst = s0 + kRingOff + st * kTileBytes, full = B(kBarKFull + fb);
                        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                        par ^= (used >> fb & 1) << fb;
                        used |= 1u << fb;
                        __syncwarp();
                        if (kPaged) {
                            if (coord >= 0)
                                tma_load_4d(dst + lane * (n_groups * 2048u), kv ? &tmap_v : &tmap_k, 0, 0, 0, coord, full);
                        } else if (lane == 0) {
                            tma_load_3d(dst, &tmap_k, 0, w.e.kv + (w.t0 + jj) * kKeys, 2 * (a.H + kv * a.Hkv + w.g), full);
                        }
                    }
                    if (!ok) break;
                    if (jj == 0) {
                        for (int s = 0; s < 2 && ok; ++s) {
                            if (!w.c[s]) continue;
                            ok = __all_sync(0xFFFFFFFFu, n_q[s] == 0 || wait(B(kBarQEmpty + s), (n_q[s] - 1) & 1));
                            if (!ok) break;
                            ++n_q[s];
                            if (lane == 0) {
                                const uint32_t dst = s0 + kQOff + s * kTileBytes, full = B(kBarQFull + s);
                                const int row = w.e.row0 + (w.dual ? 0 : s * R);
                                mbar_arrive_expect_tx(full, static_cast<uint32_t>(q_tok * G) * 256u);
                                tma_load_4d(dst, &tmap_q, 0, w.g * G, row, 0, full);
                                tma_load_4d(dst + 16384, &tmap_q, 0, w.g * G, row, 1, full);
                            }
                        }
                    }
                    coord = next;
                }
                n_kv += n;
            }
            if (!ok) {
                // loads in flight land before the CTA may exit
                for (uint32_t i = 0; i < 4 * kRing; ++i)
                    if (used >> i & 1) wait_drain(B(kBarKFull + i), par >> i & 1);
                for (int s = 0; s < 2; ++s)
                    if (n_q[s]) wait_drain(B(kBarQFull + s), (n_q[s] - 1) & 1);
            }
        } else {
            // -------------------------------------------------------- V tiles: clean and hand on
            uint32_t n_kv = 0, v_par = 0;
            bool ok = !dead;
            for (uint32_t it = 0; ok; ++it) {
                const uint32_t wi = it % kWork;
                ok = __all_sync(0xFFFFFFFFu, wait(B(kBarWorkFull + wi), (it / kWork) & 1));
                if (!ok || items[wi].last) break;
                const Item &w = items[wi];
                const int dual = w.dual, c0 = w.c[0], t0 = w.t0, t1 = w.t1, kv_len = w.kv_len, from = min(w.e.pos0 + 1, kv_len);
                for (int j = t0; j < t1 && ok; ++j) {
                    const uint32_t vi = 2 * (n_kv + j - t0) + 1, vs = vi % kRing;
                    ok = __all_sync(0xFFFFFFFFu, wait(B(kBarVFull + vs), v_par >> vs & 1));
                    if (!ok) break;
                    v_par ^= 1u << vs;
                    const int lo = max(from - j * kKeys, 0);       // rows some of the tile's queries do not see
                    if (lo < kKeys) {
                        const uint32_t tile = s0 + kRingOff + vs * kTileBytes;
                        const int end = min(max(kv_len - j * kKeys, 0), kKeys);
                        // rows behind the last key are zeroed, those before it
                        // looked over
#pragma unroll 1
                        for (int i = end * 16 + lane; i < kKeys * 16; i += 32)
                            st_shared_v4(tile + L::chunk(i >> 4, i & 15), 0, 0, 0, 0);
                        __nv_bfloat162 big = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll 1
                        for (int i0 = lo * 16 + lane; i0 < end * 16; i0 += 128) {
                            uint32_t v[4][4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int i = min(i0 + 32 * u, end * 16 - 1);
                                ld_shared_v4(tile + L::chunk(i >> 4, i & 15), v[u]);
                            }
#pragma unroll
                            for (int u = 0; u < 4 * 4; ++u)
                                big = __hmax2_nan(big, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&v[u >> 2][u & 3])));
                        }
                        const uint32_t seen = *reinterpret_cast<const uint32_t *>(&big);
                        if (__any_sync(0xFFFFFFFFu, (seen & 0x7F80u) == 0x7F80u || (seen & 0x7F800000u) == 0x7F800000u)) {
#pragma unroll 1
                            for (int i = lo * 16 + lane; i < end * 16; i += 32) {
                                const uint32_t addr = tile + L::chunk(i >> 4, i & 15);
                                uint32_t v[4];
                                ld_shared_v4(addr, v);
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    if ((v[q] & 0x7F80u) == 0x7F80u) v[q] &= 0xFFFF0000u;
                                    if ((v[q] & 0x7F800000u) == 0x7F800000u) v[q] &= 0x0000FFFFu;
                                }
                                st_shared_v4(addr, v[0], v[1], v[2], v[3]);
                            }
                            if (lane == 0) items[wi].bad = 1;
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    const int jj = j - t0;
                    if (lane == 0) mbar_arrive(B(kBarClean + (dual ? 1 + (jj & 1) : (jj < c0 ? 0 : 2)) * kRing + vs));
                }
                if (!ok) break;
                n_kv += t1 - t0;
                __syncwarp();
                if (lane == 0) mbar_arrive(B(kBarWorkEmpty + wi));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---- parts of cut items -------------------------------------------------------------------

constexpr int kCombineRows = 8;       // rows a block takes at a time: a warp each

// Block (c, y): the item that begins in CTA c's range and goes on past it.
// Its parts: c's second place, then the first place of the CTAs after c.
// Latency of three dependent reads, 5 to 7 us cold; with chunks 39 MB of parts
// lie in L2 (20 us for 148 cut items; half a warp a row takes 14, but 2 us more
// where a row has many parts).
__global__ void __launch_bounds__(32 * kCombineRows) paged_combine_kernel(const Params p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PagedAttnArgs &a = p.a;
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x;
    const Range rg = p.ranges[c];
    if (rg.cut_to == 0) return;
    const Entry en = rg.cut;
    const int g = rg.cut_g, n = rg.cut_to - c + 1;
    const bool dual = en.ntok <= p.R;
    const int64_t stride = static_cast<int64_t>(p.part_rows) * (2 + kD);
    // part k: c's second place, then the first places of the CTAs after it
    const float *base0 = p.part + (2 * static_cast<int64_t>(c) + 1) * stride;
    auto part = [&](int k) { return k == 0 ? base0 : base0 + (2 * k - 1) * stride; };
    float amax = 0.0f;
    const int rows = en.ntok * p.G;           // (token, head) pairs in order
    for (int i = blockIdx.y * kCombineRows + warp; i < rows; i += gridDim.y * kCombineRows) {
        const int tok = i / p.G, hh = i % p.G;
        const int prow = dual || tok < p.R ? i : kRows + (tok - p.R) * p.G + hh;
        // lanes take the parts' (maximum, sum); the parts' weights are then
        // handed round, and their rows are loaded eight at a time
        float m = -INFINITY, l = 0.0f;
        for (int k = lane; k < n; k += 32) m = fmaxf(m, part(k)[prow * 2]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k0 = 0; k0 < n; k0 += 32) {
            float f = 0.0f;
            if (k0 + lane < n) {
                const float2 ml = *reinterpret_cast<const float2 *>(part(k0 + lane) + prow * 2);
                // (a part without a key for this row: maximum -inf, sum and o 0
                // or, where a value was not finite, that value)
                f = ml.x > -INFINITY ? exp2f(ml.x - m) : 1.0f;
                l = fmaf(ml.y, f, l);
            }
            const int kn = min(n - k0, 32);
            for (int k = 0; k < kn; k += 8) {
                float4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    v[u] = k + u < kn ? reinterpret_cast<const float4 *>(part(k0 + k + u) + p.part_rows * 2 +
                                                                        static_cast<int64_t>(prow) * kD)[lane]
                                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float fk = __shfl_sync(0xFFFFFFFFu, f, k + u);
                    acc.x = fmaf(v[u].x, fk, acc.x);
                    acc.y = fmaf(v[u].y, fk, acc.y);
                    acc.z = fmaf(v[u].z, fk, acc.z);
                    acc.w = fmaf(v[u].w, fk, acc.w);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        const float inv = 1.0f / l;
        __nv_bfloat162 r[2] = {__floats2bfloat162_rn(acc.x * inv, acc.y * inv), __floats2bfloat162_rn(acc.z * inv, acc.w * inv)};
        reinterpret_cast<uint2 *>(a.o + static_cast<int64_t>(en.row0 + tok) * a.ldo + (g * p.G + hh) * kD)[lane] =
            *reinterpret_cast<uint2 *>(r);
#pragma unroll
        for (int q = 0; q < 2; ++q)
            amax = fmaxf(amax, fmaxf(fabsf(__bfloat162float(r[q].x)), fabsf(__bfloat162float(r[q].y))));
    }
    if (a.o_amax) {
        const unsigned u = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax));
        if (lane == 0 && u) atomicMax(reinterpret_cast<unsigned *>(a.o_amax), u);
    }
}

// ---- host -------------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = []() -> EncodeFn {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !ptr)
            return nullptr;
        return reinterpret_cast<EncodeFn>(ptr);
    }();
    return fn;
}

bool encode(CUtensorMap *m, int rank, const void *base, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    EncodeFn fn = encode_fn();
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims,
                    strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Workspace {
    size_t ent, prefix, ranges, part, total;
    int max_ent, part_rows;
};

Workspace carve(int64_t T, int64_t B, int64_t max_new, int64_t H, int64_t Hkv, bool paged, int num_sms) {
    const int64_t G = H / Hkv, R = kRows / G;
    Workspace w;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    w.max_ent = static_cast<int>(T / (2 * R) + B);
    w.ent = 256;
    w.prefix = up(w.ent + sizeof(Entry) * w.max_ent);
    w.ranges = paged ? up(w.prefix + sizeof(int64_t) * (w.max_ent + 1)) : w.prefix;
    w.part = paged ? up(w.ranges + sizeof(Range) * num_sms) : w.ranges;
    // (an even count keeps the 16-byte alignment of the rows behind the (max, sum) pairs)
    w.part_rows = paged ? static_cast<int>(max_new <= R ? (max_new * G + 1) / 2 * 2 : 2 * kRows) : 0;
    w.total = up(w.part + sizeof(float) * 2 * num_sms * w.part_rows * (2 + kD));
    return w;
}

}  // namespace


size_t attention_paged_workspace_bytes(int64_t T, int64_t B, int64_t max_new, int64_t H, int64_t Hkv, bool paged) {
    return carve(T, B, max_new, H, Hkv, paged, kMaxCtas).total;
}

template <bool kPaged>
static cudaError_t launch_kind(Params &p, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, int grid,
                               cudaStream_t s) {
    const PagedAttnArgs &a = p.a;
    const size_t prep_smem = (a.B + 1 + (kPaged ? 0 : kBins)) * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(paged_prep_kernel<kPaged>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (kPagedMaxRequests + 1 + kBins) * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(paged_attention_kernel<kPaged>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    // Few short prompts: no work list (three of 348 tokens in all: 16.3 against
    // 19.3 us with it when that was tried, 11.8 now; paged calls gained nothing,
    // their list kernel also writes the new cache rows).
    p.self = !kPaged && a.B <= 32 && (a.T / (2 * p.R) + a.B) * static_cast<int64_t>(a.Hkv) <= grid;
    if (p.self) {
        if (a.o_amax && (e = cudaMemsetAsync(a.o_amax, 0, sizeof(float), s)) != cudaSuccess) return e;
    } else {
        int prep_grid = 1;
        if (kPaged && a.slots) {
            const int64_t warps = static_cast<int64_t>(a.T) * a.Hkv;      // at most four rows a warp's turn
            prep_grid += static_cast<int>(std::min<int64_t>((warps + 4 * 32 - 1) / (4 * 32), 2 * grid));
        }
        e = launch_pdl(paged_prep_kernel<kPaged>, dim3(prep_grid), dim3(kPrepThreads), prep_smem, s, p);
        if (e != cudaSuccess) return e;
    }
    e = launch_pdl(paged_attention_kernel<kPaged>, dim3(grid), dim3(kThreads), kSmemBytes, s, tq, tk, tv, p);
    if (e != cudaSuccess) return e;
    if (kPaged) {
        const int y = (p.part_rows + kCombineRows - 1) / kCombineRows;
        e = launch_pdl(paged_combine_kernel, dim3(grid, std::min(y, 8)), dim3(32 * kCombineRows), 0, s, p);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

cudaError_t launch_attention_paged(const PagedAttnArgs &a, void *ws, unsigned *err, int num_sms, cudaStream_t s) {
    const bool paged = a.table != nullptr;
    const int grid = std::min(num_sms, kMaxCtas);
    const Workspace w = carve(a.T, a.B, a.max_new, a.H, a.Hkv, paged, kMaxCtas);
    uint8_t *base = static_cast<uint8_t *>(ws);
    Params p = {};
    p.a = a;
    p.G = a.H / a.Hkv;
    p.R = kRows / p.G;
    p.max_ent = w.max_ent;
    p.head = reinterpret_cast<Header *>(base);
    p.ent = reinterpret_cast<Entry *>(base + w.ent);
    p.prefix = reinterpret_cast<int64_t *>(base + w.prefix);
    p.ranges = reinterpret_cast<Range *>(base + w.ranges);
    p.grid = grid;
    p.part = reinterpret_cast<float *>(base + w.part);
    p.part_rows = w.part_rows;
    p.wide = reinterpret_cast<uintptr_t>(a.o) % 32 == 0 && a.ldo % 16 == 0;
    p.err = err;
    CUtensorMap tq, tk, tv;
    const cuuint64_t ld = static_cast<cuuint64_t>(a.ldqkv) * 2;
    {
        // queries as {64 columns, head, token, half}: a box is the G heads of a
        // KV head for R tokens, token-major
        const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(a.H), static_cast<cuuint64_t>(a.T), 2};
        const cuuint64_t strides[3] = {kD * 2, ld, 128};
        const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(std::min(p.R, a.max_new)), 1};
        if (!encode(&tq, 4, a.qkv, dims, strides, box)) return cudaErrorInvalidValue;
    }
    if (paged) {
        // pages as {64 columns, 8 rows, half, group of 8 rows}: a box is a page
        // of one head (128 rows of it at most)
        const cuuint64_t groups = static_cast<cuuint64_t>(a.n_pages * a.Hkv) << a.ps_shift >> 3;
        const cuuint64_t dims[4] = {64, 8, 2, groups};
        const cuuint64_t strides[3] = {kD * 2, 128, 2048};
        const cuuint32_t box[4] = {64, 8, 2, static_cast<cuuint32_t>(std::min(1 << a.ps_shift, kKeys) / 8)};
        if (!encode(&tk, 4, a.k_pages, dims, strides, box) || !encode(&tv, 4, a.v_pages, dims, strides, box))
            return cudaErrorInvalidValue;
        return launch_kind<true>(p, tq, tk, tv, grid, s);
    }
    // the batch's rows as {64 columns, row, 64-column block}
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(a.T), static_cast<cuuint64_t>(2 * (a.H + 2 * a.Hkv))};
    const cuuint64_t strides[2] = {ld, 128};
    const cuuint32_t box[3] = {64, kKeys, 2};
    if (!encode(&tk, 3, a.qkv, dims, strides, box)) return cudaErrorInvalidValue;
    return launch_kind<false>(p, tq, tk, tk, grid, s);
}

}  // namespace mq
