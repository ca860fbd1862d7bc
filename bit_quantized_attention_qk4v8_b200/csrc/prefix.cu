// Decode attention of a batch whose sequences share a prefix.
//
// The query rows of all B sequences that read one KV head (B * G * nq of them)
// multiply the same keys of the prefix, so there decode is a matrix product again:
// each K/V tile is read once for 128 rows instead of once per sequence. After it
// come each sequence's own keys, for its G * nq rows. Softmax over [prefix, own
// keys] splits into partial results with their log-sum-exp, which the merge kernel
// joins:  O = sum_s 2^(lse_s - m) O_s / sum_s 2^(lse_s - m).
//
// One persistent kernel does both. A unit is 128 query rows of a KV head (in (sequence,
// head, token) order, gathered from the packed queries): first the prefix's keys, then
// the own keys of each sequence that has rows among them, which the other rows do not
// see (their warps skip them). So own keys cost no unit, no partial result and no
// merge of their own: as units of one sequence each they took 6 us apiece, whatever
// their length. The units' 128-key tiles, laid end to end (with one tile's time for a
// unit's start and end), are cut into one equal share for each CTA; a unit that a
// share's end cuts leaves several partial results. Piece (unit, share) has slot
// unit + share, so the slots number units + shares whatever the lengths, which are on
// the device: every CTA works its share out.
//   S = Q K^T     kind::mxf4, E2M1 operands, the E8M0 scales read from TMEM.
//   O += P V      kind::f16 on bf16 operands: P from TMEM, V expanded from E4M3.
//
// Why bf16 and not the E4M3 MMAs of the other attention kernels: they write P as
// two E4M3 terms with a block scale, about 9 instructions a score, which bounds
// them. bf16 holds the same 8 significant bits in one conversion for two scores,
// needs no block scale (its exponent takes p up to 2^64 above the reference), and
// goes to TMEM without a swizzled store: about 3 instructions a score, so the
// exponentials themselves (16 a clock and SM: 1024 clk a tile of 128 x 128) become
// the bound. Rounding p to bf16 in numerator and denominator alike moves a row's
// output by at most 2^-8 of the spread of the values it averages.
// V is expanded by the tensor core: the E4M3 codes and their scales times a unit
// matrix (kind::mxf8f6f4) give fp32 in TMEM, which eight warps take to bf16, exactly
// (an E4M3 value times a power of two has 4 significant bits), and into shared
// memory. By shifts and multiplies on the codes that took 9 instructions for four
// values, as many as all of the softmax.
//
// Softmax: two sets of four warps take turns on tiles of 128 keys, one row per
// thread. A set reads its S whole (128 registers) and frees the buffer at once, so the
// next tile's S comes while P is computed, and P V is on nobody's path. What a tile costs
// beside its exponentials (waits, the reference, the store's end: some 1500 clk of short
// dependent sequences) is paid once for 128 keys. (Three sets on 64 keys each: 286 us
// where this took 278, and the 64 registers saved bought nothing.)
//
// O has one reference per row, m_O, the row max of the unit's first tile, and
// p = 2^(s - m_O). It moves only when a score passes it by 2^64 (bf16 and fp32
// keep their relative precision at any offset, so nothing is gained by moving it
// sooner): the tile's owner then scales its row of O after the P V before its own.
// The reference passes from a tile's owner to the next one's in shared memory,
// right after the row max, well before the exponentials.
// V carries a row of ones, so O column 128 sums P as rounded.
//
// Rows of several sequences share the tiles of own keys, so what one sequence's keys
// and values hold must not reach the others' rows, which take them with weight 0: their scores
// stay finite (kPxQShift), and their V goes into bf16 without infinities and NaN. 5 us of the 283.
//
// Warp roles (640 threads): warps 0..7 softmax and epilogue, 8 feeder (units, queries,
// key tiles), 9 TMEM allocator and issuer of S, 10 issuer of D, 11 issuer of P V, 12..19 V
// expansion. The softmax warps hold 128 scores and get 168 registers, the others 48
// (256 * 168 + 384 * 48 = the 640 * 96 of the launch).
//
// Measured, both launches (with a cold L2 and the events' own 5 us): 64 sequences of 64 query heads
// over 8 KV heads with 8 query tokens, 16384 shared and up to 512 own keys: 309 us, and 296 a
// call in a row of calls, 0.94 PFLOP/s; 32 sequences of 32 heads, 8192 shared and up to 1024
// own keys in pages: 42 us; 13 of 20 heads with 3 tokens, 5003 and up to 777: 29 us; 4 of 32
// heads, 1000 and up to 100: 21.5 us. In a profiler's trace, as the comparisons here and below,
// this kernel and the merge take 283 + 12, 30 + 4, 17 + 4 and 11 + 3.5 us. A tile takes 1.2 us in the long run, twice its exponentials. No one part is
// the rest: of 278 us (before V's and the scores' guards), 264 are left without the exponentials,
// 273 without the expansion, 271 with a quarter of P V, 239 without any softmax work; the roles' loops are chains of dependent
// instructions, each close to the tile's time. In the short cases 6 to 8 us are the start
// (the schedule from the lengths, page numbers, the first loads) and 1.5 us the last unit's
// partial results.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/qk4v8.h"
#include "pipeline.cuh"
#include "ptx.cuh"
#include "qk4v8_internal.h"
#include "tile_ops.cuh"

namespace qk4v8 {

namespace {

constexpr int kPxKStages = 4;
constexpr int kPxVStages = 4;
constexpr int kPxVSlots = 4;                // 64 tokens of expanded V each
constexpr int kPxSets = 2;
constexpr int kPxUnits = 8;                 // units announced at most
constexpr int kPxTiles = 8;                 // tiles described at most
constexpr int kPxSeqs = 132;                // sequences with rows among 128 consecutive ones: up to 129
constexpr int kPxSoftmaxWarps = 4 * kPxSets;
constexpr int kPxFeedWarp = kPxSoftmaxWarps;
constexpr int kPxQkWarp = kPxFeedWarp + 1;
constexpr int kPxDWarp = kPxFeedWarp + 2;
constexpr int kPxPvWarp = kPxFeedWarp + 3;
constexpr int kPxExpandWarp = kPxSoftmaxWarps + 4;
constexpr int kPxThreads = 32 * (kPxExpandWarp + 8);
constexpr float kPxMove = 64.0f;            // m_O moves once a score passes it by 2^64
constexpr float kPxClear = 126.0f;          // a move by this much and more leaves nothing of O
// The queries' scales are taken 2^-64 smaller (the softmax scale is 2^64 larger): so the scores that
// a row gets from other sequences' keys, which share its tile, stay finite even where those hold what
// the quantizer makes of an infinity or a NaN (6 * 2^126), and fma(s, scale, -inf) is -inf.
// (Scales of queries below 2^-63 count as 2^-63: scores of 2^-60 of the keys. Zeroing P of those
// rows instead: 297 us where this takes 283.)
constexpr uint32_t kPxQShift = 0x40404040u;
constexpr float kPxQScale = 18446744073709551616.0f;  // 2^64

struct PxSmem {
    static constexpr int kQBytes = 128 * 64;
    static constexpr int kQ = 0;                                  // 2 buffers, 64-byte swizzle
    static constexpr int kKBytes = 128 * 64;
    static constexpr int kK = kQ + 2 * kQBytes;                   // per stage: 128 keys x 64 B, 64-byte swizzle
    static constexpr int kVRows = 144;                            // 128 channels, the ones row, 15 zero rows
    static constexpr int kVHalf = kVRows * 128;                   // 64 tokens of bf16 per row
    static constexpr int kV = kK + kPxKStages * kKBytes;          // 4 slots of bf16 V, 128-byte swizzle
    static constexpr int kRawBytes = 128 * 128;
    static constexpr int kRaw = kV + kPxVSlots * kVHalf;          // per stage: E4M3 block, 128-byte swizzle
    static constexpr int kUnit = kRaw + kPxVStages * kRawBytes;   // 32 x 32 unit matrix, E4M3, 128-byte swizzle
    static constexpr int kSfQ = kUnit + 32 * 128;                 // 512-byte scale atoms
    static constexpr int kSfK = kSfQ + 2 * 512;
    static constexpr int kSfV = kSfK + kPxKStages * 512;
    static constexpr int kSfOne = kSfV + kPxVStages * 512;
    static constexpr int kRef = kSfOne + 512;                     // (m_O, tile) of each row
    static constexpr int kBar = kRef + 128 * 8;
    // Barriers (byte offsets).
    static constexpr int kKFull = kBar, kKEmpty = kKFull + 8 * kPxKStages;             // per stage
    static constexpr int kRawFull = kKEmpty + 8 * kPxKStages;                          // per stage
    static constexpr int kRawEmpty = kRawFull + 8 * kPxVStages;
    static constexpr int kDFull = kRawEmpty + 8 * kPxVStages, kDFree = kDFull + 16;  // per half
    static constexpr int kVFull = kDFree + 16, kVEmpty = kVFull + 8 * kPxVSlots;        // per slot
    static constexpr int kQFull = kVEmpty + 8 * kPxVSlots, kQEmpty = kQFull + 16;      // per Q buffer
    static constexpr int kSFull = kQEmpty + 16, kSFree = kSFull + 8 * kPxSets;         // per set
    static constexpr int kPFull = kSFree + 8 * kPxSets, kPvDone = kPFull + 8 * kPxSets;
    static constexpr int kOFull = kPvDone + 8 * kPxSets, kOFree = kOFull + 8, kDrain = kOFree + 8;
    static constexpr int kUnitFull = kDrain + 8, kUnitEmpty = kUnitFull + 8 * kPxUnits;
    static constexpr int kBarEnd = kUnitEmpty + 8 * kPxUnits;
    static constexpr int kMisc = (kBarEnd + 15) / 16 * 16;  // TMEM address, abort flag, tile to clear
    static constexpr int kUnits = kMisc + 16;          // PxUnit [kPxUnits]
    static constexpr int kTiles = kUnits + 64 * kPxUnits;   // PxTile [kPxTiles]
    static constexpr int kLens = kTiles + 8 * kPxTiles;     // int [kPxSeqs]: the unit's sequences
    static constexpr int kNext = (kLens + 4 * kPxSeqs + 15) / 16 * 16;  // int4 [32]: the next tiles to load
    static constexpr int kUsed = kNext + 16 * 32;  // (descriptor, K row, block)
    static constexpr int kBytes = kUsed + 1024;
};
static_assert(PxSmem::kK % 1024 == 0 && PxSmem::kV % 1024 == 0 && PxSmem::kVHalf % 1024 == 0 &&
                  PxSmem::kRaw % 1024 == 0 && PxSmem::kUnit % 1024 == 0,
              "swizzled tiles need 1024-byte alignment");
static_assert(PxSmem::kBar % 8 == 0 && PxSmem::kSfQ % 128 == 0, "alignment");
static_assert(PxSmem::kBytes <= 227 * 1024, "shared memory budget");

constexpr uint32_t kPxTmemCols = 512;
// S 128, D (V as the tensor core expands it, 2 x 32 tokens) 64, O 144, P 2 x 64, scales 16: 480.
constexpr uint32_t kPxColS = 0, kPxColD = 128, kPxColO = 192, kPxColSfQ = 464, kPxColSfK = 468, kPxColSfV = 472, kPxColOne = 476;
__device__ __forceinline__ uint32_t px_col_p(int set) { return 336u + 64u * set; }

// Block-scaled E2M1 x E2M1, N = 128 keys; block-scaled E4M3 x E4M3, N = 32; bf16 x bf16, N = 144.
constexpr uint32_t kPxIdQK = (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24);
constexpr uint32_t kPxIdD = ((32u >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24);
constexpr uint32_t kPxIdPV =
    (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t(PxSmem::kVRows) >> 3) << 17) | ((128u >> 4) << 24);
constexpr __host__ __device__ uint32_t px_sf_id(uint32_t idesc, uint32_t id) { return idesc | (id << 29) | (id << 4); }

// The issuing threads' code is short on purpose: at about 7 clk an instruction, what they
// execute between two products is what the products wait for. So barriers go by their
// shared-memory address and descriptors by their low word (the high one is constant).
constexpr uint32_t px_desc_hi(uint32_t sbo, uint32_t layout) { return (sbo >> 4) | (1u << 14) | (layout << 29); }
constexpr uint32_t kHi64B = px_desc_hi(512, 4), kHi128B = px_desc_hi(1024, 2), kHiAtom = px_desc_hi(128, 0);
__device__ __forceinline__ uint32_t px_desc_lo(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | (lbo << 12); }

// D[128, N] (+)= A B, A bf16 in TMEM (two K elements a column), B bf16 in shared memory.
template <bool kFirst>
__device__ __forceinline__ void px_mma_bf16(uint32_t d, uint32_t a, uint32_t blo, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(blo), "n"(kHi128B), "n"(kPxIdPV), "r"(kFirst ? accumulate : 1u)
        : "memory");
}

// Block-scaled products, K = 64 of E2M1 and K = 32 of E4M3, `id` the scales' byte.
template <uint32_t kIdesc>
__device__ __forceinline__ void px_mma_mxf4(uint32_t d, uint32_t alo, uint32_t blo, uint32_t sfa, uint32_t sfb,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], a, b, %4, [%5], [%6], p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "n"(kHi64B), "n"(kIdesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void px_mma_mxf8(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, 0, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], a, b, %4, [%5], [%6], p;\n\t}" ::"r"(d),
        "r"(alo), "r"(blo), "n"(kHi128B), "r"(idesc), "r"(sfa), "r"(sfb)
        : "memory");
}
__device__ __forceinline__ void px_cp_atom(uint32_t taddr, uint32_t lo) {
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
        "r"(lo), "n"(kHiAtom)
        : "memory");
}
__device__ __forceinline__ void px_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void px_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two values of V in bf16. Infinities become the largest finite values. So does a NaN of own keys
// (kPxOwnLeast): the rows of other sequences take it with weight 0, and 0 times it has to be 0. A
// NaN of the prefix, which every row averages, stays one (kPxPrefixLeast: the maximum with a NaN is
// the other value).
constexpr uint32_t kPxOwnLeast = 0xFF7FFF7Fu, kPxPrefixLeast = 0x7FFF7FFFu;
__device__ __forceinline__ uint32_t px_v_bf16x2(float lo, float hi, uint32_t least) {
    uint32_t d;
    asm("{\n\t.reg .b32 t;\n\tcvt.rn.satfinite.bf16x2.f32 t, %1, %2;\n\tmax.bf16x2 %0, t, %3;\n\t}"
        : "=r"(d)
        : "f"(hi), "f"(lo), "r"(least));
    return d;
}

// Waits for the thread's TMEM loads; r's values are not used before.
__device__ __forceinline__ void tc_wait_ld32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void tc_wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// One elected thread of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t pred;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(pred));
    return pred != 0;
}

// One look at an mbarrier phase.
__device__ __forceinline__ bool px_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait on an mbarrier phase: false past 2^31 clocks (a second), or once the CTA's abort flag is
// up. A role whose wait gave up raises the flag at its end (px_give_up), so the others
// follow at once. A dozen instructions, all of them: with waits of sixty at thirty
// places the roles' loops left the SM's instruction cache (103 misses a tile, and every
// instruction of a softmax warp took 15 clk). No time hint either: with one, a try sleeps
// well past the barrier's completion.
__device__ __forceinline__ bool px_wait(uint32_t bar, uint32_t parity, uint32_t flag) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 t0, t1, f;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra PX_DONE;\n\t"
        "mov.u32 t0, %%clock;\n\t"
        "PX_AGAIN:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra PX_DONE;\n\t"
        "ld.volatile.shared.b32 f, [%3];\n\t"
        "mov.u32 t1, %%clock;\n\t"
        "sub.u32 t1, t1, t0;\n\t"
        "setp.lt.s32 q, t1, 0;\n\t"
        "setp.ne.or.b32 q, f, 0, q;\n\t"
        "@!q bra PX_AGAIN;\n\t"
        "PX_DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(flag)
        : "memory");
    return ok != 0;
}

// The reference of a row goes from a tile's owner to the next one's as one 8-byte word with the
// tile's number. px_take: false past 2^31 clocks or once the abort flag is up.
__device__ __forceinline__ void px_pass(uint32_t at, int seqno, float m) {
    asm volatile("st.volatile.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(__float_as_uint(m)), "r"(seqno) : "memory");
}
__device__ __forceinline__ bool px_take(uint32_t at, int seqno, uint32_t flag, float &m) {
    uint32_t ok, v;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 t0, t1, f, n;\n\t"
        "ld.volatile.shared.v2.b32 {%1, n}, [%2];\n\t"
        "setp.eq.s32 p, n, %3;\n\t"
        "@p bra PX_DONE;\n\t"
        "mov.u32 t0, %%clock;\n\t"
        "PX_AGAIN:\n\t"
        "ld.volatile.shared.v2.b32 {%1, n}, [%2];\n\t"
        "setp.eq.s32 p, n, %3;\n\t"
        "@p bra PX_DONE;\n\t"
        "ld.volatile.shared.b32 f, [%4];\n\t"
        "mov.u32 t1, %%clock;\n\t"
        "sub.u32 t1, t1, t0;\n\t"
        "setp.lt.s32 q, t1, 0;\n\t"
        "setp.ne.or.b32 q, f, 0, q;\n\t"
        "@!q bra PX_AGAIN;\n\t"
        "PX_DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok), "=r"(v)
        : "r"(at), "r"(seqno), "r"(flag)
        : "memory");
    m = __uint_as_float(v);
    return ok != 0;
}

__device__ __forceinline__ void px_give_up(volatile uint32_t *flag, int32_t *status) {
    if (*flag) return;
    *flag = 1;
    if (status) atomicCAS(status, 0, QK4V8_ERR_TIMEOUT);
}

// O *= 2^-E for the row (rescale_o_lane without the call).
__device__ __forceinline__ void px_rescale(uint32_t taddr, int E) {
    const float a = E < 126 ? __uint_as_float(static_cast<uint32_t>(127 - E) << 23) : 0.f;
#pragma unroll 1
    for (int c = 0; c < PxSmem::kVRows; c += 4) {
        uint32_t o[4];
        tc_ld_32x32b_x4(taddr + c, o);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
        tc_st_32x32b_x4(taddr + c, o);
    }
    tc_wait_st();
}

// ------------------------------------------------------------------ schedule

constexpr int kPxUnitCost = 1;  // a unit's start and end, in tiles

// Sequence b's own keys.
__device__ __forceinline__ int px_own_len(const PrefixParams &p, int b) {
    return p.own ? imax(0, imin(p.seqlens[b], p.own_most)) : 0;
}

// n / d for 0 <= n < 2^30, 1 <= d <= 128, with m = ceil(2^32 / d): the product's high word is the
// quotient or one more. (A division by a variable is some forty instructions; the feeder's
// two for each query row took 12 us a unit.)
__device__ __forceinline__ int px_div(int n, int d, uint32_t m) {
    if (d == 1) return n;  // 2^32 does not fit m
    const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(n), m));
    return q - (q * d > n ? 1 : 0);
}

// Sequences with rows in row tile qt.
__device__ __forceinline__ int px_seq_lo(const PrefixParams &p, int qt) { return px_div(qt * 128, p.gq, p.m_gq); }
__device__ __forceinline__ int px_seq_hi(const PrefixParams &p, int qt) {
    return px_div(imin(qt * 128 + 128, p.rows) - 1, p.gq, p.m_gq);
}

// Tiles of a unit of row tile qt and its cost (0: no key at all).
__device__ __forceinline__ int px_span(int tiles) { return tiles > 0 ? tiles + kPxUnitCost : 0; }

// A unit's piece in the share, announced in shared memory to all roles (T = 0: no more).
struct PxUnit {
    int qt, h;       // row tile and KV head
    int row0, rows;  // its rows: row0 .. row0 + rows - 1 of the KV head
    int t0, T;       // first key tile and count
    int edge;        // 1: the piece has the unit's first tile, 2: its last one
};
static_assert(sizeof(PxUnit) <= 64, "an entry of the announced units");

// A key tile, described in shared memory by the feeder as it loads it.
struct PxTile {
    int rows;  // rows that see it: first | (last + 1) << 8; own keys: | 1 << 16
    int keys;  // keys from the tile's first on
};

// Steps through the units with a tile in this CTA's share. The whole warp calls it.
struct PxIter {
    int left, qt, h, off;  // cost left in the share; unit, and how far into it
    int tiles;             // key tiles of the units of row tile qt
    __device__ __forceinline__ static int count(const PrefixParams &p, int qt, int lane) {
        int n = 0;
        if (p.own) {
#pragma unroll 1
            for (int b = px_seq_lo(p, qt) + lane; b <= px_seq_hi(p, qt); b += 32) n += (px_own_len(p, b) + 127) >> 7;
            n = __reduce_add_sync(0xffffffffu, n);
        }
        return p.tiles + n;
    }
    __device__ __forceinline__ void begin(const PrefixParams &p, int lane) {
        // The lanes share the row tiles: L lanes to one, which add up its sequences' tiles with
        // their loads in flight together. Pass 0 finds the whole cost, pass 1 the row tile that
        // holds this share's first tile. (All of it fits 31 bits: the host has seen to it.)
        int log_l = 5;
        while (log_l > 0 && (p.row_tiles << log_l) > 32) --log_l;
        const int L = 1 << log_l, step = 32 >> log_l;
        int w = 0, r = 0, c = 0;
        left = qt = h = off = tiles = 0;
#pragma unroll 1
        for (int q0 = 0, pass = 0; pass < 2;) {
            if (pass == 0 || p.row_tiles > step) {  // else c is still there
                const int q = q0 + (lane >> log_l);
                c = 0;
                if (q < p.row_tiles && p.own) {
                    const int b1 = px_seq_hi(p, q);
#pragma unroll 4
                    for (int b = px_seq_lo(p, q) + (lane & (L - 1)); b <= b1; b += L) c += (px_own_len(p, b) + 127) >> 7;
                }
#pragma unroll 1
                for (int o = 1; o < L; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
                c = q < p.row_tiles && (lane & (L - 1)) == 0 ? px_span(p.tiles + c) * p.Hkv : 0;
            }
            if (pass == 0) {
                w += __reduce_add_sync(0xffffffffu, c);
            } else {
                int sum = c;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += v;
                }
                const int k = __popc(__ballot_sync(0xffffffffu, sum <= r));  // lane k's row tile holds r
                const int before = __shfl_sync(0xffffffffu, sum, k > 0 ? k - 1 : 0);
                if (k > 0) r -= before;
                if (k < 32) {
                    qt = q0 + (k >> log_l);
                    break;
                }
            }
            q0 += step;
            if (q0 >= p.row_tiles) {
                if (pass == 0) {
                    const int n = static_cast<int>(gridDim.x);
                    const int share = (w + n - 1) / n;
                    r = static_cast<int>(blockIdx.x) * share;
                    if (r >= w) return;
                    left = imin(share, w - r);
                }
                q0 = 0;
                ++pass;
            }
        }
        tiles = count(p, qt, lane);
        const int span = imax(1, px_span(tiles));
        h = r / span;
        off = r - h * span;
    }
    __device__ __forceinline__ bool next(const PrefixParams &p, int lane, PxUnit &u) {
#pragma unroll 1
        while (left > 0 && qt < p.row_tiles) {
            const int span = px_span(tiles);
            const int take = imin(left, span - off);
            const int lo = imax(off - kPxUnitCost, 0), hi = off + take - kPxUnitCost;
            u.qt = qt;
            u.h = h;
            u.row0 = qt * 128;
            u.rows = imin(128, p.rows - u.row0);
            u.t0 = lo;
            u.T = hi - lo;
            u.edge = (lo == 0 ? 1 : 0) | (hi == tiles ? 2 : 0);
            left -= take;
            off = 0;
            if (++h == p.Hkv) {
                h = 0;
                if (++qt < p.row_tiles) tiles = count(p, qt, lane);
            }
            if (hi > lo) return true;
        }
        u.T = 0;
        return false;
    }
};

// Row n of KV head h: its query head of [B][Hq] and token.
__device__ __forceinline__ int64_t px_row(const PrefixParams &p, int h, int n, int &t) {
    const int b = px_div(n, p.gq, p.m_gq);
    const int r = n - b * p.gq;
    const int g = px_div(r, p.nq, p.m_nq);
    t = r - g * p.nq;
    return static_cast<int64_t>(b) * p.Hq + h * p.G + g;
}

// Asynchronous copies into shared memory; zeros where there is nothing to copy.
__device__ __forceinline__ void px_copy16(uint32_t dst, const void *src, bool any) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(any ? 16 : 0) : "memory");
}
__device__ __forceinline__ void px_copy4(uint32_t dst, const void *src, bool any) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(any ? 4 : 0) : "memory");
}

// Arrives at the barrier once the thread's copies have landed.
__device__ __forceinline__ void px_arrive_copies(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Key tile `tile` of the prefix (seq < 0) or of a sequence's own keys: row and block of the
// K/V arrays. A page outside the pool reads page 0 and is reported.
__device__ __forceinline__ void px_tile(const PrefixParams &p, int h, int seq, int tile, int &row, int &blk) {
    const int32_t *table = seq < 0 ? p.prefix_table : p.block_table;
    if (!table) {
        row = seq < 0 ? h : seq * p.Hkv + h;
        blk = tile;
        return;
    }
    int page = seq < 0 ? table[tile] : table[static_cast<int64_t>(seq) * p.max_pages + tile];
    if (page < 0 || page >= p.num_pages) {
        if (p.status) atomicCAS(p.status, 0, QK4V8_ERR_INVALID_ARG);
        page = 0;
    }
    row = page * p.Hkv + h;
    blk = 0;
}

}  // namespace

__global__ void __launch_bounds__(kPxThreads, 1)
    qk4v8_prefix_kernel(const __grid_constant__ CUtensorMap tmap_pk, const __grid_constant__ CUtensorMap tmap_pv,
                        const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const __grid_constant__ PrefixParams p) {
    using S = PxSmem;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    const uint32_t sb = smem_u32(smem);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kMisc);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + S::kMisc + 4);
    const uint32_t flag = sb + S::kMisc + 4;
    auto wait = [&](uint32_t offset, uint32_t parity) { return px_wait(sb + offset, parity, flag); };
    auto wait_warp = [&](uint32_t offset, uint32_t parity) { return __all_sync(0xffffffffu, wait(offset, parity)) != 0; };

    if (threadIdx.x == 32) {
        auto init = [&](int offset, int n, uint32_t count) {
#pragma unroll 1
            for (int i = 0; i < n; ++i) mbar_init(reinterpret_cast<uint64_t *>(smem + offset + 8 * i), count);
        };
        init(S::kKFull, kPxKStages, 1);
        init(S::kKEmpty, kPxKStages, 1);
        init(S::kRawFull, kPxVStages, 1);
        init(S::kRawEmpty, kPxVStages, 1);
        init(S::kDFull, 2, 1);
        init(S::kDFree, 2, 4);
        init(S::kVFull, kPxVSlots, 8);
        init(S::kVEmpty, kPxVSlots, 1);
        init(S::kQFull, 2, 32);
        init(S::kQEmpty, 2, 1);
        init(S::kSFull, kPxSets, 1);
        init(S::kSFree, kPxSets, 4);
        init(S::kPFull, kPxSets, 4);
        init(S::kPvDone, kPxSets, 1);
        init(S::kOFull, 1, 1);
        init(S::kOFree, 1, kPxSoftmaxWarps);
        init(S::kDrain, 1, 3);
        init(S::kUnitFull, kPxUnits, 1);
        // The three issuers, the expanding and the softmax warps.
        init(S::kUnitEmpty, kPxUnits, 3 + 8 + kPxSoftmaxWarps);
        // A status already set by another launch or CTA: unwind at once, uniformly.
        *reinterpret_cast<uint32_t *>(smem + S::kMisc + 8) = 0;  // no tile to clear
        *abort_flag = (p.status && *reinterpret_cast<const volatile int32_t *>(p.status) != 0) ? 1u : 0u;
        fence_barrier_init();
    }
    if (threadIdx.x == 32 * kPxFeedWarp) {
        prefetch_tensormap(&tmap_pk);
        prefetch_tensormap(&tmap_pv);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    if (warp == kPxQkWarp) {
        tmem_alloc(tmem_slot, kPxTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x < 128) px_pass(smem_u32(smem + S::kRef) + threadIdx.x * 8, -1, 0.f);
    if (warp >= kPxExpandWarp) {
        // Constant rows of the V slots (row 128 = 1.0, rows 129..143 = 0), the unit matrix
        // (E4M3 1.0 is 0x38) and the scales of 2^0.
        const int tid = threadIdx.x - 32 * kPxExpandWarp;
#pragma unroll 1
        for (int i = tid; i < kPxVSlots * 16 * 8; i += 256) {
            const int slot = i >> 7, r = (i >> 3) & 15;
            const uint32_t v = r == 0 ? 0x3F803F80u : 0u;
            *reinterpret_cast<uint4 *>(smem + S::kV + slot * S::kVHalf + (128 + r) * 128 + (i & 7) * 16) =
                make_uint4(v, v, v, v);
        }
#pragma unroll 1
        for (int i = tid; i < 32 * 8; i += 256) {
            const int r = i >> 3, at = (i & 7) ^ (r & 7);  // row r's 16-byte chunk `at`
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            if (at == r >> 4) w[(r >> 2) & 3] = 0x38u << (8 * (r & 3));
            *reinterpret_cast<uint4 *>(smem + S::kUnit + i * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (tid < 32) reinterpret_cast<uint4 *>(smem + S::kSfOne)[tid] =
            make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        fence_proxy_async_smem();
    }
    PxIter it;
    if (warp == kPxFeedWarp) it.begin(p, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The announced units: unit c's entry once it is there, and its release.
    auto unit_at = [&](int c) { return reinterpret_cast<const PxUnit *>(smem + S::kUnits + 64 * (c & (kPxUnits - 1))); };
    auto tile_at = [&](int g) { return reinterpret_cast<const PxTile *>(smem + S::kTiles + 8 * (g & (kPxTiles - 1))); };
    auto unit_wait = [&](int c) { return wait(S::kUnitFull + 8 * (c & (kPxUnits - 1)), (c / kPxUnits) & 1); };
    auto unit_done = [&](int c) { px_arrive(sb + S::kUnitEmpty + 8 * (c & (kPxUnits - 1))); };

    // Rows r0 .. r1 - 1 of a unit's queries into buffer qb by the warp, four lanes to a row: copies
    // that need no register, all in flight (a spilled register goes to L2, as shared memory leaves
    // next to no L1: the gather by loads took 12 us a unit). Rows past the unit's are zero.
    auto gather = [&](const PxUnit &u, int qb, int r0, int r1) {
        const int chunk = lane & 3;
#pragma unroll 1
        for (int r = r0 + (lane >> 2); r < r1; r += 8) {
            const bool any = r < u.rows;
            int t = 0;
            const int64_t bh = any ? px_row(p, u.h, u.row0 + r, t) : 0;
            px_copy16(sb + S::kQ + qb * S::kQBytes + r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4),
                      p.q_codes + (bh * p.q_cap + t) * 64 + chunk * 16, any);
            if (chunk == 0)
                px_copy4(sb + S::kSfQ + qb * 512 + (r & 31) * 16 + (r >> 5) * 4,
                         p.q_scales + bh * (p.q_cap / 128) * 512 + t * 16, any);
        }
    };

    if (warp < kPxSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        // ------------------------------------------------------------------ softmax
        const int quarter = warp & 3, set = warp >> 2;
        const int row = quarter * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_base + kPxColS;
        const uint32_t a_ref = smem_u32(smem + S::kRef) + row * 8;
        const float sc = p.scale_log2 * kPxQScale;
        int k = 0;        // tiles of this set so far
        int first = set;  // how far this set's next tile lies in its unit
        int gt = 0;       // tiles of the units so far
        bool ok = true;
#pragma unroll 1
        for (int c = 0; ok; ++c) {  // units
            ok = __all_sync(0xffffffffu, unit_wait(c));
            const PxUnit &u = *unit_at(c);
            if (!ok || u.T == 0) break;
            const int n = u.T;
            const int late = p.nq - 1 - (u.row0 + row - px_div(u.row0 + row, p.nq, p.m_nq) * p.nq);  // own keys after this row's token
            float m = -INFINITY;  // m_O as of this warp's last tile; -inf: no key yet
            int i = first;
#pragma unroll 1
            for (; i < n; i += kPxSets, ++k) {
                // (A wait that gave up lets the warp go on with whatever is there, to one vote at
                // the tile's end: a vote after each was a tenth of the loop.)
                ok = wait(S::kSFull + 8 * set, k & 1);
                tc_fence_after();
                const PxTile tile = *tile_at(gt + i);
                const int lo = tile.rows & 0xFF, hi = (tile.rows >> 8) & 0xFF;
                const bool active = lo < quarter * 32 + 32 && hi > quarter * 32;  // a row of the warp sees it
                uint32_t s[4][32];
                // Keys j < jv of the tile are seen; a row of another sequence sees none.
                const bool mine = row >= lo && row < hi;
                int jv = tile.keys;
                if (p.causal && (tile.rows >> 16)) jv -= late;
                if (__builtin_expect(active && __any_sync(0xffffffffu, mine && jv < 128), 0)) {
                    // Masked in place, in a short loop: unrolled over the registers it took 2.7 KB
                    // of the instruction cache that all roles share.
#pragma unroll 1
                    for (int j0 = 0; j0 < 128; j0 += 16) {
                        uint32_t v[16];
                        tc_ld_32x32b_x16(tS + j0, v);
                        tc_wait_ld16(v);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (j0 + j >= jv) v[j] = 0xFF800000u;
                        tc_st_32x32b_x16(tS + j0, v);
                    }
                    tc_wait_st();
                }
                if (active) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc_ld_32x32b_x32(tS + 32 * q, s[q]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc_wait_ld32(s[q]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) px_arrive(sb + S::kSFree + 8 * set);  // the next S of this set, while P is computed
                float hm = -INFINITY;
                if (active) {
                    hm = sc * fmaxf(fmaxf(max32(s[0]), max32(s[1])), fmaxf(max32(s[2]), max32(s[3])));
                    if (!mine) hm = -INFINITY;
                }
                // The reference, after the last tile's owner.
                int E = 0;
                const int ps = set == 0 ? kPxSets - 1 : set - 1;
                const int seqno = gt + i;  // the tile's number in the share
                if (i > 0) ok &= px_take(a_ref, seqno - 1, flag, m);
                if (i == 0 || (hm > m && (m == -INFINITY || hm - m > kPxMove))) {
                    if (m > -INFINITY) {
                        // By whole binades, which O can be scaled by; further than those reach, to the
                        // score itself, and O is cleared: the move has no limit, so p stays below 2^64.
                        const float up = hm - m;
                        E = static_cast<int>(ceilf(fminf(up, kPxClear)));
                        m = up < kPxClear ? m + static_cast<float>(E) : hm;
                    } else {
                        m = hm;
                    }
                }
                px_pass(a_ref, seqno, m);
                // This set's P is free once P V of its last tile is done. A warp without rows
                // waits as well: else it could arrive at p_full a second time before the set's
                // other warps have once.
                ok &= wait(S::kPvDone + 8 * set, (k & 1) ^ 1);
                if (i > 0 && __builtin_expect(__any_sync(0xffffffffu, E != 0), 0)) {
                    // O holds the tiles before this one: scale its rows before P V. (The phase
                    // before the awaited one is complete: P V of this set's last tile came
                    // after it.)
                    ok &= wait(S::kPvDone + 8 * ps, (set == 0 ? k - 1 : k) & 1);
                    __syncwarp();
                    tc_fence_after();
                    px_rescale(tmem + lane_base + kPxColO, E);
                }
                __syncwarp();
                tc_fence_after();
                if (!active) {
                    const uint32_t zero[16] = {};
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc_st_32x32b_x16(tmem + lane_base + px_col_p(set) + 16 * q, zero);
                    tc_wait_st();
                } else {
                    // p = 2^(s - m); 0 for a row that sees nothing here (hm = -inf), whose scores are
                    // finite whatever the keys (kPxQShift).
                    const float nm = hm > -INFINITY ? -m : -INFINITY;
                    const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(nm, nm);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 a = ffma2(
                                make_float2(__uint_as_float(s[q][4 * e]), __uint_as_float(s[q][4 * e + 1])), sc2, nm2);
                            const float2 b = ffma2(
                                make_float2(__uint_as_float(s[q][4 * e + 2]), __uint_as_float(s[q][4 * e + 3])), sc2, nm2);
                            w[2 * e] = cvt_bf16x2(exp2_approx(a.x), exp2_approx(a.y));
                            w[2 * e + 1] = cvt_bf16x2(exp2_approx(b.x), exp2_approx(b.y));
                        }
                        tc_st_32x32b_x16(tmem + lane_base + px_col_p(set) + 16 * q, w);
                    }
                    tc_wait_st();
                }
                tc_fence_before();
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) px_arrive(sb + S::kPFull + 8 * set);
            }
            const bool owns_last = i == n + kPxSets - 1;  // this set had the unit's last tile
            first = i - n;
            gt += u.T;
            if (!ok) break;
            // -------------------------------------------------------------- epilogue
            ok = wait_warp(S::kOFull, c & 1);
            if (!ok) break;
            if (quarter * 32 < u.rows) {
                tc_fence_after();
                const float l = __uint_as_float(tc_ld_32x32b_x1(tmem + lane_base + kPxColO + 128));
                tc_wait_ld();
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const int un = u.qt * p.Hkv + u.h;
                const int64_t slot = un + static_cast<int>(blockIdx.x);
                // [slot][32 chunks of 4 channels][128 rows][4]: a warp stores its 32 rows side by side.
                float4 *dst = reinterpret_cast<float4 *>(p.part_o) + slot * (32 * 128) + row;
#pragma unroll 1
                for (int q = set; q < 8; q += kPxSets) {  // 16 channels at a time
                    uint32_t o[16];
                    tc_ld_32x32b_x16(tmem + lane_base + kPxColO + 16 * q, o);
                    tc_wait_ld16(o);
                    if (row < u.rows) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[(4 * q + e) * 128] =
                                make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                            __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
                    }
                }
                // The owner of the unit's last tile has m_O of its end.
                if (owns_last && row < u.rows) p.part_lse[slot * 128 + row] = l > 0.f ? log2f(l) + m : -INFINITY;
                if (threadIdx.x == 0) {
                    if (u.edge & 1) p.first[un] = static_cast<int>(blockIdx.x);
                    if (u.edge & 2) p.last[un] = static_cast<int>(blockIdx.x);
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) {
                px_arrive(sb + S::kOFree);
                unit_done(c);
            }
        }
        if (!ok && lane == 0) px_give_up(abort_flag, p.status);
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kPxFeedWarp) {
        // --------------------------------------------------------------------- feeder
        // Announces the units, gathers each one's query rows (the warp) and loads its key
        // tiles. A unit's rows come before its keys, so they are there when the unit
        // before ends.
        int announced = 0;
        auto announce = [&]() -> bool {
            const int e = announced & (kPxUnits - 1);
            if (!wait_warp(S::kUnitEmpty + 8 * e, ((announced / kPxUnits) & 1) ^ 1)) return false;
            PxUnit v{};
            (void)it.next(p, lane, v);
            if (lane == 0) {
                *reinterpret_cast<PxUnit *>(smem + S::kUnits + 64 * e) = v;
                px_arrive(sb + S::kUnitFull + 8 * e);
            }
            __syncwarp();
            ++announced;
            return true;
        };
        int k_issued = 0, v_issued = 0;  // tiles
        // The tile that comes next: of the prefix (seq < 0) or of sequence seq, whose own keys
        // are len.
        int *lens = reinterpret_cast<int *>(smem + S::kLens);
        int seq = -1, tile = 0, len = 0;
        // `ahead` tiles on, in a unit with rows of the sequences b0 .. b1.
        auto walk = [&](int b0, int b1, int ahead) {
#pragma unroll 1
            for (;;) {
                const int left = ((len + 127) >> 7) - tile;  // of the sequence's tiles
                if (ahead < left || !p.own || seq == b1) break;
                ahead -= left;
                seq = seq < 0 ? b0 : seq + 1;
                len = lens[seq - b0];
                tile = 0;
            }
            tile += ahead;
        };
        // To the piece's first tile, by the warp.
        auto seek = [&](const PxUnit &u) {
            const int b0 = px_seq_lo(p, u.qt), b1 = px_seq_hi(p, u.qt);
            if (p.own)
#pragma unroll 1
                for (int b = b0 + lane; b <= b1; b += 32) lens[b - b0] = px_own_len(p, b);
            __syncwarp();
            seq = -1;
            tile = 0;
            len = p.len;
            walk(b0, b1, u.t0);
        };
        // `count` more tiles of unit u. The lanes look 32 tiles up at once (a page's number
        // takes a trip to memory, and one after the other those took longer than the tiles),
        // lane 0 loads them.
        int4 *next = reinterpret_cast<int4 *>(smem + S::kNext);
        auto load = [&](const PxUnit &u, int count) -> bool {
            const int b0 = px_seq_lo(p, u.qt), b1 = px_seq_hi(p, u.qt);
            bool ok = true;
#pragma unroll 1
            for (int i0 = 0; i0 < count && ok; i0 += 32) {
                const int n = imin(32, count - i0);
                // Lane l goes l tiles ahead; all start the next 32 from n ahead.
                const int mine = imin(lane, n - 1);
                walk(b0, b1, mine);
                int row, blk;
                px_tile(p, u.h, seq, tile, row, blk);
                // Rows of the row tile that see it, keys from its first on, K/V row and block.
                const bool sees = seq < 0;  // all rows do
                const int lo = sees ? 0 : imax(seq * p.gq - u.row0, 0), hi = sees ? 128 : imin((seq + 1) * p.gq - u.row0, 128);
                next[mine] = make_int4(lo | (hi << 8) | (sees ? 0 : 1 << 16), len - tile * 128, row, blk);
                walk(b0, b1, n - mine);
                __syncwarp();
                if (lane == 0) {
#pragma unroll 1
                    for (int i = 0; i < n; ++i) {
                        const int4 d = next[i];
                        const bool own = (d.x >> 16) != 0;
                        const CUtensorMap *mk = own ? &tmap_k : &tmap_pk, *mv = own ? &tmap_v : &tmap_pv;
                        const int vt = d.z * (own ? p.own_blocks : p.prefix_blocks) + d.w;
                        const int64_t at = static_cast<int64_t>(vt) * 512;
                        const int gi = k_issued;
                        const int st = gi & (kPxKStages - 1), sv = gi & (kPxVStages - 1);
                        uint64_t *kf = reinterpret_cast<uint64_t *>(smem + S::kKFull + 8 * st);
                        uint64_t *rf = reinterpret_cast<uint64_t *>(smem + S::kRawFull + 8 * sv);
                        ok = wait(S::kKEmpty + 8 * st, ((gi / kPxKStages) & 1) ^ 1);
                        if (!ok) break;
                        // (The tile eight before is done with: S of the one four before is in the
                        // tensor core's past, so every set has gone on from the eighth.)
                        *reinterpret_cast<PxTile *>(smem + S::kTiles + 8 * (gi & (kPxTiles - 1))) = PxTile{d.x, d.y};
                        mbar_arrive_expect_tx(kf, S::kKBytes + 512);
                        tma_load_3d(smem + S::kK + st * S::kKBytes, mk, 0, d.w * 128, d.z, kf);
                        bulk_load(smem + S::kSfK + st * 512, (own ? p.k_scales : p.p_k_scales) + at, 512, kf);
                        k_issued = gi + 1;
                        ok = wait(S::kRawEmpty + 8 * sv, ((gi / kPxVStages) & 1) ^ 1);
                        if (!ok) break;
                        mbar_arrive_expect_tx(rf, S::kRawBytes + 512);
                        tma_load_3d(smem + S::kRaw + sv * S::kRawBytes, mv, 0, 0, vt, rf);
                        bulk_load(smem + S::kSfV + sv * 512, (own ? p.v_scales : p.p_v_scales) + at, 512, rf);
                        v_issued = gi + 1;
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
            }
            return ok;
        };
        bool ok = true;
#pragma unroll 1
        for (int c = 0; ok; ++c) {
#pragma unroll 1
            while (ok && announced <= c) ok = announce();
            const PxUnit &u = *unit_at(c);
            if (!ok || u.T == 0) break;
            const int qb = c & 1;
            ok = wait_warp(S::kQEmpty + 8 * qb, ((c >> 1) & 1) ^ 1);
            if (!ok) break;
            // q_full completes with the copies; its waiter makes them visible to the tensor core.
            // The first unit's rows are the expanding warps', which wait for V then.
            if (c > 0) {
                gather(u, qb, 0, 128);
                px_arrive_copies(sb + S::kQFull + 8 * qb);
            }
            seek(u);
            ok = load(u, u.T);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (lane == 0) {
            if (!ok) px_give_up(abort_flag, p.status);
            // Let every issued copy land before the CTA can retire.
            auto settle = [&](uint32_t bar, uint32_t parity) {
                const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
                while (!px_try(bar, parity))
                    if (globaltimer_ns() - t0 > kWaitTimeoutNs) break;
            };
#pragma unroll 1
            for (int i = imax(0, k_issued - kPxKStages); i < k_issued; ++i)
                settle(sb + S::kKFull + 8 * (i % kPxKStages), (i / kPxKStages) & 1);
#pragma unroll 1
            for (int i = imax(0, v_issued - kPxVStages); i < v_issued; ++i)
                settle(sb + S::kRawFull + 8 * (i % kPxVStages), (i / kPxVStages) & 1);
        }
        __syncwarp();
    } else if (warp == kPxQkWarp) {
        // ------------------------------------------------------------- Q K^T issuer
        // Each of the three products (S, P V, D) has an issuing thread of its own.
        const uint32_t tSfQ = tmem + kPxColSfQ, tSfK = tmem + kPxColSfK, tS = tmem + kPxColS;
        int g = 0;  // tiles
        bool ok = true;
#pragma unroll 1
        for (int c = 0; ok; ++c) {
            const int qb = c & 1;
            ok = __all_sync(0xffffffffu, unit_wait(c));
            const int T = unit_at(c)->T;
            if (!ok || T == 0) break;
            ok = wait_warp(S::kQFull + 8 * qb, (c >> 1) & 1);
            if (!ok) break;
            {
                uint4 *sf = reinterpret_cast<uint4 *>(smem + S::kSfQ + qb * 512) + lane;
                uint4 v = *sf;
                v.x = __vsubus4(v.x, kPxQShift), v.y = __vsubus4(v.y, kPxQShift);
                v.z = __vsubus4(v.z, kPxQShift), v.w = __vsubus4(v.w, kPxQShift);
                *sf = v;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (elect_one()) {
                unit_done(c);
                tc_fence_after();
                const uint32_t dQ = px_desc_lo(sb + S::kQ + qb * S::kQBytes, 16);
                px_cp_atom(tSfQ, px_desc_lo(sb + S::kSfQ + qb * 512, 0));
#pragma unroll 1
                for (int j = g; j < g + T; ++j) {
                    const int st = j & (kPxKStages - 1);
                    ok = wait(S::kKFull + 8 * st, (j / kPxKStages) & 1);
                    // The set of the tile before has read S.
                    if (j > 0) ok &= wait(S::kSFree + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    px_cp_atom(tSfK, px_desc_lo(sb + S::kSfK, 0) + st * 32);
                    const uint32_t dK = px_desc_lo(sb + S::kK, 16) + st * (S::kKBytes >> 4);
                    px_mma_mxf4<px_sf_id(kPxIdQK, 0)>(tS, dQ, dK, tSfQ, tSfK, 0u);
                    px_mma_mxf4<px_sf_id(kPxIdQK, 2)>(tS, dQ + 2, dK + 2, tSfQ | (2u << 30), tSfK | (2u << 30), 1u);
                    px_commit(sb + S::kSFull + 8 * (j & 1));
                    px_commit(sb + S::kKEmpty + 8 * st);
                }
                if (ok) px_commit(sb + S::kQEmpty + 8 * qb);
            }
            g += T;
            ok = __all_sync(0xffffffffu, ok);
        }
        if (elect_one()) {
            if (!ok) px_give_up(abort_flag, p.status);
            // Every tcgen05 operation of the issuers has completed once `drain` does. (Of this warp
            // the elected thread issues them all.)
            px_commit(sb + S::kDrain);
        }
        __syncwarp();
        (void)wait_peers(reinterpret_cast<uint64_t *>(smem + S::kDrain), 0);
    } else if (warp == kPxPvWarp) {
        // --------------------------------------------------------------- P V issuer
        if (elect_one()) {
            const uint32_t tO = tmem + kPxColO, dV0 = px_desc_lo(sb + S::kV, 16);
            int g = 0;  // tiles
            bool ok = true;
#pragma unroll 1
            for (int c = 0; ok; ++c) {
                ok = unit_wait(c);
                const int T = unit_at(c)->T;
                if (!ok || T == 0) break;
                unit_done(c);
#pragma unroll 1
                for (int i = 0; i < T; ++i, ++g) {
                    const int set = g & 1;
                    if (i == 0 && c >= 1) ok = wait(S::kOFree, (c - 1) & 1);
                    ok = ok && wait(S::kPFull + 8 * set, (g >> 1) & 1);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {  // 64 keys
                        const int slot = (2 * g + half) & (kPxVSlots - 1);
                        ok = ok && wait(S::kVFull + 8 * slot, ((2 * g + half) / kPxVSlots) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t dV = dV0 + slot * (S::kVHalf >> 4), tP = tmem + px_col_p(set) + 32 * half;
                        if (half == 0)
                            px_mma_bf16<true>(tO, tP, dV, i > 0 ? 1u : 0u);
                        else
                            px_mma_bf16<false>(tO, tP, dV, 1u);
#pragma unroll
                        for (int q = 1; q < 4; ++q) px_mma_bf16<false>(tO, tP + 8 * q, dV + 2 * q, 1u);
                        px_commit(sb + S::kVEmpty + 8 * slot);
                    }
                    if (!ok) break;
                    px_commit(sb + S::kPvDone + 8 * set);
                }
                if (!ok) break;
                px_commit(sb + S::kOFull);
            }
            if (!ok) px_give_up(abort_flag, p.status);
            px_commit(sb + S::kDrain);
        }
        __syncwarp();
    } else if (warp == kPxDWarp) {
        // ----------------------------------------------------------------- D issuer
        // D = V of 64 tokens, a channel per TMEM lane and a token per column: the E4M3 codes
        // times a unit matrix, which the tensor core expands with their scales.
        const uint32_t tD = tmem + kPxColD, tSfV = tmem + kPxColSfV, tOne = tmem + kPxColOne;
        const uint32_t dUnit = px_desc_lo(sb + S::kUnit, 16);
        // (One thread and few instructions a tile: its loop is what the expansion waits for. With
        // the warp in it, for the tiles that end early, it took 1350 clk from tile to tile.)
        if (elect_one()) {
            px_cp_atom(tOne, px_desc_lo(sb + S::kSfOne, 0));
            int g = 0;
            uint32_t p0 = 0;  // uses of D's first half so far, mod 2
            bool ok = true;
#pragma unroll 1
            for (int c = 0; ok; ++c) {
                ok = unit_wait(c);
                const int T = unit_at(c)->T;
                if (!ok || T == 0) break;
                unit_done(c);
#pragma unroll 1
                for (int i = 0; i < T; ++i, ++g) {
                    const int sv = g & (kPxVStages - 1);
                    ok = wait(S::kRawFull + 8 * sv, (g / kPxVStages) & 1);
                    // The four warps have read what the half held (its use before this one).
                    ok &= wait(S::kDFree, p0 ^ 1);
                    if (!ok) break;
                    if (__builtin_expect(tile_at(g)->keys < 128, 0)) {
                        // The expanding warps clear what lies past the last token; they take the
                        // request for a use of the half.
                        sts32(sb + S::kMisc + 8, static_cast<uint32_t>(g + 1));
                        px_arrive(sb + S::kDFull);
                        p0 ^= 1;
                        ok = wait(S::kDFree, p0 ^ 1);
                        if (!ok) break;
                    }
                    tc_fence_after();
                    px_cp_atom(tSfV, px_desc_lo(sb + S::kSfV, 0) + sv * 32);
                    const uint32_t dRaw = px_desc_lo(sb + S::kRaw, 16) + sv * (S::kRawBytes >> 4);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {  // 32 tokens, into the halves of D in turn
                        if (q > 0) ok = wait(S::kDFree + 8 * (q & 1), q == 2 ? p0 : q == 1 ? 1u : 0u);
                        if (!ok) break;
                        tc_fence_after();
                        px_mma_mxf8(tD + 32 * (q & 1), dRaw + 2 * q, dUnit, px_sf_id(kPxIdD, q),
                                    tSfV | (static_cast<uint32_t>(q) << 30), tOne | (static_cast<uint32_t>(q) << 30));
                        px_commit(sb + S::kDFull + 8 * (q & 1));
                    }
                    if (!ok) break;
                    px_commit(sb + S::kRawEmpty + 8 * sv);
                }
            }
            if (!ok) px_give_up(abort_flag, p.status);
            px_commit(sb + S::kDrain);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------------- V expansion
        // A thread takes its channel's 32 values of D to bf16, one conversion for two, and into
        // the swizzled K-major row that P V reads.
        // Four warps take D's first half, four its second: with four for both, they were what
        // P V waited for (1100 clk for 64 tokens).
        const int quarter = warp & 3, ch = quarter * 32 + lane, q = (warp - kPxExpandWarp) >> 2;
        const uint32_t tD = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kPxColD + 32 * q;
        const uint32_t full = S::kDFull + 8 * q, free = S::kDFree + 8 * q;
        int k = 0;
        uint32_t f = 0;  // the parity of what comes next
        bool ok = true;
#pragma unroll 1
        for (int c = 0; ok; ++c) {
            ok = __all_sync(0xffffffffu, unit_wait(c));
            const int n = 2 * unit_at(c)->T;
            if (!ok || n == 0) break;
            if (c == 0) {  // the first unit's queries, 16 rows a warp
                const int r0 = 16 * (warp - kPxExpandWarp);
                gather(*unit_at(0), 0, r0, r0 + 16);
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                if (lane < 4 && !p.test_stall) px_arrive(sb + S::kQFull);  // 32 in all, as from the feeder
            }
            __syncwarp();
            if (lane == 0) unit_done(c);
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++k) {
                const int slot = k & (kPxVSlots - 1);
                ok = wait(full, f);
                f ^= 1;
                if (q == 0 && (k & 1) == 0 && lds32(sb + S::kMisc + 8) == (k >> 1) + 1u) {
                    // This tile ends early, and D is not there yet. Codes past the last token may be
                    // anything (a NaN would spread): zeros, in the thread's channel.
                    const int sv = (k >> 1) & (kPxVStages - 1), jv = tile_at(k >> 1)->keys;
                    uint8_t *codes = smem + S::kRaw + sv * S::kRawBytes + ch * 128;
#pragma unroll 1
                    for (int at = jv >> 4; at < 8; ++at) {
                        uint8_t *chunk = codes + ((at ^ (ch & 7)) << 4);
                        if (16 * at >= jv) {
                            *reinterpret_cast<uint4 *>(chunk) = make_uint4(0, 0, 0, 0);
                        } else {
#pragma unroll 1
                            for (int e = jv - 16 * at; e < 16; ++e) chunk[e] = 0;
                        }
                    }
                    uint8_t *sfv = smem + S::kSfV + sv * 512 + (ch & 31) * 16 + (ch >> 5) * 4;
#pragma unroll 1
                    for (int at = (jv + 31) >> 5; at < 4; ++at) sfv[at] = 0;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) px_arrive(sb + free);
                    ok &= wait(full, f);
                    f ^= 1;
                }
                // (The entry is the tile's until the warps have read its D.)
                const uint32_t least = tile_at(k >> 1)->rows >> 16 ? kPxOwnLeast : kPxPrefixLeast;
                ok &= wait(S::kVEmpty + 8 * slot, ((k / kPxVSlots) & 1) ^ 1);
                tc_fence_after();
                __syncwarp();
                const uint32_t row = sb + S::kV + slot * S::kVHalf + ch * 128;
#pragma unroll
                for (int e0 = 0; e0 < 2; ++e0) {  // 16 tokens
                    uint32_t d[16];
                    tc_ld_32x32b_x16(tD + 16 * e0, d);
                    tc_wait_ld16(d);
                    if (e0 == 1) {
                        tc_fence_before();
                        if (lane == 0) px_arrive(sb + free);
                    }
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e] = px_v_bf16x2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1]), least);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        sts128(row + (((4 * q + 2 * e0 + e) ^ (ch & 7)) << 4), w[4 * e], w[4 * e + 1], w[4 * e + 2],
                               w[4 * e + 3]);
                }
                fence_proxy_async_smem();
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) px_arrive(sb + S::kVFull + 8 * slot);
            }
        }
        if (!ok && lane == 0) px_give_up(abort_flag, p.status);
    }
    }
    teardown_tmem(warp == kPxQkWarp, tmem, kPxTmemCols);
}

// Joins the partial results of each query row: those of its unit, one for each share the
// unit has a part in, in slots unit + share. A CTA takes 32 rows and 32 channels of a unit,
// a warp four channels, a lane a row, as they are stored; then through shared memory to
// whole rows. kBatch partials are in flight: 8 where the units are fewer than the shares (a
// unit has several then; 3.9 us for 18 of them, 9 us one after the other), 2 where they are
// more, with as many threads again on the SM.
template <int kBatch>
__global__ void __launch_bounds__(256, kBatch == 2 ? 6 : 4)
    qk4v8_prefix_merge_kernel(const PrefixParams p, __nv_bfloat16 *__restrict__ out, float *__restrict__ lse) {
    __shared__ uint2 tile[32][9];  // [row][chunk], 4 bf16
    const int un = static_cast<int>(blockIdx.x >> 4);
    const int row0 = (blockIdx.x >> 2 & 3) * 32;  // of the unit
    const int chunk0 = (blockIdx.x & 3) * 8;
    const int qt = un / p.Hkv, h = un - qt * p.Hkv;
    if (qt * 128 + row0 >= p.rows) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = row0 + lane;
    const int n = qt * 128 + row;  // of the KV head
    // (A row without a key may belong to a unit without a tile, which nobody wrote. The counts are
    // held to the shares there are: a kernel that gave up leaves none.)
    const bool in = n < p.rows;
    const int c0 = imax(0, imin(p.first[un], p.shares - 1));
    const int np = imax(0, imin(p.last[un], p.shares - 1) - c0 + 1);
    const bool keys = in && (p.tiles > 0 || px_own_len(p, px_div(n, p.gq, p.m_gq)) > 0);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f, m = -INFINITY;
    if (keys) {
        const float *lp = p.part_lse + static_cast<int64_t>(un + c0) * 128 + row;
        const float4 *po = reinterpret_cast<const float4 *>(p.part_o) + static_cast<int64_t>(un + c0) * (32 * 128) +
                           (chunk0 + warp) * 128 + row;
        for (int s0 = 0; s0 < np; s0 += kBatch) {
            float l[kBatch];
            float4 v[kBatch];
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                l[s] = -INFINITY;
                v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s0 + s < np) {
                    l[s] = lp[(s0 + s) * 128];
                    v[s] = po[static_cast<int64_t>(s0 + s) * (32 * 128)];
                }
            }
            float top = m;
#pragma unroll
            for (int s = 0; s < kBatch; ++s) top = fmaxf(top, l[s]);
            if (top == -INFINITY) continue;
            const float w0 = exp2f(m - top);
            m = top;
            sum *= w0;
            acc.x *= w0, acc.y *= w0, acc.z *= w0, acc.w *= w0;
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                const float w = exp2f(l[s] - m);
                sum += w;
                acc.x += w * v[s].x;
                acc.y += w * v[s].y;
                acc.z += w * v[s].z;
                acc.w += w * v[s].w;
            }
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    tile[lane][warp] = make_uint2(cvt_bf16x2(acc.x * inv, acc.y * inv), cvt_bf16x2(acc.z * inv, acc.w * inv));
    int t;
    if (lse && chunk0 + warp == 0 && in) {
        const int64_t bh = px_row(p, h, n, t);
        lse[bh * p.nq + t] = sum > 0.f ? (log2f(sum) + m) * 0.6931471805599453f : -INFINITY;
    }
    __syncthreads();
    const int r = threadIdx.x >> 3, c = threadIdx.x & 7;
    if (qt * 128 + row0 + r >= p.rows) return;
    const int64_t bh = px_row(p, h, qt * 128 + row0 + r, t);
    const int64_t b = bh / p.Hq;
    reinterpret_cast<uint2 *>(out + ((b * p.nq + t) * p.Hq + (bh - b * p.Hq)) * 128)[chunk0 + c] = tile[r][c];
}

cudaError_t launch_prefix(const CUtensorMap &pk, const CUtensorMap &pv, const CUtensorMap &k, const CUtensorMap &v,
                          const PrefixParams &p, void *out, float *lse, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static bool configured[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !configured[dev]) {
        e = cudaFuncSetAttribute(qk4v8_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PxSmem::kBytes);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) configured[dev] = true;
    }
    if (p.shares > 0) {
        qk4v8_prefix_kernel<<<p.shares, kPxThreads, PxSmem::kBytes, stream>>>(pk, pv, k, v, p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const unsigned units = static_cast<unsigned>(p.row_tiles) * static_cast<unsigned>(p.Hkv);
    auto *o = static_cast<__nv_bfloat16 *>(out);
    if (units < static_cast<unsigned>(p.shares))
        qk4v8_prefix_merge_kernel<8><<<16u * units, 256, 0, stream>>>(p, o, lse);
    else
        qk4v8_prefix_merge_kernel<2><<<16u * units, 256, 0, stream>>>(p, o, lse);
    return cudaGetLastError();
}

}  // namespace qk4v8
