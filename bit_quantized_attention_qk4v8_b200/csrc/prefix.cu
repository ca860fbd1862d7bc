// Attention of a whole batch over the prefix that its sequences share.
//
// With a shared prefix, the query rows of all B sequences that read one KV head
// (B * G * nq of them) multiply the same keys, so decode over the prefix is a matrix
// product again: each K/V tile is read once for 128 rows instead of once per
// sequence. softmax over [prefix, own keys] splits into two partial results with
// their log-sum-exp, which qk4v8_prefix_merge_kernel joins:
//   O = sum_s 2^(lse_s - m) O_s / sum_s 2^(lse_s - m).
//
// One CTA takes 128 query rows of a KV head (rows in (sequence, head, token) order,
// gathered from the packed queries) against a split of the prefix, 128 keys a tile:
//   S = Q K^T     kind::mxf4, E2M1 operands, the E8M0 scales read from TMEM.
//   O += P V      kind::f16 on bf16 operands: P from TMEM, V expanded from E4M3.
//
// Why bf16 and not the E4M3 MMAs of the other attention kernels: they write P as
// two E4M3 terms with a block scale, about 9 instructions a score, which bounds
// them. bf16 holds the same 8 significant bits in one conversion for two scores,
// needs no block scale (its exponent takes p up to 2^64 above the reference), and
// goes to TMEM without a swizzled store: about 3 instructions a score, so the
// exponentials themselves (16 a clock and SM: 1024 clk a tile) become the bound.
// V costs 2.3 instructions an element to expand, exactly (an E4M3 value times a
// power of two has 4 significant bits), shared by the tile's 128 rows, on warps of
// their own.
//
// Softmax: two sets of four warps take alternate key tiles, one row per thread, all
// 128 keys. P (64 columns) overwrites the front of S in the same buffer; S of tile i + 2 is issued behind P V of tile i, so the tensor
// pipe's own order protects it. O has one reference per row, the row max of the
// unit's first tile; p = 2^(s - m_O). It moves only when a later score passes it by
// 2^64 (bf16 and fp32 keep their relative precision at any offset, so nothing is
// gained by moving it sooner): the tile's owner then scales its row of O after the
// P V before its own. The reference passes from a tile's owner to the next one's in
// shared memory, right after the row max, well before the exponentials.
// V carries a row of ones, so O column 128 sums P as rounded.
//
// Warp roles (512 threads): warps 0..7 softmax and epilogue, 8 K/V producer, 9 TMEM
// allocator and MMA issuer, 10 query gather, 12..15 V expansion.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pipeline.cuh"
#include "ptx.cuh"
#include "qk4v8_internal.h"
#include "tile_ops.cuh"

namespace qk4v8 {

namespace {

constexpr int kPxKStages = 6;
constexpr int kPxVStages = 4;
constexpr int kPxThreads = 512;
constexpr int kPxProducerWarp = 8;
constexpr int kPxMmaWarp = 9;
constexpr int kPxQWarp = 10;
constexpr int kPxExpandWarp = 12;
constexpr float kPxMove = 64.0f;      // m_O moves once a score passes it by 2^64
constexpr float kPxMaxMove = 65536.0f;

struct PxSmem {
    static constexpr int kQBytes = 128 * 64;
    static constexpr int kQ = 0;                                  // 2 buffers, 64-byte swizzle
    static constexpr int kKBytes = 128 * 64;
    static constexpr int kK = kQ + 2 * kQBytes;                   // per stage: 128 keys x 64 B, 64-byte swizzle
    static constexpr int kVRows = 144;                            // 128 channels, the ones row, 15 zero rows
    static constexpr int kVHalf = kVRows * 128;                   // 64 tokens of bf16 per row
    static constexpr int kVBytes = 2 * kVHalf;
    static constexpr int kV = kK + kPxKStages * kKBytes;          // 2 buffers of bf16 V, 128-byte swizzle
    static constexpr int kRawBytes = 128 * 128;
    static constexpr int kRaw = kV + 2 * kVBytes;                 // per stage: E4M3 block, channel rows
    static constexpr int kSfQ = kRaw + kPxVStages * kRawBytes;    // 512-byte scale atoms
    static constexpr int kSfK = kSfQ + 2 * 512;
    static constexpr int kSfV = kSfK + kPxKStages * 512;
    static constexpr int kRef = kSfV + kPxVStages * 512;          // float [2][128]: m_O by tile parity
    static constexpr int kBar = kRef + 2 * 128 * 4;
    // k_full/k_empty, raw_full/raw_empty per stage; v_full/v_empty per bf16 buffer;
    // q_full/q_empty per Q buffer; s_full, p_full, pv_done per set; o_full, o_free,
    // drain; reference [4 quarters][2].
    static constexpr int kNumBars = 2 * kPxKStages + 2 * kPxVStages + 4 + 4 + 6 + 3 + 8;
    static constexpr int kMisc = kBar + kNumBars * 8;
    static constexpr int kUsed = kMisc + 16;
    static constexpr int kBytes = kUsed + 1024;
};
static_assert(PxSmem::kK % 1024 == 0 && PxSmem::kV % 1024 == 0 && PxSmem::kVHalf % 1024 == 0,
              "swizzled tiles need 1024-byte alignment");
static_assert(PxSmem::kBar % 8 == 0 && PxSmem::kRaw % 16 == 0, "alignment");
static_assert(PxSmem::kBytes <= 227 * 1024, "shared memory budget");

constexpr uint32_t kPxTmemCols = 512;
constexpr uint32_t kPxColO = 256;  // 144 columns
__device__ __forceinline__ uint32_t px_col_s(int set) { return 128u * set; }  // P in its first 64 columns
__device__ __forceinline__ uint32_t px_col_sf_q(int qb) { return 400u + 4u * qb; }
__device__ __forceinline__ uint32_t px_col_sf_k(int set) { return 408u + 4u * set; }

// Block-scaled E2M1 x E2M1, N = 128 keys; bf16 x bf16 into fp32, N = 144.
constexpr uint32_t kPxIdQK = (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24);
constexpr uint32_t kPxIdPV =
    (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t(PxSmem::kVRows) >> 3) << 17) | ((128u >> 4) << 24);
__device__ __forceinline__ uint32_t px_sf_id(uint32_t idesc, uint32_t id) { return idesc | (id << 29) | (id << 4); }

// D[128, N] (+)= A B, A bf16 in TMEM (two K elements a column), B bf16 in shared memory.
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Waits for the thread's TMEM loads; r's values are not used before.
__device__ __forceinline__ void tc_wait_ld32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// One elected thread of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t pred;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(pred));
    return pred != 0;
}

struct PxUnit {
    int h, q0, split, t0, T;  // KV head, first row, split, its first key tile and count
};

// Units that run side by side share a split's keys (consecutive row tiles).
__device__ __forceinline__ PxUnit px_unit(const PrefixParams &p, int idx) {
    PxUnit u;
    const int qt = idx % p.row_tiles;
    idx /= p.row_tiles;
    u.h = idx % p.Hkv;
    u.split = idx / p.Hkv;
    u.q0 = qt * 128;
    u.t0 = static_cast<int>(static_cast<int64_t>(u.split) * p.tiles / p.splits);
    u.T = static_cast<int>(static_cast<int64_t>(u.split + 1) * p.tiles / p.splits) - u.t0;
    return u;
}

// Row n of KV head h: query head, sequence and token; returns the row of [B][Hq][nq].
__device__ __forceinline__ int64_t px_row(const PrefixParams &p, int h, int n, int64_t &bh, int &t) {
    t = n % p.nq;
    const int bg = n / p.nq;
    const int b = bg / p.G;
    bh = static_cast<int64_t>(b) * p.Hq + h * p.G + (bg - b * p.G);
    return bh * p.nq + t;
}

// The prefix's tile `tile` of head h: row and block of the K/V arrays. A page outside
// the pool reads page 0 and is reported.
__device__ __forceinline__ void px_tile(const PrefixParams &p, int h, int tile, int &row, int &blk) {
    if (!p.table) {
        row = h;
        blk = tile;
        return;
    }
    int page = p.table[tile];
    if (page < 0 || page >= p.num_pages) {
        if (p.status) atomicCAS(p.status, 0, 1);
        page = 0;
    }
    row = page * p.Hkv + h;
    blk = 0;
}

}  // namespace

__global__ void __launch_bounds__(kPxThreads, 1)
    qk4v8_prefix_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ PrefixParams p) {
    using S = PxSmem;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kBar);
    uint64_t *k_full = bars;
    uint64_t *k_empty = k_full + kPxKStages;
    uint64_t *raw_full = k_empty + kPxKStages;
    uint64_t *raw_empty = raw_full + kPxVStages;
    uint64_t *v_full = raw_empty + kPxVStages;  // [bf16 buffer]
    uint64_t *v_empty = v_full + 2;
    uint64_t *q_full = v_empty + 2;             // [Q buffer]
    uint64_t *q_empty = q_full + 2;
    uint64_t *s_full = q_empty + 2;             // [set]
    uint64_t *p_full = s_full + 2;              // [set]
    uint64_t *pv_done = p_full + 2;             // [set]
    uint64_t *o_full = pv_done + 2;
    uint64_t *o_free = o_full + 1;
    uint64_t *drain = o_free + 1;
    uint64_t *ref_bar = drain + 1;              // [quarter][tile parity]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kMisc);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + S::kMisc + 4);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPxKStages; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < kPxVStages; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&v_full[s], 4);
            mbar_init(&v_empty[s], 1);
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&pv_done[s], 1);
        }
        mbar_init(o_full, 1);
        mbar_init(o_free, 8);
        mbar_init(drain, 1);
        for (int g = 0; g < 8; ++g) mbar_init(&ref_bar[g], 1);
        // A status already set by another launch or CTA: unwind at once, uniformly.
        *abort_flag = (p.status && *reinterpret_cast<const volatile int32_t *>(p.status) != 0) ? 1u : 0u;
        fence_barrier_init();
    }
    if (warp == kPxMmaWarp) {
        tmem_alloc(tmem_slot, kPxTmemCols);
        tmem_relinquish();
    }
    if (warp >= kPxExpandWarp) {
        // Constant rows of both V buffers: row 128 = 1.0, rows 129..143 = 0.
        for (int i = threadIdx.x - 32 * kPxExpandWarp; i < 2 * 2 * 16 * 8; i += 128) {
            const int half = i >> 7, r = (i >> 3) & 15;
            const uint32_t v = r == 0 ? 0x3F803F80u : 0u;
            *reinterpret_cast<uint4 *>(smem + S::kV + half * S::kVHalf + (128 + r) * 128 + (i & 7) * 16) =
                make_uint4(v, v, v, v);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == kPxProducerWarp) {
        // ------------------------------------------------------------- K/V producer
        if (elect_one()) {
            prefetch_tensormap(&tmap_k);
            int g = 0;                   // tiles so far
            int k_issued = 0, v_issued = 0;
            bool ok = true;
            for (int un = blockIdx.x; un < p.units && ok; un += gridDim.x) {
                const PxUnit u = px_unit(p, un);
                int row, blk;
                px_tile(p, u.h, u.t0, row, blk);
                for (int i = 0; i < u.T; ++i) {
                    int nrow = 0, nblk = 0;
                    if (i + 1 < u.T) px_tile(p, u.h, u.t0 + i + 1, nrow, nblk);  // ahead of the waits
                    const int gi = g + i;
                    const int st = gi % kPxKStages, sv = gi % kPxVStages;
                    const int64_t at = static_cast<int64_t>(row) * p.row_blocks + blk;
                    ok = wait_bar(&k_empty[st], ((gi / kPxKStages) & 1) ^ 1, abort_flag, p.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&k_full[st], S::kKBytes + 512);
                    tma_load_3d(smem + S::kK + st * S::kKBytes, &tmap_k, 0, blk * 128, row, &k_full[st]);
                    bulk_load(smem + S::kSfK + st * 512, p.k_scales + at * 512, 512, &k_full[st]);
                    k_issued = gi + 1;
                    ok = wait_bar(&raw_empty[sv], ((gi / kPxVStages) & 1) ^ 1, abort_flag, p.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&raw_full[sv], S::kRawBytes + 512);
                    bulk_load(smem + S::kRaw + sv * S::kRawBytes, p.v_codes + at * S::kRawBytes, S::kRawBytes,
                              &raw_full[sv]);
                    bulk_load(smem + S::kSfV + sv * 512, p.v_scales + at * 512, 512, &raw_full[sv]);
                    v_issued = gi + 1;
                    row = nrow;
                    blk = nblk;
                }
                g += u.T;
            }
            // Let every issued copy land before the CTA can retire.
            auto settle = [&](uint64_t *bar, uint32_t parity) {
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(bar, parity))
                    if (globaltimer_ns() - t0 > kWaitTimeoutNs) break;
            };
            for (int i = imax(0, k_issued - kPxKStages); i < k_issued; ++i)
                settle(&k_full[i % kPxKStages], (i / kPxKStages) & 1);
            for (int i = imax(0, v_issued - kPxVStages); i < v_issued; ++i)
                settle(&raw_full[i % kPxVStages], (i / kPxVStages) & 1);
        }
        __syncwarp();
    } else if (warp == kPxQWarp) {
        // ------------------------------------------------------------- query gather
        int c = 0;  // units so far
        for (int un = blockIdx.x; un < p.units; un += gridDim.x, ++c) {
            const PxUnit u = px_unit(p, un);
            const int qb = c & 1;
            if (!__all_sync(0xffffffffu, wait_bar(&q_empty[qb], ((c >> 1) & 1) ^ 1, abort_flag, p.status))) break;
            uint8_t *qbuf = smem + S::kQ + qb * S::kQBytes;
            uint8_t *sfq = smem + S::kSfQ + qb * 512;
            // Rows lane / 4 + 8 i, 16-byte chunk lane % 4: four loads of a lane in flight.
#pragma unroll 1
            for (int i0 = 0; i0 < 16; i0 += 4) {
                uint4 code[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = u.q0 + (lane >> 2) + 8 * (i0 + i);
                    code[i] = make_uint4(0, 0, 0, 0);
                    if (n < p.rows) {
                        int64_t bh;
                        int t;
                        px_row(p, u.h, n, bh, t);
                        code[i] = *reinterpret_cast<const uint4 *>(p.q_codes + (bh * p.q_cap + t) * 64 + (lane & 3) * 16);
                    }
                }
                const int rs = u.q0 + lane + 8 * i0;  // scale word of row lane + 32 (i0 / 4)
                uint32_t sf = 0;
                if (rs < p.rows) {
                    int64_t bh;
                    int t;
                    px_row(p, u.h, rs, bh, t);
                    sf = *reinterpret_cast<const uint32_t *>(p.q_scales + bh * (p.q_cap / 128) * 512 + t * 16);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = (lane >> 2) + 8 * (i0 + i);
                    *reinterpret_cast<uint4 *>(qbuf + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4)) = code[i];
                }
                *reinterpret_cast<uint32_t *>(sfq + lane * 16 + i0) = sf;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && !(p.test_stall && c == 0)) mbar_arrive(&q_full[qb]);
        }
    } else if (warp == kPxMmaWarp) {
        // -------------------------------------------------------------- MMA issuer
        if (elect_one()) {
            const uint32_t sb = smem_u32(smem);
            const uint64_t dQ0 = smem_desc(sb + S::kQ, 16, 512, 4);
            const uint64_t dK0 = smem_desc(sb + S::kK, 16, 512, 4);
            const uint64_t dV0 = smem_desc(sb + S::kV, 16, 1024, 2);
            const uint64_t dSfQ0 = smem_desc(sb + S::kSfQ, 0, 128, 0);
            const uint64_t dSfK0 = smem_desc(sb + S::kSfK, 0, 128, 0);
            const uint32_t tO = tmem + kPxColO;
            bool ok = true;
            int g = 0, c = 0;
            for (int un = blockIdx.x; un < p.units && ok; un += gridDim.x) {
                const int T = px_unit(p, un).T;
                const int qb = c & 1;
                ok = wait_bar(&q_full[qb], (c >> 1) & 1, abort_flag, p.status);
                if (!ok) break;
                tc_fence_after();
                const uint32_t tSfQ = tmem + px_col_sf_q(qb);
                const uint64_t dQ = dQ0 + static_cast<uint64_t>(qb * (S::kQBytes >> 4));
                tc_cp_32x128b_warpx4(tSfQ, dSfQ0 + static_cast<uint64_t>(qb * 32));
                // S(gi) into buffer gi & 1: behind P V(gi - 2) in the tensor pipe, and the
                // warps read S(gi - 2) before they wrote that P.
                auto issue_qk = [&](int i) -> bool {
                    const int gi = g + i, st = gi % kPxKStages;
                    if (!wait_bar(&k_full[st], (gi / kPxKStages) & 1, abort_flag, p.status)) return false;
                    tc_fence_after();
                    const uint32_t tSfK = tmem + px_col_sf_k(gi & 1), tS = tmem + px_col_s(gi & 1);
                    const uint64_t dK = dK0 + static_cast<uint64_t>(st * (S::kKBytes >> 4));
                    tc_cp_32x128b_warpx4(tSfK, dSfK0 + static_cast<uint64_t>(st * 32));
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        tc_mma_mxf4(tS, dQ + 2 * k, dK + 2 * k, px_sf_id(kPxIdQK, 2 * k), tSfQ | ((2u * k) << 30),
                                    tSfK | ((2u * k) << 30), k > 0 ? 1u : 0u);
                    tc_commit(&s_full[gi & 1]);
                    tc_commit(&k_empty[st]);
                    return true;
                };
                auto issue_pv = [&](int i) -> bool {
                    const int gi = g + i, vb = gi & 1;
                    if (!wait_bar(&v_full[vb], (gi >> 1) & 1, abort_flag, p.status)) return false;
                    if (i == 0 && c >= 1 && !wait_bar(o_free, (c - 1) & 1, abort_flag, p.status)) return false;
                    if (!wait_bar(&p_full[gi & 1], (gi >> 1) & 1, abort_flag, p.status)) return false;
                    tc_fence_after();
                    const uint32_t tP = tmem + px_col_s(gi & 1);
                    const uint64_t dV = dV0 + static_cast<uint64_t>(vb * (S::kVBytes >> 4));
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tc_mma_bf16_ts(tO, tP + 8 * k, dV + static_cast<uint64_t>((k >> 2) * (S::kVHalf >> 4) + 2 * (k & 3)),
                                       kPxIdPV, (i > 0 || k > 0) ? 1u : 0u);
                    tc_commit(&pv_done[gi & 1]);
                    tc_commit(&v_empty[vb]);
                    return true;
                };
                ok = issue_qk(0);
                if (ok && T > 1) ok = issue_qk(1);
                for (int i = 0; i < T && ok; ++i) {
                    ok = issue_pv(i);
                    if (ok && i + 2 < T) ok = issue_qk(i + 2);
                }
                if (!ok) break;
                tc_commit(&q_empty[qb]);
                tc_commit(o_full);
                g += T;
                ++c;
            }
            // Every tcgen05 operation issued above has completed once `drain` does.
            tc_commit(drain);
        }
        __syncwarp();
        (void)wait_peers(drain, 0);
    } else if (warp >= kPxExpandWarp) {
        // -------------------------------------------------------------- V expansion
        // E4M3 byte s eeee mmm -> bf16 s 0000eeee mmm0000, which is the value times 2^-120
        // (subnormals too), then times 2^(X + 120): exact. A thread takes 16 tokens of a
        // channel at a time; of each four the order becomes 0, 2, 1, 3, the order in
        // which P's columns are written.
        const int tid = threadIdx.x - 32 * kPxExpandWarp;
        const int j = tid & 7;  // 16-token chunk of the channel row
        int g = 0;
        bool ok = true;
        for (int un = blockIdx.x; un < p.units && ok; un += gridDim.x) {
            const PxUnit u = px_unit(p, un);
            for (int i = 0; i < u.T; ++i) {
                const int gi = g + i, sv = gi % kPxVStages, vb = gi & 1;
                ok = wait_bar(&raw_full[sv], (gi / kPxVStages) & 1, abort_flag, p.status);
                ok = __all_sync(0xffffffffu, ok && wait_bar(&v_empty[vb], ((gi >> 1) & 1) ^ 1, abort_flag, p.status));
                if (!ok) break;
                const uint32_t raw = smem_u32(smem + S::kRaw + sv * S::kRawBytes) + j * 16;
                const uint8_t *sfv = smem + S::kSfV + sv * 512 + (j >> 1);
                const uint32_t out = smem_u32(smem + S::kV + vb * S::kVBytes) + (j >> 2) * S::kVHalf;
                // Tokens past the prefix may hold anything: their codes become zero.
                const int left = p.len - (u.t0 + i) * 128 - 16 * j;  // valid tokens from this chunk's first on
#pragma unroll 4
                for (int it = 0; it < 8; ++it) {
                    const int c = it * 16 + (tid >> 3);
                    const uint4 v4 = lds128(raw + c * 128);
                    uint32_t w[4] = {v4.x, v4.y, v4.z, v4.w};
                    int e = sfv[(c & 31) * 16 + (c >> 5) * 4] + 120;  // exponent field of 2^(X + 120)
                    if (left < 16) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int n = left - 4 * q;  // valid bytes of the word
                            w[q] = n <= 0 ? 0u : n >= 4 ? w[q] : w[q] & ((1u << (8 * n)) - 1u);
                        }
                        if (left <= 0) e = 127;
                    }
                    const int e1 = imin(e, 254);
                    const uint32_t f = static_cast<uint32_t>(e1) * 0x00800080u;
                    uint32_t o[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[2 * q] = mul_bf16x2(((w[q] << 4) & 0x07F007F0u) | ((w[q] << 8) & 0x80008000u), f);
                        o[2 * q + 1] = mul_bf16x2(((w[q] >> 4) & 0x07F007F0u) | (w[q] & 0x80008000u), f);
                    }
                    if (e > 254) {  // values past 2^16: the rest of the power in a second factor
                        const uint32_t f2 = static_cast<uint32_t>(e - 254 + 127) * 0x00800080u;
#pragma unroll
                        for (int q = 0; q < 8; ++q) o[q] = mul_bf16x2(o[q], f2);
                    }
                    // 16-byte pieces 2 (j % 4) and + 1 of the row; odd and even halves of the
                    // lanes write them in opposite order, so 8 lanes meet 8 different banks.
                    const uint32_t dst = out + c * 128;
                    const int q0 = 2 * (j & 3), sw = c & 7, flip = j >> 2;
                    const uint32_t a0 = dst + (((q0 + flip) ^ sw) << 4), a1 = dst + (((q0 + 1 - flip) ^ sw) << 4);
                    sts128(a0, flip ? o[4] : o[0], flip ? o[5] : o[1], flip ? o[6] : o[2], flip ? o[7] : o[3]);
                    sts128(a1, flip ? o[0] : o[4], flip ? o[1] : o[5], flip ? o[2] : o[6], flip ? o[3] : o[7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&v_full[vb]);
                    mbar_arrive(&raw_empty[sv]);
                }
            }
            g += u.T;
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------------ softmax
        const int quarter = warp & 3, set = warp >> 2;
        const int row = quarter * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_base + px_col_s(set);
        const uint32_t a_ref = smem_u32(smem + S::kRef) + row * 4;
        uint64_t *ref = ref_bar + quarter * 2;
        const float sc = p.scale_log2;
        int g = 0, c = 0;
        bool ok = true;
        for (int un = blockIdx.x; un < p.units && ok; un += gridDim.x) {
            const PxUnit u = px_unit(p, un);
            const int T = u.T;
            float m = 0.f;  // m_O as of this warp's last tile
            for (int i = (set - g) & 1; i < T; i += 2) {
                const int gi = g + i, k = gi >> 1;
                ok = __all_sync(0xffffffffu, wait_bar(&s_full[set], k & 1, abort_flag, p.status));
                if (!ok) break;
                // The reference as the last tile's owner left it (posted long ago as a rule).
                float prev = 0.f;
                if (gi > 0) {
                    ok = __all_sync(0xffffffffu, wait_bar(&ref[(gi - 1) & 1], ((gi - 1) >> 1) & 1, abort_flag, p.status));
                    if (!ok) break;
                    prev = __uint_as_float(lds32(a_ref + ((gi - 1) & 1) * 512));
                }
                tc_fence_after();
                const int jv = p.len - (u.t0 + i) * 128;  // keys of the tile, at least 1
                // 32 scores of the row; keys past the prefix are -inf.
                auto load_scores = [&](int q, uint32_t (&s)[32]) { tc_ld_32x32b_x32(tS + 32 * q, s); };
                auto mask = [&](int q, uint32_t (&s)[32]) {
                    if (jv < 32 * q + 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (32 * q + j >= jv) s[j] = 0xFF800000u;
                    }
                };
                // The row max first, in a pass of its own: the scores are read from TMEM
                // again for the exponentials rather than held (128 of the 128 registers).
                float hm = -INFINITY;
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    uint32_t s0[32], s1[32];
                    load_scores(q, s0);
                    load_scores(q + 1, s1);
                    tc_wait_ld32(s0);
                    tc_wait_ld32(s1);
                    mask(q, s0);
                    mask(q + 1, s1);
                    hm = fmax3(hm, max32(s0), max32(s1));
                }
                hm *= sc;
                int E = 0;
                if (i == 0) {
                    m = hm > -INFINITY ? hm : 0.f;
                } else {
                    m = prev;
                    if (hm - m > kPxMove) {
                        const float up = ceilf(fminf(hm - m, kPxMaxMove));
                        E = static_cast<int>(up);
                        m += up;
                    }
                }
                sts32(a_ref + (gi & 1) * 512, __float_as_uint(m));
                __syncwarp();
                if (lane == 0) mbar_arrive(&ref[gi & 1]);
                if (i > 0 && __any_sync(0xffffffffu, E != 0)) {
                    // O holds the tiles before this one: scale its rows before P V(gi).
                    ok = __all_sync(0xffffffffu,
                                    wait_bar(&pv_done[(gi - 1) & 1], ((gi - 1) >> 1) & 1, abort_flag, p.status));
                    if (!ok) break;
                    tc_fence_after();
                    rescale_o_lane(tmem + lane_base + kPxColO, S::kVRows, E);
                }
                const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-m, -m);
                uint32_t s[2][32];
                load_scores(0, s[0]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t (&cur)[32] = s[q & 1];
                    tc_wait_ld32(cur);
                    if (q < 3) load_scores(q + 1, s[(q + 1) & 1]);
                    mask(q, cur);
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 a = ffma2(make_float2(__uint_as_float(cur[4 * e]), __uint_as_float(cur[4 * e + 1])),
                                               sc2, nm2);
                        const float2 b = ffma2(
                            make_float2(__uint_as_float(cur[4 * e + 2]), __uint_as_float(cur[4 * e + 3])), sc2, nm2);
                        const float p0 = exp2_approx(a.x), p1 = exp2_approx(a.y);
                        const float p2 = exp2_approx(b.x), p3 = exp2_approx(b.y);
                        w[2 * e] = cvt_bf16x2(p0, p2);
                        w[2 * e + 1] = cvt_bf16x2(p1, p3);
                    }
                    // Columns [16 q, 16 q + 16) hold scores that have been read (q >= 1: 16 q + 16
                    // <= 32 q).
                    tc_st_32x32b_x16(tS + 16 * q, w);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[set]);
            }
            if (!ok) break;
            // -------------------------------------------------------------- epilogue
            ok = __all_sync(0xffffffffu, wait_bar(o_full, c & 1, abort_flag, p.status));
            if (!ok) break;
            tc_fence_after();
            const float l = __uint_as_float(tc_ld_32x32b_x1(tmem + lane_base + kPxColO + 128));
            tc_wait_ld();
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const int n = u.q0 + row;
            int64_t bh;
            int t;
            const int64_t part = px_row(p, u.h, n, bh, t) * p.splits + u.split;
            float4 *dst = reinterpret_cast<float4 *>(p.ws_o + part * 128 + 64 * set);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t o[32];
                tc_ld_32x32b_x32(tmem + lane_base + kPxColO + 64 * set + 32 * hh, o);
                tc_wait_ld32(o);
                if (n < p.rows) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        dst[8 * hh + q] = make_float4(__uint_as_float(o[4 * q]) * inv, __uint_as_float(o[4 * q + 1]) * inv,
                                                      __uint_as_float(o[4 * q + 2]) * inv,
                                                      __uint_as_float(o[4 * q + 3]) * inv);
                }
            }
            if (n < p.rows && ((g + T - 1) & 1) == set) p.ws_lse[part] = l > 0.f ? log2f(l) + m : -INFINITY;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            g += T;
            ++c;
        }
    }
    teardown_tmem(warp == kPxMmaWarp, tmem, kPxTmemCols);
}

// Joins the partial results of each query row: `splits` of the prefix and `own_splits` of
// its own keys (either may be 0). One warp per row, four channels a lane.
__global__ void __launch_bounds__(256) qk4v8_prefix_merge_kernel(const float *__restrict__ o, const float *__restrict__ l,
                                                                 int splits, const float *__restrict__ own_o,
                                                                 const float *__restrict__ own_l, int own_splits,
                                                                 int64_t rows, int Hq, int nq,
                                                                 __nv_bfloat16 *__restrict__ out,
                                                                 float *__restrict__ lse) {
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    const int lane = threadIdx.x & 31;
    const float *lp = l + r * splits, *lo = own_l + r * own_splits;
    float m = -INFINITY;
    for (int s = lane; s < splits + own_splits; s += 32) m = fmaxf(m, s < splits ? lp[s] : lo[s - splits]);
    m = warp_max_f32(m);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    if (m > -INFINITY) {
        auto add = [&](const float *po, float ls) {
            const float w = exp2f(ls - m);
            const float4 v = *reinterpret_cast<const float4 *>(po + lane * 4);
            sum += w;
            acc.x += w * v.x;
            acc.y += w * v.y;
            acc.z += w * v.z;
            acc.w += w * v.w;
        };
#pragma unroll 4
        for (int s = 0; s < splits; ++s) add(o + (r * splits + s) * 128, lp[s]);
#pragma unroll 4
        for (int s = 0; s < own_splits; ++s) add(own_o + (r * own_splits + s) * 128, lo[s]);
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int64_t bh = r / nq;
    const int t = static_cast<int>(r - bh * nq);
    const int64_t b = bh / Hq;
    const int h = static_cast<int>(bh - b * Hq);
    uint2 w;
    w.x = cvt_bf16x2(acc.x * inv, acc.y * inv);
    w.y = cvt_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2 *>(out + ((b * nq + t) * Hq + h) * 128 + lane * 4) = w;
    if (lse && lane == 0) lse[r] = sum > 0.f ? (log2f(sum) + m) * 0.6931471805599453f : -INFINITY;
}

cudaError_t launch_prefix(const CUtensorMap &tk, const PrefixParams &p, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static bool configured[kMaxDevices] = {};
    static int sm_count[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int sms = dev < kMaxDevices ? sm_count[dev] : 0;
    if (dev >= kMaxDevices || !configured[dev]) {
        e = cudaFuncSetAttribute(qk4v8_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PxSmem::kBytes);
        if (e != cudaSuccess) return e;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) {
            sm_count[dev] = sms;
            configured[dev] = true;
        }
    }
    const int grid = p.units < sms ? p.units : sms;
    qk4v8_prefix_kernel<<<grid, kPxThreads, PxSmem::kBytes, stream>>>(tk, p);
    return cudaGetLastError();
}

cudaError_t launch_prefix_merge(const float *o, const float *l, int splits, const float *own_o, const float *own_l,
                                int own_splits, int B, int Hq, int nq, void *out, float *lse, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(B) * Hq * nq;
    const int64_t grid = (rows + 7) / 8;
    if (grid >= (int64_t{1} << 31)) return cudaErrorInvalidValue;
    qk4v8_prefix_merge_kernel<<<static_cast<unsigned>(grid), 256, 0, stream>>>(
        o, l, splits, own_o, own_l, own_splits, rows, Hq, nq, static_cast<__nv_bfloat16 *>(out), lse);
    return cudaGetLastError();
}

}  // namespace qk4v8
