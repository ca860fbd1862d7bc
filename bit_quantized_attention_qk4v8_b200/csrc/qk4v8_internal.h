// Internal declarations shared by the CUDA translation units of libqk4v8.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace qk4v8 {

// Limit on any single pipeline wait inside a kernel before it gives up, sets
// the timeout status and unwinds (nanoseconds).
constexpr uint64_t kWaitTimeoutNs = 1000000000ull;

struct AttnParams {
    const uint8_t *q_codes;   // [B][Hq][q_cap][64]
    // Swap-AB decode only: when q_bf16 is set, the kernel quantizes the query
    // rows itself from bf16 [b][t][h][128] (element strides q_sb, q_st, q_sh)
    // and q_codes / q_scales are unused.
    const __nv_bfloat16 *q_bf16;
    int64_t q_sb, q_st, q_sh;
    const uint8_t *q_scales;  // [B][Hq][q_cap/128][512]
    const uint8_t *k_scales;  // [B][Hkv][kv_cap/128][512]
    const uint8_t *v_scales;  // [B][Hkv][kv_cap/128][512]
    const int32_t *seqlens;   // [B] or null
    int B, Hq, Hkv, G;
    int Sq;                   // query tokens per sequence (prefill length, or nq when decoding)
    int q_cap, kv_cap;
    int Lk;                   // KV length when seqlens is null
    int causal;
    // Decode only: > 0 limits every query row of a sequence of L keys to keys
    // j >= L - Sq - window (the last `window` keys before the Sq-token block, and
    // the block); 0: no lower bound.
    int window;
    // Decode only: paged K/V when non-null. Key tile t of sequence b is page
    // block_table[b * max_pages + t] of pools [num_pages][Hkv][128 tokens]
    // (kv_cap is then max_pages * 128); null: contiguous [B][Hkv][kv_cap].
    const int32_t *block_table;
    int max_pages, num_pages;
    // Decode only: V is MXFP4 (E2M1 codes [B][Hkv][128][kv_cap / 2], the QK4V4
    // comparison point) instead of MXFP8.
    int v_fp4;
    float scale_log2;         // softmax_scale * log2(e)
    int decode;               // 0: units (b, h_q, q tile); 1: units (b, h_kv, split)
    int n_qtiles;
    int num_splits, split_tiles;
    __nv_bfloat16 *out;       // prefill [B][Sq][Hq][128]
    float *lse;               // prefill [B][Hq][Sq] (natural log), nullable
    float *ws_o;              // decode partial outputs [B][Hq][nq][splits][128]
    float *ws_lse;            // decode partial log2-sum-exp [B][Hq][nq][splits]
    int direct_out;           // decode: write out [B][nq][Hq][128] and lse directly
    int32_t *piece_counts;    // GQA decode with splits: [B][Hkv] pieces of each sequence (0: written whole)
    int32_t *status;          // nullable
    int test_stall;           // test hook: the producer withholds the Q-ready signal
    float *test_dump_s;       // test hook: CTA 0 writes its first raw score tile [128 lanes][128 keys]
};

// pad_to_cap: write all `cap` token rows of each sequence (rows past the valid
// length get zero codes and scales); otherwise only the S input rows.
// rotate: quantize each row after its rotation by H / sqrt(128).
cudaError_t launch_quantize_qk(const void *x, int B, int S, int H, int64_t sb, int64_t ss, int64_t sh,
                               const int32_t *seqlens, int cap, uint8_t *codes, uint8_t *scales,
                               cudaStream_t stream, bool pad_to_cap = true, bool rotate = false);
cudaError_t launch_quantize_v(const void *v, int B, int S, int H, int64_t sb, int64_t ss, int64_t sh,
                              const int32_t *seqlens, int cap, uint8_t *codes, uint8_t *scales,
                              cudaStream_t stream);
cudaError_t launch_quantize_qkv(const void *q, const void *k, const void *v, int B, int Sq, int Sk, int Hq, int Hkv,
                                const int32_t *seqlens_k, int q_cap, int kv_cap, uint8_t *q_codes, uint8_t *q_scales,
                                uint8_t *k_codes, uint8_t *k_scales, uint8_t *v_codes, uint8_t *v_scales,
                                cudaStream_t stream);
cudaError_t launch_quantize_v4(const void *v, int B, int S, int H, int64_t sb, int64_t ss, int64_t sh,
                               const int32_t *seqlens, int cap, uint8_t *codes, uint8_t *scales,
                               cudaStream_t stream);
cudaError_t launch_attention(const CUtensorMap &tmap_k, const CUtensorMap &tmap_v, const AttnParams &p,
                             int grid, cudaStream_t stream);
// Prefill kernel (persistent: one CTA per SM over the (sequence, query head,
// 128-token query tile) units), and its QK^T-stage-only build over the same
// schedule. tmap_q maps the packed Q codes like tmap_k the K codes.
cudaError_t launch_prefill(const CUtensorMap &tmap_q, const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                           const AttnParams &p, cudaStream_t stream);
cudaError_t launch_prefill_stage_qk(const CUtensorMap &tmap_q, const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                                    const AttnParams &p, cudaStream_t stream);
// Tensor-pipe peak run of one block-scaled MMA shape (measurement aid).
cudaError_t launch_mma_peak(int kind, int ctas, int iters, int32_t *status, cudaStream_t stream);
// Swap-AB split-KV decode kernel; handles G*nq <= kDecodeMaxRows query rows.
constexpr int kDecodeMaxRows = 64;
cudaError_t launch_decode(const CUtensorMap &tmap_k, const CUtensorMap &tmap_v, const AttnParams &p, int grid,
                          cudaStream_t stream);
// GQA decode kernel for kGqaMinRows..kDecodeMaxRows query rows per KV head
// (persistent, one CTA per SM; packed MXFP4 queries), followed, for a
// direct-output call with splits, by the merge of the cut sequences.
constexpr int kGqaMinRows = 33;
cudaError_t launch_gqa_decode(const CUtensorMap &tmap_k, const CUtensorMap &tmap_v, const AttnParams &p,
                              cudaStream_t stream);
// Merge of the sequences a persistent decode kernel cut (direct output, splits >= 2,
// <= 64 rows per KV head), from the partials and the recorded piece counts.
cudaError_t launch_cut_merge(const AttnParams &p, cudaStream_t stream);
// Paged KV append (K and V of n_new tokens per sequence at positions
// seqlens[b] ..; V groups re-encoded from the staging buffer `tail`), then
// seqlens_out[b] = seqlens[b] + n_new (seqlens_out may be seqlens).
cudaError_t launch_kv_append(const void *k, const void *v, int B, int n_new, int H, int64_t sb, int64_t st,
                             int64_t sh, const int32_t *seqlens, const int32_t *block_table, int max_pages,
                             int num_pages, uint8_t *k_codes, uint8_t *k_scales, uint8_t *v_codes,
                             uint8_t *v_scales, void *tail, bool rotate_k, int32_t *seqlens_out, int32_t *status,
                             cudaStream_t stream);
// Shared-prefix decode (prefix.cu).
struct PrefixParams {
    const uint8_t *q_codes, *q_scales;            // [B][Hq][q_cap]
    int Hq, Hkv, G, nq, q_cap;
    int gq;                                       // G * nq
    uint32_t m_gq, m_nq;                          // ceil(2^32 / gq), ceil(2^32 / nq), for px_div
    int rows, row_tiles;                          // query rows of a KV head (B * G * nq), and 128-row tiles
    float scale_log2;
    int causal;
    // The prefix: tokens and 128-key tiles (0: none); scales [rows][prefix_blocks] blocks of
    // 128 tokens; pages of its tiles (null: contiguous, [1][Hkv]).
    int len, tiles, prefix_blocks;
    const uint8_t *p_k_scales, *p_v_scales;
    const int32_t *prefix_table;
    // The sequences' own keys (own = 0: none), contiguous [B][Hkv][own_blocks * 128] or paged;
    // lengths past own_most are cut to it.
    int own, own_most, own_blocks;
    const uint8_t *k_scales, *v_scales;
    const int32_t *block_table, *seqlens;
    int max_pages, num_pages;
    // Partial results of unit u = row_tile * Hkv + head in share c, slot u + c: O
    // [slot][32 chunks of 4 channels][128 rows][4] and log2-sum-exp [slot][128]; the first and last share of each unit.
    int shares;
    float *part_o, *part_lse;
    int32_t *first, *last;
    int32_t *status;
    int test_stall;
};
// The kernel over the prefix and the own keys on p.shares CTAs (0: no keys at all), then the merge.
cudaError_t launch_prefix(const CUtensorMap &pk, const CUtensorMap &pv, const CUtensorMap &k, const CUtensorMap &v,
                          const PrefixParams &p, void *out, float *lse, cudaStream_t stream);
// Rotary positions of a call, as the kernels take them (rope.cuh).
struct RopeParams {
    const float *table;         // (cos, sin) [max_pos][rotary / 2][2]
    int max_pos, rotary;        // rotary: a multiple of 16, up to 128
    int adjacent;               // pairs (2i, 2i + 1) instead of (i, i + rotary / 2)
    int n_axes;                 // 1..4
    uint64_t pair_axis[2];      // two bits per pair
    const int32_t *positions;   // null: the same token index on every axis
    int64_t pos_sa, pos_sb, pos_st;
};
// MXFP4 of the rotated rows (after the Hadamard rotation with `rotate`). pad: write
// all `cap` token rows, else the S given ones.
cudaError_t launch_quantize_qk_rope(const void *x, int B, int S, int H, int64_t sb, int64_t ss, int64_t sh,
                                    const int32_t *seqlens, const int32_t *start, int cap, const RopeParams &rope,
                                    bool rotate, bool pad, uint8_t *codes, uint8_t *scales, int32_t *status,
                                    cudaStream_t stream);
// Paged append with K rotated, new_lens[b] (null: n) tokens of each sequence; ks, vs:
// strides of batch, token and head.
cudaError_t launch_kv_append_rope(const void *k, const void *v, int B, int n, int H, const int64_t (&ks)[3],
                                  const int64_t (&vs)[3], const int32_t *seqlens, const int32_t *new_lens,
                                  int32_t *seqlens_out, const int32_t *block_table, int max_pages, int num_pages,
                                  uint8_t *k_codes, uint8_t *k_scales, uint8_t *v_codes, uint8_t *v_scales,
                                  void *tail, const RopeParams &rope, bool hadamard_k, int32_t *status,
                                  cudaStream_t stream);
cudaError_t launch_decode_merge(const float *ws_o, const float *ws_lse, int B, int Hq, int nq, int splits,
                                __nv_bfloat16 *out, float *lse, cudaStream_t stream);

}  // namespace qk4v8
