// Paged KV cache append with online scale update.
//
// MpFA QK4V8 article, section 3.2: the block scales are computed online, from
// the data of the block itself, with no calibration; section 6.1: the QK4V8
// attention runs over a quantized KV cache. Decode appends tokens to that
// cache one step at a time (1 token, or the 8 tokens of a verified draft
// block), into pages of 128 tokens taken from a pool (paged attention).
//
// K is quantized per token (one MXFP4 scale per 32 channels), so a new token's
// K row is encoded on its own and written into its page. V is quantized per
// channel over groups of 32 tokens along the sequence: a token that lands in a
// group that already holds tokens changes that group's amax, so the group's
// scale is recomputed and every code of the group re-encoded. To do that
// exactly (the result is identical to quantizing the whole sequence at once),
// the bf16 values of the open group, the last, partly filled group of each
// (sequence, KV head), are kept in a small staging buffer ("tail", 32 tokens x
// 128 channels of bf16) that the append reads and refreshes.
//
// Page layout (one page = 128 tokens of one KV head, as the contiguous layout
// with capacity 128):
//   K codes  [pages][Hkv][128][64],  K scales [pages][Hkv][512]
//   V codes  [pages][Hkv][128][128] (channel rows, token-contiguous),
//   V scales [pages][Hkv][512]
// Token t of sequence b lives in page block_table[b][t / 128] at row t % 128.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/qk4v8.h"
#include "mx_encode.cuh"
#include "ptx.cuh"
#include "qk4v8_internal.h"
#include "rope.cuh"

namespace qk4v8 {

namespace {

__device__ __forceinline__ void flag_bad_page(int32_t *status) {
    if (status) atomicCAS(status, 0, QK4V8_ERR_INVALID_ARG);
}

// Page of token position pos of sequence b, or -1 if the block table has no
// valid page there.
__device__ __forceinline__ int page_of(const int32_t *__restrict__ block_table, int max_pages, int num_pages, int b,
                                       int pos) {
    const int slot = pos >> 7;
    if (pos < 0 || slot >= max_pages) return -1;
    const int page = block_table[static_cast<int64_t>(b) * max_pages + slot];
    return (page >= 0 && page < num_pages) ? page : -1;
}

}  // namespace

// One kernel does the whole append. CTA (b, h, chunk), 128 threads:
//  - K: the chunk's share of the n_new rows of head h, 16 lanes per row (two
//    rows per warp step), with the quantization kernels' encoder (identical
//    bytes), optionally after the Hadamard rotation of the row;
//  - V: thread c = channel c; the chunk's share of the 32-token groups the new
//    tokens touch. A group's tokens come from the staging buffer (those before
//    the append, only in the first touched group) and from the new rows; the
//    channel's amax over them fixes the E8M0 scale, all of the group's codes
//    are (re)written, and codes past the new length are zero;
//  - chunk 0 then refreshes the staging buffer with the open group after the
//    append. It is also the only reader of the old staging (the first touched
//    group is its own), and thread c reads and writes only column c, so the
//    refresh needs no barrier;
//  - with a separate seqlens_out, CTA (b, 0, 0) writes the new length (no CTA
//    reads seqlens_out). When the two are the same array, a second launch
//    advances the lengths after every reader.
template <bool kRotate>
__global__ void __launch_bounds__(128) kv_append_kernel(const __nv_bfloat16 *__restrict__ k,
                                                        const __nv_bfloat16 *__restrict__ v, int n_new, int H,
                                                        int64_t sb, int64_t st, int64_t sh,
                                                        const int32_t *__restrict__ seqlens,
                                                        const int32_t *__restrict__ block_table, int max_pages,
                                                        int num_pages, uint8_t *__restrict__ k_codes,
                                                        uint8_t *__restrict__ k_scales, uint8_t *__restrict__ v_codes,
                                                        uint8_t *__restrict__ v_scales, __nv_bfloat16 *__restrict__ tail,
                                                        int chunks, int32_t *seqlens_out, int32_t *status) {
    const int ci = static_cast<int>(blockIdx.x % chunks);
    const int h = static_cast<int>((blockIdx.x / chunks) % H);
    const int b = static_cast<int>(blockIdx.x / (static_cast<int64_t>(chunks) * H));
    const int L0 = seqlens[b];
    const int L1 = L0 + n_new;
    const int c = threadIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    // ---- K rows [r_begin, r_end) of this chunk
    const int rows_per_chunk = (n_new + chunks - 1) / chunks;
    const int r_begin = ci * rows_per_chunk;
    const int r_end = r_begin + rows_per_chunk < n_new ? r_begin + rows_per_chunk : n_new;
    const int sub = lane & 15;
    // The loop bound is per warp, so all 32 lanes reach the encoder's shuffles.
    for (int r0 = r_begin + 2 * warp; r0 < r_end; r0 += 8) {
        const int t = r0 + (lane >> 4);
        const bool in = t < r_end;
        const int pos = L0 + t;
        int page = -1;
        if (in) {
            page = page_of(block_table, max_pages, num_pages, b, pos);
            if (page < 0 && sub == 0) flag_bad_page(status);
        }
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (page >= 0) raw = *reinterpret_cast<const uint4 *>(k + b * sb + t * st + h * sh + sub * 8);
        int X;
        uint32_t packed;
        if (kRotate) {
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
            hadamard128_rows(x, sub);
            packed = mxfp4_encode8_f32(x, true, X);
        } else {
            packed = mxfp4_encode8(raw, true, X);
        }
        if (page >= 0) {
            const int64_t row = static_cast<int64_t>(page) * H + h;
            const int rr = pos & 127;
            reinterpret_cast<uint32_t *>(k_codes + (row * 128 + rr) * 64)[sub] = packed;
            if ((sub & 3) == 0)
                k_scales[row * 512 + (rr & 31) * 16 + (rr >> 5) * 4 + (sub >> 2)] = static_cast<uint8_t>(X + 127);
        }
    }

    // ---- V groups L0 / 32 + ci, + chunks, ... touched by the new tokens
    uint16_t *tail_bh = reinterpret_cast<uint16_t *>(tail) + ((static_cast<int64_t>(b) * H + h) * 32) * 128;
    const uint16_t *vin = reinterpret_cast<const uint16_t *>(v) + b * sb + h * sh + c;
    for (int G = L0 / 32 + ci; G * 32 < L1; G += chunks) {
        const int t0 = G * 32;
        const int page = page_of(block_table, max_pages, num_pages, b, t0);
        if (page < 0) {
            if (c == 0) flag_bad_page(status);
            continue;
        }
        uint16_t x[32];
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int t = t0 + j;
            uint16_t bits = 0;
            if (t < L0)
                bits = tail_bh[j * 128 + c];  // staged before this append
            else if (t < L1)
                bits = vin[(t - L0) * st];
            x[j] = bits;
            amax = fmaxf(amax, fabsf(__uint_as_float(static_cast<uint32_t>(bits) << 16)));
        }
        const int X = shared_exponent(amax, 8);
        const float f = pow2_neg(X);
        // x / 2^X is exact; the conversion keeps the sign bit, also of a value
        // that rounds to zero. Tokens past L1 encode as zero.
        uint32_t words[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t lo = cvt_e4m3x2(__uint_as_float(static_cast<uint32_t>(x[4 * q]) << 16) * f,
                                           __uint_as_float(static_cast<uint32_t>(x[4 * q + 1]) << 16) * f);
            const uint32_t hi = cvt_e4m3x2(__uint_as_float(static_cast<uint32_t>(x[4 * q + 2]) << 16) * f,
                                           __uint_as_float(static_cast<uint32_t>(x[4 * q + 3]) << 16) * f);
            words[q] = lo | (hi << 16);
        }
        const int64_t row = static_cast<int64_t>(page) * H + h;
        uint4 *dst = reinterpret_cast<uint4 *>(v_codes + (row * 128 + c) * 128 + (t0 & 127));
        dst[0] = make_uint4(words[0], words[1], words[2], words[3]);
        dst[1] = make_uint4(words[4], words[5], words[6], words[7]);
        v_scales[row * 512 + (c & 31) * 16 + (c >> 5) * 4 + ((t0 >> 5) & 3)] = static_cast<uint8_t>(X + 127);
    }

    // ---- the open group after the append, staged in slots t % 32 (its tokens
    // from before the append are in place already)
    if (ci == 0 && (L1 & 31) != 0) {
        const int t0 = L1 & ~31;
        for (int t = t0 > L0 ? t0 : L0; t < L1; ++t) tail_bh[(t - t0) * 128 + c] = vin[(t - L0) * st];
    }
    if (seqlens_out && ci == 0 && h == 0 && c == 0) seqlens_out[b] = L1;
}

// seqlens[b] += n_new in place, after every reader of seqlens ran.
__global__ void kv_advance_lengths_kernel(int32_t *seqlens, int B, int n_new) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < B) seqlens[b] += n_new;
}

cudaError_t launch_kv_append(const void *k, const void *v, int B, int n_new, int H, int64_t sb, int64_t st,
                             int64_t sh, const int32_t *seqlens, const int32_t *block_table, int max_pages,
                             int num_pages, uint8_t *k_codes, uint8_t *k_scales, uint8_t *v_codes,
                             uint8_t *v_scales, void *tail, bool rotate_k, int32_t *seqlens_out, int32_t *status,
                             cudaStream_t stream) {
    // Chunks per (sequence, head): at most 8 touched V groups and 256 K rows
    // per CTA (one chunk for a decode step of up to 32 tokens).
    const int groups = (n_new + 31) / 32 + 1;  // the open group and those the new tokens fill
    int chunks = (groups + 7) / 8;
    const int chunks_k = (n_new + 255) / 256;
    if (chunks_k > chunks) chunks = chunks_k;
    const int64_t grid = static_cast<int64_t>(B) * H * chunks;
    if (grid >= (int64_t{1} << 31)) return cudaErrorInvalidValue;
    const bool in_place = seqlens_out && seqlens_out == seqlens;
    int32_t *direct_out = in_place ? nullptr : seqlens_out;
    const __nv_bfloat16 *kk = static_cast<const __nv_bfloat16 *>(k);
    const __nv_bfloat16 *vv = static_cast<const __nv_bfloat16 *>(v);
    __nv_bfloat16 *tl = static_cast<__nv_bfloat16 *>(tail);
    if (rotate_k)
        kv_append_kernel<true><<<static_cast<unsigned>(grid), 128, 0, stream>>>(
            kk, vv, n_new, H, sb, st, sh, seqlens, block_table, max_pages, num_pages, k_codes, k_scales, v_codes,
            v_scales, tl, chunks, direct_out, status);
    else
        kv_append_kernel<false><<<static_cast<unsigned>(grid), 128, 0, stream>>>(
            kk, vv, n_new, H, sb, st, sh, seqlens, block_table, max_pages, num_pages, k_codes, k_scales, v_codes,
            v_scales, tl, chunks, direct_out, status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !in_place) return e;
    kv_advance_lengths_kernel<<<(B + 255) / 256, 256, 0, stream>>>(seqlens_out, B, n_new);
    return cudaGetLastError();
}

// ------------------------------------------------ append with the position rotation

// The append of a model with rotary positions: K rows are rotated (rope.cuh) on
// their way into MXFP4, V is packed as above, and every sequence may bring its own
// number of new tokens (a padded batch).
//
// One launch, two kinds of CTA of 256 threads:
//  - K: a warp takes a few tokens by up to 32 heads, eight lanes per row, so that a
//    token's cosines and sines are read once for its heads;
//  - V: CTA (b, h, page) takes the 32-token groups of one page that the new tokens
//    touch. It stages their bf16 rows in shared memory (16-byte loads along the
//    channels; rows from before the append come from the staging buffer), and
//    thread (channel pair, group) encodes 32 tokens of two channels from there. The
//    codes go out through shared memory as whole 32-byte sectors, so a full page is
//    16 KiB contiguous. (The append above loads two bytes per thread and token.)
//    The CTA of the first page is the only reader of the staging rows, so it also
//    refreshes them, after its own reads.
//
// 512 bytes read and 200 written per new token and head; a single token of a sequence
// rewrites its open group, 4 KB per head. A long append is bound by the K rows'
// instructions and the V pages' trips to memory, which is why the two kinds of CTA lie
// evenly among each other: 8192 tokens of 8 heads and 4 sequences take 52 us a call in a row of
// calls (0.60 of the copy peak), 58 with a cold L2. (In a profiler's trace 53.6, and 66.5 with
// the V pages last and one token by four heads a K step.) One token of 64 sequences and 8
// heads: 11 us with a cold L2, 5 of them the events' own, a chain of length, page and row.
struct KvAppendRopeArgs {
    const __nv_bfloat16 *k, *v;
    int B, n, H;
    int64_t ksb, kst, ksh, vsb, vst, vsh;
    const int32_t *seqlens, *new_lens;
    int32_t *seqlens_out;  // null, or another array than seqlens
    const int32_t *block_table;
    int max_pages, num_pages;
    uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    __nv_bfloat16 *tail;
    int32_t *status;
    RopeParams rope;
    RopeTiling tile;
    uint32_t v_ratio;  // ceil(2^32 * V pages' CTAs / all CTAs)
    int v_pages;  // pages that n tokens can touch
};

// A length that sequences can have; the others' are skipped and keep theirs.
__device__ __forceinline__ bool append_length_ok(int L0, int max_pages) { return L0 >= 0 && L0 <= max_pages * 128; }

// New tokens of sequence b: new_lens[b] (none: all n), held to 0..n.
__device__ __forceinline__ int append_count(const KvAppendRopeArgs &a, int b) {
    if (!a.new_lens) return a.n;
    const int m = a.new_lens[b];
    if (m >= 0 && m <= a.n) return m;
    flag_bad_page(a.status);
    return m < 0 ? 0 : a.n;
}

template <bool kAdjacent, bool kHadamard>
__device__ __forceinline__ void append_k_rows(const KvAppendRopeArgs &a, uint32_t cta) {
    const int item = static_cast<int>(cta * 8 + (threadIdx.x >> 5));
    const int per_b = a.tile.token_groups * a.tile.head_chunks;
    const int b = item / per_b;
    if (b >= a.B) return;
    const int rem = item - b * per_b;
    const int tg = rem / a.tile.head_chunks, hc = rem - tg * a.tile.head_chunks;
    const int lane = threadIdx.x & 31, j = lane & 7, slot = lane >> 3;
    const int hs = 1 << a.tile.hs_log2;
    const int t = tg * (4 >> a.tile.hs_log2) + (slot >> a.tile.hs_log2);
    const int h_end = min(a.H, (hc + 1) * a.tile.heads);
    const int L0 = a.seqlens[b];
    const int nrot = a.rope.rotary >> 4;
    int k0, k1;
    rope_chunks(kAdjacent, nrot, j, k0, k1);
    // The lane's two chunks of head h; each step goes hs heads on. The first are read before
    // the page and the position are known.
    int h = hc * a.tile.heads + (slot & (hs - 1));
    const __nv_bfloat16 *x0 = a.k + b * a.ksb + static_cast<int64_t>(t) * a.kst + h * a.ksh + k0 * 8;
    const int64_t xstep = hs * a.ksh;
    const int xsecond = (k1 - k0) * 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 r0 = zero, r1 = zero;
    const bool mine = t < append_count(a, b);
    if (mine && h < h_end) {
        r0 = *reinterpret_cast<const uint4 *>(x0);
        r1 = *reinterpret_cast<const uint4 *>(x0 + xsecond);
    }
    int page = -1;
    // (L0 + t cannot pass 2^31 within the pages: L0 < max_pages * 128 < 2^31 - n.)
    if (mine) {
        page = append_length_ok(L0, a.max_pages) ? page_of(a.block_table, a.max_pages, a.num_pages, b, L0 + t) : -1;
        if (page < 0 && j == 0) flag_bad_page(a.status);
    }
    const bool live = page >= 0;
    RopeTrig g;
    rope_load<kAdjacent>(a.rope, b, t, L0, j, live, a.status, g);
    const int rr = (L0 + t) & 127;
    const int64_t row = static_cast<int64_t>(page) * a.H + h;
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.k_codes + (row * 128 + rr) * 64) + j;
    uint32_t *dsf = reinterpret_cast<uint32_t *>(a.k_scales + row * 512 + (rr & 31) * 16 + (rr >> 5) * 4);
    for (int h0 = hc * a.tile.heads; h0 < h_end; h0 += hs) {
        uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
        const bool store = live && h < h_end;
        h += hs;
        x0 += xstep;
        if (live && h < h_end) {
            r0 = *reinterpret_cast<const uint4 *>(x0);
            r1 = *reinterpret_cast<const uint4 *>(x0 + xsecond);
        }
        rope_row<kAdjacent>(g, nrot, j, w0, w1);
        uint32_t c0, c1, sf;
        mxfp4_row8<kHadamard>(w0, w1, j, c0, c1, sf);
        if (store) {
            dst[0] = c0;
            dst[8] = c1;
            if (j == 0) *dsf = sf;
        }
        dst += hs * (128 * 16);
        dsf += hs * 128;
    }
}

__device__ __forceinline__ void append_v_page(const KvAppendRopeArgs &a, int idx) {
    constexpr int kPitch = 136;   // bf16 elements per staged token row (16 bytes of padding)
    constexpr int kCPitch = 144;  // bytes per staged code row
    __shared__ __align__(16) uint16_t tile[128 * kPitch];
    __shared__ __align__(4) uint8_t atom[512];
    uint8_t *ctile = reinterpret_cast<uint8_t *>(tile);
    const int bh = idx / a.v_pages, pg = idx - bh * a.v_pages;
    const int b = bh / a.H, h = bh - b * a.H;
    const int L0 = a.seqlens[b];
    const int m = append_count(a, b);
    const bool length_ok = append_length_ok(L0, a.max_pages);
    if (pg == 0 && h == 0 && threadIdx.x == 0 && a.seqlens_out) a.seqlens_out[b] = length_ok ? L0 + m : L0;
    if (m == 0) return;
    if (!length_ok) {
        if (threadIdx.x == 0) flag_bad_page(a.status);
        return;
    }
    const int L1 = L0 + m;
    const int p0 = ((L0 >> 7) + pg) * 128;  // first token of the page
    if (p0 >= L1) return;
    const int lo = max(L0 & ~31, p0), hi = min((L1 + 31) & ~31, p0 + 128);  // touched groups' tokens
    uint16_t *tail = reinterpret_cast<uint16_t *>(a.tail) + static_cast<int64_t>(bh) * (32 * 128);
    const uint16_t *vin = reinterpret_cast<const uint16_t *>(a.v) + b * a.vsb + h * a.vsh;
    uint4 raw[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // every load of the thread before its first store
        const int i = threadIdx.x + 256 * k;
        const int t = p0 + (i >> 4), ch = (i & 15) * 8;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (t >= lo && t < hi) {
            if (t < L0)
                raw[k] = *reinterpret_cast<const uint4 *>(tail + (t & 31) * 128 + ch);
            else if (t < L1)
                raw[k] = *reinterpret_cast<const uint4 *>(vin + static_cast<int64_t>(t - L0) * a.vst + ch);
        }
    }
    const int page = page_of(a.block_table, a.max_pages, a.num_pages, b, p0);  // during the loads
    if (page < 0 && threadIdx.x == 0) flag_bad_page(a.status);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int i = threadIdx.x + 256 * k;
        const int tk = i >> 4;
        if (p0 + tk >= lo && p0 + tk < hi)
            *reinterpret_cast<uint4 *>(&tile[tk * kPitch + (i & 15) * 8]) = raw[k];
    }
    __syncthreads();
    if (pg == 0 && (L1 & 31) != 0) {
        // The open group after the append, in slots t % 32. (Its rows from before the
        // append are in place; the old rows were read above.)
        const int t0 = max(L1 & ~31, L0);
        for (int i = threadIdx.x; i < (L1 - t0) * 16; i += 256) {
            const int t = t0 + (i >> 4), ch = (i & 15) * 8;
            *reinterpret_cast<uint4 *>(tail + (t & 31) * 128 + ch) =
                *reinterpret_cast<const uint4 *>(vin + static_cast<int64_t>(t - L0) * a.vst + ch);
        }
    }
    if (page < 0) return;
    const int cp = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const bool on = p0 + grp * 32 >= lo && p0 + grp * 32 < hi;
    uint32_t words[2][8];
    int X[2] = {-127, -127};
    if (on) {
        const uint32_t *t32 = reinterpret_cast<const uint32_t *>(tile);
        uint32_t w[32];
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            w[i] = t32[(grp * 32 + i) * (kPitch / 2) + cp];
            mx = max_abs_number_bf16x2(w[i], mx);  // (a NaN does not set its group's scale)
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            X[q] = shared_exponent(fabsf(q ? bf16_hi(mx) : bf16_lo(mx)), 8);
            const float f = pow2_neg(X[q]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // x / 2^X is exact; the conversion keeps the sign, also of a value that
                // rounds to zero.
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = (q ? bf16_hi(w[4 * i + e]) : bf16_lo(w[4 * i + e])) * f;
                words[q][i] = cvt_e4m3x2(y[0], y[1]) | (static_cast<uint32_t>(cvt_e4m3x2(y[2], y[3])) << 16);
            }
        }
    }
    __syncthreads();  // the staged rows have been read
    if (on) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int c = 2 * cp + q;
            // Staged code rows: channel 2cp at row cp, 2cp + 1 at row 64 + cp, so that a
            // warp stores to consecutive rows.
            uint4 *dst = reinterpret_cast<uint4 *>(&ctile[(cp + 64 * q) * kCPitch + grp * 32]);
            dst[0] = make_uint4(words[q][0], words[q][1], words[q][2], words[q][3]);
            dst[1] = make_uint4(words[q][4], words[q][5], words[q][6], words[q][7]);
            atom[(c & 31) * 16 + (c >> 5) * 4 + grp] = static_cast<uint8_t>(X[q] + 127);
        }
    }
    __syncthreads();
    const int64_t row = static_cast<int64_t>(page) * a.H + h;
    uint8_t *block = a.v_codes + row * (128 * 128);
    const int g0 = (lo - p0) >> 5, ng = (hi - lo) >> 5;  // touched groups: [g0, g0 + ng)
    for (int i = threadIdx.x; i < 128 * 8; i += 256) {
        const int c = i >> 3, ch = i & 7;
        if ((ch >> 1) >= g0 && (ch >> 1) < g0 + ng)
            *reinterpret_cast<uint4 *>(block + c * 128 + ch * 16) =
                *reinterpret_cast<const uint4 *>(&ctile[((c >> 1) + (c & 1) * 64) * kCPitch + ch * 16]);
    }
    if (threadIdx.x < 128) {  // the channel's four scale bytes, those of the touched groups
        const int at = (threadIdx.x & 31) * 16 + (threadIdx.x >> 5) * 4;
        uint8_t *dst = a.v_scales + row * 512 + at;
        if (ng == 4)
            *reinterpret_cast<uint32_t *>(dst) = *reinterpret_cast<const uint32_t *>(atom + at);
        else
            for (int g = g0; g < g0 + ng; ++g) dst[g] = atom[at + g];
    }
}

template <bool kAdjacent, bool kHadamard>
__global__ void __launch_bounds__(256, 3) kv_append_rope_kernel(const __grid_constant__ KvAppendRopeArgs a) {
    // The V pages' CTAs lie evenly among the K rows': those wait for memory, these for the ALU.
    const uint32_t v = __umulhi(blockIdx.x, a.v_ratio);
    if (__umulhi(blockIdx.x + 1, a.v_ratio) == v)
        append_k_rows<kAdjacent, kHadamard>(a, blockIdx.x - v);
    else
        append_v_page(a, static_cast<int>(v));
}

// seqlens[b] += new_lens[b] (held to 0..n) in place, after every reader of seqlens ran.
__global__ void kv_advance_ragged_kernel(int32_t *seqlens, const int32_t *new_lens, int B, int n, int max_pages) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < B && append_length_ok(seqlens[b], max_pages)) seqlens[b] += new_lens ? min(max(new_lens[b], 0), n) : n;
}

cudaError_t launch_kv_append_rope(const void *k, const void *v, int B, int n, int H, const int64_t (&ks)[3],
                                  const int64_t (&vs)[3], const int32_t *seqlens, const int32_t *new_lens,
                                  int32_t *seqlens_out, const int32_t *block_table, int max_pages, int num_pages,
                                  uint8_t *k_codes, uint8_t *k_scales, uint8_t *v_codes, uint8_t *v_scales,
                                  void *tail, const RopeParams &rope, bool hadamard_k, int32_t *status,
                                  cudaStream_t stream) {
    const bool in_place = seqlens_out == seqlens;
    KvAppendRopeArgs a{};
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.B = B;
    a.n = n;
    a.H = H;
    a.ksb = ks[0];
    a.kst = ks[1];
    a.ksh = ks[2];
    a.vsb = vs[0];
    a.vst = vs[1];
    a.vsh = vs[2];
    a.seqlens = seqlens;
    a.new_lens = new_lens;
    a.seqlens_out = in_place ? nullptr : seqlens_out;
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.k_codes = k_codes;
    a.k_scales = k_scales;
    a.v_codes = v_codes;
    a.v_scales = v_scales;
    a.tail = static_cast<__nv_bfloat16 *>(tail);
    a.status = status;
    a.rope = rope;
    a.tile = rope_tiling(B, n, H);
    const int64_t items = static_cast<int64_t>(B) * a.tile.token_groups * a.tile.head_chunks;
    a.v_pages = (n + 126) / 128 + 1;
    const int64_t v_ctas = static_cast<int64_t>(B) * H * a.v_pages, grid = (items + 7) / 8 + v_ctas;
    // (Past these, K alone would be 500 GB.)
    if (items >= (int64_t{1} << 31) - 8 || grid >= (int64_t{1} << 31)) return cudaErrorInvalidValue;
    a.v_ratio = static_cast<uint32_t>(((static_cast<uint64_t>(v_ctas) << 32) + grid - 1) / grid);
    const unsigned g = static_cast<unsigned>(grid);
    if (rope.adjacent) {
        if (hadamard_k)
            kv_append_rope_kernel<true, true><<<g, 256, 0, stream>>>(a);
        else
            kv_append_rope_kernel<true, false><<<g, 256, 0, stream>>>(a);
    } else {
        if (hadamard_k)
            kv_append_rope_kernel<false, true><<<g, 256, 0, stream>>>(a);
        else
            kv_append_rope_kernel<false, false><<<g, 256, 0, stream>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !in_place) return e;
    kv_advance_ragged_kernel<<<(B + 255) / 256, 256, 0, stream>>>(seqlens_out, new_lens, B, n, max_pages);
    return cudaGetLastError();
}

}  // namespace qk4v8
