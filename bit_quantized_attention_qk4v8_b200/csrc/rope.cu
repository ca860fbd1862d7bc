// Q or K through the rotary position embedding into MXFP4 in one pass
// (rope.cuh has the rotation and its rounding; the scale rule is the one of
// quantize.cu). Without it a user rotates in bf16 and quantizes after: the
// rotated tensor is written and read once more (512 of 836 bytes a row).
//
// A row of 128 channels is 256 bytes in and 68 out; the table row of a token
// (4 * rotary bytes) is read once for up to 32 heads. Bound by its instructions (the rotation's
// exact rounding, the two unpackings, the encoder: 250 a step of four rows, ALU pipe 0.66
// and issue 0.72 busy at 24 warps an SM): 4 x 8192 tokens of 32 heads 93 us a call in a row of
// calls, 0.59 of the copy peak. With a cold L2, the events' own 5 us in them: that call 99
// us; 2047 tokens of 64 heads, half of the channels rotated, 24; 3 x 1601 tokens of 8
// heads with three axes and the Hadamard rotation 15; one token of 32 sequences and 32 heads 9.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rope.cuh"

namespace qk4v8 {

struct QkRopeArgs {
    const __nv_bfloat16 *x;
    int B, S, H;
    int64_t sb, ss, sh;
    const int32_t *seqlens, *start;
    int cap, row_len;
    uint8_t *codes, *scales;
    int32_t *status;
    RopeParams rope;
    RopeTiling tile;
};

// One warp per item (batch entry, TS tokens, up to 32 heads), eight lanes per row.
template <bool kAdjacent, bool kHadamard>
__global__ void __launch_bounds__(256, 3) quantize_qk_rope_kernel(const __grid_constant__ QkRopeArgs a) {
    const int item = static_cast<int>(blockIdx.x * 8 + (threadIdx.x >> 5));
    const int per_b = a.tile.token_groups * a.tile.head_chunks;
    const int b = item / per_b;
    if (b >= a.B) return;
    const int rem = item - b * per_b;
    const int tg = rem / a.tile.head_chunks, hc = rem - tg * a.tile.head_chunks;
    const int lane = threadIdx.x & 31, j = lane & 7, slot = lane >> 3;
    const int hs = 1 << a.tile.hs_log2;
    const int t = tg * (4 >> a.tile.hs_log2) + (slot >> a.tile.hs_log2);
    const int h_end = min(a.H, (hc + 1) * a.tile.heads);
    int len = a.S;
    if (a.seqlens) len = min(len, a.seqlens[b]);
    const bool live = t < len;  // else padding: zero codes and scales
    const int nrot = a.rope.rotary >> 4;
    int k0, k1;
    rope_chunks(kAdjacent, nrot, j, k0, k1);
    const int nblk = a.cap / 128;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    int h = hc * a.tile.heads + (slot & (hs - 1));
    // The lane's two chunks of head h, its code words and scales: each step goes hs heads on.
    const __nv_bfloat16 *x0 = a.x + b * a.sb + static_cast<int64_t>(t) * a.ss + h * a.sh + k0 * 8;
    const int64_t xstep = hs * a.sh;
    const int xsecond = (k1 - k0) * 8;
    const int64_t head = static_cast<int64_t>(b) * a.H + h;
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.codes + (head * a.cap + t) * 64) + j;
    const int64_t cstep = static_cast<int64_t>(hs) * a.cap * 16;
    uint32_t *dsf = reinterpret_cast<uint32_t *>(a.scales + (head * nblk + t / 128) * 512 + (t & 31) * 16 +
                                                 ((t & 127) >> 5) * 4);
    const int64_t sstep = static_cast<int64_t>(hs) * nblk * 128;
    uint4 r0 = zero, r1 = zero;
    if (live && h < h_end) {
        r0 = *reinterpret_cast<const uint4 *>(x0);
        r1 = *reinterpret_cast<const uint4 *>(x0 + xsecond);
    }
    RopeTrig g;  // (after the rows: the position and then the table's row are a trip to memory each)
    rope_load<kAdjacent>(a.rope, b, t, a.start ? a.start[b] : 0, j, live, a.status, g);
    const bool store = t < a.row_len;
    // The trip count is the same for all lanes of the warp (its row helpers shuffle). Padding
    // stays zero on the way through: zero codes and scales.
    for (int h0 = hc * a.tile.heads; h0 < h_end; h0 += hs) {
        uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
        const bool mine = h < h_end;
        h += hs;
        x0 += xstep;
        if (live && h < h_end) {  // the next heads' rows, while these are encoded
            r0 = *reinterpret_cast<const uint4 *>(x0);
            r1 = *reinterpret_cast<const uint4 *>(x0 + xsecond);
        }
        rope_row<kAdjacent>(g, nrot, j, w0, w1);
        uint32_t c0, c1, sf;
        mxfp4_row8<kHadamard>(w0, w1, j, c0, c1, sf);
        if (store && mine) {
            dst[0] = c0;
            dst[8] = c1;
            if (j == 0) *dsf = sf;
        }
        dst += cstep;
        dsf += sstep;
    }
}

cudaError_t launch_quantize_qk_rope(const void *x, int B, int S, int H, int64_t sb, int64_t ss, int64_t sh,
                                    const int32_t *seqlens, const int32_t *start, int cap, const RopeParams &rope,
                                    bool rotate, bool pad, uint8_t *codes, uint8_t *scales, int32_t *status,
                                    cudaStream_t stream) {
    QkRopeArgs a{};
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.B = B;
    a.S = S;
    a.H = H;
    a.sb = sb;
    a.ss = ss;
    a.sh = sh;
    a.seqlens = seqlens;
    a.start = start;
    a.cap = cap;
    a.row_len = pad ? cap : S;
    a.codes = codes;
    a.scales = scales;
    a.status = status;
    a.rope = rope;
    if (a.row_len == 0) return cudaSuccess;
    a.tile = rope_tiling(B, a.row_len, H);
    const int64_t items = static_cast<int64_t>(B) * a.tile.token_groups * a.tile.head_chunks;
    if (items >= (int64_t{1} << 31) - 8) return cudaErrorInvalidValue;  // (500 GB of rows)
    const unsigned n = static_cast<unsigned>((items + 7) / 8);
    if (rope.adjacent) {
        if (rotate)
            quantize_qk_rope_kernel<true, true><<<n, 256, 0, stream>>>(a);
        else
            quantize_qk_rope_kernel<true, false><<<n, 256, 0, stream>>>(a);
    } else {
        if (rotate)
            quantize_qk_rope_kernel<false, true><<<n, 256, 0, stream>>>(a);
        else
            quantize_qk_rope_kernel<false, false><<<n, 256, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace qk4v8
