"""Rotating MXFP4 quantizer against a rotation in 64 bits and the plain quantizer: the bytes must be equal."""
import numpy as np
import pytest
import torch

import bit_quantized_attention_qk4v8_b200 as qk
import oracle
from gpu_util import to_dev
from layouts import qk_scales_logical, unpack_e2m1
from ref_positions import angles, f32_to_bf16, rotate

pytestmark = pytest.mark.gpu


def rand_bits(rng, shape, spread=4.0):
    return f32_to_bf16((rng.standard_normal(shape) * np.exp2(rng.uniform(-spread, spread, shape[:-1] + (1,)))).astype(np.float32))


def expected(bits, table, pos, axis, adjacent, hadamard):
    y = rotate(bits, table, pos, axis, adjacent)
    return oracle.quantize_qk_hadamard(y) if hadamard else oracle.quantize_qk(y)


def check(packed, want, T):
    codes, scales = want
    assert np.array_equal(unpack_e2m1(packed.codes.cpu().numpy()[:, :, :T]), codes)
    assert np.array_equal(qk_scales_logical(packed.scales.cpu().numpy(), T), scales)


@pytest.mark.parametrize("B,T,H,rotary,adjacent,n_axes,hadamard", [
    (1, 1, 1, 128, False, 1, False), (3, 1, 32, 128, False, 1, False), (1, 1, 2, 128, True, 1, True),
    (2, 129, 3, 64, False, 1, False), (1, 37, 5, 16, False, 1, True), (2, 33, 2, 112, False, 1, False),
    (1, 200, 4, 48, False, 1, False), (1, 130, 7, 96, True, 1, False), (2, 5, 9, 16, True, 1, True),
    (1, 64, 2, 128, True, 2, False), (2, 50, 3, 128, False, 3, True), (1, 31, 6, 80, False, 4, False),
    (1, 3, 33, 32, False, 1, False), (5, 257, 1, 128, False, 1, False), (1, 2, 64, 128, False, 3, False),
    (40, 130, 8, 128, False, 1, True),
])
def test_equals_rotation_then_quantization(B, T, H, rotary, adjacent, n_axes, hadamard):
    rng = np.random.default_rng(B * 1000 + T + rotary)
    bits = rand_bits(rng, (B, T, H, 128))
    table = angles(500, rotary)
    axis = rng.integers(0, n_axes, rotary // 2)
    axis[:n_axes] = np.arange(n_axes)
    pos = rng.integers(0, 500, (n_axes, B, T)).astype(np.int32)
    rope = qk.Rope(torch.from_numpy(table).cuda(), adjacent=adjacent, pair_axis=axis.tolist() if n_axes > 1 else None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qk.quantize_qk_rope(to_dev(bits), rope, positions=torch.from_numpy(pos).cuda(), hadamard=hadamard,
                              dev_status=status)
    check(got, expected(bits, table, pos, axis, adjacent, hadamard), T)
    assert not got.codes[:, :, T:].any() and int(status) == 0
    assert not qk_scales_logical(got.scales.cpu().numpy(), got.cap)[:, :, T:].any()


@pytest.mark.parametrize("adjacent", [False, True])
def test_values_on_and_near_the_rounding_borders(adjacent):
    """Cosines and sines of a few bits: many results lie on the middle between two bf16 values, or one fp32 unit beside it."""
    rng = np.random.default_rng(7)
    B, T, H = 2, 64, 8
    bits = rand_bits(rng, (B, T, H, 128), spread=1.0)
    table = (rng.integers(-16, 17, (64, 64, 2)) / 16.0).astype(np.float32)
    table[1::2] *= np.float32(1 + 2.0 ** -20)
    table[2::4] = np.nextafter(table[2::4], np.float32(2))
    pos = np.arange(T, dtype=np.int32)[None, None].repeat(B, 1)
    got = qk.quantize_qk_rope(to_dev(bits), qk.Rope(torch.from_numpy(table).cuda(), adjacent=adjacent))
    y = rotate(bits, table, pos, None, adjacent)
    exact = 0
    x = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    for i in range(64):  # how many results are ties
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + 64)
        c, s = (table[pos[0], i, e].astype(np.float64)[:, :, None] for e in (0, 1))
        u = (x[..., a] * c - x[..., b] * s).astype(np.float32).view(np.uint32) & 0xFFFF
        exact += int((np.abs(u.astype(np.int64) - 0x8000) <= 4).sum())
    assert exact > 100
    check(got, oracle.quantize_qk(y), T)


@pytest.mark.parametrize("case", ["zeros", "tiny", "large", "cancel"])
def test_special_values(case):
    rng = np.random.default_rng(3)
    B, T, H = 1, 40, 4
    bits = rand_bits(rng, (B, T, H, 128))
    table = angles(T, 128)
    if case == "zeros":       # zeros of both signs, and rows of nothing else
        bits[..., ::3] = 0x8000
        bits[..., 1::3] = 0
        bits[:, 5] = 0x8000
        bits[:, 6] = 0
    elif case == "tiny":      # subnormal inputs and results
        bits = (rng.integers(0, 0x0180, bits.shape) | (rng.integers(0, 2, bits.shape) << 15)).astype(np.uint16)
    elif case == "large":     # close to the largest bf16 value, and half the range below it
        bits[:, ::2] = (0x7E00 + rng.integers(0, 0x80, bits[:, ::2].shape)).astype(np.uint16)
    else:                     # x_a c - x_b s cancels to a few bits
        table[:, :, 0] = np.float32(0.70710677)
        table[:, :, 1] = np.nextafter(np.float32(0.70710677), np.float32(1))
        bits[..., 64:] = bits[..., :64]
    pos = np.arange(T, dtype=np.int32)[None, None]
    for hadamard in (False, True) if case != "large" else (False,):
        got = qk.quantize_qk_rope(to_dev(bits), qk.Rope(torch.from_numpy(table).cuda()), hadamard=hadamard)
        check(got, expected(bits, table, pos, None, False, hadamard), T)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("others", [0x0000, 0x3F80])
def test_results_that_underflow_keep_their_sign(adjacent, others):
    """x_a c - x_b s = -2^-152 and its like: below what fp32 holds, so the code is a zero, whose sign is the exact value's."""
    rng = np.random.default_rng(17)
    B, T, H = 2, 16, 5
    bits = np.full((B, T, H, 128), others, np.uint16)
    at = np.arange(0, 64, 3)
    table = np.zeros((T, 64, 2), np.float32)
    table[..., 0], table[..., 1] = 1.0, 0.0
    # Subnormal values of up to two bits with cosines and sines of 2^-14 .. 2^-22: results of 2^-155 .. 2^-144, both signs.
    small = lambda: (rng.integers(1, 4, (B, T, H, len(at))) | (rng.integers(0, 2, (B, T, H, len(at))) << 15)).astype(np.uint16)
    a, b = (2 * at, 2 * at + 1) if adjacent else (at, at + 64)
    bits[..., a], bits[..., b] = small(), small()
    table[:, at] = np.ldexp(rng.choice([-1.0, 1.0], (T, len(at), 2)), -rng.integers(14, 23, (T, len(at), 2))).astype(np.float32)
    pos = np.arange(T, dtype=np.int32)[None, None].repeat(B, 1)
    got = qk.quantize_qk_rope(to_dev(bits), qk.Rope(torch.from_numpy(table).cuda(), adjacent=adjacent))
    check(got, oracle.quantize_qk(rotate(bits, table, pos, None, adjacent)), T)


def test_strides_positions_and_starts():
    """Heads of a fused projection, positions of every shape, starts: the same rows."""
    rng = np.random.default_rng(11)
    B, T, H = 3, 21, 4
    table = angles(300, 128)
    rope = qk.Rope(torch.from_numpy(table).cuda())
    fused = rand_bits(rng, (B, T, 3 * H, 128))
    x = to_dev(fused)[:, :, H:2 * H]
    bits = fused[:, :, H:2 * H]
    start = np.array([0, 7, 279], np.int32)
    pos = (start[:, None] + np.arange(T)).astype(np.int32)[None]
    want = expected(bits, table, pos, None, False, False)
    check(qk.quantize_qk_rope(x, rope, start=torch.from_numpy(start).cuda()), want, T)
    check(qk.quantize_qk_rope(x, rope, positions=torch.from_numpy(pos[0]).cuda()), want, T)
    wide = torch.zeros((1, T, 5, B), dtype=torch.int32, device="cuda")
    wide[:, :, 2] = torch.from_numpy(pos.transpose(0, 2, 1)).cuda()
    check(qk.quantize_qk_rope(x, rope, positions=wide[:, :, 2].permute(0, 2, 1)), want, T)
    same = torch.arange(T, dtype=torch.int32, device="cuda")[None].expand(B, T)
    check(qk.quantize_qk_rope(x, rope, positions=same),
          expected(bits, table, np.broadcast_to(np.arange(T), (1, B, T)), None, False, False), T)
    # A permuted input: [B, H, T, 128] in memory.
    y = to_dev(bits).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    check(qk.quantize_qk_rope(y, rope, positions=torch.from_numpy(pos[0]).cuda()), want, T)


def test_padding_and_kept_buffers():
    rng = np.random.default_rng(12)
    B, T, H = 2, 3, 5
    table = angles(64, 128)
    rope = qk.Rope(torch.from_numpy(table).cuda())
    bits = rand_bits(rng, (B, T, H, 128))
    pos = np.broadcast_to(np.arange(T), (1, B, T))
    codes, scales = expected(bits, table, pos, None, False, False)
    kept = qk.MXFP4(torch.full((B, H, 256, 64), 0xA5, dtype=torch.uint8, device="cuda"),
                    torch.full((B, H, 2, 512), 0x5A, dtype=torch.uint8, device="cuda"), B, H, 256, 256)
    lens = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    for pad in (False, True):
        got = qk.quantize_qk_rope(to_dev(bits), rope, out=kept, pad=pad, seqlens=lens)
        assert got is kept and got.length == T
        c = unpack_e2m1(got.codes.cpu().numpy())
        s = qk_scales_logical(got.scales.cpu().numpy(), 256)
        assert np.array_equal(c[0, :, :3], codes[0]) and np.array_equal(c[1, :, :1], codes[1, :, :1])
        assert np.array_equal(s[0, :, :3], scales[0]) and np.array_equal(s[1, :, :1], scales[1, :, :1])
        assert not c[1, :, 1:3].any() and not s[1, :, 1:3].any()
        if pad:
            assert not c[:, :, 3:].any() and not s[:, :, 3:].any()
        else:
            assert (got.codes[:, :, 3:] == 0xA5).all() and (torch.from_numpy(s[:, :, 3:]) == 0x5A).all()


def test_positions_outside_the_table_are_reported_and_read_its_first_row():
    rng = np.random.default_rng(13)
    bits = rand_bits(rng, (1, 4, 2, 128))
    table = angles(16, 128)
    rope = qk.Rope(torch.from_numpy(table).cuda())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = torch.tensor([[3, -1, 16, 15]], dtype=torch.int32, device="cuda")
    got = qk.quantize_qk_rope(to_dev(bits), rope, positions=bad, dev_status=status)
    assert int(status) == 1
    check(got, expected(bits, table, np.array([[[3, 0, 0, 15]]]), None, False, False), 4)
    # Padding rows have no position: theirs may be anything.
    status.zero_()
    got = qk.quantize_qk_rope(to_dev(bits), rope, positions=torch.tensor([[3, 15, 99, -7]], dtype=torch.int32, device="cuda"),
                              seqlens=torch.tensor([2]), dev_status=status)
    assert int(status) == 0 and not got.codes[:, :, 2:].any()


def test_empty_input_and_python_refusals():
    rope = qk.Rope(torch.from_numpy(angles(16, 128)).cuda())
    x = torch.zeros((2, 0, 3, 128), dtype=torch.bfloat16, device="cuda")
    kept = qk.MXFP4(torch.full((2, 3, 128, 64), 9, dtype=torch.uint8, device="cuda"),
                    torch.full((2, 3, 1, 512), 9, dtype=torch.uint8, device="cuda"), 2, 3, 128, 0)
    qk.quantize_qk_rope(x, rope, out=kept, pad=False)
    assert (kept.codes == 9).all() and (kept.scales == 9).all()
    qk.quantize_qk_rope(x, rope, out=kept)
    assert not kept.codes.any() and not kept.scales.any()
    y = torch.zeros((2, 3, 3, 128), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(positions=torch.zeros((2, 4), dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros((2, 3), dtype=torch.int64, device="cuda")),
                dict(positions=torch.zeros((2, 3), dtype=torch.int32)), dict(start=torch.zeros(2, dtype=torch.int32)),
                dict(start=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(out=kept, cap=256)):
        with pytest.raises(ValueError):
            qk.quantize_qk_rope(y, rope, **bad)
    for bad in (torch.zeros(16, 64, 2), torch.zeros((16, 128), device="cuda"),
                torch.zeros((16, 64, 2), dtype=torch.float16, device="cuda"), torch.zeros((16, 64, 4), device="cuda")[..., ::2]):
        with pytest.raises(ValueError):
            qk.Rope(bad)
    with pytest.raises(ValueError):
        qk.Rope(torch.zeros((16, 64, 2), device="cuda"), pair_axis=[0] * 63)
    with pytest.raises(qk.QK4V8Error):
        qk.quantize_qk_rope(y, qk.Rope(torch.zeros((16, 60, 2), device="cuda")))


def test_captured_call_follows_its_inputs_on_another_stream():
    rng = np.random.default_rng(14)
    B, T, H = 4, 2, 8
    table = angles(100, 128)
    rope = qk.Rope(torch.from_numpy(table).cuda())
    x = torch.zeros((B, T, H, 128), dtype=torch.bfloat16, device="cuda")
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = qk.quantize_qk_rope(x, rope)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        qk.quantize_qk_rope(x, rope, start=start, out=kept, pad=False)
    for step in range(3):
        bits = rand_bits(rng, (B, T, H, 128))
        at = rng.integers(0, 98, B).astype(np.int32)
        x.copy_(to_dev(bits))
        start.copy_(torch.from_numpy(at))
        graph.replay()
        torch.cuda.synchronize()
        check(kept, expected(bits, table, (at[:, None] + np.arange(T))[None], None, False, False), T)


def test_table_of_the_package():
    t = qk.rope_table(1000, 64, base=500000.0).cpu().double()
    want = torch.from_numpy(np.arange(1000)[:, None] * 500000.0 ** (-2.0 * np.arange(32) / 64))
    # fp64 angles, one rounding to fp32 (half an eps of values up to 1).
    assert (t[..., 0] - want.cos()).abs().max() <= 2.0 ** -24 and (t[..., 1] - want.sin()).abs().max() <= 2.0 ** -24
