"""Rotating append into pages: after any run of appends, by this call and by kv_append, each sequence's pages hold the
bytes of quantizing the whole (rotated) sequence at once, and everything else is as it was."""
import numpy as np
import pytest
import torch

import bit_quantized_attention_qk4v8_b200 as qk
import oracle
from gpu_util import to_dev
from layouts import gather_pages, qk_scales_logical, unpack_e2m1, v_scales_logical
from ref_positions import angles, f32_to_bf16, rotate

pytestmark = pytest.mark.gpu
FILL = 0xA7


def make(B, H, T, rotary, adjacent, n_axes, hadamard, seed, max_pages, num_pages):
    rng = np.random.default_rng(seed)
    k = f32_to_bf16(rng.standard_normal((B, T, H, 128)).astype(np.float32))
    v = f32_to_bf16((rng.standard_normal((B, T, H, 128)) * np.exp2(rng.uniform(-6, 6, (B, 1, H, 128)))).astype(np.float32))
    table = angles(T + 40, rotary)
    axis = rng.integers(0, n_axes, rotary // 2)
    axis[:n_axes] = np.arange(n_axes)
    pos = rng.integers(0, T + 40, (n_axes, B, T)).astype(np.int32)
    rope = qk.Rope(torch.from_numpy(table).cuda(), adjacent, axis.tolist() if n_axes > 1 else None)
    bt = rng.permutation(num_pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    cache = qk.paged_kv(B, H, num_pages, torch.from_numpy(bt), hadamard_k=hadamard)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(FILL)
    return k, v, table, axis, pos, rope, cache


def check(cache, turned, v, lens, hadamard=False):
    bt = cache.block_table.cpu().numpy()
    B, max_pages = bt.shape
    pools = [t.cpu().numpy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    kc, ks = gather_pages(pools[0], pools[1], bt, max_pages)
    vc, vs = gather_pages(pools[2], pools[3], bt, max_pages)
    cap = max_pages * 128
    ksl, vsl = qk_scales_logical(ks, cap), v_scales_logical(vs, cap)
    for b, L in enumerate(lens):
        top = (L + 31) // 32 * 32
        if L:
            rows = turned[b:b + 1, :L]
            oc, os_ = oracle.quantize_qk_hadamard(rows) if hadamard else oracle.quantize_qk(rows)
            assert np.array_equal(unpack_e2m1(kc[b:b + 1, :, :L]), oc), (b, L)
            assert np.array_equal(ksl[b:b + 1, :, :L], os_), (b, L)
            oc, os_ = oracle.quantize_v(v[b:b + 1, :L], np.full((1,), L, np.int32))
            assert np.array_equal(vc[b:b + 1, ..., :L], oc[..., :L]), (b, L)
            assert np.array_equal(vsl[b:b + 1, :, :, :top // 32], os_[..., :top // 32]), (b, L)
            assert not vc[b, ..., L:top].any()
        # Behind the sequence: as it was.
        assert (kc[b, :, L:] == FILL).all() and (ksl[b, :, L:] == FILL).all(), (b, L)
        assert (vc[b, ..., top:] == FILL).all() and (vsl[b, :, :, top // 32:] == FILL).all(), (b, L)
    others = np.setdiff1d(np.arange(pools[0].shape[0]), bt.reshape(-1))
    assert all((p[others] == FILL).all() for p in pools)


@pytest.mark.parametrize("H,rotary,adjacent,n_axes,hadamard", [
    (1, 128, False, 1, False), (3, 128, False, 1, True), (2, 64, True, 1, False), (8, 128, False, 3, False),
    (5, 48, False, 2, True)])
def test_ragged_appends(H, rotary, adjacent, n_axes, hadamard):
    B, T = 5, 300
    k, v, table, axis, pos, rope, cache = make(B, H, T, rotary, adjacent, n_axes, hadamard, 31 + H, 3, 20)
    turned = rotate(k, table, pos, axis, adjacent)
    kd, vd, pd, td = to_dev(k), to_dev(v), torch.from_numpy(pos).cuda(), to_dev(turned)
    rng = np.random.default_rng(5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = np.zeros(B, int)
    for step in range(9):
        n = int([1, 8, 40, 1, 33, 7, 1, 90, 64][step])
        new = rng.integers(0, n + 1, B)
        new[step % B] = 0
        new = np.minimum(new, T - lens)
        kn, vn = torch.zeros((B, n, H, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, n, H, 128),
                                                                                              dtype=torch.bfloat16, device="cuda")
        pn = torch.zeros((n_axes, B, n), dtype=torch.int32, device="cuda")
        kn.fill_(float("nan"))   # rows past new_lens are not read as tokens
        vn.fill_(float("nan"))
        pn.fill_(-5)
        for b in range(B):
            a, e = lens[b], lens[b] + new[b]
            kn[b, :new[b]], vn[b, :new[b]], pn[:, b, :new[b]] = kd[b, a:e], vd[b, a:e], pd[:, b, a:e]
        qk.kv_append_rope(cache, kn, vn, rope, positions=pn, new_lens=torch.from_numpy(new.astype(np.int32)).cuda(),
                          dev_status=status)
        lens = lens + new
        assert int(status) == 0 and cache.seqlens.cpu().tolist() == lens.tolist()
        check(cache, turned, v, lens, hadamard)


def test_runs_with_the_plain_append():
    """Tokens by turns from the two calls (the plain one given rotated K), equal lengths, K and V with strides of their own."""
    B, H, T = 2, 4, 280
    k, v, table, axis, pos, rope, cache = make(B, H, T, 128, False, 1, False, 77, 3, 9)
    pos[:] = np.arange(T)
    turned = rotate(k, table, pos, axis)
    fused = torch.cat((to_dev(k), to_dev(v)), 2)                  # one projection's [K | V]
    vt = to_dev(v).permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    td, vd = to_dev(turned), to_dev(v)
    L = 0
    for i, n in enumerate([5, 120, 3, 1, 31, 64, 1, 40]):
        if i % 2:
            qk.kv_append(cache, td[:, L:L + n], vd[:, L:L + n])
        elif i % 4:
            qk.kv_append_rope(cache, fused[:, L:L + n, :H], fused[:, L:L + n, H:], rope)
        else:
            qk.kv_append_rope(cache, to_dev(k)[:, L:L + n], vt[:, L:L + n], rope)
        L += n
        check(cache, turned, v, [L] * B)


def test_whole_prompt_and_lengths_beside():
    """Pages filled in one call, the new lengths in an array of their own, then one token past the pages."""
    B, H, T = 3, 2, 384
    k, v, table, axis, pos, rope, cache = make(B, H, T, 128, False, 1, False, 78, 3, 9)
    pos[:] = np.arange(T)
    turned = rotate(k, table, pos, axis)
    out = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qk.kv_append_rope(cache, to_dev(k), to_dev(v), rope, seqlens_out=out, dev_status=status)
    assert out.cpu().tolist() == [T] * B and cache.seqlens.cpu().tolist() == [0] * B and int(status) == 0
    check(cache, turned, v, [T] * B)
    cache.seqlens.copy_(out)
    qk.kv_append_rope(cache, to_dev(k)[:, :1], to_dev(v)[:, :1], rope, seqlens_out=out, dev_status=status)
    assert int(status) == 1
    check(cache, turned, v, [T] * B)


def test_bad_pages_lengths_and_counts_are_reported_and_skipped():
    B, H, T = 6, 2, 50
    k, v, table, axis, pos, rope, cache = make(B, H, T, 128, False, 1, False, 79, 2, 12)
    pos[:] = np.arange(T)
    turned = rotate(k, table, pos, axis)
    clean = cache.block_table.clone()
    cache.block_table[1, 0] = -1
    cache.block_table[2, 0] = 12
    cache.seqlens[3] = -4
    cache.seqlens[4] = 2 * 128 + 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(B, dtype=torch.int32, device="cuda")
    qk.kv_append_rope(cache, to_dev(k), to_dev(v), rope, dev_status=status, seqlens_out=out)
    assert int(status) == 1
    cache.block_table.copy_(clean)
    check(cache, turned, v, [T, 0, 0, 0, 0, T])
    # Counts outside 0..n are held to it.
    cache.seqlens.copy_(torch.tensor([T, 0, 0, 0, 0, T]))
    status.zero_()
    new = torch.tensor([-3, 2, 99, 0, 1, 0], dtype=torch.int32, device="cuda")
    qk.kv_append_rope(cache, to_dev(k)[:, :4], to_dev(v)[:, :4], rope, new_lens=new, dev_status=status)
    assert int(status) == 1 and cache.seqlens.cpu().tolist() == [T, 2, 4, 0, 1, T]
    check(cache, turned, v, [T, 2, 4, 0, 1, T])


def test_values_that_are_not_finite_are_packed_as_by_the_plain_append():
    """A NaN or an infinity of a value leaves the rest of its group of 32 as kv_append and quantize_v pack it."""
    B, H, T = 2, 3, 70
    k, v, table, axis, pos, rope, cache = make(B, H, T, 128, False, 1, False, 84, 1, 2)
    pos[:] = np.arange(T)
    v[0, 5, 1, ::7] = 0x7FC0
    v[0, 40, 2, 3:9] = 0xFFC1
    v[1, 69, 0, ::2] = 0x7F80
    v[1, 33] = 0xFF80
    other = qk.paged_kv(B, H, 2, cache.block_table)
    for a, b in zip((other.k_codes, other.k_scales, other.v_codes, other.v_scales), (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)):
        a.copy_(b)
    turned = to_dev(rotate(k, table, pos, axis))
    kd, vd = to_dev(k), to_dev(v)
    for a, b in ((0, 20), (20, 21), (21, 66), (66, T)):
        qk.kv_append_rope(cache, kd[:, a:b], vd[:, a:b], rope)
        qk.kv_append(other, turned[:, a:b], vd[:, a:b])
    whole = qk.quantize_v(vd)
    for b in range(B):
        page = int(cache.block_table[b, 0])
        assert torch.equal(other.v_codes[page, ..., :96], whole.codes[b, :, 0, :, :96])
        assert torch.equal(cache.v_codes[page], other.v_codes[page]) and torch.equal(cache.v_scales[page], other.v_scales[page])


@pytest.mark.parametrize("in_place", [False, True])
def test_lengths_after_sequences_and_tokens_that_were_skipped(in_place):
    """A sequence that is skipped (its length below 0 or past its pages) keeps its length; tokens without a page count, as
    kv_append's do: the caller sees the status and has the numbers that it asked for."""
    B, H, T = 6, 2, 50
    k, v, table, axis, pos, rope, cache = make(B, H, T, 128, False, 1, False, 83, 2, 12)
    cache.block_table[5, 0] = -1
    lens = [0, -4, 2 * 128 + 1, 2 * 128, 230, 0]
    cache.seqlens.copy_(torch.tensor(lens))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cache.seqlens if in_place else torch.full((B,), -77, dtype=torch.int32, device="cuda")
    new = torch.tensor([T, 7, 7, 3, T, 20], dtype=torch.int32, device="cuda")
    rope = qk.Rope(torch.from_numpy(angles(300, 128)).cuda())
    qk.kv_append_rope(cache, to_dev(k), to_dev(v), rope, new_lens=new, dev_status=status,
                      seqlens_out=None if in_place else out)
    assert int(status) == 1
    assert out.cpu().tolist() == [T, -4, 2 * 128 + 1, 2 * 128 + 3, 230 + T, 20]
    assert in_place or cache.seqlens.cpu().tolist() == lens


def test_captured_appends():
    """A captured append, replayed for one token after the other on a stream of its own."""
    B, H, T = 4, 8, 70
    k, v, table, axis, pos, rope, cache = make(B, H, T, 128, False, 1, True, 80, 1, 5)
    pos[:] = np.arange(T)
    turned = rotate(k, table, pos, axis)
    kd, vd = to_dev(k), to_dev(v)
    kn, vn = kd[:, :1].clone(), vd[:, :1].clone()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        qk.kv_append_rope(cache, kn, vn, rope)
    assert cache.seqlens.cpu().tolist() == [0] * B
    with torch.cuda.stream(stream):
        for t in range(T):
            kn.copy_(kd[:, t:t + 1])
            vn.copy_(vd[:, t:t + 1])
            graph.replay()
    torch.cuda.synchronize()
    check(cache, turned, v, [T] * B, hadamard=True)


def test_python_refusals():
    _, _, _, _, _, rope, cache = make(2, 2, 10, 128, False, 1, False, 81, 1, 4)
    x = torch.zeros((2, 3, 2, 128), dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for args, kw in (((x, x[:, :2]), {}), ((x[:1], x[:1]), {}), ((x[:, :, :1], x[:, :, :1]), {}), ((x.float(), x), {}),
                     ((x, x), dict(new_lens=lens[:1])), ((x, x), dict(new_lens=lens.long())),
                     ((x, x), dict(seqlens_out=lens.cpu())), ((x, x), dict(positions=lens))):
        with pytest.raises(ValueError):
            qk.kv_append_rope(cache, *args, rope, **kw)
