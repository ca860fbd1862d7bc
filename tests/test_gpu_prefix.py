"""Decode over a shared prefix against attention in 64 bits over the prefix and each sequence's own keys. The bounds on
the differences are derived in ref_positions.attention_row."""
import numpy as np
import pytest
import torch

import bit_quantized_attention_qk4v8_b200 as qk
from bit_quantized_attention_qk4v8_b200 import _lib
from gpu_util import to_dev
from layouts import fill_v_bytes
from ref_positions import angles, dequantize_qk, dequantize_v, f32_to_bf16, prefix_attention, rotate

pytestmark = pytest.mark.gpu


class Problem:
    def __init__(self, B, Hq, Hkv, nq, prefix, lens, seed=1, paged=False, q_mult=1.0, k_mult=None, cap=None):
        rng = np.random.default_rng(seed)
        self.B, self.Hq, self.Hkv, self.nq, self.prefix, self.lens = B, Hq, Hkv, nq, prefix, list(lens)
        self.most = max(self.lens)
        bits = lambda *s: f32_to_bf16(rng.standard_normal(s).astype(np.float32))
        self.q = f32_to_bf16((rng.standard_normal((B, nq, Hq, 128)) * q_mult).astype(np.float32))
        T = max(self.most, 1)
        self.pk, self.pv, self.k, self.v = bits(1, max(prefix, 1), Hkv, 128), bits(1, max(prefix, 1), Hkv, 128), bits(
            B, T, Hkv, 128), bits(B, T, Hkv, 128)
        if k_mult is not None:  # keys grow along the sequence
            f = lambda x, r: f32_to_bf16(((x.astype(np.uint32) << 16).view(np.float32) * r[None, :, None, None]).astype(np.float32))
            self.pk = f(self.pk, k_mult(np.arange(self.pk.shape[1])))
            self.k = f(self.k, k_mult(prefix + np.arange(T)))
        sl = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.sl = sl
        self.qp = qk.quantize_qk(to_dev(self.q))
        self.cap = cap or max(128, -(-T // 128) * 128)
        pcap = max(128, -(-prefix // 128) * 128)
        self.pkp = qk.quantize_qk(to_dev(self.pk), cap=pcap, seqlens=torch.tensor([prefix]))
        self.pvp = qk.quantize_v(to_dev(self.pv), cap=pcap, seqlens=torch.tensor([prefix]))
        self.kp = qk.quantize_qk(to_dev(self.k), cap=self.cap, seqlens=sl)
        self.vp = qk.quantize_v(to_dev(self.v), cap=self.cap, seqlens=sl)
        self.paged = paged
        if paged:
            nb, np_ = self.cap // 128, pcap // 128
            num = B * nb + np_ + 3
            perm = rng.permutation(num).astype(np.int32)
            self.prefix_table = torch.from_numpy(perm[:np_].copy()).cuda()
            bt = torch.from_numpy(perm[np_:np_ + B * nb].reshape(B, nb).copy())
            c = self.cache = qk.paged_kv(B, Hkv, num, bt)
            for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
                t.fill_(0xFF)
            for pages, kk, vv in ((self.prefix_table.long()[None], self.pkp, self.pvp), (bt.long().cuda(), self.kp, self.vp)):
                for i in range(pages.shape[1]):
                    c.k_codes[pages[:, i]] = kk.codes[:, :, i * 128:(i + 1) * 128]
                    c.k_scales[pages[:, i]] = kk.scales[:, :, i]
                    c.v_codes[pages[:, i]] = vv.codes[:, :, i]
                    c.v_scales[pages[:, i]] = vv.scales[:, :, i]
            c.seqlens.copy_(sl)

    def run(self, **kw):
        kw.setdefault("max_seqlen", self.most)
        kw.setdefault("return_lse", True)
        if self.paged:
            return qk.attention_decode_prefix_paged(self.qp, self.cache, self.prefix_table, self.prefix, **kw)
        return qk.attention_decode_prefix(self.qp, self.pkp, self.pvp, self.kp, self.vp, self.sl, prefix_len=self.prefix, **kw)

    def reference(self, causal=True, lens=None, scale=None):
        lens = self.lens if lens is None else lens
        none = np.zeros((self.Hkv, 0, 128))   # (the scales of V are those of the whole sequence)
        dk = [dequantize_qk(self.k[b:b + 1, :n])[0] if n else none for b, n in enumerate(lens)]
        dv = [dequantize_v(self.v[b:b + 1, :self.lens[b]])[0][:, :n] if n else none for b, n in enumerate(lens)]
        pk = dequantize_qk(self.pk)[0][:, :self.prefix]
        pv = dequantize_v(self.pv[:, :self.prefix])[0] if self.prefix else np.zeros((self.Hkv, 0, 128))
        return prefix_attention(dequantize_qk(self.q), pk, pv, dk, dv, causal, scale)


def check(got, want):
    out, lse = got
    ref, rl, tol, ltol = want
    d = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    assert np.isfinite(d).all()
    assert (d <= tol).all(), f"out: worst {np.max(d / tol):.3g} of its bound"
    g = lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(g), empty)
    e = np.abs(g[~empty] - rl[~empty])
    assert (e <= ltol[~empty]).all(), f"lse: worst {np.max(e / ltol[~empty]):.3g} of its bound"


CASES = [
    # B, Hq, Hkv, nq, prefix, own lengths
    (1, 1, 1, 1, 1, [0]), (1, 1, 1, 1, 0, [1]), (1, 1, 1, 1, 1, [1]), (2, 4, 2, 1, 127, [3, 0]),
    (3, 8, 2, 1, 128, [1, 128, 129]), (2, 4, 4, 2, 129, [2, 63]), (1, 8, 8, 8, 300, [8]), (4, 16, 1, 8, 200, [8, 9, 64, 65]),
    (3, 15, 3, 3, 257, [0, 1, 2]),               # fewer own keys than query tokens
    (13, 20, 4, 3, 500, [0, 1, 3, 130, 0, 200, 64, 0, 0, 5, 127, 128, 0]),  # rows straddle the row tiles
    (130, 2, 2, 1, 64, [i % 7 for i in range(130)]),                        # 128 sequences in a row tile
    (20, 8, 1, 1, 0, [0] * 20), (5, 4, 2, 2, 700, [0] * 5), (6, 4, 2, 4, 0, [0, 3, 300, 0, 1, 129]),
    (1, 6, 2, 5, 1500, [700]), (700, 8, 1, 1, 40, [i % 3 for i in range(700)]),   # 44 row tiles
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])))
def test_against_64_bits(case, paged):
    p = Problem(*case, paged=paged)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = p.run(dev_status=status)
    assert int(status) == 0
    check(got, p.reference())


def test_rows_without_a_key():
    out, lse = Problem(20, 8, 1, 1, 0, [0] * 20).run()
    assert not out.any() and torch.isneginf(lse).all()
    p = Problem(3, 4, 2, 3, 0, [1, 0, 3])
    out, lse = p.run()
    assert not out[1].any() and not out[0, :2].any() and torch.isneginf(lse[0, :, :2]).all() and out[0, 2].any()
    check((out, lse), p.reference())


@pytest.mark.parametrize("causal", [False, True])
def test_draft_blocks_see_all_own_keys_or_those_before_them(causal):
    p = Problem(5, 12, 2, 7, 150, [7, 0, 70, 3, 260], seed=4)
    check(p.run(causal_in_block=causal), p.reference(causal))


def test_softmax_scale():
    p = Problem(3, 8, 2, 2, 333, [5, 100, 0], seed=6)
    check(p.run(softmax_scale=0.3), p.reference(scale=0.3))


@pytest.mark.parametrize("order", ["up", "down", "jump", "zigzag"])
@pytest.mark.parametrize("prefix,lens", [(1000, [300, 0, 64]), (0, [500, 200, 129])])
def test_scores_that_pass_the_reference_by_far(order, prefix, lens):
    """The row's reference moves when a score passes it by 2^64: scores of hundreds, along the keys in every order."""
    n = prefix + max(lens)
    f = {"up": lambda j: 0.01 + 3.0 * j / n, "down": lambda j: 3.0 - 2.9 * j / n, "jump": lambda j: np.where(j < 90, 1e-3, 3.0),
         "zigzag": lambda j: np.where(j // 64 % 2 == 0, 1e-3, 1.0 + j / n)}[order]
    p = Problem(3, 8, 2, 2, prefix, lens, seed=8, q_mult=30.0, k_mult=f)
    assert np.abs(p.reference()[1]).max() > 200
    check(p.run(), p.reference())


# Enough tiles that every CTA has a run of several: of a long prefix, and of the own keys of many sequences.
RUNS = [(2, 8, 8, 1, 12000, [300, 0]), (24, 4, 4, 2, 128, [600 - 9 * i for i in range(24)])]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("case", RUNS, ids=["prefix", "own"])
@pytest.mark.parametrize("q_mult", [8.0, 30.0])
def test_references_that_move_within_a_run_of_tiles(q_mult, case, paged):
    """Every second tile's keys are small, and the others grow: a run's first maxima are passed by tens to hundreds of
    binades again and again, by more and by less than O can be scaled by (2^-126)."""
    p = Problem(*case, seed=40, paged=paged, q_mult=q_mult, k_mult=lambda j: np.where(j // 128 % 2 == 0, 1e-2, 0.2 + j / 4000))
    check(p.run(), p.reference())


def one_hot(p):
    """Whether each row's softmax is one key's: the gap from its largest score to the next passes by 100 (e^-100 is lost in
    any rounding here) what the two can be off by, 16 * 2^-24 of their terms' magnitudes each as in
    ref_positions.attention_row. Also the least step up, in binades, from the keys of the even tiles to the odd ones'."""
    q, none = dequantize_qk(p.q), np.zeros((p.Hkv, 0, 128))
    pk = dequantize_qk(p.pk)[0][:, :p.prefix] if p.prefix else none
    step = np.inf
    for b, n in enumerate(p.lens):
        own = dequantize_qk(p.k[b:b + 1, :n])[0] if n else none
        odd = np.arange(p.prefix + n) // 128 % 2 == 1
        for h in range(p.Hq):
            kv = h // (p.Hq // p.Hkv)
            for t in range(p.nq):
                m = max(0, n - p.nq + t + 1)
                k = np.concatenate((pk[kv], own[kv, :m]))
                s = k @ q[b, h, t] / np.sqrt(128)
                mag = (np.abs(k) @ np.abs(q[b, h, t])).max() / np.sqrt(128)
                top = np.sort(s)[-2:]
                if top[1] - top[0] < 100 + 2 * 16 * 2.0 ** -24 * mag:
                    return False, 0.0
                step = min(step, (top[1] - s[~odd[:len(s)]].max()) * np.log2(np.e))
    return True, step


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("case", RUNS, ids=["prefix", "own"])
def test_scores_that_jump_further_than_an_exponent_reaches(case, paged):
    """Queries and keys of N(0, 1000^2), but the keys of every second tile a millionth as large: the largest scores pass a
    run's first ones by a million binades. The softmax of such a row is one key's, so the output is that key's value,
    rounded to bf16 once (the general bound, whose spread of values is 0 here)."""
    p = Problem(*case, seed=41, paged=paged, q_mult=1000.0, k_mult=lambda j: np.where(j // 128 % 2 == 0, 1e-3, 1e3))
    alone, step = one_hot(p)
    assert alone and step > 3e5
    check(p.run(), p.reference())


@pytest.mark.parametrize("paged", [False, True])
def test_nothing_behind_the_last_token_is_seen(paged):
    """NaN codes and NaN scales behind the lengths: not a bit of the result changes."""
    p = Problem(4, 8, 2, 2, 333, [5, 100, 0, 161], paged=paged, seed=9)
    clean = p.run()
    def spoil(kc, ks, vc, vs, b, n):
        """Contiguous [B, H, ...] views."""
        cap = kc.shape[2]
        kc[b, :, n:] = 0xFF
        at = np.array([(t // 128) * 512 + (t % 32) * 16 + (t % 128) // 32 * 4 + g for t in range(n, cap) for g in range(4)])
        ks.view(ks.shape[0], ks.shape[1], -1)[b][:, torch.from_numpy(at).cuda()] = 0xFF
        fill_v_bytes(vc, b, n, 0xFF)
        ch = np.arange(128)
        at = np.array([(g // 4) * 512 + (c % 32) * 16 + c // 32 * 4 + g % 4 for g in range((n + 31) // 32, cap // 32) for c in ch], int)
        vs.view(vs.shape[0], vs.shape[1], -1)[b][:, torch.from_numpy(at).cuda()] = 0xFF
    spoil(p.pkp.codes, p.pkp.scales, p.pvp.codes, p.pvp.scales, 0, p.prefix)
    for b, n in enumerate(p.lens):
        spoil(p.kp.codes, p.kp.scales, p.vp.codes, p.vp.scales, b, n)
    p.qp.codes[:, :, 2:] = 0xFF
    if paged:
        for pages, kk, vv in ((p.prefix_table.long()[None], p.pkp, p.pvp), (p.cache.block_table.long(), p.kp, p.vp)):
            for i in range(pages.shape[1]):
                p.cache.k_codes[pages[:, i]] = kk.codes[:, :, i * 128:(i + 1) * 128]
                p.cache.k_scales[pages[:, i]] = kk.scales[:, :, i]
                p.cache.v_codes[pages[:, i]] = vv.codes[:, :, i]
                p.cache.v_scales[pages[:, i]] = vv.scales[:, :, i]
    got = p.run()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("where", ["k", "v", "v_scale", "k_scale"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_one_sequence_does_not_reach_another(where, bad):
    """NaN or infinity in sequence 2's own keys or values: the others' bits stay, though their rows share its tiles.
    (Key scales are the quantizer's, whose largest is 2^126, byte 0xFD; a value scale may be anything.)"""
    lens, nq = [70, 200, 130, 5, 64, 129], 2
    p = Problem(6, 8, 2, nq, 260, lens, seed=31)
    clean = p.run()
    if where in ("k", "v"):
        x = (p.k if where == "k" else p.v).copy()
        x[2, 100] = 0x7FC0 if bad == "nan" else 0x7F80
        x[2, 129, :, ::3] = 0xFF80
        d = to_dev(x)
        if where == "k":
            p.kp = qk.quantize_qk(d, cap=p.cap, seqlens=p.sl)
        else:
            p.vp = qk.quantize_v(d, cap=p.cap, seqlens=p.sl)
    else:
        t = (p.kp if where == "k_scale" else p.vp).scales
        t[2, :, 0, :] = 0xFD if where == "k_scale" else 0xFF if bad == "nan" else 0xFE
    out, lse = p.run()
    others = [b for b in range(6) if b != 2]
    assert torch.equal(out[others], clean[0][others]) and torch.equal(lse[others], clean[1][others])


@pytest.mark.parametrize("paged", [False, True])
def test_a_nan_in_the_prefix_reaches_every_row_that_averages_it(paged):
    """Every row sees the prefix, so a NaN among its values is in every row's output, in its head and channel, and nowhere
    else; as in the other decode calls."""
    def problem(bad):
        p = Problem(4, 8, 2, 2, 333, [5, 100, 0, 161], seed=12)
        if bad:
            p.pv[0, 70, 1, 9] = p.pv[0, 300, 0, 127] = 0x7FC0
        q = Problem.__new__(Problem)
        q.__dict__.update(p.__dict__)
        q.pvp = qk.quantize_v(to_dev(p.pv), cap=p.pkp.cap, seqlens=torch.tensor([p.prefix]))
        if paged:
            pages = 3 + 4 * 2
            q.paged, q.prefix_table = True, torch.tensor([7, 0, 9], dtype=torch.int32, device="cuda")
            bt = torch.tensor([[1, 2], [3, 4], [5, 6], [8, 10]], dtype=torch.int32)
            c = q.cache = qk.paged_kv(4, 2, pages, bt)
            for at, kk, vv in ((q.prefix_table.long()[None], q.pkp, q.pvp), (bt.long().cuda(), q.kp, q.vp)):
                for i in range(at.shape[1]):
                    c.k_codes[at[:, i]] = kk.codes[:, :, i * 128:(i + 1) * 128]
                    c.k_scales[at[:, i]] = kk.scales[:, :, i]
                    c.v_codes[at[:, i]] = vv.codes[:, :, i]
                    c.v_scales[at[:, i]] = vv.scales[:, :, i]
            c.seqlens.copy_(q.sl)
        return q
    clean, (out, lse) = problem(False).run(), problem(True).run()
    bad = torch.zeros(8, 128, dtype=torch.bool, device="cuda")
    bad[4:, 9] = bad[:4, 127] = True
    assert torch.isnan(out[:, :, bad]).all()
    assert torch.equal(out[:, :, ~bad], clean[0][:, :, ~bad]) and torch.equal(lse, clean[1])


def test_bounds_that_are_loose_or_cut():
    p = Problem(4, 8, 2, 1, 200, [5, 100, 0, 161], cap=1024)
    check(p.run(max_seqlen=1024), p.reference())
    check(p.run(max_seqlen=90), p.reference(lens=[5, 90, 0, 90]))
    check(p.run(max_seqlen=0), p.reference(lens=[0] * 4))
    p.sl.copy_(torch.tensor([-9, 100, 2**31 - 1, 161]))   # below 0: none; past the bound: cut to it
    got = p.run(max_seqlen=100)
    check((got[0][[0, 1, 3]], got[1][[0, 1, 3]]), [x[[0, 1, 3]] for x in p.reference(lens=[0, 100, 0, 100])])


def test_the_same_bits_each_time_from_pages_in_any_order():
    a, b = Problem(9, 16, 2, 3, 700, [i * 31 for i in range(9)]), Problem(9, 16, 2, 3, 700, [i * 31 for i in range(9)], paged=True)
    first = a.run()
    for p in (a, b, a):
        got = p.run()
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_buffers_of_the_caller():
    p = Problem(4, 8, 2, 2, 300, [5, 100, 0, 161])
    need = qk.decode_prefix_workspace_bytes(4, 8, 2, 2, 300, p.most)
    guard = torch.full((need + 512,), 0x5C, dtype=torch.uint8, device="cuda")
    out = torch.empty((4, 2, 8, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((4, 8, 2), device="cuda")
    got = p.run(workspace=guard[256:256 + need], out=out, lse=lse)
    assert got[0] is out and got[1] is lse and (guard[:256] == 0x5C).all() and (guard[256 + need:] == 0x5C).all()
    check(got, p.reference())
    only = p.run(return_lse=False)
    assert torch.equal(only, out)
    with pytest.raises(qk.QK4V8Error):
        p.run(workspace=guard[:need - 16])
    for bad in (dict(out=out.float()), dict(out=out[:, :1]), dict(out=out.cpu()), dict(out=out.transpose(1, 2)),
                dict(lse=lse.half()), dict(lse=lse[:2]), dict(lse=lse.cpu()), dict(workspace=guard.cpu()),
                dict(workspace=guard[::2])):
        with pytest.raises(ValueError):
            p.run(**bad)
    for bad in (dict(k=p.pkp), dict(v=p.kp), dict(pk=p.kp), dict(v=qk.MXFP8V(p.vp.codes[..., ::2], p.vp.scales, 4, 2, p.vp.cap, 1))):
        a = dict(pk=p.pkp, pv=p.pvp, k=p.kp, v=p.vp)
        a.update(bad)
        with pytest.raises(ValueError):
            qk.attention_decode_prefix(p.qp, a["pk"], a["pv"], a["k"], a["v"], p.sl)


def test_pages_outside_the_pool_are_reported():
    for where in ("prefix_table", "block_table"):
        for bad in (-1, 1 << 20):
            p = Problem(2, 4, 2, 1, 300, [200, 40], paged=True)
            t = p.prefix_table if where == "prefix_table" else p.cache.block_table
            t.view(-1)[1] = bad
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            p.run(dev_status=status)
            assert int(status) == 1
    p = Problem(2, 4, 2, 1, 300, [100, 40], paged=True, cap=256)
    p.cache.block_table[:, 1] = -1   # behind the lengths: not looked at
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(p.run(dev_status=status), p.reference())
    assert int(status) == 0


def test_two_captured_calls_replayed_with_new_lengths():
    a, b = Problem(6, 8, 2, 2, 500, [200] * 6, seed=1), Problem(3, 4, 4, 1, 90, [150] * 3, seed=2)
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)], []
    for p, s, g in zip((a, b), streams, graphs):
        ws = torch.empty(qk.decode_prefix_workspace_bytes(p.B, p.Hq, p.Hkv, p.nq, p.prefix, p.most), dtype=torch.uint8,
                         device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            outs.append(p.run(workspace=ws))
    for la, lb in (([200, 0, 1, 64, 65, 130], [0, 0, 0]), ([0] * 6, [150, 2, 64]), ([2, 3, 4, 199, 128, 127], [1, 1, 128])):
        a.sl.copy_(torch.tensor(la))
        b.sl.copy_(torch.tensor(lb))
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):   # both in flight, on streams of their own
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        check(outs[0], a.reference(lens=la))
        check(outs[1], b.reference(lens=lb))


@pytest.mark.timeout(120)
def test_a_wait_that_runs_out_is_reported_and_the_context_survives():
    p = Problem(4, 8, 2, 2, 300, [5, 100, 0, 161])
    ref = p.run()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _lib.lib().qk4v8_test_set_stall(1)
    try:
        p.run(dev_status=status)
        torch.cuda.synchronize()
    finally:
        _lib.lib().qk4v8_test_set_stall(0)
    assert int(status) == 4
    again = p.run()
    assert torch.equal(again[0], ref[0]) and torch.equal(again[1], ref[1])


@pytest.mark.parametrize("Hq,Hkv,nq,hadamard", [(8, 2, 1, False), (12, 4, 3, True)])
def test_serving_steps_of_all_of_it(Hq, Hkv, nq, hadamard):
    """A prefix appended once, then steps: Q rotated into a kept buffer, K rotated and V appended behind the prefix's
    positions, attention over prefix and pages, some sequences idle; against 64 bits on all tokens."""
    B, prefix, steps = 5, 300, 4
    rng = np.random.default_rng(21)
    T = nq * steps
    mk = lambda *s: f32_to_bf16(rng.standard_normal(s).astype(np.float32))
    pk, pv, k, v, q = mk(1, prefix, Hkv, 128), mk(1, prefix, Hkv, 128), mk(B, T, Hkv, 128), mk(B, T, Hkv, 128), mk(B, T, Hq, 128)
    table = angles(prefix + T, 128)
    rope = qk.Rope(torch.from_numpy(table).cuda())
    num = 3 + B + 2
    perm = rng.permutation(num).astype(np.int32)
    prefix_table = torch.from_numpy(perm[:3].copy()).cuda()
    cache = qk.paged_kv(B, Hkv, num, torch.from_numpy(perm[3:3 + B].reshape(B, 1).copy()), hadamard_k=hadamard)
    head = qk.PagedKV(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales,
                      torch.zeros((1, Hkv, 32, 128), dtype=torch.bfloat16, device="cuda"), prefix_table[None],
                      torch.zeros(1, dtype=torch.int32, device="cuda"), hadamard)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qk.kv_append_rope(head, to_dev(pk), to_dev(pv), rope, dev_status=status)
    kept = qk.MXFP4(torch.empty((B, Hq, 128, 64), dtype=torch.uint8, device="cuda"),
                    torch.empty((B, Hq, 1, 512), dtype=torch.uint8, device="cuda"), B, Hq, 128, nq)
    lens = np.zeros(B, int)
    seen_k, seen_v = [np.zeros((0, Hkv, 128), np.uint16)] * B, [np.zeros((0, Hkv, 128), np.uint16)] * B
    at = lambda n: (prefix + lens[:, None] + np.arange(n)).astype(np.int32)
    deq = lambda x: dequantize_qk_maybe(x, hadamard)
    for s in range(steps):
        go = np.ones(B, int) * nq
        go[s % B] = 0                       # an idle sequence: attends with what it has
        qs, ks, vs = (x[:, s * nq:(s + 1) * nq] for x in (q, k, v))
        pos = at(nq)
        qk.quantize_qk_rope(to_dev(qs), rope, start=(prefix + cache.seqlens).int(), out=kept, pad=False, hadamard=hadamard,
                            dev_status=status)
        qk.kv_append_rope(cache, to_dev(ks), to_dev(vs), rope, positions=torch.from_numpy(pos).cuda(),
                          new_lens=torch.from_numpy(go.astype(np.int32)).cuda(), dev_status=status)
        got = qk.attention_decode_prefix_paged(kept, cache, prefix_table, prefix, max_seqlen=128, return_lse=True,
                                               dev_status=status)
        turned = rotate(ks, table, pos[None])
        for b in range(B):
            if go[b]:
                seen_k[b], seen_v[b] = np.concatenate((seen_k[b], turned[b])), np.concatenate((seen_v[b], vs[b]))
        lens += go
        assert int(status) == 0 and cache.seqlens.cpu().tolist() == lens.tolist()
        want = prefix_attention(deq(rotate(qs, table, pos[None])), deq(rotate(pk, table, np.arange(prefix)[None, None]))[0],
                                dequantize_v(pv)[0], [deq(x[None])[0] if len(x) else np.zeros((Hkv, 0, 128)) for x in seen_k],
                                [dequantize_v(x[None])[0] if len(x) else np.zeros((Hkv, 0, 128)) for x in seen_v])
        check(got, want)


def test_the_documented_loop_over_a_shared_prefix():
    """The user guide's lines, from the rotary positions to the attention, run as they stand for three steps of a batch:
    against 64 bits with each token at its place behind the prefix."""
    import re
    from pathlib import Path
    text = (Path(qk.__file__).resolve().parents[1] / "README.md").read_text()
    lines = re.search(r"^rope = qk\.Rope\(.*?^out = qk\.attention_decode_prefix_paged\([^\n]*$", text, re.S | re.M).group(0)
    B, Hq, Hkv, nq, prefix, steps, max_pos = 4, 8, 2, 2, 300, 3, 512
    rng = np.random.default_rng(23)
    mk = lambda *s: f32_to_bf16(rng.standard_normal(s).astype(np.float32))
    pk, pv, k, v, q = mk(1, prefix, Hkv, 128), mk(1, prefix, Hkv, 128), mk(B, nq * steps, Hkv, 128), mk(
        B, nq * steps, Hkv, 128), mk(B, nq * steps, Hq, 128)
    pages = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")
    cache = qk.paged_kv(B, Hkv, 8, torch.tensor([[1], [3], [4], [6]], dtype=torch.int32))
    head = qk.PagedKV(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales,
                      torch.zeros((1, Hkv, 32, 128), dtype=torch.bfloat16, device="cuda"), pages[None],
                      torch.zeros(1, dtype=torch.int32, device="cuda"))
    qk.kv_append_rope(head, to_dev(pk), to_dev(pv), qk.Rope(qk.rope_table(max_pos)))
    table = qk.rope_table(max_pos).cpu().numpy()
    n = torch.full((B,), nq, dtype=torch.int32, device="cuda")
    turned = rotate(k, table, (prefix + np.arange(nq * steps))[None, None].repeat(B, 1))
    for s in range(steps):
        at = slice(s * nq, (s + 1) * nq)
        env = dict(qk=qk, torch=torch, cache=cache, max_pos=max_pos, q_step=to_dev(q[:, at]), k_step=to_dev(k[:, at]),
                   v_step=to_dev(v[:, at]), n=n, prefix_pages=pages, prefix_len=prefix, max_seqlen=128, B=B, Hq=Hq, Hkv=Hkv,
                   nq=nq)
        exec(lines, env)
        seen = (s + 1) * nq
        assert cache.seqlens.cpu().tolist() == [seen] * B
        pos = (prefix + np.arange(s * nq, seen))[None, None].repeat(B, 1)
        want = prefix_attention(dequantize_qk(rotate(q[:, at], table, pos)),
                                dequantize_qk(rotate(pk, table, np.arange(prefix)[None, None]))[0], dequantize_v(pv)[0],
                                [dequantize_qk(turned[b:b + 1, :seen])[0] for b in range(B)],
                                [dequantize_v(v[b:b + 1, :seen])[0] for b in range(B)])
        d = np.abs(env["out"].float().cpu().numpy().astype(np.float64) - want[0])
        assert (d <= want[2]).all(), f"step {s}: worst {np.max(d / want[2]):.3g} of its bound"


def test_pages_far_into_a_large_pool():
    """Pages whose bytes lie past 2^32 of the pool: appended and attended to bit for bit as in a small pool."""
    B, Hkv, Hq, nq, prefix, T = 3, 8, 16, 2, 200, 300
    pages = (1 << 32) // (Hkv * 128 * 128) + 64          # 4.3 GB of V
    if torch.cuda.mem_get_info()[0] < 9 << 30:
        pytest.skip("needs 9 GB")
    rng = np.random.default_rng(3)
    mk = lambda *s: to_dev(f32_to_bf16(rng.standard_normal(s).astype(np.float32)))
    pk, pv, k, v, q = mk(1, prefix, Hkv, 128), mk(1, prefix, Hkv, 128), mk(B, T, Hkv, 128), mk(B, T, Hkv, 128), mk(B, nq, Hq, 128)
    rope = qk.Rope(torch.from_numpy(angles(prefix + T, 128)).cuda())
    qp = qk.quantize_qk_rope(q, rope, start=torch.full((B,), prefix + T - nq, dtype=torch.int32, device="cuda"))
    outs = []
    for num in (16, pages):
        perm = torch.arange(num - 1, num - 15, -1, dtype=torch.int32)
        cache = qk.paged_kv(B, Hkv, num, perm[2:2 + 3 * B].reshape(B, 3))
        head = qk.PagedKV(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales,
                          torch.zeros((1, Hkv, 32, 128), dtype=torch.bfloat16, device="cuda"), perm[None, :2].cuda(),
                          torch.zeros(1, dtype=torch.int32, device="cuda"))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        qk.kv_append_rope(head, pk, pv, rope, dev_status=status)
        pos = torch.arange(prefix, prefix + T, dtype=torch.int32, device="cuda")[None].expand(B, T)
        qk.kv_append_rope(cache, k, v, rope, positions=pos, dev_status=status)
        outs.append(qk.attention_decode_prefix_paged(qp, cache, perm[:2].cuda(), prefix, max_seqlen=384, return_lse=True,
                                                     dev_status=status))
        assert int(status) == 0
        if num == pages:
            assert cache.v_codes.numel() > 1 << 32
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def dequantize_qk_maybe(bits, hadamard):
    """What the packed rows hold; rotated by the Hadamard matrix on both sides, Q K^T is what it is."""
    if not hadamard:
        return dequantize_qk(bits)
    import oracle
    from ref_positions import E2M1
    c, s = oracle.quantize_qk_hadamard(bits)
    return E2M1[c] * np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, -1)
