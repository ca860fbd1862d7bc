"""What is measured of the position-rotating quantizers and of the shared-prefix decode attention.

Three operators of one serving step over the packed KV cache (MXFP4 Q and K, MXFP8-E4M3 V):

  rope    rotary positions of one or several axes, applied to Q or K on the way into MXFP4
          (quantize_qk_rope);
  append  new keys and values into the pages of the cache, the keys rotated on the way
          (kv_append_rope);
  prefix  decode attention of a batch whose sequences share one prefix, contiguous or paged
          (attention_decode_prefix, attention_decode_prefix_paged).

The plain forms below are elementary torch operations. The rotation is taken in 64 bits, since a
rotated value next to a rounding border of a 4-bit code decides that code; attention is taken in 32.

Packed outputs: E4M3 codes and E8M0 scales are returned under their own torch types, which stand for
their values. Two E2M1 codes share a byte, for which torch has no type that it can read; those bytes
are returned as the whole numbers they are and have to be equal.
"""
import math

import torch

own = False

D = 128
PAGE = 128


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step's queries, of the B = 32, 32-head GQA decode workload, into the buffer that a decode
        # loop keeps: only the rows of the step are written, not the capacity.
        dict(name="rope_q_step", op="rope", B=32, T=1, H=32, rotary=128, adjacent=False, axes=1, hadamard=False,
             pad=False),
        # Keys of three images: three position axes shared by the batch, an odd token count, the outlier rotation.
        dict(name="rope_k_images", op="rope", B=3, T=1601, H=8, rotary=128, adjacent=False, axes=3, hadamard=True,
             pad=True),
        # A prompt whose model rotates half of each head, adjacent pairs.
        dict(name="rope_q_partial", op="rope", B=1, T=2047, H=64, rotary=64, adjacent=True, axes=1, hadamard=False,
             pad=True),
        # The queries of the S = 8192 prefill.
        dict(name="rope_q_prompt", op="rope", B=4, T=8192, H=32, rotary=128, adjacent=False, axes=1, hadamard=False,
             pad=True),
        # One token for each of 64 sequences of mixed lengths.
        dict(name="append_step", op="append", B=64, n=1, H=8, rotary=128, adjacent=False, axes=1, hadamard=False,
             ragged=False, start=2000),
        # A verified draft block: up to 8 tokens are kept of each sequence, some keep none.
        dict(name="append_verify", op="append", B=64, n=8, H=8, rotary=128, adjacent=False, axes=1, hadamard=False,
             ragged=True, start=1500),
        # Prompts with images, three axes, of different lengths in one padded batch.
        dict(name="append_images", op="append", B=5, n=1601, H=4, rotary=128, adjacent=False, axes=3, hadamard=True,
             ragged=True, start=0),
        # The S = 8192 prompts into empty pages.
        dict(name="append_prompt", op="append", B=4, n=8192, H=8, rotary=128, adjacent=False, axes=1, hadamard=False,
             ragged=False, start=0),
        # A few chats after a short system prompt, early in their answers.
        dict(name="prefix_small", op="prefix", B=4, G=4, H=8, nq=1, prefix=1000, suffix=100, empties=False,
             paged=False),
        # 32 requests on one 8192-token context, mixed answer lengths.
        dict(name="prefix_step", op="prefix", B=32, G=4, H=8, nq=1, prefix=8192, suffix=1024, empties=False,
             paged=True),
        # Odd everything: 13 sequences, groups of 5 heads, blocks of 3 tokens, some with no key of their own yet.
        dict(name="prefix_odd", op="prefix", B=13, G=5, H=4, nq=3, prefix=5003, suffix=777, empties=True, paged=True),
        # 8-token verify of 64 sequences, 64 heads, over a 16384-token prefix.
        dict(name="prefix_verify", op="prefix", B=64, G=8, H=8, nq=8, prefix=16384, suffix=512, empties=False,
             paged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


MAX_ROPE = 4 * 8192 * 32          # rows of rope_q_prompt
MAX_APPEND = 4 * 8192 * 8         # token rows of append_prompt
MAX_SCORES = 64 * 8 * 8 * 8 * 16384
MAX_SUFFIX = 64 * 8 * 512         # own key rows of prefix_verify


def draw(rng):
    op = rng.choice(["rope", "append", "prefix"])
    if op == "prefix":
        B, H, G = _log(rng, 1, 128), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8])
        nq = rng.choice([1, 1, 2, 3, 5, 8])
        rows = B * G * H * nq
        prefix = _log(rng, 1, max(1, min(131072, MAX_SCORES // rows - 2048)))
        suffix = _log(rng, nq, max(nq, min(4096, MAX_SUFFIX // (B * H))))
        return dict(op=op, B=B, G=G, H=H, nq=nq, prefix=prefix, suffix=suffix, empties=rng.random() < 0.3,
                    paged=rng.random() < 0.5)
    H = rng.choice([1, 2, 4, 5, 8, 16] if op == "append" else [1, 2, 5, 8, 16, 32, 40, 64])
    most = MAX_APPEND if op == "append" else MAX_ROPE
    B = _log(rng, 1, 64)
    n = _log(rng, 1, min(8192, most // (B * H)))
    if rng.random() < 0.25:
        n = min(n, 8)
    case = dict(op=op, B=B, H=H, rotary=rng.choice([32, 64, 96, 128, 128]), adjacent=rng.random() < 0.3,
                axes=rng.choice([1, 1, 2, 3]), hadamard=rng.random() < 0.3)
    if op == "rope":
        return dict(case, T=n, pad=n > 8)
    return dict(case, n=n, ragged=rng.random() < 0.5, start=rng.choice([0, 31, 500, 2000]))


# --------------------------------------------------------------------------------------- packed formats

def _e2m1_codes(y):
    """E2M1 codes of y / 2^X already scaled: nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                       (5.0, False)):
        code += (a >= border) if up else (a > border)
    return code | (torch.signbit(y).to(torch.uint8) << 3)


def _shared_exponent(amax, emax):
    """floor(log2 amax) - emax, at least -127, from the exponent field of a 32-bit amax."""
    return ((amax.view(torch.int32) >> 23) - 127 - emax).clamp(-127, 127)


def _pow2(x):
    return torch.ldexp(torch.ones_like(x, dtype=torch.float32), x)


def _atoms(rows4):
    """[..., 128 rows, 4] bytes -> [..., 512]: row r, byte g at (r % 32) * 16 + (r / 32) * 4 + g."""
    s = rows4.shape[:-2]
    return rows4.reshape(*s, 4, 32, 4).transpose(-3, -2).reshape(*s, 512)


def _rows4(atoms):
    s = atoms.shape[:-1]
    return atoms.reshape(*s, 32, 4, 4).transpose(-3, -2).reshape(*s, 128, 4)


def _pack_rows(x):
    """MXFP4 of rows [..., 128] (float): packed codes [..., 64] and E8M0 bytes [..., 4]."""
    g = x.float().reshape(*x.shape[:-1], 4, 32)
    X = _shared_exponent(g.abs().amax(-1), 2)
    codes = _e2m1_codes(g * _pow2(-X).unsqueeze(-1)).reshape(*x.shape[:-1], 64, 2)
    return codes[..., 0] | (codes[..., 1] << 4), (X + 127).to(torch.uint8)


def _pack_groups(g):
    """MXFP8 of groups [..., 32] of V along the tokens: codes [..., 32] and E8M0 bytes [...]."""
    g = g.float()
    X = _shared_exponent(g.abs().amax(-1), 8)
    codes = (g * _pow2(-X).unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (X + 127).to(torch.uint8)


def _pack_qk(x, cap):
    """[B, T, H, 128] -> codes [B, H, cap, 64], scales [B, H, cap / 128, 512]; padding is zero."""
    B, T, H, _ = x.shape
    codes, scales = _pack_rows(x.transpose(1, 2))
    codes = torch.nn.functional.pad(codes, (0, 0, 0, cap - T))
    scales = torch.nn.functional.pad(scales, (0, 0, 0, cap - T))
    return codes, _atoms(scales.reshape(B, H, cap // 128, 128, 4))


def _pack_v(x, cap):
    """[B, T, H, 128] -> codes [B, H, cap / 128, 128, 128] (channel rows), scales [B, H, cap / 128, 512]."""
    B, T, H, _ = x.shape
    y = torch.nn.functional.pad(x.permute(0, 2, 3, 1), (0, cap - T)).reshape(B, H, D, cap // 128, 4, 32)
    codes, scales = _pack_groups(y.transpose(2, 3))
    return codes.reshape(B, H, cap // 128, D, 128), _atoms(scales)


def _unpack_rows(codes, scales4):
    """Values (32 bits) of MXFP4 rows: codes [..., 64], scale bytes [..., 4] -> [..., 128]."""
    both = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 4, 32)
    m = (both & 7).float()
    mag = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, m * 2 - 8))
    v = torch.where(both >= 8, -mag, mag) * _pow2(scales4.int() - 127).unsqueeze(-1)
    return v.reshape(*codes.shape[:-1], 128)


def _unpack_v(codes, atoms):
    """Values of MXFP8 V blocks: codes [..., 128 channels, 128 tokens], atoms [..., 512] -> the same shape."""
    s = _pow2(_rows4(atoms).int() - 127)
    v = codes.view(torch.float8_e4m3fn).float().reshape(*codes.shape[:-1], 4, 32)
    return (v * s.unsqueeze(-1)).reshape(codes.shape)


# ---------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _activations(g, B, T, H, outliers):
    """bf16 N(0, 1), with `outliers` channels of each head 16 times larger, as keys and queries have them."""
    x = torch.randn((B, T, H, D), generator=g, device="cuda", dtype=torch.float32)
    if outliers:
        at = torch.randint(0, D, (H, outliers), generator=g, device="cuda")
        x = x * torch.ones((H, D), device="cuda").scatter_(1, at, 16.0)
    return x.to(torch.bfloat16)


def _table(max_pos, rotary):
    """(cos, sin) of pos * 10000^(-2 i / rotary), taken in 64 bits, held in 32: [max_pos, rotary / 2, 2]."""
    i = torch.arange(rotary // 2, device="cuda", dtype=torch.float64)
    angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / rotary)
    return torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()


def _pair_axes(axes, pairs):
    """Axis of each pair: the first quarter of the pairs for axis 0, the others shared evenly (one axis: all)."""
    first = pairs if axes == 1 else pairs // 4
    return [0 if i < first else 1 + (i - first) * (axes - 1) // (pairs - first) for i in range(pairs)]


def _grid_positions(axes, T, base):
    """Positions of T tokens: text order for one axis; (time, row, column) of frames 40 tokens wide for more."""
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    if axes == 1:
        return base[None, :, None] + t
    kinds = torch.stack((t // 1600, (t % 1600) // 40, t % 40))[3 - axes:]
    return (base[None, :, None] + kinds[:, None, :]).contiguous()


def _rope_state(case, g, B, T, base):
    pairs = case["rotary"] // 2
    positions = _grid_positions(case["axes"], T, base).to(torch.int32)
    if case["op"] == "rope" and case["axes"] > 1:
        positions = positions[:, :1].expand(-1, B, -1)   # the same for every sequence, held once
    return dict(table=_table(int(base.max()) + T + 1, case["rotary"]), positions=positions,
                axis_list=_pair_axes(case["axes"], pairs),
                pair_axis=torch.tensor(_pair_axes(case["axes"], pairs), device="cuda"))


def _prepare_rope(case, g):
    B, T = case["B"], case["T"]
    base = torch.randint(0, 4000, (B,), generator=g, device="cuda", dtype=torch.int32)
    s = dict(case=case, x=_activations(g, B, T, case["H"], 4), cap=max(128, -(-T // 128) * 128),
             **_rope_state(case, g, B, T, base))
    if not case["pad"]:
        u8 = dict(dtype=torch.uint8, device="cuda")
        s["codes"] = torch.zeros((B, case["H"], s["cap"], 64), **u8)
        s["scales"] = torch.zeros((B, case["H"], s["cap"] // 128, 512), **u8)
    if own:
        import bit_quantized_attention_qk4v8_b200 as qk
        s["rope"] = qk.Rope(s["table"], adjacent=case["adjacent"], pair_axis=s["axis_list"])
        s["kept"] = None if case["pad"] else qk.MXFP4(s["codes"], s["scales"], B, case["H"], s["cap"], T)
    return s


def _prepare_append(case, g):
    B, n, H = case["B"], case["n"], case["H"]
    # Lengths such that a pass that is run again finds the staged rows that it reads as they were: single
    # tokens at any length, blocks inside one group of 32 tokens, longer pieces from a group's start.
    lens = torch.randint(case["start"] // 2, case["start"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens = lens - torch.where(lens % 32 + n > 32, lens % 32, 0)
    new = torch.full((B,), n, device="cuda", dtype=torch.int32)
    if case["ragged"]:
        new = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    pages = -(-(case["start"] + n) // PAGE)
    total = B * pages
    order = torch.randperm(total, generator=g, device="cuda").reshape(B, pages).to(torch.int32)
    u8 = dict(dtype=torch.uint8, device="cuda")
    # The plain form writes what is to be skipped to a page behind the pool.
    s = dict(case=case, k=_activations(g, B, n, H, 4), v=_activations(g, B, n, H, 0), lens=lens, new=new,
             block_table=order, k_codes=torch.zeros((total + 1, H, PAGE, 64), **u8),
             k_scales=torch.zeros((total + 1, H, 512), **u8), v_codes=torch.zeros((total + 1, H, D, PAGE), **u8),
             v_scales=torch.zeros((total + 1, H, 512), **u8),
             tail=_activations(g, B, 32, H, 0).transpose(1, 2).contiguous(),
             lens_out=torch.zeros((B,), dtype=torch.int32, device="cuda"),
             **_rope_state(case, g, B, n, lens))
    if own:
        import bit_quantized_attention_qk4v8_b200 as qk
        s["rope"] = qk.Rope(s["table"], adjacent=case["adjacent"], pair_axis=s["axis_list"])
        s["cache"] = qk.PagedKV(s["k_codes"][:-1], s["k_scales"][:-1], s["v_codes"][:-1], s["v_scales"][:-1],
                                s["tail"], order, lens, hadamard_k=case["hadamard"])
    return s


def _cap(n):
    return max(128, -(-n // 128) * 128)


def _prepare_prefix(case, g):
    B, H, G, nq, prefix, suffix = (case[k] for k in ("B", "H", "G", "nq", "prefix", "suffix"))
    q = _pack_qk(_activations(g, B, nq, H * G, 4), 128)
    lens = torch.randint(nq, suffix + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if case["empties"]:
        lens = lens * (torch.rand((B,), generator=g, device="cuda") < 0.7)
    lens = lens.to(torch.int32)
    kp, ksp = _pack_qk(_activations(g, 1, prefix, H, 4), _cap(prefix))
    vp, vsp = _pack_v(_activations(g, 1, prefix, H, 0), _cap(prefix))
    seen = (torch.arange(suffix, device="cuda")[None] < lens[:, None])[..., None, None]
    k, ks = _pack_qk(_activations(g, B, suffix, H, 4) * seen, _cap(suffix))
    v, vs = _pack_v(_activations(g, B, suffix, H, 0) * seen, _cap(suffix))
    s = dict(case=case, q=q[0], qs=q[1], lens=lens)
    if not case["paged"]:
        s.update(kp=kp, ksp=ksp, vp=vp, vsp=vsp, k=k, ks=ks, v=v, vs=vs)
    else:
        np_, ns = _cap(prefix) // 128, _cap(suffix) // 128
        order = torch.randperm(np_ + B * ns, generator=g, device="cuda")
        back = torch.argsort(order)

        def pool(a, b, block):  # [1, H, np, *block], [B, H, ns, *block] -> [pages, H, *block]
            a = a.reshape(H, np_, *block).transpose(0, 1)
            b = b.reshape(B, H, ns, *block).transpose(1, 2).reshape(B * ns, H, *block)
            return torch.cat((a, b))[back].contiguous()

        s.update(pk=pool(kp, k, (128, 64)), pks=pool(ksp, ks, (512,)), pv=pool(vp, v, (128, 128)),
                 pvs=pool(vsp, vs, (512,)), prefix_table=order[:np_].to(torch.int32),
                 block_table=order[np_:].reshape(B, ns).to(torch.int32).contiguous())
    if own:
        import bit_quantized_attention_qk4v8_b200 as qk
        s["packed_q"] = qk.MXFP4(s["q"].contiguous(), s["qs"].contiguous(), B, H * G, 128, nq)
        if case["paged"]:
            s["cache"] = qk.PagedKV(s["pk"], s["pks"], s["pv"], s["pvs"], None, s["block_table"], lens)
        else:
            # The packed buffers of a program are dense; the ones made above may be permuted views.
            kp, ksp, vp, vsp, k, ks, v, vs = (a.contiguous() for a in (kp, ksp, vp, vsp, k, ks, v, vs))
            s["prefix_kv"] = (qk.MXFP4(kp, ksp, 1, H, _cap(prefix), prefix), qk.MXFP8V(vp, vsp, 1, H, _cap(prefix), prefix))
            s["own_kv"] = (qk.MXFP4(k, ks, B, H, _cap(suffix), suffix), qk.MXFP8V(v, vs, B, H, _cap(suffix), suffix))
    return s


def prepare(case, seed):
    g = _gen(seed)
    return {"rope": _prepare_rope, "append": _prepare_append, "prefix": _prepare_prefix}[case["op"]](case, g)


# ---------------------------------------------------------------------------------------- plain forms

def _rotate(x, s, case):
    """bf16 [B, T, H, 128] -> the rotated rows in bf16, each value rounded once from 64 (by way of 32) bits."""
    R = case["rotary"]
    pos = s["positions"][s["pair_axis"]].permute(1, 2, 0).expand(x.shape[0], -1, -1).long()   # [B, T, pairs]
    cs = s["table"][pos, torch.arange(R // 2, device=x.device)].double()[:, :, None]
    c, sn = cs[..., 0], cs[..., 1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if case["adjacent"] else (x[..., :R // 2], x[..., R // 2:R])
    a, b = a.double(), b.double()
    ya, yb = (a * c - b * sn).float().bfloat16(), (b * c + a * sn).float().bfloat16()
    y = torch.stack((ya, yb), -1).flatten(-2) if case["adjacent"] else torch.cat((ya, yb), -1)
    y = torch.cat((y, x[..., R:]), -1)
    return _hadamard(y) if case["hadamard"] else y


def _hadamard(x):
    """Rows times the Sylvester matrix / sqrt(128), in 32 bits, butterflies of stride 1, 2, .. 64."""
    y = x.float()
    for stride in (1, 2, 4, 8, 16, 32, 64):
        p = y.reshape(*x.shape[:-1], 128 // (2 * stride), 2, stride)
        a, b = p[..., 0, :], p[..., 1, :]
        y = torch.stack((a + b, a - b), -2).reshape(x.shape)
    return y * torch.tensor(2.0 ** -3.5, dtype=torch.float32, device=x.device)


def _plain_rope(s):
    y = _rotate(s["x"], s, s["case"])
    if s["case"]["pad"]:
        return _pack_qk(y, s["cap"])
    codes, scales = _pack_rows(y.transpose(1, 2))
    t = torch.arange(y.shape[1], device=y.device)
    s["codes"][:, :, :y.shape[1]] = codes
    s["scales"].view(*s["scales"].shape[:3], 32, 4, 4)[:, :, t // 128, t % 32, t % 128 // 32] = scales
    return s["codes"], s["scales"]


def _plain_append(s):
    case = s["case"]
    B, n, H = case["B"], case["n"], case["H"]
    dev = s["k"].device
    L0, L1, skip = s["lens"].long()[:, None], (s["lens"] + s["new"]).long()[:, None], s["k_codes"].shape[0] - 1
    table = s["block_table"].long()

    def page_of(pos, wanted):
        at = (pos // PAGE).clamp(max=table.shape[1] - 1)
        return torch.where(wanted, table.gather(1, at), skip)

    # Keys: each row on its own.
    t = torch.arange(n, device=dev)[None]
    pos = L0 + t
    page, row = page_of(pos, pos < L1), pos % PAGE
    codes, scales = _pack_rows(_rotate(s["k"], s, case))
    s["k_codes"][page, :, row] = codes
    s["k_scales"].view(-1, H, 32, 4, 4)[page, :, row % 32, row // 32] = scales
    # Values: every group of 32 tokens that the new ones touch, whole.
    groups = (n + 31) // 32 + 1
    tg = (L0 // 32 * 32) + torch.arange(groups * 32, device=dev)[None]
    fresh = s["v"].transpose(1, 2).gather(2, (tg - L0).clamp(0, n - 1)[:, None, :, None].expand(B, H, -1, D))
    staged = s["tail"].gather(2, (tg % 32)[:, None, :, None].expand(B, H, -1, D))
    keep = lambda m: m[:, None, :, None]  # noqa: E731
    vals = torch.where(keep(tg < L0), staged, torch.where(keep(tg < L1), fresh, 0))
    codes, scales = _pack_groups(vals.reshape(B, H, groups, 32, D).transpose(-1, -2))   # [B, H, groups, 128, 32]
    first = tg[:, ::32]
    page, slot = page_of(first, (first < L1) & (L1 > L0)), first % PAGE // 32
    s["v_codes"].view(-1, H, D, 4, 32)[page, :, :, slot] = codes.transpose(1, 2)
    s["v_scales"].view(-1, H, 32, 4, 4)[page, :, :, :, slot] = scales.transpose(1, 2).reshape(
        B, groups, H, 4, 32).transpose(-1, -2)
    # The open group's values, staged for the next append.
    tt = (L1 // 32 * 32) + torch.arange(32, device=dev)[None]
    fresh = s["v"].transpose(1, 2).gather(2, (tt - L0).clamp(0, n - 1)[:, None, :, None].expand(B, H, -1, D))
    s["tail"].copy_(torch.where(keep((tt >= L0) & (tt < L1)), fresh, s["tail"]))
    s["lens_out"].copy_(s["lens"] + s["new"])
    return _append_outputs(s)


def _append_outputs(s):
    return dict(k_codes=s["k_codes"][:-1], k_scales=s["k_scales"][:-1].view(torch.float8_e8m0fnu),
                v_codes=s["v_codes"][:-1].view(torch.float8_e4m3fn),
                v_scales=s["v_scales"][:-1].view(torch.float8_e8m0fnu), tail=s["tail"], lens=s["lens_out"])


def _prefix_caches(s):
    """The prefix and own caches of a state as contiguous [B, H, blocks, ...] arrays."""
    if not s["case"]["paged"]:
        return tuple(s[k] for k in ("kp", "ksp", "vp", "vsp", "k", "ks", "v", "vs"))
    pt, bt = s["prefix_table"].long()[None], s["block_table"].long()
    flat = lambda c: c.reshape(c.shape[0], c.shape[1], -1, 64)  # noqa: E731
    got = [s[k][t].transpose(1, 2) for t in (pt, bt) for k in ("pk", "pks", "pv", "pvs")]
    got[0], got[4] = flat(got[0]), flat(got[4])
    return tuple(got)


def _plain_prefix(s):
    case = s["case"]
    B, H, G, nq, prefix = (case[k] for k in ("B", "H", "G", "nq", "prefix"))
    kp, ksp, vp, vsp, k, ks, v, vs = _prefix_caches(s)
    scale = 1.0 / math.sqrt(D)

    def rows(c, a):
        return _unpack_rows(c, _rows4(a).reshape(*c.shape[:-1], 4))

    def channels(c, a):  # [B, H, 128, tokens]
        return _unpack_v(c, a).transpose(2, 3).flatten(3)

    q = _unpack_rows(s["q"][:, :, :nq], _rows4(s["qs"])[:, :, 0, :nq])
    q = q.reshape(B, H, G * nq, D) * scale
    # Scores against the prefix, all sequences' rows of a KV head at once, and against the own keys.
    qa = q.transpose(0, 1).reshape(H, B * G * nq, D)
    sp = qa @ rows(kp, ksp)[0, :, :prefix].transpose(1, 2)
    so = q @ rows(k, ks).transpose(2, 3)
    t = torch.arange(G * nq, device=q.device) % nq
    bound = s["lens"].long()[:, None] - nq + t[None] + 1
    cols = torch.arange(so.shape[-1], device=q.device)
    so = so.masked_fill(cols >= bound[:, None, :, None], -math.inf)
    mp = sp.amax(-1, keepdim=True).reshape(H, B, G * nq, 1).transpose(0, 1)
    m = torch.maximum(mp, so.amax(-1, keepdim=True))
    pp = (sp - m.transpose(0, 1).reshape(H, B * G * nq, 1)).exp_()
    po = (so - m).exp_()
    den = pp.sum(-1, keepdim=True).reshape(H, B, G * nq, 1).transpose(0, 1) + po.sum(-1, keepdim=True)
    num = (pp @ channels(vp, vsp)[0, :, :, :prefix].transpose(1, 2)).reshape(H, B, G * nq, D).transpose(0, 1)
    num = num + po @ channels(v, vs).transpose(2, 3)
    out = (num / den).reshape(B, H * G, nq, D).transpose(1, 2)
    return out.to(torch.bfloat16).contiguous()


# --------------------------------------------------------------------------------------- own operators

def _own_rope(s):
    import bit_quantized_attention_qk4v8_b200 as qk
    p = qk.quantize_qk_rope(s["x"], s["rope"], positions=s["positions"], hadamard=s["case"]["hadamard"],
                            out=s["kept"], pad=s["case"]["pad"])
    return p.codes, p.scales


def _own_append(s):
    import bit_quantized_attention_qk4v8_b200 as qk
    qk.kv_append_rope(s["cache"], s["k"], s["v"], s["rope"], positions=s["positions"], new_lens=s["new"],
                      seqlens_out=s["lens_out"])
    return _append_outputs(s)


def _own_prefix(s):
    import bit_quantized_attention_qk4v8_b200 as qk
    case = s["case"]
    if case["paged"]:
        return qk.attention_decode_prefix_paged(s["packed_q"], s["cache"], s["prefix_table"], case["prefix"],
                                                max_seqlen=case["suffix"])
    return qk.attention_decode_prefix(s["packed_q"], *s["prefix_kv"], *s["own_kv"], s["lens"],
                                      max_seqlen=case["suffix"])


def run(state):
    op = state["case"]["op"]
    if own:
        got = {"rope": _own_rope, "append": _own_append, "prefix": _own_prefix}[op](state)
    else:
        got = {"rope": _plain_rope, "append": _plain_append, "prefix": _plain_prefix}[op](state)
    return (got[0], got[1].view(torch.float8_e8m0fnu)) if op == "rope" else got


# ------------------------------------------------------------------------------------------------ work

def work(case):
    if case["op"] == "rope":
        rows = case["B"] * case["T"] * case["H"]
        tokens = case["B"] * case["T"]
        written = max(128, -(-case["T"] // 128) * 128) * case["B"] * case["H"] if case["pad"] else rows
        return dict(bytes=256 * rows + 68 * written + tokens * (4 * case["axes"] + 4 * case["rotary"]),
                    flops=rows * (3 * case["rotary"] + 4 * D + (7 * D if case["hadamard"] else 0)))
    if case["op"] == "append":
        mean = case["n"] / 2 if case["ragged"] else case["n"]
        rows = case["B"] * mean * case["H"]
        # The open group: about half of it staged before, its codes written whole, its new rows staged.
        tail = case["B"] * case["H"] * (min(1.0, mean) * (16 * 256 * (case["start"] > 0) + 16 * D) + min(mean, 16) * 256)
        return dict(bytes=512 * rows + 200 * rows + tail + case["B"] * mean * (4 * case["axes"] + 4 * case["rotary"]),
                    flops=rows * (3 * case["rotary"] + 8 * D + (7 * D if case["hadamard"] else 0)))
    rows = case["B"] * case["G"] * case["H"] * case["nq"]
    mean = (case["nq"] + case["suffix"]) / 2 * (0.7 if case["empties"] else 1.0)
    return dict(bytes=(68 + 256) * rows + 200 * case["H"] * (case["prefix"] + case["B"] * mean),
                flops=4 * D * rows * (case["prefix"] + mean))


# ----------------------------------------------------------------------------------------------- exact

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _byte_of(r, g):
    return (r % 32) * 16 + (r // 32) * 4 + g


def _turn(rows, positions, s, case):
    """Rows [T, H, 128] of one sequence at positions [axes, T], rotated in 64 bits pair by pair, rounded to bf16."""
    R = case["rotary"]
    y = rows.double().clone()
    for i, axis in enumerate(s["axis_list"]):
        a, b = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + R // 2)
        cs = s["table"][positions[axis].long(), i].double()
        z = torch.complex(rows[..., a].double(), rows[..., b].double()) * torch.complex(cs[:, 0], cs[:, 1])[:, None]
        y[..., a], y[..., b] = z.real, z.imag
    y = y.float().bfloat16().double()
    if case["hadamard"]:
        i = torch.arange(128, device=y.device)
        bits = i[:, None] & i[None]
        parity = sum((bits >> k) & 1 for k in range(7)) % 2
        y = y @ ((1.0 - 2.0 * parity.double()) / math.sqrt(128.0))
    return y


def _block_scale(x, emax):
    """2^X of groups [..., 32] in 64 bits; 2^-127 for an empty one."""
    top = x.abs().amax(-1)
    _, e = torch.frexp(top)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), (e - 1 - emax).clamp(-127, 127)),
                       torch.full_like(top, 2.0 ** -127))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        B, T, H = case["B"], case["T"], case["H"]
        scales = torch.full((B, H, s["cap"] // 128, 512), 2.0 ** -127, dtype=torch.float64, device="cuda")
        t = torch.arange(T, device="cuda")
        for b in range(B):
            y = _turn(s["x"][b], s["positions"][:, b], s, case)
            for g in range(4):
                scales[b, :, t // 128, _byte_of(t % 128, g)] = _block_scale(y[..., 32 * g:32 * g + 32], 2).T
        return None, scales
    if case["op"] == "append":
        return _exact_append(case, s)
    return _exact_prefix(case, s)


def _exact_append(case, s):
    B, H = case["B"], case["H"]
    P = s["k_codes"].shape[0] - 1
    f64 = dict(dtype=torch.float64, device="cuda")
    ks, vs = torch.full((P, H, 512), 2.0 ** -127, **f64), torch.full((P, H, 512), 2.0 ** -127, **f64)
    vc = torch.zeros((P, H, D, PAGE), **f64)
    tail = s["tail"].double()
    lens, new, bt = s["lens"].tolist(), s["new"].tolist(), s["block_table"].tolist()
    c = torch.arange(D, device="cuda")
    for b in range(B):
        L0, L1 = lens[b], lens[b] + new[b]
        if L1 == L0:
            continue
        y = _turn(s["k"][b, :new[b]], s["positions"][:, b, :new[b]], s, case)
        v = s["v"][b, :new[b]].double()
        for p in range(L0 // PAGE, (L1 + PAGE - 1) // PAGE):
            lo, hi = max(L0, p * PAGE), min(L1, (p + 1) * PAGE)
            r = torch.arange(lo, hi, device="cuda") % PAGE
            for g in range(4):
                ks[bt[b][p], :, _byte_of(r, g)] = _block_scale(y[lo - L0:hi - L0, :, 32 * g:32 * g + 32], 2).T
        for first in range(L0 // 32 * 32, L1, 32):
            group = torch.zeros((H, D, 32), **f64)
            if first < L0:
                group[:, :, :L0 - first] = s["tail"][b, :, :L0 - first].double().transpose(1, 2)
            lo, hi = max(first, L0), min(first + 32, L1)
            group[:, :, lo - first:hi - first] = v[lo - L0:hi - L0].permute(1, 2, 0)
            scale = _block_scale(group, 8)
            page, slot = bt[b][first // PAGE], first % PAGE // 32
            vs[page, :, _byte_of(c, slot)] = scale
            vc[page, :, :, slot * 32:slot * 32 + 32] = (group / scale[..., None]).clamp(-448, 448)
        for t in range(max(L0, L1 // 32 * 32), L1):
            tail[b, :, t % 32] = v[t - L0]
    return dict(k_codes=None, k_scales=ks, v_codes=vc, v_scales=vs, tail=tail, lens=None)


def _exact_prefix(case, s):
    B, H, G, nq, prefix = (case[k] for k in ("B", "H", "G", "nq", "prefix"))
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    r, gq = torch.arange(128, device="cuda")[:, None], torch.arange(4, device="cuda")[None]
    at = _byte_of(r, gq)

    def power(byte):
        return torch.pow(2.0, byte.double() - 127)

    def keys(codes, atoms, n):  # [blocks * 128, 64], [blocks, 512] -> [n, 128]
        c = codes.reshape(-1, 64)[:n].long()
        v = torch.stack((grid[c & 15], grid[c >> 4]), -1).reshape(n, 4, 32)
        return (v * power(atoms[:, at].reshape(-1, 4)[:n])[..., None]).reshape(n, 128)

    def values(codes, atoms, n):  # [blocks, 128, 128], [blocks, 512] -> [n, 128]
        v = codes.view(torch.float8_e4m3fn).double().reshape(-1, 128, 4, 32) * power(atoms[:, at])[..., None]
        return v.reshape(-1, 128, 128).transpose(1, 2).reshape(-1, 128)[:n]

    lens = s["lens"].tolist()
    paged = case["paged"]
    out = torch.empty((B, nq, H * G, D), dtype=torch.float64, device="cuda")
    for h in range(H):
        if paged:
            pt = s["prefix_table"].long()
            kp, vp = keys(s["pk"][pt, h], s["pks"][pt, h], prefix), values(s["pv"][pt, h], s["pvs"][pt, h], prefix)
        else:
            kp, vp = keys(s["kp"][0, h], s["ksp"][0, h], prefix), values(s["vp"][0, h], s["vsp"][0, h], prefix)
        for b in range(B):
            L = lens[b]
            if paged:
                bt = s["block_table"][b].long()
                ko, vo = keys(s["pk"][bt, h], s["pks"][bt, h], L), values(s["pv"][bt, h], s["pvs"][bt, h], L)
            else:
                ko, vo = keys(s["k"][b, h], s["ks"][b, h], L), values(s["v"][b, h], s["vs"][b, h], L)
            q = torch.stack([keys(s["q"][b, h * G + i], s["qs"][b, h * G + i], nq) for i in range(G)])  # [G, nq, 128]
            sees = torch.arange(prefix + L, device="cuda")[None] < (
                prefix + (L - nq + 1 + torch.arange(nq, device="cuda")).clamp(min=0))[:, None]
            w = q @ torch.cat((kp, ko)).T / math.sqrt(D)
            w = torch.softmax(w.masked_fill(~sees, -math.inf), -1)
            out[b, :, h * G:(h + 1) * G] = (w @ torch.cat((vp, vo))).transpose(0, 1)
    return out
