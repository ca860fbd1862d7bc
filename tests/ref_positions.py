"""Plain numpy forms, in 64 bits, of the rotating quantizers and of attention over a shared prefix (test code only)."""
import numpy as np

import oracle

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
E4M3 = np.array([oracle.decode(oracle.E4M3, c) for c in range(256)])


def bf16_to_f64(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f32_to_bf16(x):
    """To nearest, ties to even, of finite values (no overflow)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def rotate(bits, table, positions, axis=None, adjacent=False):
    """bf16 bits [B, T, H, 128] rotated: table f32 [max_pos, R/2, 2], positions int [axes, B, T], axis [R/2]."""
    half = table.shape[1]
    axis = np.zeros(half, int) if axis is None else np.asarray(axis)
    x = bf16_to_f64(bits)
    out = bits.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        cs = table[positions[axis[i]], i].astype(np.float64)[:, :, None]  # [B, T, 1, 2]
        c, s = cs[..., 0], cs[..., 1]
        out[..., a] = f32_to_bf16((x[..., a] * c - x[..., b] * s).astype(np.float32))
        out[..., b] = f32_to_bf16((x[..., b] * c + x[..., a] * s).astype(np.float32))
    return out


def angles(max_pos, rotary, base=10000.0):
    a = np.arange(max_pos)[:, None] * base ** (-2.0 * np.arange(rotary // 2) / rotary)
    return np.stack((np.cos(a), np.sin(a)), -1).astype(np.float32)


def dequantize_qk(bits):
    """bf16 bits [B, T, H, 128] -> what MXFP4 holds of them, f64 [B, H, T, 128]."""
    c, s = oracle.quantize_qk(bits)
    return E2M1[c] * np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, -1)


def dequantize_v(bits):
    """bf16 bits [B, T, H, 128] -> what MXFP8 holds of them, f64 [B, H, T, 128]."""
    T = bits.shape[1]
    c, s = oracle.quantize_v(bits, np.full((bits.shape[0],), T, np.int32))
    scale = np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, -1)[..., :T]
    return np.swapaxes(E4M3[c[..., :T]] * scale, 2, 3)


def attention_row(q, k, v, scale):
    """q f64 [n, 128], k, v f64 [m, 128] -> out [n, 128], natural log-sum-exp [n], and the bound on the kernel's error.

    The kernel's departures from this, relative to a row's weights p / sum p: each p is rounded to bf16 in the
    numerator and the denominator alike (at most 2^-8), its exponent has an error e of a few fp32 units in the last
    place of the row's largest score magnitude A (the product's sum, the scaling, the offset: 8 * 2^-24 * A each way),
    ex2.approx is within 2^-22. Together (w) they move the mean of v by at most w * sum p |v - out| / sum p to first
    order; w < 1/100, so (1 + 4 w) covers the rest. The output is rounded to bf16 (2^-8 of its value)."""
    s = (q @ k.T) * scale
    mag = (np.abs(q) @ np.abs(k).T).max(1) * scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    o = p @ v / l
    spread = np.stack([p[i] @ np.abs(v - o[i]) / l[i, 0] for i in range(len(q))])
    w = 2.0 ** -8 + 2.0 ** -22 + 16 * 2.0 ** -24 * mag[:, None]
    moved = w * (1 + 4 * w) * spread
    return o, (m + np.log(l))[:, 0], moved + 2.0 ** -8 * (np.abs(o) + moved) + 1e-37, (w * (1 + 4 * w))[:, 0]


def prefix_attention(q, pk, pv, ks, vs, causal=True, scale=None):
    """q f64 [B, Hq, nq, 128]; pk, pv f64 [Hkv, prefix, 128]; ks, vs: a list of the sequences' own [Hkv, len, 128].

    Returns out [B, nq, Hq, 128], lse [B, Hq, nq] and the bounds on their errors."""
    B, Hq, nq, _ = q.shape
    Hkv = pk.shape[0]
    scale = 128 ** -0.5 if scale is None else scale
    out = np.zeros((B, nq, Hq, 128))
    tol = np.full((B, nq, Hq, 128), 1e-37)
    lse = np.full((B, Hq, nq), -np.inf)
    ltol = np.zeros((B, Hq, nq))
    for b in range(B):
        n = ks[b].shape[1]
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            for t in range(nq):
                own = max(0, n - nq + t + 1) if causal else n
                k = np.concatenate((pk[kv], ks[b][kv, :own]))
                v = np.concatenate((pv[kv], vs[b][kv, :own]))
                if len(k):
                    o, s, e, w = attention_row(q[b, h, t:t + 1], k, v, scale)
                    out[b, t, h], lse[b, h, t], tol[b, t, h], ltol[b, h, t] = o[0], s[0], e[0], w[0] + 1e-5 + 1e-6 * abs(s[0])
    return out, lse, tol, ltol
