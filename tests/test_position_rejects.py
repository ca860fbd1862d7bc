"""Refusals of the rotating quantizer and append and of shared-prefix decode, without a GPU: every bad argument is
named before any device work, and the workspace's size follows from the sizes."""
import ctypes

import pytest

from bit_quantized_attention_qk4v8_b200 import _lib
from bit_quantized_attention_qk4v8_b200 import build as qkbuild

FAKE = 0x10000  # never dereferenced: the calls are refused first
INVALID = 1


@pytest.fixture(scope="module")
def lib():
    qkbuild.build()
    return _lib.lib()


def rope_struct(axes=None, **kw):
    f = dict(table=FAKE, max_pos=100, rotary_dim=128, adjacent=0, n_axes=1, pair_axis=None, positions=None,
             pos_stride_axis=0, pos_stride_b=0, pos_stride_t=1)
    f.update(kw)
    if axes is not None:
        f["pair_axis"] = ctypes.addressof(axes)
    return _lib.RopeStruct(*f.values())


def quantize(lib, rope=None, **kw):
    a = dict(x=FAKE, B=1, S=10, H=2, d=128, sb=2560, ss=256, sh=128, sl=None, start=None, rope=rope or rope_struct(),
             hadamard=0, cap=128, pad=1, codes=FAKE, scales=FAKE, status=None, stream=None)
    a.update(kw)
    a["rope"] = None if a["rope"] == "none" else ctypes.addressof(a["rope"])
    return lib.qk4v8_quantize_qk_rope(*a.values())


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(codes=None), dict(scales=None), dict(rope="none"), dict(B=0), dict(S=-1), dict(H=0), dict(d=64),
    dict(cap=100), dict(cap=0), dict(S=129), dict(sb=2561), dict(ss=252), dict(sh=-128), dict(x=FAKE + 2),
    dict(codes=FAKE + 8), dict(scales=FAKE + 4)])
def test_quantize_refuses(lib, kw):
    assert quantize(lib, **kw) == INVALID
    assert lib.qk4v8_last_error()


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(table=FAKE + 4), dict(max_pos=0), dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=120),
    dict(rotary_dim=144), dict(n_axes=0), dict(n_axes=5), dict(positions=FAKE, pos_stride_t=-1),
    dict(positions=FAKE, pos_stride_b=-8), dict(positions=FAKE, pos_stride_axis=-1)])
def test_rope_refuses(lib, kw):
    assert quantize(lib, rope=rope_struct(**kw)) == INVALID
    assert append(lib, rope=rope_struct(**kw)) == INVALID


def test_pair_on_an_axis_that_is_not_there(lib):
    axes = (ctypes.c_uint8 * 64)(*([0] * 63 + [2]))
    assert quantize(lib, rope=rope_struct(axes, n_axes=2, positions=FAKE)) == INVALID
    assert b"axis 2" in lib.qk4v8_last_error()


def append(lib, rope=None, **kw):
    s3 = ctypes.c_int64 * 3
    ks, vs = s3(*kw.pop("ks", (2560, 256, 128))), s3(*kw.pop("vs", (2560, 256, 128)))
    a = dict(k=FAKE, v=FAKE, B=1, n=10, H=2, d=128, ks=ctypes.addressof(ks), vs=ctypes.addressof(vs), lens=FAKE, new=None,
             out=FAKE, rope=rope or rope_struct(), table=FAKE, max_pages=4, num_pages=8, kc=FAKE, ksc=FAKE, vc=FAKE,
             vsc=FAKE, tail=FAKE, hadamard=0, status=None, stream=None)
    a.update(kw)
    a["rope"] = None if a["rope"] == "none" else ctypes.addressof(a["rope"])
    return lib.qk4v8_kv_append_rope(*a.values())


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(lens=None), dict(table=None), dict(kc=None), dict(ksc=None), dict(vc=None),
    dict(vsc=None), dict(tail=None), dict(rope="none"), dict(B=0), dict(n=0), dict(n=1 << 30), dict(H=0), dict(d=96),
    dict(max_pages=0), dict(max_pages=1 << 23), dict(num_pages=0), dict(num_pages=1 << 30), dict(ks=(2560, 256, 4)),
    dict(vs=(2560, -256, 128)), dict(k=FAKE + 2), dict(v=FAKE + 8), dict(kc=FAKE + 1), dict(tail=FAKE + 4),
    dict(vsc=FAKE + 8)])
def test_append_refuses(lib, kw):
    assert append(lib, **kw) == INVALID


def prefix(lib, **kw):
    a = dict(qc=FAKE, qs=FAKE, B=2, Hq=8, nq=1, q_cap=128, pkc=FAKE, pks=FAKE, pvc=FAKE, pvs=FAKE, plen=300, pcap=384,
             kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, Hkv=2, cap=256, lens=FAKE, most=200, causal=1, scale=0.0, ws=FAKE,
             wsb=1 << 40, out=FAKE, lse=None, status=None, stream=None)
    a.update(kw)
    return lib.qk4v8_attention_decode_prefix(*a.values())


@pytest.mark.parametrize("kw", [
    dict(qc=None), dict(qs=None), dict(pkc=None), dict(pvs=None), dict(kc=None), dict(vs=None), dict(lens=None),
    dict(out=None), dict(ws=None), dict(wsb=16), dict(B=0), dict(Hq=7), dict(Hkv=0), dict(nq=0), dict(nq=9),
    dict(Hq=64, Hkv=1, nq=4), dict(q_cap=100), dict(plen=-1), dict(plen=400), dict(pcap=300), dict(most=-1), dict(most=257),
    dict(cap=200), dict(qc=FAKE + 4), dict(pvc=FAKE + 8), dict(ws=FAKE + 8), dict(out=FAKE + 2), dict(B=1 << 28)])
def test_prefix_refuses(lib, kw):
    assert prefix(lib, **kw) == INVALID
    assert lib.qk4v8_last_error()


def paged(lib, **kw):
    a = dict(qc=FAKE, qs=FAKE, B=2, Hq=8, nq=1, q_cap=128, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, Hkv=2, pages=64, ptab=FAKE,
             plen=300, table=FAKE, max_pages=4, lens=FAKE, most=200, causal=1, scale=0.0, ws=FAKE, wsb=1 << 40, out=FAKE,
             lse=None, status=None, stream=None)
    a.update(kw)
    return lib.qk4v8_attention_decode_prefix_paged(*a.values())


@pytest.mark.parametrize("kw", [
    dict(ptab=None), dict(table=None), dict(max_pages=0), dict(max_pages=1 << 24), dict(pages=0), dict(pages=1 << 30),
    dict(most=513), dict(lens=None), dict(Hkv=0), dict(wsb=0), dict(plen=2**31 - 1)])
def test_paged_prefix_refuses(lib, kw):
    assert paged(lib, **kw) == INVALID


def test_workspace_size(lib):
    """Partial results of 128 rows (fp32 O, and a log-sum-exp each) for every unit (128 rows of a KV head) and share (148
    SMs without a device; no more than tiles), and two ints a unit, each array rounded up to 16 bytes."""
    size = lib.qk4v8_decode_prefix_workspace_bytes

    def want(units, shares):
        slots = units + shares if shares else 0
        return slots * 128 * 129 * 4 + 2 * ((units * 4 + 15) // 16 * 16)

    assert size(64, 64, 8, 8, 16384, 512) == want(32 * 8, 148)
    assert size(2, 8, 2, 1, 300, 0) == want(2, 3 * 2 + 2)            # 8 rows of each KV head: one row tile
    assert size(1, 1, 1, 1, 0, 1) == want(1, 2 + 1)                  # (a sequence may touch two row tiles)
    assert size(3, 4, 4, 2, 0, 0) == want(4, 0)
    for bad in ((0, 8, 2, 1, 1, 1), (1, 7, 2, 1, 1, 1), (1, 8, 2, 9, 1, 1), (1, 8, 2, 1, -1, 1), (1, 256, 1, 1, 1, 1),
                (1 << 20, 8, 8, 1, 2**31 - 1, 0)):
        assert size(*bad) == 0


@pytest.mark.parametrize("kw", [
    dict(out=FAKE + 4, lens=FAKE, B=2), dict(out=FAKE, lens=FAKE + 4, B=2), dict(out=FAKE + 64, new=FAKE + 64),
    dict(out=FAKE + 64, new=FAKE + 68, B=2), dict(out=FAKE, lens=FAKE, new=FAKE + 4, B=2)])
def test_lengths_that_would_be_read_and_written_at_once(lib, kw):
    """seqlens_out over a part of seqlens, or over new_lens: other blocks still read those while they are written."""
    assert append(lib, **kw) == INVALID
    assert b"seqlens_out" in lib.qk4v8_last_error()
