"""Buffers of another type, size, device or layout than a call reads and writes are refused before it. Without a GPU: the
tensors are fake ones, which have all of that but no memory, and a stand-in for the library notes what would be called."""
import contextlib
import warnings

import pytest
import torch
from torch._subclasses import FakeTensorMode

import bit_quantized_attention_qk4v8_b200 as qk

B, H, HQ, P, MAX, CAP, N = 3, 2, 4, 10, 2, 256, 5


@pytest.fixture
def calls(monkeypatch):
    """Names of the library's functions that were called."""
    got = []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                got.append(name)
                return 1 << 20 if name.endswith("workspace_bytes") else 0
            return call
    monkeypatch.setattr(qk, "lib", Library)
    monkeypatch.setattr(qk, "_on", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(qk, "_stream", lambda device: 0)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")   # a fake tensor's address is 0
        yield got


def u8(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda:0")


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda:0")


def bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda:0")


def cache():
    return qk.PagedKV(u8(P, H, 128, 64), u8(P, H, 512), u8(P, H, 128, 128), u8(P, H, 512), bf16(B, H, 32, 128), i32(B, MAX),
                      i32(B))


def packed(b=B, h=H, length=200):
    return qk.MXFP4(u8(b, h, CAP, 64), u8(b, h, CAP // 128, 512), b, h, CAP, length)


def packed_v(b=B):
    return qk.MXFP8V(u8(b, H, CAP // 128, 128, 128), u8(b, H, CAP // 128, 512), b, H, CAP, 200)


def rope():
    return qk.Rope(torch.empty((300, 64, 2), dtype=torch.float32, device="cuda:0"))


def append(c, **kw):
    return qk.kv_append_rope(c, bf16(B, N, H, 128), bf16(B, N, H, 128), rope(), **kw)


def attend_paged(c, q=None, **kw):
    return qk.attention_decode_prefix_paged(q or packed(h=HQ, length=1), c, i32(2), 200, max_seqlen=200, **kw)


def attend(q=None, pk=None, pv=None, k=None, v=None, **kw):
    return qk.attention_decode_prefix(q or packed(h=HQ, length=1), pk or packed(1), pv or packed_v(1), k or packed(),
                                      v or packed_v(), i32(B), **kw)


def rotate(**kw):
    return qk.quantize_qk_rope(bf16(B, N, H, 128), rope(), **kw)


def change(x, field, f):
    setattr(x, field, f(getattr(x, field)))
    return x


WRONG = {
    "int64": lambda t: t.long(), "half the rows": lambda t: t[: t.shape[0] // 2], "a row more": lambda t: torch.cat((t, t[:1])),
    "every second": lambda t: torch.cat((t, t), -1)[..., ::2],
    "host": lambda t: torch.empty(t.shape, dtype=t.dtype),
}


def test_what_fits_is_called(calls):
    append(cache())
    append(cache(), dev_status=i32(1))
    attend_paged(cache(), dev_status=i32(1))
    c = cache()
    c.v_tail = None          # attention reads none
    attend_paged(c)
    attend()
    rotate(out=packed(), dev_status=i32(1))
    rotate()
    assert [n for n in calls if not n.endswith("bytes")] == [
        "qk4v8_kv_append_rope"] * 2 + ["qk4v8_attention_decode_prefix_paged"] * 2 + ["qk4v8_attention_decode_prefix"] + [
        "qk4v8_quantize_qk_rope"] * 2


def refused(calls, f, *args, **kw):
    before = len(calls)
    with pytest.raises(ValueError):
        f(*args, **kw)
    assert [n for n in calls[before:] if not n.endswith("bytes")] == []


@pytest.mark.parametrize("wrong", WRONG)
@pytest.mark.parametrize("field", ["k_codes", "k_scales", "v_codes", "v_scales", "v_tail", "block_table", "seqlens"])
def test_cache(calls, field, wrong):
    refused(calls, append, change(cache(), field, WRONG[wrong]))
    if field != "v_tail":
        refused(calls, attend_paged, change(cache(), field, WRONG[wrong]))


def test_arrays_without_their_axes(calls):
    for field in ("k_codes", "block_table"):
        for f in (append, attend_paged):
            refused(calls, f, change(cache(), field, lambda t: t.reshape(-1)))


def test_append_without_a_tail(calls):
    refused(calls, append, change(cache(), "v_tail", lambda _: None))


@pytest.mark.parametrize("wrong", WRONG)
@pytest.mark.parametrize("field", ["codes", "scales"])
def test_packed(calls, field, wrong):
    f = WRONG[wrong]
    refused(calls, rotate, out=change(packed(), field, f))
    refused(calls, attend_paged, cache(), q=change(packed(h=HQ, length=1), field, f))
    refused(calls, attend, q=change(packed(h=HQ, length=1), field, f))
    for name, make in (("pk", lambda: packed(1)), ("pv", lambda: packed_v(1)), ("k", packed), ("v", packed_v)):
        refused(calls, attend, **{name: change(make(), field, f)})


@pytest.mark.parametrize("field,value", [("cap", 384), ("H", 1), ("B", 2)])
def test_numbers_that_are_not_the_buffers(calls, field, value):
    for f, kw in ((attend, dict(k=change(packed(), field, lambda _: value), v=change(packed_v(), field, lambda _: value))),
                  (attend, dict(q=change(packed(h=HQ, length=1), field, lambda _: value))),
                  (rotate, dict(out=change(packed(), field, lambda _: value)))):
        refused(calls, f, **kw)


@pytest.mark.parametrize("status", ["host", "float", "empty"])
def test_status(calls, status):
    s = {"host": lambda: torch.zeros(1, dtype=torch.int32), "float": lambda: i32(1).float(), "empty": lambda: i32(0)}[status]()
    refused(calls, append, cache(), dev_status=s)
    refused(calls, attend_paged, cache(), dev_status=s)
    refused(calls, attend, dev_status=s)
    refused(calls, rotate, dev_status=s)


def test_a_rope_that_is_changed_later(calls):
    """The table and the pairs' axes are checked against each other whenever one is set, as at first: the library reads an
    axis for each pair of the table."""
    f32 = lambda *s: torch.empty(s, dtype=torch.float32, device="cuda:0")
    r = qk.Rope(f32(300, 32, 2), pair_axis=[0] * 16 + [1] * 16)
    for name, value in (("table", f32(300, 64, 2)), ("table", f32(300, 32, 2).double()), ("table", torch.empty(300, 32, 2)),
                        ("table", f32(32, 300, 2).transpose(0, 1)), ("pair_axis", [0] * 31), ("pair_axis", [4] * 32)):
        old = getattr(r, name)
        with pytest.raises(ValueError):
            setattr(r, name, value)
        assert getattr(r, name) is old and r.n_axes == 2 and r.rotary_dim == 64
    r.pair_axis = None
    assert r.n_axes == 1
    r.table = f32(500, 64, 2)
    r.pair_axis = [2] * 64
    assert r.n_axes == 3 and r.rotary_dim == 128
    rotate_by = lambda: qk.quantize_qk_rope(bf16(B, N, H, 128), r, positions=i32(3, B, N))
    rotate_by()
    r.pair_axis = [3] * 64
    refused(calls, rotate_by)      # positions on three axes
