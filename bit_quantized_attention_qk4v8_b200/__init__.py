"""QK4V8 mixed-precision attention for B200 (sm_100a).

This is the Python binding of libqk4v8.so. It marshals arguments only: torch
provides device memory and the current stream, and every step of the
computation runs in the library's CUDA kernels. Function names follow the C
entry points in include/qk4v8.h.

Method (MpFA QK4V8 article, mhpn.cn):
  - Q and K are quantized to MXFP4 and V to MXFP8-E4M3, with one E8M0 scale
    per 32 values computed online.
  - Attention then runs tile by tile with an FP32 online softmax, on
    block-scaled tcgen05 tensor-core MMAs.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from dataclasses import dataclass, field
from typing import Optional, Sequence

import torch

from ._lib import QK4V8Error, RopeStruct, check, lib

__all__ = [
    "MXFP4", "MXFP4V", "MXFP8V", "PagedKV", "QK4V8Error", "lib", "round_cap",
    "quantize_qk", "quantize_v", "quantize", "attention_prefill", "attention_decode",
    "decode_workspace_bytes", "decode_default_splits", "decode_plan_splits", "attention_decode_splitkv",
    "decode_merge",
    "attention_decode_bf16", "decode_bf16_workspace_bytes",
    "paged_kv", "kv_append", "attention_decode_paged", "attention_decode_bf16_paged", "quantize_v4",
    "Rope", "rope_table", "quantize_qk_rope", "kv_append_rope",
    "attention_decode_prefix", "attention_decode_prefix_paged", "decode_prefix_workspace_bytes",
]

D = 128


def round_cap(n: int) -> int:
    """Smallest multiple of 128 that holds n tokens (at least 128)."""
    return max(128, (int(n) + 127) // 128 * 128)


@dataclass
class MXFP4:
    """Packed MXFP4 tensor (Q or K): codes uint8 [B][H][cap][64], scales uint8 [B][H][cap/128][512]."""
    codes: torch.Tensor
    scales: torch.Tensor
    B: int
    H: int
    cap: int
    length: int


@dataclass
class MXFP4V:
    """Packed MXFP4 V (the QK4V4 comparison point): codes uint8 [B][H][cap/128][128][64]
    (128-token blocks of channel rows, two tokens per byte), scales uint8 [B][H][cap/128][512]."""
    codes: torch.Tensor
    scales: torch.Tensor
    B: int
    H: int
    cap: int
    length: int


@dataclass
class MXFP8V:
    """Packed MXFP8-E4M3 V: codes uint8 [B][H][cap/128][128][128] (128-token blocks of
    channel rows), scales uint8 [B][H][cap/128][512]."""
    codes: torch.Tensor
    scales: torch.Tensor
    B: int
    H: int
    cap: int
    length: int


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    """The current stream's handle (without a Stream object around it: 2 us of host time)."""
    if device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


_HERE = contextlib.nullcontext()


def _on(device):
    """The device as the current one; no switch (1.5 us of host time) when it is that already."""
    return _HERE if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)


def _check_bf16(x: torch.Tensor, name: str):
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 4 or x.shape[-1] != D or x.stride(-1) != 1:
        raise ValueError(f"{name} must be a CUDA bf16 tensor [B, T, H, 128] with unit channel stride")


def _seqlens(seqlens, B, device):
    if seqlens is None:
        return None
    if torch.is_tensor(seqlens) and seqlens.dtype is torch.int32 and seqlens.device == device and seqlens.numel() == B and \
            seqlens.is_contiguous():
        return seqlens
    if not torch.is_tensor(seqlens):
        seqlens = torch.tensor(seqlens, dtype=torch.int32)
    seqlens = seqlens.to(device=device, dtype=torch.int32).contiguous()
    if seqlens.numel() != B:
        raise ValueError("seqlens must have B entries")
    return seqlens


def quantize_qk(x: torch.Tensor, cap: Optional[int] = None, seqlens=None, out: Optional[MXFP4] = None,
                hadamard: bool = False) -> MXFP4:
    """MXFP4-quantize Q or K ([B, T, H, 128] bf16) into the packed layout.

    hadamard=True rotates each row by H/sqrt(128) first (qk4v8_quantize_qk_hadamard);
    rotate both Q and K, or neither."""
    _check_bf16(x, "x")
    B, T, H, _ = x.shape
    cap = round_cap(T) if cap is None else int(cap)
    sl = _seqlens(seqlens, B, x.device)
    if out is None:
        out = MXFP4(torch.empty((B, H, cap, 64), dtype=torch.uint8, device=x.device),
                    torch.empty((B, H, cap // 128, 512), dtype=torch.uint8, device=x.device), B, H, cap, T)
    fn, name = ((lib().qk4v8_quantize_qk_hadamard, "qk4v8_quantize_qk_hadamard") if hadamard
                else (lib().qk4v8_quantize_qk, "qk4v8_quantize_qk"))
    check(fn(x.data_ptr(), B, T, H, D, x.stride(0), x.stride(1), x.stride(2), _ptr(sl), cap,
             out.codes.data_ptr(), out.scales.data_ptr(), _stream(x.device)), name)
    out.length = T
    return out


def quantize_v(v: torch.Tensor, cap: Optional[int] = None, seqlens=None, out: Optional[MXFP8V] = None) -> MXFP8V:
    """MXFP8-E4M3-quantize V ([B, T, H, 128] bf16), groups of 32 along T."""
    _check_bf16(v, "v")
    B, T, H, _ = v.shape
    cap = round_cap(T) if cap is None else int(cap)
    sl = _seqlens(seqlens, B, v.device)
    if out is None:
        out = MXFP8V(torch.empty((B, H, cap // 128, D, 128), dtype=torch.uint8, device=v.device),
                     torch.empty((B, H, cap // 128, 512), dtype=torch.uint8, device=v.device), B, H, cap, T)
    check(lib().qk4v8_quantize_v(v.data_ptr(), B, T, H, D, v.stride(0), v.stride(1), v.stride(2), _ptr(sl), cap,
                                 out.codes.data_ptr(), out.scales.data_ptr(), _stream(v.device)), "qk4v8_quantize_v")
    out.length = T
    return out


def quantize_v4(v: torch.Tensor, cap: Optional[int] = None, seqlens=None, out: Optional[MXFP4V] = None) -> MXFP4V:
    """MXFP4-quantize V ([B, T, H, 128] bf16), groups of 32 along T (qk4v8_quantize_v4, QK4V4)."""
    _check_bf16(v, "v")
    B, T, H, _ = v.shape
    cap = round_cap(T) if cap is None else int(cap)
    sl = _seqlens(seqlens, B, v.device)
    if out is None:
        out = MXFP4V(torch.empty((B, H, cap // 128, D, 64), dtype=torch.uint8, device=v.device),
                     torch.empty((B, H, cap // 128, 512), dtype=torch.uint8, device=v.device), B, H, cap, T)
    check(lib().qk4v8_quantize_v4(v.data_ptr(), B, T, H, D, v.stride(0), v.stride(1), v.stride(2), _ptr(sl), cap,
                                  out.codes.data_ptr(), out.scales.data_ptr(), _stream(v.device)), "qk4v8_quantize_v4")
    out.length = T
    return out


def quantize(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seqlens_k=None, q_cap=None, kv_cap=None,
             hadamard: bool = False):
    """Quantize contiguous Q [B,Sq,Hq,128], K and V [B,Sk,Hkv,128] in one library call.

    hadamard=True quantizes Q and K after their Hadamard rotation (three launches:
    qk4v8_quantize_qk_hadamard for Q and K, qk4v8_quantize_v for V)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check_bf16(t, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous for qk4v8_quantize")
    B, Sq, Hq, _ = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    q_cap = round_cap(Sq) if q_cap is None else int(q_cap)
    kv_cap = round_cap(Sk) if kv_cap is None else int(kv_cap)
    dev = q.device
    sl = _seqlens(seqlens_k, B, dev)
    if hadamard:
        qp = quantize_qk(q, cap=q_cap, hadamard=True)
        kp = quantize_qk(k, cap=kv_cap, seqlens=sl, hadamard=True)
        vp = quantize_v(v, cap=kv_cap, seqlens=sl)
        return qp, kp, vp
    qp = MXFP4(torch.empty((B, Hq, q_cap, 64), dtype=torch.uint8, device=dev),
               torch.empty((B, Hq, q_cap // 128, 512), dtype=torch.uint8, device=dev), B, Hq, q_cap, Sq)
    kp = MXFP4(torch.empty((B, Hkv, kv_cap, 64), dtype=torch.uint8, device=dev),
               torch.empty((B, Hkv, kv_cap // 128, 512), dtype=torch.uint8, device=dev), B, Hkv, kv_cap, Sk)
    vp = MXFP8V(torch.empty((B, Hkv, kv_cap // 128, D, 128), dtype=torch.uint8, device=dev),
                torch.empty((B, Hkv, kv_cap // 128, 512), dtype=torch.uint8, device=dev), B, Hkv, kv_cap, Sk)
    check(lib().qk4v8_quantize(q.data_ptr(), k.data_ptr(), v.data_ptr(), B, Sq, Sk, Hq, Hkv, D, _ptr(sl), q_cap,
                               kv_cap, qp.codes.data_ptr(), qp.scales.data_ptr(), kp.codes.data_ptr(),
                               kp.scales.data_ptr(), vp.codes.data_ptr(), vp.scales.data_ptr(), _stream(dev)),
          "qk4v8_quantize")
    return qp, kp, vp


def attention_prefill(q: MXFP4, k: MXFP4, v: MXFP8V, seqlens_k=None, causal: bool = True,
                      softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                      dev_status: Optional[torch.Tensor] = None):
    """QK4V8 prefill attention. Returns out bf16 [B, Sq, Hq, 128] (and lse [B, Hq, Sq])."""
    dev = q.codes.device
    B, Hq, Sq = q.B, q.H, q.length
    sl = _seqlens(seqlens_k, B, dev)
    if out is None:
        out = torch.empty((B, Sq, Hq, D), dtype=torch.bfloat16, device=dev)
    if return_lse and lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=dev)
    check(lib().qk4v8_attention_prefill(q.codes.data_ptr(), q.scales.data_ptr(), B, Hq, Sq, q.cap,
                                        k.codes.data_ptr(), k.scales.data_ptr(), v.codes.data_ptr(),
                                        v.scales.data_ptr(), k.H, k.length, k.cap, _ptr(sl), int(bool(causal)),
                                        float(softmax_scale or 0.0), out.data_ptr(), _ptr(lse), _ptr(dev_status),
                                        _stream(dev)), "qk4v8_attention_prefill")
    return (out, lse) if return_lse else out


def decode_workspace_bytes(B: int, Hq: int, nq: int, num_splits: int) -> int:
    return int(lib().qk4v8_decode_workspace_bytes(B, Hq, nq, num_splits))


def decode_default_splits(B: int, Hq: int, Hkv: int, nq: int, max_seqlen: int, window: int = 0) -> int:
    if window:
        return int(lib().qk4v8_decode_default_splits_window(B, Hq, Hkv, nq, max_seqlen, int(window)))
    return int(lib().qk4v8_decode_default_splits(B, Hq, Hkv, nq, max_seqlen))


def decode_plan_splits(B: int, Hq: int, Hkv: int, nq: int, seqlens, window: int = 0) -> int:
    """Split count from the host-side sequence lengths (qk4v8_decode_plan_splits)."""
    import numpy as np
    lens = np.ascontiguousarray(np.asarray(seqlens if not torch.is_tensor(seqlens) else seqlens.cpu().numpy()),
                                dtype=np.int32)
    if lens.size != B:
        raise ValueError("seqlens must have B entries")
    return int(lib().qk4v8_decode_plan_splits(B, Hq, Hkv, nq, lens.ctypes.data, int(window)))


def attention_decode(q: MXFP4, k: MXFP4, v, seqlens_k, max_seqlen: Optional[int] = None,
                     causal_in_block: bool = True, softmax_scale: Optional[float] = None, num_splits: int = 0,
                     workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                     dev_status: Optional[torch.Tensor] = None, window: int = 0):
    """Split-KV decode / speculative verify over a packed cache. Returns out bf16 [B, nq, Hq, 128].

    window > 0: draft-block attention, each query row sees only the last `window`
    keys before the nq-token block and the block (qk4v8_attention_decode_window)."""
    dev = q.codes.device
    B, Hq, nq = q.B, q.H, q.length
    sl = _seqlens(seqlens_k, B, dev)
    if max_seqlen is None:
        max_seqlen = k.cap
    splits = num_splits if num_splits > 0 else decode_default_splits(B, Hq, k.H, nq, max_seqlen, window)
    need = decode_workspace_bytes(B, Hq, nq, splits)
    if workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty((B, nq, Hq, D), dtype=torch.bfloat16, device=dev)
    if return_lse and lse is None:
        lse = torch.empty((B, Hq, nq), dtype=torch.float32, device=dev)
    head = (q.codes.data_ptr(), q.scales.data_ptr(), B, Hq, nq, q.cap, k.codes.data_ptr(), k.scales.data_ptr(),
            v.codes.data_ptr(), v.scales.data_ptr(), k.H, k.cap, _ptr(sl), int(max_seqlen),
            int(bool(causal_in_block)))
    tail = (float(softmax_scale or 0.0), int(splits), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), out.data_ptr(), _ptr(lse), _ptr(dev_status), _stream(dev))
    if isinstance(v, MXFP4V):
        check(lib().qk4v8_attention_decode_v4(*head, int(window), *tail), "qk4v8_attention_decode_v4")
    elif window:
        check(lib().qk4v8_attention_decode_window(*head, int(window), *tail), "qk4v8_attention_decode_window")
    else:
        check(lib().qk4v8_attention_decode(*head, *tail), "qk4v8_attention_decode")
    return (out, lse) if return_lse else out


def decode_bf16_workspace_bytes(B: int, Hq: int, Hkv: int, nq: int, num_splits: int) -> int:
    return int(lib().qk4v8_decode_bf16_workspace_bytes(B, Hq, Hkv, nq, num_splits))


def attention_decode_bf16(q: torch.Tensor, k: MXFP4, v, seqlens_k, max_seqlen: Optional[int] = None,
                          causal_in_block: bool = True, softmax_scale: Optional[float] = None, num_splits: int = 0,
                          workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                          dev_status: Optional[torch.Tensor] = None, window: int = 0):
    """Decode step from bf16 queries q [B, nq, Hq, 128]; the query is MXFP4-quantized inside the call.
    Returns out bf16 [B, nq, Hq, 128] (and lse [B, Hq, nq]). window as for attention_decode."""
    _check_bf16(q, "q")
    dev = q.device
    B, nq, Hq, _ = q.shape
    sl = _seqlens(seqlens_k, B, dev)
    if max_seqlen is None:
        max_seqlen = k.cap
    splits = num_splits if num_splits > 0 else decode_default_splits(B, Hq, k.H, nq, max_seqlen, window)
    need = decode_bf16_workspace_bytes(B, Hq, k.H, nq, splits)
    if workspace is None and need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty((B, nq, Hq, D), dtype=torch.bfloat16, device=dev)
    if return_lse and lse is None:
        lse = torch.empty((B, Hq, nq), dtype=torch.float32, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    head = (q.data_ptr(), B, Hq, nq, q.stride(0), q.stride(1), q.stride(2), k.codes.data_ptr(), k.scales.data_ptr(),
            v.codes.data_ptr(), v.scales.data_ptr(), k.H, k.cap, _ptr(sl), int(max_seqlen),
            int(bool(causal_in_block)))
    tail = (float(softmax_scale or 0.0), int(splits), _ptr(workspace), ws_bytes, out.data_ptr(), _ptr(lse),
            _ptr(dev_status), _stream(dev))
    if isinstance(v, MXFP4V):
        check(lib().qk4v8_attention_decode_bf16_v4(*head, int(window), *tail), "qk4v8_attention_decode_bf16_v4")
    elif window:
        check(lib().qk4v8_attention_decode_bf16_window(*head, int(window), *tail), "qk4v8_attention_decode_bf16_window")
    else:
        check(lib().qk4v8_attention_decode_bf16(*head, *tail), "qk4v8_attention_decode_bf16")
    return (out, lse) if return_lse else out


def attention_decode_splitkv(q: MXFP4, k: MXFP4, v: MXFP8V, seqlens_k: torch.Tensor, max_seqlen: int,
                             num_splits: int, workspace: torch.Tensor, causal_in_block: bool = True,
                             softmax_scale: Optional[float] = None, dev_status: Optional[torch.Tensor] = None):
    """First decode stage: per-split partial (O, lse2) into `workspace` (num_splits must be > 0)."""
    dev = q.codes.device
    check(lib().qk4v8_attention_decode_splitkv(q.codes.data_ptr(), q.scales.data_ptr(), q.B, q.H, q.length, q.cap,
                                               k.codes.data_ptr(), k.scales.data_ptr(), v.codes.data_ptr(),
                                               v.scales.data_ptr(), k.H, k.cap, seqlens_k.data_ptr(),
                                               int(max_seqlen), int(bool(causal_in_block)),
                                               float(softmax_scale or 0.0), int(num_splits), workspace.data_ptr(),
                                               workspace.numel() * workspace.element_size(), _ptr(dev_status),
                                               _stream(dev)), "qk4v8_attention_decode_splitkv")


def decode_merge(workspace: torch.Tensor, B: int, Hq: int, nq: int, num_splits: int, out: torch.Tensor,
                 lse: Optional[torch.Tensor] = None):
    """Second decode stage: merge the split partials into out bf16 [B, nq, Hq, 128]."""
    check(lib().qk4v8_decode_merge(workspace.data_ptr(), workspace.numel() * workspace.element_size(), B, Hq, nq,
                                   num_splits, out.data_ptr(), _ptr(lse), _stream(out.device)), "qk4v8_decode_merge")
    return out


def default_scale() -> float:
    return 1.0 / math.sqrt(D)


# ----------------------------------------------------------------------------------------------------------
# Measurement hooks (include/qk4v8_test.h): not part of the attention API.

def prefill_stage_qk(q: MXFP4, k: MXFP4, seqlens_k=None, causal: bool = True,
                     softmax_scale: Optional[float] = None, row_max: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The QK^T stage of the prefill kernel alone (same tile schedule, no exp / P / PV).

    Returns row_max float32 [B, Hq, Sq]: each query row's largest allowed score
    times softmax_scale * log2(e) (-inf for a row with no allowed key).
    """
    dev = q.codes.device
    B, Hq, Sq = q.B, q.H, q.length
    sl = _seqlens(seqlens_k, B, dev)
    if row_max is None:
        row_max = torch.empty((B, Hq, Sq), dtype=torch.float32, device=dev)
    check(lib().qk4v8_test_prefill_stage_qk(q.codes.data_ptr(), q.scales.data_ptr(), B, Hq, Sq, q.cap,
                                            k.codes.data_ptr(), k.scales.data_ptr(), k.H, k.length, k.cap, _ptr(sl),
                                            int(bool(causal)), float(softmax_scale or 0.0), row_max.data_ptr(),
                                            _ptr(dev_status), _stream(dev)), "qk4v8_test_prefill_stage_qk")
    return row_max


MMA_PEAK_SHAPES = {0: ("mxf4", 128, 128, 64), 1: ("mxf8f6f4", 128, 144, 32),
                   2: ("mxf8f6f4", 128, 256, 32), 3: ("mxf4", 128, 256, 64)}


def mma_peak_run(kind: int, ctas: int, iters: int, device=None, dev_status: Optional[torch.Tensor] = None) -> int:
    """Enqueue one tensor-pipe peak run; returns its FLOP count (2*M*N*K per instruction)."""
    dev = torch.device(device or "cuda")
    check(lib().qk4v8_test_mma_peak(int(kind), int(ctas), int(iters), _ptr(dev_status), _stream(dev)),
          "qk4v8_test_mma_peak")
    _, m, n, kk = MMA_PEAK_SHAPES[int(kind)]
    return 2 * m * n * kk * int(ctas) * int(iters)


# ----------------------------------------------------------------------------------------------------------
# Paged KV cache (include/qk4v8.h: qk4v8_kv_append, qk4v8_attention_decode_paged).

@dataclass
class PagedKV:
    """Packed KV cache in pools of 128-token pages, and the per-sequence state.

    k_codes uint8 [P, Hkv, 128, 64], k_scales uint8 [P, Hkv, 512],
    v_codes uint8 [P, Hkv, 128, 128], v_scales uint8 [P, Hkv, 512] (P pages);
    block_table int32 [B, max_pages]: page of each 128-token block of a sequence;
    seqlens int32 [B]: tokens held; v_tail bf16 [B, Hkv, 32, 128]: the open V
    group of each sequence and head, which every append reads and refreshes."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor
    v_tail: torch.Tensor
    block_table: torch.Tensor
    seqlens: torch.Tensor
    hadamard_k: bool = False

    @property
    def num_pages(self) -> int:
        return self.k_codes.shape[0]

    @property
    def Hkv(self) -> int:
        return self.k_codes.shape[1]

    @property
    def B(self) -> int:
        return self.block_table.shape[0]

    @property
    def max_pages(self) -> int:
        return self.block_table.shape[1]


def paged_kv(B: int, Hkv: int, num_pages: int, block_table: torch.Tensor, device="cuda",
             hadamard_k: bool = False) -> PagedKV:
    """An empty paged cache (every sequence of length 0) over a new pool of num_pages pages.
    block_table: int32 [B, max_pages] page indices, owned by the caller's page allocator."""
    dev = torch.device(device)
    bt = block_table.to(device=dev, dtype=torch.int32).contiguous()
    if bt.dim() != 2 or bt.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    u8 = torch.uint8
    return PagedKV(k_codes=torch.empty((num_pages, Hkv, 128, 64), dtype=u8, device=dev),
                   k_scales=torch.empty((num_pages, Hkv, 512), dtype=u8, device=dev),
                   v_codes=torch.empty((num_pages, Hkv, 128, 128), dtype=u8, device=dev),
                   v_scales=torch.empty((num_pages, Hkv, 512), dtype=u8, device=dev),
                   v_tail=torch.empty((B, Hkv, 32, 128), dtype=torch.bfloat16, device=dev),
                   block_table=bt, seqlens=torch.zeros((B,), dtype=torch.int32, device=dev), hadamard_k=hadamard_k)


def kv_append(cache: PagedKV, k_new: torch.Tensor, v_new: torch.Tensor, dev_status: Optional[torch.Tensor] = None):
    """Append k_new, v_new (bf16 [B, n_new, Hkv, 128], same strides) to every sequence
    (qk4v8_kv_append); cache.seqlens advances by n_new on the device."""
    _check_bf16(k_new, "k_new")
    _check_bf16(v_new, "v_new")
    if k_new.shape != v_new.shape or k_new.stride() != v_new.stride():
        raise ValueError("k_new and v_new must have the same shape and strides")
    B, n_new, Hkv, _ = k_new.shape
    check(lib().qk4v8_kv_append(k_new.data_ptr(), v_new.data_ptr(), B, n_new, Hkv, D, k_new.stride(0),
                                k_new.stride(1), k_new.stride(2), cache.seqlens.data_ptr(),
                                cache.seqlens.data_ptr(), cache.block_table.data_ptr(), cache.max_pages,
                                cache.num_pages, cache.k_codes.data_ptr(), cache.k_scales.data_ptr(),
                                cache.v_codes.data_ptr(), cache.v_scales.data_ptr(), cache.v_tail.data_ptr(),
                                int(cache.hadamard_k), _ptr(dev_status), _stream(k_new.device)), "qk4v8_kv_append")
    return cache


def _paged_call_args(cache: PagedKV):
    return (cache.k_codes.data_ptr(), cache.k_scales.data_ptr(), cache.v_codes.data_ptr(), cache.v_scales.data_ptr(),
            cache.Hkv, cache.num_pages, cache.block_table.data_ptr(), cache.max_pages, cache.seqlens.data_ptr())


def attention_decode_paged(q: MXFP4, cache: PagedKV, max_seqlen: int, causal_in_block: bool = True,
                           window: int = 0, softmax_scale: Optional[float] = None, num_splits: int = 0,
                           workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                           dev_status: Optional[torch.Tensor] = None):
    """Decode / verify / draft-block attention over a paged cache (qk4v8_attention_decode_paged)."""
    dev = q.codes.device
    B, Hq, nq = q.B, q.H, q.length
    splits = num_splits if num_splits > 0 else decode_default_splits(B, Hq, cache.Hkv, nq, max_seqlen, window)
    if workspace is None:
        workspace = torch.empty((max(16, decode_workspace_bytes(B, Hq, nq, splits)),), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty((B, nq, Hq, D), dtype=torch.bfloat16, device=dev)
    if return_lse and lse is None:
        lse = torch.empty((B, Hq, nq), dtype=torch.float32, device=dev)
    check(lib().qk4v8_attention_decode_paged(q.codes.data_ptr(), q.scales.data_ptr(), B, Hq, nq, q.cap,
                                             *_paged_call_args(cache), int(max_seqlen), int(bool(causal_in_block)),
                                             int(window), float(softmax_scale or 0.0), int(splits),
                                             workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                             out.data_ptr(), _ptr(lse), _ptr(dev_status), _stream(dev)),
          "qk4v8_attention_decode_paged")
    return (out, lse) if return_lse else out


def attention_decode_bf16_paged(q: torch.Tensor, cache: PagedKV, max_seqlen: int, causal_in_block: bool = True,
                                window: int = 0, softmax_scale: Optional[float] = None, num_splits: int = 0,
                                workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                                lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                                dev_status: Optional[torch.Tensor] = None):
    """Decode step from bf16 queries q [B, nq, Hq, 128] over a paged cache (qk4v8_attention_decode_bf16_paged)."""
    _check_bf16(q, "q")
    dev = q.device
    B, nq, Hq, _ = q.shape
    splits = num_splits if num_splits > 0 else decode_default_splits(B, Hq, cache.Hkv, nq, max_seqlen, window)
    need = decode_bf16_workspace_bytes(B, Hq, cache.Hkv, nq, splits)
    if workspace is None and need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty((B, nq, Hq, D), dtype=torch.bfloat16, device=dev)
    if return_lse and lse is None:
        lse = torch.empty((B, Hq, nq), dtype=torch.float32, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib().qk4v8_attention_decode_bf16_paged(q.data_ptr(), B, Hq, nq, q.stride(0), q.stride(1), q.stride(2),
                                                  *_paged_call_args(cache), int(max_seqlen),
                                                  int(bool(causal_in_block)), int(window),
                                                  float(softmax_scale or 0.0), int(splits), _ptr(workspace), ws_bytes,
                                                  out.data_ptr(), _ptr(lse), _ptr(dev_status), _stream(dev)),
          "qk4v8_attention_decode_bf16_paged")
    return (out, lse) if return_lse else out


def _empty(dtype, device, a, b, c, d):
    """torch.empty of [a, b, c, d], as empty_strided (less host time)."""
    return torch.empty_strided((a, b, c, d), (b * c * d, c * d, d, 1), dtype=dtype, device=device)


_I32, _BF16 = torch.int32, torch.bfloat16


def _misfit(device, name, t, what, nbytes):
    got = "none" if t is None else f"{t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}"
    return ValueError(f"{name} must be a contiguous {what} tensor of {nbytes} bytes on {device}, got {got}")


def _check_packed(device, name, x, row):
    """codes (row bytes a token) and scales of a packed tensor: that what the call reads or writes is there. (By their
    bytes, in one expression: half of a short call's host time went to comparing types and shapes one by one.)"""
    c, s, i = x.codes, x.scales, device.index
    n = x.B * x.H * x.cap
    if c.nbytes == n * row and s.nbytes == n * 4 and c.get_device() == i and s.get_device() == i and \
            c.is_contiguous() and s.is_contiguous():
        return
    for part, t, need in ((name + ".codes", c, n * row), (name + ".scales", s, n * 4)):
        if t.nbytes != need or t.device != device or not t.is_contiguous():
            raise _misfit(device, part, t, "uint8", need)


def _check_cache(device, cache, tail):
    """A paged cache's buffers (the staged rows if `tail`), as _check_packed; its pages, heads, sequences and pages of a
    sequence."""
    kc, ks, vc, vs, bt, sl = cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, cache.block_table, cache.seqlens
    if kc.dim() != 4 or bt.dim() != 2:
        raise ValueError("the cache must have k_codes [pages, Hkv, 128, 64] and block_table [B, max_pages]")
    P, H, _, _ = kc.shape
    B, most = bt.shape
    i, n, t = device.index, P * H, cache.v_tail if tail else None
    if bt.dtype is _I32 and sl.dtype is _I32 and kc.nbytes == n * 8192 and ks.nbytes == n * 512 and \
            vc.nbytes == n * 16384 and vs.nbytes == n * 512 and sl.nbytes == B * 4 and kc.get_device() == i and \
            ks.get_device() == i and vc.get_device() == i and vs.get_device() == i and bt.get_device() == i and \
            sl.get_device() == i and kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and \
            vs.is_contiguous() and bt.is_contiguous() and sl.is_contiguous() and (
                not tail or (t is not None and t.dtype is _BF16 and t.nbytes == B * H * 8192 and t.get_device() == i and
                             t.is_contiguous())):
        return P, H, B, most
    for name, x, dtype, need in (("k_codes", kc, kc.dtype, n * 8192), ("k_scales", ks, ks.dtype, n * 512),
                                 ("v_codes", vc, vc.dtype, n * 16384), ("v_scales", vs, vs.dtype, n * 512),
                                 ("block_table", bt, _I32, B * most * 4), ("seqlens", sl, _I32, B * 4)):
        if x.dtype is not dtype or x.nbytes != need or x.device != device or not x.is_contiguous():
            raise _misfit(device, "the cache's " + name, x, "int32" if dtype is _I32 else "uint8", need)
    raise _misfit(device, "the cache's v_tail", t, "bfloat16", B * H * 8192)


def _status(t: Optional[torch.Tensor], device):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.device != device or t.numel() < 1:
        raise ValueError("dev_status must be an int32 tensor on the inputs' device")
    return t.data_ptr()


# ----------------------------------------------------------------------------------------------------------
# Rotary positions (include/qk4v8.h: qk4v8_rope, qk4v8_quantize_qk_rope, qk4v8_kv_append_rope).

@dataclass
class Rope:
    """A model's rotary positions: what a program makes once and gives to every call.

    table float32 [max_pos, rotary_dim / 2, 2] (CUDA, contiguous): cosine and sine of
    position p for pair i (rope_table makes the usual one); adjacent: pairs (2i, 2i + 1)
    instead of (i, i + rotary_dim / 2); pair_axis: axis of each pair (rotary_dim / 2
    entries of 0..3) when positions have several axes."""
    table: torch.Tensor
    adjacent: bool = False
    pair_axis: Optional[Sequence[int]] = None
    n_axes: int = field(init=False)
    _axes: object = field(init=False, repr=False)

    def __post_init__(self):
        t = self.table
        if t.dtype != torch.float32 or not t.is_cuda or t.dim() != 3 or t.shape[2] != 2 or not t.is_contiguous():
            raise ValueError("table must be a contiguous CUDA float32 tensor [max_pos, rotary_dim / 2, 2]")
        self._axes, self.n_axes = None, 1
        if self.pair_axis is not None:
            axes = [int(a) for a in self.pair_axis]
            if len(axes) != t.shape[1] or min(axes) < 0 or max(axes) > 3:
                raise ValueError("pair_axis must have rotary_dim / 2 entries of 0..3")
            self._axes, self.n_axes = (ctypes.c_uint8 * len(axes))(*axes), max(axes) + 1

    def __setattr__(self, name, value):
        """A table or axes set later are checked as the first ones (the library reads an axis for each pair of the table)."""
        later = name in ("table", "pair_axis") and "_axes" in self.__dict__
        before = self.__dict__.copy()
        self.__dict__[name] = value
        if later:
            try:
                self.__post_init__()
            except Exception:
                self.__dict__.update(before)
                raise

    @property
    def rotary_dim(self) -> int:
        return 2 * self.table.shape[1]


def rope_table(max_pos: int, rotary_dim: int = D, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Rope.table with angles p * base^(-2 i / rotary_dim), taken in fp64 (far positions) and held in fp32."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    p = torch.arange(max_pos, dtype=torch.float64, device=device)
    angle = p[:, None] * (float(base) ** (-2.0 * i / rotary_dim))
    return torch.stack((angle.cos(), angle.sin()), -1).to(torch.float32).contiguous()


def _rope_struct(rope: Rope, positions: Optional[torch.Tensor], B: int, T: int, device) -> RopeStruct:
    if rope.table.device != device:
        raise ValueError("rope.table must be on the inputs' device")
    s = RopeStruct(rope.table.data_ptr(), rope.table.shape[0], 2 * rope.table.shape[1], int(rope.adjacent),
                   rope.n_axes, None if rope._axes is None else ctypes.addressof(rope._axes))
    if positions is not None:
        if positions.dim() == 2:
            positions = positions.unsqueeze(0)
        if positions.dtype != torch.int32 or positions.device != device or positions.dim() != 3 or \
                positions.shape[0] < rope.n_axes or tuple(positions.shape[1:]) != (B, T):
            raise ValueError("positions must be an int32 tensor [B, T] or [axes, B, T] on the inputs' device, with an "
                             "axis for each one that rope.pair_axis names")
        s.positions = positions.data_ptr()
        s.pos_stride_axis, s.pos_stride_b, s.pos_stride_t = positions.stride()
    return s


def _int32_on(t: Optional[torch.Tensor], B: int, device, name: str) -> Optional[int]:
    if t is None:
        return None
    if t.dtype != torch.int32 or t.device != device or tuple(t.shape) != (B,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor [B] on the inputs' device")
    return t.data_ptr()


def quantize_qk_rope(x: torch.Tensor, rope: Rope, positions: Optional[torch.Tensor] = None,
                     start: Optional[torch.Tensor] = None, cap: Optional[int] = None, seqlens=None,
                     out: Optional[MXFP4] = None, hadamard: bool = False, pad: bool = True,
                     dev_status: Optional[torch.Tensor] = None) -> MXFP4:
    """Rotate Q or K ([B, T, H, 128] bf16) by their positions and MXFP4-quantize them, in one pass
    (qk4v8_quantize_qk_rope).

    positions: int32 [B, T] or [axes, B, T], any strides (an expanded one is read in place); without them
    token t of sequence b is at start[b] + t (start: int32 [B], None: 0). pad=False writes the T given rows
    and leaves the rest of `out` (a buffer kept over the decode steps) as it is."""
    _check_bf16(x, "x")
    B, T, H, _ = x.shape
    dev = x.device
    if out is not None:
        if out.B != B or out.H != H or (cap is not None and cap != out.cap):
            raise ValueError("out must be a packed tensor of the same B, H and capacity")
        _check_packed(dev, "out", out, 64)
        cap = out.cap
    elif cap is None:
        cap = round_cap(T)
    sl = _seqlens(seqlens, B, dev)
    rs = _rope_struct(rope, positions, B, T, dev)
    st = _int32_on(start, B, dev, "start")
    if out is None:
        out = MXFP4(_empty(torch.uint8, dev, B, H, cap, 64), _empty(torch.uint8, dev, B, H, cap // 128, 512), B, H, cap, T)
    with _on(dev):
        # (An empty x has a null pointer; no row of it is read.)
        check(lib().qk4v8_quantize_qk_rope(x.data_ptr() or out.codes.data_ptr(), B, T, H, D, x.stride(0), x.stride(1),
                                           x.stride(2), _ptr(sl), st, ctypes.addressof(rs), int(bool(hadamard)), cap,
                                           int(bool(pad)), out.codes.data_ptr(), out.scales.data_ptr(),
                                           _status(dev_status, dev), _stream(dev)), "qk4v8_quantize_qk_rope")
    out.length = T
    return out


_Strides = ctypes.c_int64 * 3


def kv_append_rope(cache: PagedKV, k_new: torch.Tensor, v_new: torch.Tensor, rope: Rope,
                   positions: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
                   seqlens_out: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None) -> PagedKV:
    """Append k_new (rotated by its positions) and v_new (bf16 [B, n_new, Hkv, 128], strides of their own) to the
    sequences (qk4v8_kv_append_rope).

    new_lens: int32 [B], the sequence's first new_lens[b] tokens are appended (None: all n_new).
    positions as for quantize_qk_rope; without them a token is at its place in the sequence, which is its position unless
    the sequence goes on behind a prefix held elsewhere (attention_decode_prefix_paged): then give prefix_len + place.
    cache.seqlens advances on the device, unless seqlens_out (int32 [B]) receives the new lengths."""
    _check_bf16(k_new, "k_new")
    shape, dev = k_new.shape, k_new.device
    B, n_new, Hkv, _ = shape
    if v_new.dtype is not _BF16 or v_new.shape != shape or v_new.device != dev or v_new.stride(3) != 1:
        raise ValueError("v_new must be a bf16 tensor with k_new's shape and device and unit channel stride")
    num_pages, heads, rows, max_pages = _check_cache(dev, cache, True)
    if B != rows or Hkv != heads:
        raise ValueError("k_new must be [cache.B, n_new, cache.Hkv, 128]")
    rs = _rope_struct(rope, positions, B, n_new, dev)
    nl = _int32_on(new_lens, B, dev, "new_lens")
    lens = cache.seqlens.data_ptr()
    so = lens if seqlens_out is None else _int32_on(seqlens_out, B, dev, "seqlens_out")
    ks, vs = _Strides(*k_new.stride()[:3]), _Strides(*v_new.stride()[:3])
    with _on(dev):
        check(lib().qk4v8_kv_append_rope(k_new.data_ptr(), v_new.data_ptr(), B, n_new, Hkv, D, ctypes.addressof(ks),
                                         ctypes.addressof(vs), lens, nl, so, ctypes.addressof(rs),
                                         cache.block_table.data_ptr(), max_pages, num_pages,
                                         cache.k_codes.data_ptr(), cache.k_scales.data_ptr(),
                                         cache.v_codes.data_ptr(), cache.v_scales.data_ptr(), cache.v_tail.data_ptr(),
                                         int(cache.hadamard_k), _status(dev_status, dev), _stream(dev)),
              "qk4v8_kv_append_rope")
    return cache


# ----------------------------------------------------------------------------------------------------------
# Decode over a shared prefix (include/qk4v8.h: qk4v8_attention_decode_prefix).

def decode_prefix_workspace_bytes(B: int, Hq: int, Hkv: int, nq: int, prefix_len: int, max_seqlen: int) -> int:
    return int(lib().qk4v8_decode_prefix_workspace_bytes(B, Hq, Hkv, nq, prefix_len, max_seqlen))


def _prefix_buffers(q: MXFP4, Hkv: int, prefix_len: int, max_seqlen: int, workspace, out, lse, return_lse):
    dev = q.codes.device
    if workspace is None:
        need = decode_prefix_workspace_bytes(q.B, q.H, Hkv, q.length, prefix_len, max_seqlen)
        workspace = torch.empty_strided((max(16, need),), (1,), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on q's device")
    if out is None:
        out = _empty(torch.bfloat16, dev, q.B, q.length, q.H, D)
    elif out.dtype != torch.bfloat16 or out.device != dev or tuple(out.shape) != (q.B, q.length, q.H, D) or \
            not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor [B, nq, Hq, 128] on q's device")
    if lse is not None:
        if lse.dtype != torch.float32 or lse.device != dev or tuple(lse.shape) != (q.B, q.H, q.length) or \
                not lse.is_contiguous():
            raise ValueError("lse must be a contiguous float32 tensor [B, Hq, nq] on q's device")
    elif return_lse:
        lse = torch.empty((q.B, q.H, q.length), dtype=torch.float32, device=dev)
    return workspace, workspace.numel() * workspace.element_size(), out, lse


def attention_decode_prefix(q: MXFP4, k_prefix: MXFP4, v_prefix: MXFP8V, k: MXFP4, v: MXFP8V, seqlens_k,
                            max_seqlen: Optional[int] = None, prefix_len: Optional[int] = None,
                            causal_in_block: bool = True, softmax_scale: Optional[float] = None,
                            workspace: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            return_lse: bool = False, dev_status: Optional[torch.Tensor] = None):
    """Decode / verify of sequences that share a prefix (k_prefix, v_prefix: packed with B = 1), followed by their
    own keys (k, v, seqlens_k as for attention_decode; a length may be 0). The prefix is read once for all
    (qk4v8_attention_decode_prefix). Returns out bf16 [B, nq, Hq, 128] (and lse [B, Hq, nq])."""
    dev = q.codes.device
    B, Hq, nq = q.B, q.H, q.length
    if k_prefix.B != 1 or v_prefix.B != 1 or k_prefix.H != k.H or v_prefix.H != k.H or k_prefix.cap != v_prefix.cap:
        raise ValueError("k_prefix and v_prefix must be packed tensors with B = 1, the KV heads of k and one capacity")
    if k.B != B or v.B != B or v.H != k.H or k.cap != v.cap:
        raise ValueError("k and v must be packed tensors of q's batch with the same heads and capacity")
    if not isinstance(v, MXFP8V) or not isinstance(v_prefix, MXFP8V):
        raise ValueError("v and v_prefix must be MXFP8 (MXFP8V)")
    _check_packed(dev, "q", q, 64)
    _check_packed(dev, "k_prefix", k_prefix, 64)
    _check_packed(dev, "v_prefix", v_prefix, D)
    _check_packed(dev, "k", k, 64)
    _check_packed(dev, "v", v, D)
    prefix_len = k_prefix.length if prefix_len is None else int(prefix_len)
    max_seqlen = k.cap if max_seqlen is None else int(max_seqlen)
    sl = _seqlens(seqlens_k, B, dev)
    ws, ws_bytes, out, lse = _prefix_buffers(q, k.H, prefix_len, max_seqlen, workspace, out, lse, return_lse)
    with _on(dev):
        check(lib().qk4v8_attention_decode_prefix(
            q.codes.data_ptr(), q.scales.data_ptr(), B, Hq, nq, q.cap, k_prefix.codes.data_ptr(),
            k_prefix.scales.data_ptr(), v_prefix.codes.data_ptr(), v_prefix.scales.data_ptr(), prefix_len, k_prefix.cap,
            k.codes.data_ptr(), k.scales.data_ptr(), v.codes.data_ptr(), v.scales.data_ptr(), k.H, k.cap, _ptr(sl),
            max_seqlen, int(bool(causal_in_block)), float(softmax_scale or 0.0), ws.data_ptr(), ws_bytes, out.data_ptr(),
            _ptr(lse), _status(dev_status, dev), _stream(dev)), "qk4v8_attention_decode_prefix")
    return (out, lse) if return_lse else out


def attention_decode_prefix_paged(q: MXFP4, cache: PagedKV, prefix_table: torch.Tensor, prefix_len: int,
                                  max_seqlen: int, causal_in_block: bool = True,
                                  softmax_scale: Optional[float] = None,
                                  workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                                  lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                                  dev_status: Optional[torch.Tensor] = None):
    """attention_decode_prefix over a page pool: prefix_table int32 [pages] lists the prefix's pages, the cache's
    block_table and seqlens hold the sequences' own tokens (qk4v8_attention_decode_prefix_paged), whose keys stand at
    positions from prefix_len on: kv_append_rope into such a cache needs its `positions`."""
    dev = q.codes.device
    B, Hq, nq = q.B, q.H, q.length
    prefix_len, max_seqlen = int(prefix_len), int(max_seqlen)
    num_pages, Hkv, rows, max_pages = _check_cache(dev, cache, False)
    if rows != B:
        raise ValueError("the cache must hold q's batch")
    _check_packed(dev, "q", q, 64)
    if prefix_table.dtype != torch.int32 or prefix_table.device != dev or prefix_table.dim() != 1 or \
            not prefix_table.is_contiguous() or prefix_table.shape[0] * 128 < prefix_len:
        raise ValueError("prefix_table must be a contiguous int32 tensor of the prefix's pages on q's device")
    ws, ws_bytes, out, lse = _prefix_buffers(q, Hkv, prefix_len, max_seqlen, workspace, out, lse, return_lse)
    with _on(dev):
        check(lib().qk4v8_attention_decode_prefix_paged(
            q.codes.data_ptr(), q.scales.data_ptr(), B, Hq, nq, q.cap, cache.k_codes.data_ptr(),
            cache.k_scales.data_ptr(), cache.v_codes.data_ptr(), cache.v_scales.data_ptr(), Hkv, num_pages,
            prefix_table.data_ptr(), prefix_len, cache.block_table.data_ptr(), max_pages,
            cache.seqlens.data_ptr(), max_seqlen, int(bool(causal_in_block)), float(softmax_scale or 0.0),
            ws.data_ptr(), ws_bytes, out.data_ptr(), _ptr(lse), _status(dev_status, dev), _stream(dev)),
            "qk4v8_attention_decode_prefix_paged")
    return (out, lse) if return_lse else out
