"""Times of the cases that perf/operators.py lists, on this machine's GPU: `python perf/times.py [--plain] [name ...]`.

Three columns, in microseconds:
  call    one call of a row of them from Python on three sets of inputs in turn, host and device overlapping as in
          a program's loop, the L2 holding what the calls before left in it
  device  the device's part of one call with a cold L2: events around the call, queued behind a write of 1 GiB whose 0.15 ms
          outlast the host's work (median of 30)
  plain   as `call`, of the operator's plain form in torch (with --plain)

`python perf/times.py --shared` compares decode over a shared prefix with attention_decode_paged, whose block tables list the
prefix's pages in front of each sequence's own (one pool, pages in random order): `device` times of both.

`python perf/times.py --once name [size=value ...]` makes three calls of the case, with other sizes where given, and times
none: for a profiler.
"""
import os
import statistics
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch  # noqa: E402

from perf import operators  # noqa: E402


def call_us(states, least_s=0.2):
    def rounds(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        for i in range(n):
            operators.run(states[i % len(states)])
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) * 1e3 / n
    us = rounds(12)
    return min(rounds(max(12, int(least_s / 3 / us * 1e6))) for _ in range(3))


def device_us(call, flush, repeats=30):
    got = []
    for i in range(repeats + 3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        flush.fill_(i)
        a.record()
        call(i)
        b.record()
        torch.cuda.synchronize()
        got.append(a.elapsed_time(b) * 1e3)
    return statistics.median(got[3:])


def main(names, plain):
    flush = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    for case in operators.listed():
        if names and case["name"] not in names:
            continue
        line = f"{case['name']:16}"
        for own in (True, False) if plain else (True,):
            operators.own = own
            states = [operators.prepare(case, seed) for seed in (1, 2, 3)]
            for s in states:
                operators.run(s)
            line += f"  {'call' if own else 'plain'} {call_us(states):8.1f}"
            if own:
                line += f"  device {device_us(lambda i: operators.run(states[i % 3]), flush):8.1f}"
            del states
        print(line, flush=True)


# Sequences, query heads, KV heads, query tokens, prefix tokens, own tokens.
SHARED = [(4, 32, 8, 1, 1000, 100), (16, 32, 8, 1, 1000, 100), (64, 32, 8, 1, 1000, 100), (32, 32, 8, 1, 512, 4096),
          (32, 32, 8, 1, 4096, 4096), (32, 32, 8, 1, 8192, 128), (32, 32, 8, 1, 8192, 1024), (8, 32, 8, 1, 32768, 1024),
          (13, 20, 4, 3, 5003, 777), (64, 64, 8, 8, 16384, 512), (64, 64, 8, 8, 2048, 2048)]


def shared():
    import bit_quantized_attention_qk4v8_b200 as qk
    flush = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    for B, Hq, Hkv, nq, prefix, own in SHARED:
        g = torch.Generator(device="cuda").manual_seed(B * 1000 + prefix)
        pp, po = -(-prefix // 128), -(-own // 128)
        order = torch.randperm(pp + B * po, generator=g, device="cuda").to(torch.int32)
        table = order[pp:].reshape(B, po).contiguous()
        # Prefixes of whole pages, so that the own tokens go on where the other call's table has them.
        prefix = pp * 128
        cache = qk.paged_kv(B, Hkv, pp + B * po, table)
        whole = qk.PagedKV(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, cache.v_tail,
                           torch.cat((order[:pp].expand(B, pp), table), 1).contiguous(),
                           torch.full((B,), prefix + own, dtype=torch.int32, device="cuda"))
        for codes in (cache.k_codes, cache.v_codes):
            codes.random_(0, 64, generator=g)
        cache.k_scales.fill_(127)
        cache.v_scales.fill_(127)
        cache.seqlens.fill_(own)
        q = qk.quantize_qk(torch.randn((B, nq, Hq, 128), generator=g, device="cuda").to(torch.bfloat16))
        a = device_us(lambda i: qk.attention_decode_prefix_paged(q, cache, order[:pp], prefix, max_seqlen=own), flush)
        b = device_us(lambda i: qk.attention_decode_paged(q, whole, max_seqlen=prefix + own), flush)
        print(f"{B:3} sequences, {Hq} / {Hkv} heads, {nq} tokens, {prefix:5} shared + {own:4} own:  shared {a:7.1f}  "
              f"each its own {b:7.1f}", flush=True)


def once(name, *sizes):
    case = next(c for c in operators.listed() if c["name"] == name)
    case.update((k, int(v)) for k, v in (s.split("=") for s in sizes))
    operators.own = True
    state = operators.prepare(case, 1)
    for _ in range(3):
        operators.run(state)
    torch.cuda.synchronize()


if __name__ == "__main__":
    args = sys.argv[1:]
    if args[:1] == ["--once"]:
        once(*args[1:])
    elif args == ["--shared"]:
        shared()
    else:
        main([a for a in args if a != "--plain"], "--plain" in args)
