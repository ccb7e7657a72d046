"""Runs the kernels a few times at one shape (for profilers).

    python -m continuous_softmax_attention_gb300.run_case --B 1 --H 24 --T 8192 --d 128
    python -m continuous_softmax_attention_gb300.run_case --decode --B 4 --H 32 --T 8192
    python -m continuous_softmax_attention_gb300.run_case --paged --B 16 --H 32 --kv-heads 8 --T 4096
    python -m continuous_softmax_attention_gb300.run_case --paged --draft 16 --kind e4m3 --B 16 --H 32 --kv-heads 8

Inputs come from the seeded generator; each iteration launches the
continuous kernel once and, unless --no-std, the standard kernel once.
With --decode each iteration is one decode step (lengths drawn from
[T/2, T]); with --backward one forward pass, then each iteration is one
backward pass; with --paged one step of a server over a paged cache: room
reserved for a token of each sequence, its key and value appended with rotary
positions, and the decode step (lengths drawn from [T/2, T]).  --kind e4m3 or
int8 holds the cache in 8 bits; --draft N drafts a tree of N tokens per
sequence instead: appended at their depths, attended, and the branch of the
last one kept.
"""
from __future__ import annotations

import argparse
import math

import torch

import continuous_softmax_attention_gb300 as csa
from continuous_softmax_attention_gb300.inputs import make_inputs


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--B", type=int, default=1)
    ap.add_argument("--H", type=int, default=24)
    ap.add_argument("--T", type=int, default=8192)
    ap.add_argument("--d", type=int, default=128)
    ap.add_argument("--mode", type=int, default=0)
    ap.add_argument("--iters", type=int, default=2)
    ap.add_argument("--no-std", action="store_true")
    ap.add_argument("--decode", action="store_true")
    ap.add_argument("--backward", action="store_true")
    ap.add_argument("--short-conv", action="store_true",
                    help="the first-order (eq. (13)) form instead of the exact one")
    ap.add_argument("--log-domain", action="store_true",
                    help="the exact form's weights formed in the log domain")
    ap.add_argument("--paged", action="store_true")
    ap.add_argument("--kv-heads", type=int, default=0, help="cached heads (default: H)")
    ap.add_argument("--page", type=int, default=64, help="rows per page")
    ap.add_argument("--kind", choices=["bf16", "e4m3", "int8"], default="bf16", help="the cache's elements")
    ap.add_argument("--draft", type=int, default=0, help="drafted tokens per sequence and step (at most 64)")
    a = ap.parse_args()
    if a.paged:
        return run_paged(a)
    if a.decode:
        return run_decode(a)
    if a.backward:
        return run_backward(a)
    x = make_inputs(a.B, a.H, a.T, a.d, "bf16", seed=0)
    g = {k: v.cuda() for k, v in x.items()}
    scale = 1.0 / math.sqrt(a.d)
    for _ in range(a.iters):
        o, lse = csa.forward(g["q"], g["k"], g["v"], g["k0"], g["v0"], mode=a.mode, scale=scale,
                             short_conv=a.short_conv, log_domain=a.log_domain)
        if not a.no_std:
            csa.std_forward(g["q"], g["k"], g["v"], scale=scale)
    torch.cuda.synchronize()
    st = csa.device_status()
    print(f"ok status={st} o_mean={o.float().abs().mean().item():.5f}")
    if st != 0:
        raise SystemExit(1)


def run_backward(a):
    x = make_inputs(a.B, a.H, a.T, a.d, "bf16", seed=0)
    g = {k: v.cuda() for k, v in x.items()}
    scale = 1.0 / math.sqrt(a.d)
    o, lse = csa.forward(g["q"], g["k"], g["v"], g["k0"], g["v0"], mode=a.mode, scale=scale)
    dout = torch.randn(a.B, a.H, a.T, a.d, generator=torch.Generator().manual_seed(1))
    dout = dout.to(torch.bfloat16).cuda()
    for _ in range(a.iters):
        dq, dk, dv, _, _ = csa.backward(g["q"], g["k"], g["v"], o, lse, dout, g["k0"], g["v0"],
                                        mode=a.mode, scale=scale)
    torch.cuda.synchronize()
    st = csa.device_status()
    print(f"ok status={st} dq_mean={dq.float().abs().mean().item():.5f}")
    if st != 0:
        raise SystemExit(1)


def run_decode(a):
    from continuous_softmax_attention_gb300.inputs import make_decode_inputs

    x = make_decode_inputs(a.B, a.H, a.T, a.d, seed=0, len_lo=max(1, a.T // 2))
    g = {k: v.cuda() for k, v in x.items()}
    for _ in range(a.iters):
        o, lse = csa.decode(g["q"], g["k"], g["v"], g["k0"], g["v0"], seqlens=g["seqlens"],
                            mode=a.mode)
    torch.cuda.synchronize()
    st = csa.device_status()
    print(f"ok status={st} o_mean={o.float().abs().mean().item():.5f}")
    if st != 0:
        raise SystemExit(1)


def run_paged(a):
    kv, T = a.kv_heads or a.H, a.draft or 1
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(max(1, a.T // 2), a.T + 1, (a.B,), generator=g, dtype=torch.int32).cuda()
    M = -(-(a.T + a.iters * T) // a.page)
    P = a.B * M
    bf = lambda *shape: torch.randn(*shape, device="cuda", dtype=torch.bfloat16)
    k, v, x = bf(P, kv, a.page, a.d), bf(P, kv, a.page, a.d), bf(a.B, a.H + 2 * kv, T, a.d)
    cache = {}
    if a.kind != "bf16":
        k, v = ((t * 32).to(torch.float8_e4m3fn if a.kind == "e4m3" else torch.int8) for t in (k, v))
        cache["row_scales"] = torch.full((P, kv, a.page, 2), 1 / 32, device="cuda")
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    table = torch.full((a.B, M), -1, dtype=torch.int32, device="cuda")
    held = torch.zeros(a.B, dtype=torch.int32, device="cuda")
    new = torch.full((a.B,), T, dtype=torch.int32, device="cuda")
    sink = dict(k0=bf(kv, a.d), v0=bf(kv, a.d)) if a.mode == csa.GIVEN else {}
    plan = csa.RopeAxes(a.d, (a.d // 2,))
    # a tree with two continuations of each token
    depth = torch.tensor([int(math.log2(t + 1)) for t in range(T)], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[(t + 1) // 2 - 1 for t in range(T)]] * a.B, dtype=torch.int32, device="cuda")
    short = csa.cache_reserve(refs, table, held, a.page, lens)
    for _ in range(a.iters):
        short += csa.cache_reserve(refs, table, held, a.page, new)
        q = csa.cache_append(x[:, a.H:a.H + kv], x[:, a.H + kv:], k, v, table, held, rope=plan, q=x[:, :a.H],
                             positions=(held - T)[:, None] + depth if a.draft else None, **cache)
        if a.draft:
            o, lse = csa.decode_tree(q, k, v, table, held, parents, mode=a.mode, **sink, **cache)
            src, dst = csa.cache_accept(refs, table, held, a.page, new - 1, T, parents=parents)
            csa.cache_copy_rows(k, v, src, dst, **cache)
        else:
            o, lse = csa.decode_paged(q[:, :, 0], k, v, table, held, mode=a.mode, **sink, **cache)
    torch.cuda.synchronize()
    st = csa.device_status()
    print(f"ok status={st} short={short.item()} o_mean={o.float().abs().mean().item():.5f}")
    if st != 0 or short.item() != 0:
        raise SystemExit(1)


if __name__ == "__main__":
    main()
