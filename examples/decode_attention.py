"""The attention half of a decode layer, as a serving loop runs it: QKV
projection, append with rotary positions, attention over the paged 4-bit
cache, O projection, captured once in a graph and replayed for every token.

    python examples/decode_attention.py [--live 16] [--context 4096] [--steps 64]

The layer is the Qwen3-14B-shaped one of ``workloads.py`` (5120 wide, 40 query
and 8 key/value heads of 128) with random weights and activations.  Each
session gets a prompt's worth of random keys and values first, put into the
cache by the same append.  Prints the time of a step and what its parts read.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_weight_streaming_q8_amd as q8  # noqa: E402

HIDDEN, N_Q, N_KV, DIM, BASE, PAGE = 5120, 40, 8, 128, 1e6, 64
N_QKV = (N_Q + 2 * N_KV) * DIM


def packed(n: int, k: int) -> torch.Tensor:
    w = q8.empty_packed_weights(n, k)
    q8.q8_pack_weights(torch.randn(n, k, device="cuda") * 0.02, n, k, w)
    return w


class Layer:
    """Weights, cache and buffers of one layer for ``live`` sessions of up to
    ``capacity`` tokens."""

    def __init__(self, live: int, capacity: int):
        self.live = live
        self.wqkv, self.wo = packed(N_QKV, HIDDEN), packed(HIDDEN, N_Q * DIM)
        self.ws_qkv = q8.zeroed_workspace(N_QKV, HIDDEN)
        self.ws_o = q8.zeroed_workspace(HIDDEN, N_Q * DIM)
        pages = -(-capacity // PAGE)
        table = torch.randperm(live * pages, device="cuda").int().reshape(live, pages)
        self.cache = q8.KV4Cache(live * pages, PAGE, N_KV, DIM, table)
        self.rotary = q8.rotary_plan(DIM, base=BASE)
        self.ws_attend = q8.kv4_attend_workspace(self.cache, live, 1, N_Q)
        self.slots = torch.arange(live, device="cuda").int()  # activation slots and cache slots
        self.pos = torch.zeros(live, dtype=torch.int32, device="cuda")
        self.x = torch.randn(live, HIDDEN, device="cuda")
        self.xq, self.aq = q8.empty_act_slots(HIDDEN), q8.empty_act_slots(N_Q * DIM)
        self.qkv = torch.empty(live, N_QKV, device="cuda")
        self.q = torch.empty(live, N_Q * DIM, device="cuda")
        self.attended = torch.empty(live, N_Q * DIM, device="cuda")
        self.y = torch.empty(live, HIDDEN, device="cuda")

    def prompt(self, tokens: int) -> None:
        """Random keys and values at positions 0 .. tokens - 1 of every session."""
        width = 2 * N_KV * DIM
        for s in range(self.live):
            at = torch.arange(tokens, device="cuda").int()
            q8.q8_kv4_append(self.cache, torch.randn(tokens, width, device="cuda"), tokens, width,
                             torch.full_like(at, s), at, rotary=self.rotary)
        self.pos.fill_(tokens)

    def step(self) -> None:
        n = self.live
        q8.q8_quantize_acts(self.x, n, HIDDEN, self.xq)
        q8.q8_matmul_narrow_ws(self.wqkv, self.xq, self.slots, n, N_QKV, HIDDEN, self.qkv, self.ws_qkv)
        q8.q8_kv4_append(self.cache, self.qkv, n, N_QKV, self.slots, self.pos, rotary=self.rotary,
                         n_q_heads=N_Q, Q=self.q)
        q8.q8_kv4_attend(self.cache, self.q, n, 1, N_Q, self.slots, self.pos, self.attended, self.ws_attend)
        q8.q8_quantize_acts(self.attended, n, N_Q * DIM, self.aq)
        q8.q8_matmul_narrow_ws(self.wo, self.aq, self.slots, n, HIDDEN, N_Q * DIM, self.y, self.ws_o)
        self.pos.add_(1)


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser()
    ap.add_argument("--live", type=int, default=16, help="sessions, 1..16")
    ap.add_argument("--context", type=int, default=4096, help="tokens cached before the first step")
    ap.add_argument("--steps", type=int, default=64)
    args = ap.parse_args(argv)
    if not 1 <= args.live <= q8.Q8_MAX_SLOTS or args.context < 1 or args.steps < 1:
        ap.error("--live has to be in 1..16, --context and --steps at least 1")
    torch.manual_seed(0)
    layer = Layer(args.live, args.context + args.steps + 2)
    layer.prompt(args.context)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.step()  # warm up
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = begin.elapsed_time(end) * 1e3 / args.steps
    cached = args.live * args.context * layer.cache.page_bytes // PAGE
    out = {"live": args.live, "context": args.context, "steps": args.steps, "us_per_step": round(us, 2),
           "cache_MB_read": round(cached / 1e6, 1), "finite": bool(torch.isfinite(layer.y).all()),
           "position": int(layer.pos[0])}
    print(out)
    return out


if __name__ == "__main__":
    main()
