"""The feed-forward half of a decode layer, as a serving loop runs it: the
attention's output joins the residual stream and is normed into 8-bit blocks,
the gated block and the down projection run on 4-bit weights, their output joins
the stream, and the next layer's norm leaves q8_0 slots for its QKV
projection.  Captured once in a graph and replayed for every token.

    python examples/decode_feed_forward.py [--live 16] [--steps 64] [--format mx8]

The layer is the Qwen3-14B-shaped one of ``workloads.py`` (5120 wide, 17408
inner features) with random weights and activations.  Prints the time of a step
and the bytes of its weights.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_weight_streaming_q8_amd as q8  # noqa: E402

HIDDEN, INNER, N_QKV, EPS = 5120, 17408, 7168, 1e-6


def mx4(n: int, k: int) -> q8.MX4Weights:
    w = q8.MX4Weights(n, k)
    q8.q8_mx4_pack_weights(torch.randn(n, k, device="cuda") * k ** -0.5, w)
    return w


class Layer:
    """Weights and buffers of one layer's feed-forward half and of the next
    layer's QKV projection, for ``live`` sessions."""

    def __init__(self, live: int, form: str):
        self.live = live
        self.gate, self.up, self.down = mx4(INNER, HIDDEN), mx4(INNER, HIDDEN), mx4(HIDDEN, INNER)
        self.wqkv = q8.empty_packed_weights(N_QKV, HIDDEN)
        q8.q8_pack_weights(torch.randn(N_QKV, HIDDEN, device="cuda") * 0.02, N_QKV, HIDDEN, self.wqkv)
        self.ws_qkv = q8.zeroed_workspace(N_QKV, HIDDEN)
        self.norms = [q8.Norm(HIDDEN, "rms", 1 + 0.1 * torch.randn(HIDDEN, device="cuda"), eps=EPS)
                      for _ in range(2)]
        self.x = q8.Acts(live, HIDDEN, form)
        self.h = q8.Acts(live, INNER, form)
        self.next = q8.Acts(q8.Q8_MAX_SLOTS, HIDDEN, "q8_0")
        self.slots = torch.arange(live, device="cuda").int()
        self.attended = torch.randn(live, HIDDEN, device="cuda")
        self.stream = torch.randn(live, HIDDEN, device="cuda")
        self.y = torch.empty(live, HIDDEN, device="cuda")
        self.qkv = torch.empty(live, N_QKV, device="cuda")

    def step(self) -> None:
        n = self.live
        q8.q8_norm_step(self.attended, n, HIDDEN, residual=self.stream, residual_out=self.stream, pre=self.norms[0],
                        acts=self.x)
        q8.q8_mx4_gated(self.gate, self.up, self.x, None, n, h_acts=self.h)
        q8.q8_mx4_matmul(self.down, self.h, None, n, self.y)
        q8.q8_norm_step(self.y, n, HIDDEN, residual=self.stream, residual_out=self.stream, pre=self.norms[1],
                        acts=self.next)
        q8.q8_matmul_narrow_ws(self.wqkv, self.next.data, self.slots, n, N_QKV, HIDDEN, self.qkv, self.ws_qkv)


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser()
    ap.add_argument("--live", type=int, default=16, help="sessions, 1..16")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--format", default="mx8", choices=("mx4", "mx6", "mx8"), help="of the activations")
    args = ap.parse_args(argv)
    if not 1 <= args.live <= q8.Q8_MAX_SLOTS or args.steps < 1:
        ap.error("--live has to be in 1..16 and --steps at least 1")
    torch.manual_seed(0)
    layer = Layer(args.live, args.format)
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
    weights = layer.gate.nbytes + layer.up.nbytes + layer.down.nbytes + layer.wqkv.nbytes
    out = {"live": args.live, "steps": args.steps, "format": args.format, "us_per_step": round(us, 2),
           "weights_MB_read": round(weights / 1e6, 1), "finite": bool(torch.isfinite(layer.qkv).all())}
    print(out)
    return out


if __name__ == "__main__":
    main()
