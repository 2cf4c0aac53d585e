"""Decode steps of a small hybrid stack: KDA layers with a full attention layer
behind every third, on the library's operators.

    python examples/hybrid_decode.py            # builds the libraries if needed; wants a GB300

A KDA layer:        x -> q, k, v, gates -> kda_decode_step -> kda_head_norm -> projection
An attention layer: x -> q, k, v -> kda_kv4_append -> kda_kv4_attend -> projection
Between blocks:     kda_block_norm: the block's output is normed, gated, scaled
                    and added to the residual stream, and the next block's
                    input is the norm of that

Projections are plain library matrix products.  A step is captured into one CUDA
graph; contexts grow in place (ctx_len is incremented on the device).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_linear_attention_gated_gb300 as kda  # noqa: E402


class HybridStack:
    """Random weights; `n` requests, each with its own state slot and pages."""

    def __init__(self, n=8, layers=4, hidden=512, hv=4, dim=128, h_q=8, h_kv=2, page=64, max_len=512, seed=0, device="cuda"):
        self.n, self.hidden, self.hv, self.dim, self.h_q, self.h_kv = n, hidden, hv, dim, h_q, h_kv
        self.lib = kda.KdaLibrary(torch.float32)
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g) * cols ** -0.5).to(torch.bfloat16).to(device)

        def near_one(m):
            return (1 + 0.1 * torch.randn(m, generator=g)).to(device)

        f32, bf, i32 = torch.float32, torch.bfloat16, torch.int32
        cols = -(-max_len // page)
        self.layers = []
        for i in range(layers):
            attention = i % 3 == 2
            w = {"attention": attention, "post": near_one(hidden), "pre": near_one(hidden), "gate": weight(hidden, hidden)}
            if attention:
                width = (h_q + 2 * h_kv) * dim
                w["in"], w["out"] = weight(width, hidden), weight(hidden, h_q * dim)
                w["pages"] = torch.zeros(n * cols, h_kv, page // 16, 18 * dim, dtype=torch.uint8, device=device)
            else:
                width = 4 * hv * dim       # q, k, v and the output gate
                w["in"], w["out"] = weight(width, hidden), weight(hidden, hv * dim)
                w["decay"], w["beta"] = weight(hv * dim, hidden), weight(hv, hidden)
                w["norm"] = near_one(dim)
                w["pool"] = torch.zeros(n, hv, dim, dim, dtype=f32, device=device)
            self.layers.append(w)
        self.first = near_one(hidden)
        self.slots = torch.randperm(n, generator=g).to(i32).to(device)
        self.table = torch.randperm(n * cols, generator=g).to(i32).view(n, cols).to(device)
        self.ctx = torch.zeros(n, dtype=i32, device=device)
        f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
        angle = torch.arange(max_len, dtype=torch.float64)[:, None] * f
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)
        self.status = torch.zeros(1, dtype=i32, device=device)
        self.workspace = torch.zeros(kda.KDA_KV4_WORKSPACE_BYTES, dtype=torch.uint8, device=device)
        self.x = torch.zeros(n, hidden, dtype=bf, device=device)          # a step's input
        self.residual = torch.empty(n, hidden, dtype=f32, device=device)
        self.h = torch.empty(n, hidden, dtype=bf, device=device)          # a block's input; at last the step's output

    def step(self, flags=0) -> torch.Tensor:
        """One token of every request: self.x in, the normed last hidden state out."""
        n, L = self.n, self.lib
        self.residual.copy_(self.x)
        L.kda_block_norm(self.residual, None, None, w_pre=self.first, x=self.h, flags=flags)
        for w in self.layers:
            p = self.h @ w["in"].T
            if w["attention"]:
                p = p.view(n, -1, self.dim)
                q, k, v = p[:, :self.h_q], p[:, self.h_q:self.h_q + self.h_kv], p[:, self.h_q + self.h_kv:]
                o = torch.empty(n, self.h_q, self.dim, dtype=torch.bfloat16, device=q.device)
                L.kda_kv4_append(w["pages"], self.table, self.ctx, k, v, self.status, cos=self.cos, sin=self.sin, flags=flags)
                L.kda_kv4_attend(w["pages"], self.table, self.ctx, q, o, self.workspace, self.status, cos=self.cos, sin=self.sin, flags=flags)
            else:
                p = p.view(n, 4, self.hv, self.dim)
                q, k, v = (p[:, i].contiguous() for i in range(3))
                decay = (self.h @ w["decay"].T).float().view(n, self.hv, self.dim)
                beta = (self.h @ w["beta"].T).float()
                raw = torch.empty(n, self.hv, self.dim, device=q.device)
                L.kda_decode_step(w["pool"], self.slots, q, k, v, decay, beta, raw, self.status)
                o = torch.empty(n, self.hv, self.dim, dtype=torch.bfloat16, device=q.device)
                L.kda_head_norm(raw, w["norm"], o, gate=p[:, 3], flags=flags)
            y = o.view(n, -1) @ w["out"].T
            L.kda_block_norm(self.residual, y, self.residual, w_post=w["post"], gate=self.h @ w["gate"].T, w_pre=w["pre"], x=self.h,
                             branch_scale=0.5, flags=flags)
        self.ctx += 1
        return self.h

    def capture(self) -> torch.cuda.CUDAGraph:
        """The step as a graph; the warm-up step it takes is undone (states, pages behind ctx_len and ctx_len itself)."""
        keep = [w["pool"].clone() for w in self.layers if not w["attention"]]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
            self.ctx -= 1
            for w, pool in zip((w for w in self.layers if not w["attention"]), keep):
                w["pool"].copy_(pool)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def main() -> None:
    kda.build()
    stack = HybridStack(n=64, layers=6, hidden=1536, hv=12, h_q=12, max_len=1024)
    graph = stack.capture()
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    steps = 200
    for i in range(steps + 20):
        if i == 20:
            start.record()
        stack.x.copy_(stack.h)       # a model would embed the sampled token here
        graph.replay()
    stop.record()
    torch.cuda.synchronize()
    assert stack.status.item() == 0
    print(f"{len(stack.layers)} layers, {stack.n} requests, contexts up to {stack.ctx.max().item()} tokens: "
          f"{start.elapsed_time(stop) / steps * 1e3:.1f} us a step")


if __name__ == "__main__":
    main()
