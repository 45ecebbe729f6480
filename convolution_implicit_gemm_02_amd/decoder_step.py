"""A small decoder on low-bit numbers, which runs the operators of llm.py together as a server would: RMS norm with the residual,
products on 4-bit weights with int8 rows, keys and values into a paged int8 cache, attention over it.  Prompts go in chunks; the
step of one new token a sequence is captured into a graph, whose lengths, slots and rows stay on the GPU.

    python -m convolution_implicit_gemm_02_amd.decoder_step --layers 8 --seqs 8 --prompt 1000 --tokens 64

Weights are random and there is neither a vocabulary nor a position encoding: a step's output rows are the next step's input,
scaled to unit size.
"""
from __future__ import annotations

import argparse
import time
from dataclasses import dataclass

import torch

from . import llm


@dataclass
class Config:
    hidden: int = 2048
    heads: int = 16
    kv_heads: int = 4
    head_dim: int = 128
    ffn: int = 8192
    layers: int = 8
    group: int = 128
    page: int = 32
    window: int = 0


def pack4(w, group=128, scale_dtype=torch.float16):
    """4-bit codes [n][round_up(ceil(k / 2), 16)] and scales [ceil(k / group)][n] of a weight [n][k], zero point 8: the layout of
    cbs_w4_linear.  A group's largest magnitude is 7 steps."""
    n, k = w.shape
    groups = -(-k // group)
    parts = torch.nn.functional.pad(w.float(), (0, groups * group - k)).view(n, groups, group)
    scales = (parts.abs().amax(2) / 7).to(scale_dtype)
    step = scales.float()
    codes = (parts / torch.where(step == 0, 1.0, step)[..., None]).round_().clamp_(-8, 7).add_(8).to(torch.uint8).view(n, -1)
    wide = -(-k // 32) * 32
    codes = torch.nn.functional.pad(codes, (0, max(0, wide - codes.shape[1])), value=8)[:, :wide]
    return (codes[:, 0::2] | codes[:, 1::2] << 4).contiguous(), scales.t().contiguous()


class Decoder:
    """Weights, caches and workspaces of a stack of blocks for up to max_seqs sequences of up to max_len tokens, max_rows new
    tokens a step in all."""

    def __init__(self, cfg: Config, max_seqs, max_len, max_rows, seed=0):
        self.cfg, self.max_seqs = cfg, max_seqs
        c, dev = cfg, torch.device("cuda")
        g = torch.Generator(device=dev).manual_seed(seed)
        qkv, both = (c.heads + 2 * c.kv_heads) * c.head_dim, c.heads * c.head_dim
        self.sizes = {"qkv": (c.hidden, qkv), "o": (both, c.hidden), "up": (c.hidden, 2 * c.ffn), "down": (c.ffn, c.hidden)}

        def weight(k, n):
            return pack4(torch.randn(n, k, generator=g, device=dev) * k**-0.5, c.group)

        def norm():
            return (1 + 0.1 * torch.randn(c.hidden, generator=g, device=dev)).bfloat16()

        columns = -(-max_len // c.page)
        pages = max_seqs * columns
        self.table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(max_seqs, columns)
        self.kv_len = torch.zeros(max_seqs, dtype=torch.int32, device=dev)
        self.layers = [dict({name: weight(k, n) for name, (k, n) in self.sizes.items()}, norm1=norm(), norm2=norm(),
                            k=torch.zeros(pages, c.kv_heads, c.page, c.head_dim, dtype=torch.int8, device=dev),
                            v=torch.zeros(pages, c.kv_heads, c.head_dim, c.page, dtype=torch.int8, device=dev),
                            ks=torch.zeros(pages, c.kv_heads, c.page, device=dev), vs=torch.zeros(pages, c.kv_heads, c.page, device=dev))
                       for _ in range(c.layers)]
        self.last = norm()
        # Descriptors, the attention's workspace and the buffers between the operators: made once.
        self.to_i8 = llm.make_rms_desc(c.hidden, dtype=llm.CBS_BF16, out_dtype=llm.CBS_I8)
        self.to_bf16 = llm.make_rms_desc(c.hidden, dtype=llm.CBS_BF16)
        self.w4 = {name: llm.make_w4_desc(k, n, c.group, dtype=llm.CBS_I8 if name in ("qkv", "up") else llm.CBS_BF16) for name, (k, n) in self.sizes.items()}
        self.kv = llm.make_kv_desc(c.kv_heads, c.head_dim, c.page)
        self.attn = llm.cbs_attn_create(llm.make_attn_desc(c.heads, c.kv_heads, c.head_dim, c.page, window=c.window, max_seqs=max_seqs))
        self.codes = torch.empty(max_rows, c.hidden, dtype=torch.int8, device=dev)
        self.scale = torch.empty(max_rows, device=dev)
        self.rows = {name: torch.empty(max_rows, n, dtype=torch.bfloat16, device=dev) for name, (_, n) in self.sizes.items()}
        self.heads_out = torch.empty(max_rows, c.heads, c.head_dim, dtype=torch.bfloat16, device=dev)
        self.sum = torch.empty(max_rows, c.hidden, dtype=torch.bfloat16, device=dev)
        self.gated = torch.empty(max_rows, c.ffn, dtype=torch.bfloat16, device=dev)
        self.out = torch.empty(max_rows, c.hidden, dtype=torch.bfloat16, device=dev)

    def slots(self, seq, place):
        """Cache slots of sequences' places (tensors of one shape on the GPU); past max_len's pages -1, which is not written."""
        page, columns = self.cfg.page, self.table.shape[1]
        column = place // page
        return torch.where(column < columns, self.table[seq, column.clamp(max=columns - 1)].long() * page + place % page, -1)

    def forward(self, x, q_start, kv_len, table, slots, max_new, max_kv):
        """The blocks over rows x of new tokens, whose keys and values go to `slots`; returns a buffer's rows."""
        c, n = self.cfg, x.shape[0]
        codes, scale, heads_out, hidden = self.codes[:n], self.scale[:n], self.heads_out[:n], self.sum[:n]
        qkv, o, up, down = (self.rows[name][:n] for name in ("qkv", "o", "up", "down"))
        q, k, v = qkv.view(n, -1, c.head_dim).split((c.heads, c.kv_heads, c.kv_heads), 1)
        residual, added = None, x
        for at in self.layers:
            llm.cbs_rms_norm(self.to_i8, added, at["norm1"], codes, residual=residual, residual_out=None if residual is None else hidden, out_scale=scale)
            llm.cbs_w4_linear(self.w4["qkv"], codes, *at["qkv"], qkv, x_scale=scale)
            llm.cbs_kv_write(self.kv, k, v, slots, at["k"], at["v"], at["ks"], at["vs"])
            llm.cbs_attn_run(self.attn, q, q_start, kv_len, table, at["k"], at["v"], heads_out, at["ks"], at["vs"], max_new=max_new, max_kv=max_kv)
            llm.cbs_w4_linear(self.w4["o"], heads_out.view(n, -1), *at["o"], o)
            llm.cbs_rms_norm(self.to_i8, o, at["norm2"], codes, residual=x if residual is None else residual, residual_out=hidden, out_scale=scale)
            residual = hidden
            llm.cbs_w4_linear(self.w4["up"], codes, *at["up"], up, x_scale=scale)
            gate, values = up.split(c.ffn, 1)
            torch.mul(torch.nn.functional.silu(gate), values, out=self.gated[:n])
            llm.cbs_w4_linear(self.w4["down"], self.gated[:n], *at["down"], down)
            added = down
        out = self.out[:n]
        llm.cbs_rms_norm(self.to_bf16, added, self.last, out, residual=residual)
        return out

    def prompt(self, seq, x, chunk=512):
        """A sequence's rows x in chunks after what is cached of it; returns the last row."""
        have, last = int(self.kv_len[seq]), None
        if have + x.shape[0] > self.table.shape[1] * self.cfg.page:
            raise ValueError("%d tokens after %d: there is room for %d" % (x.shape[0], have, self.table.shape[1] * self.cfg.page))
        for at in range(0, x.shape[0], chunk):
            part = x[at : at + chunk]
            n, first = part.shape[0], have + at
            place = torch.arange(first, first + n, device=x.device)
            last = self.forward(part, torch.tensor([0, n], dtype=torch.int32, device=x.device), torch.tensor([first + n], dtype=torch.int32, device=x.device),
                                self.table[seq : seq + 1], self.slots(torch.full_like(place, seq), place), n, first + n)[-1].clone()
        self.kv_len[seq] = have + x.shape[0]
        return last

    def single(self, rows):
        """One new token in every sequence: rows [max_seqs][hidden] become the outputs.  Lengths and slots are computed on the
        GPU, so that the call can be captured and replayed.  A sequence that has no room left keeps what is cached, and its lengths."""
        seq = torch.arange(self.max_seqs, device=rows.device)
        slots = self.slots(seq, self.kv_len.long())
        self.kv_len.add_(1).clamp_(max=self.table.shape[1] * self.cfg.page)
        starts = torch.arange(self.max_seqs + 1, dtype=torch.int32, device=rows.device)
        rows.copy_(self.forward(rows, starts, self.kv_len, self.table, slots, 1, self.table.shape[1] * self.cfg.page))

    def cached(self, layer, seq):
        """What a layer's cache holds of a sequence: keys and values [tokens][kv_heads][head_dim]."""
        at, place = self.layers[layer], torch.arange(int(self.kv_len[seq]), device=self.table.device)
        k = torch.empty(len(place), self.cfg.kv_heads, self.cfg.head_dim, dtype=torch.bfloat16, device=place.device)
        v = torch.empty_like(k)
        llm.cbs_kv_read(self.kv, self.slots(torch.full_like(place, seq), place), at["k"], at["v"], k, v, at["ks"], at["vs"])
        return k, v


def capture(decoder, rows):
    """A graph of single(rows), captured on a stream of its own."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        decoder.single(rows)
    torch.cuda.current_stream().wait_stream(side)
    return graph


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("layers", 8), ("seqs", 8), ("prompt", 1000), ("tokens", 64), ("hidden", 2048), ("heads", 16), ("kv-heads", 4), ("head-dim", 128), ("ffn", 8192)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    cfg = Config(hidden=a.hidden, heads=a.heads, kv_heads=a.kv_heads, head_dim=a.head_dim, ffn=a.ffn, layers=a.layers)
    decoder = Decoder(cfg, a.seqs, a.prompt + a.tokens + 2, max(512, a.seqs))
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randn(a.seqs, a.prompt, a.hidden, generator=g, device="cuda").bfloat16()
    rows = torch.empty(a.seqs, a.hidden, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for s in range(a.seqs):
        rows[s] = decoder.prompt(s, prompts[s])
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    decoder.single(rows)  # once before the capture: it loads the kernels
    graph = capture(decoder, rows)
    graph.replay()
    torch.cuda.synchronize()
    t2 = time.perf_counter()
    for _ in range(a.tokens):
        graph.replay()
    torch.cuda.synchronize()
    t3 = time.perf_counter()
    print("prompts: %d tokens in %.1f ms;  single tokens: %.0f us a step, %.0f tokens/s;  rows finite: %s"
          % (a.seqs * a.prompt, (t1 - t0) * 1e3, (t3 - t2) / a.tokens * 1e6, a.seqs * a.tokens / (t3 - t2), bool(rows.isfinite().all())))


if __name__ == "__main__":
    main()
