"""A served batch from its prompts to its last tokens, with everything that differs from
request to request on the device: pages, adapters, sampling.

    python examples/serve_batch.py [--requests 16] [--steps 32]

One attention layer with an NVFP4 projection between an embedding and an NVFP4 head, all
with random weights.  The prompts run as one ragged batch, in which every token attends
through a table of its own; then each step takes one token of every request, in a CUDA
graph: room in the cache, the layer with the requests' adapters, the next token.  A request
that draws the end token gives its pages back.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w4a16_nvfp4_weight_gb300 as nv  # noqa: E402
from examples.decode_layer import random_weight  # noqa: E402


class Batch:
    """Requests of one batch: their page tables, adapters and settings."""

    def __init__(self, requests, width, pages, page, adapters, temperature, top_k, top_p):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.page = page
        self.lengths, self.table = torch.zeros(requests, **i32), torch.zeros(requests, width, **i32)
        self.free_pages, self.free_count = torch.randperm(pages, device="cuda", dtype=torch.int32), torch.tensor([pages], **i32)
        self.adapters = adapters
        self.how = dict(temperature=temperature, top_k=top_k, top_p=top_p)

    def extend(self, new_tokens, rows, row_tables=False):
        return nv.extend_tables(self.lengths, new_tokens, self.table, self.free_pages, self.free_count, self.page, rows,
                                row_tables=row_tables, in_place=True)

    def end(self, ended):
        """Requests where `ended` is true keep no token."""
        keep = torch.where(ended, 0, self.lengths)
        nv.trim_tables(self.lengths, keep, self.table, self.free_pages, self.free_count, self.page, in_place=True)


class Model:
    """Embedding, norm, qkv with adapters, attention, output projection, head."""

    def __init__(self, V, H, Hq, Hkv, D, rank, adapters, most, g):
        def randn(*shape, std=1.0):
            return (torch.randn(shape, device="cuda", generator=g) * std).bfloat16()
        N = (Hq + 2 * Hkv) * D
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.embedding, self.norm = randn(V, H), torch.ones(H, dtype=torch.bfloat16, device="cuda")
        self.qkv, self.o, self.head = random_weight(N, H, g), random_weight(H, Hq * D, g), random_weight(V, H, g)
        self.a, self.b = randn(adapters, rank, H, std=H ** -0.5), randn(adapters, N, rank, std=0.1)
        self.rope = nv.rope_table(most, D)

    def logits(self, tokens, adapters, positions, slots, table, lengths, cache):
        """Rows of tokens (-1: none), each with its adapter, position, slot, page table and length."""
        h = self.embedding[tokens.clamp(min=0)]
        x = nv.rms_norm(h, self.norm)
        y = nv.gemm(x, self.qkv)
        qkv = nv.lora_add(y, x, self.a, self.b, adapters, out=y).view(-1, self.Hq + 2 * self.Hkv, self.D)
        q = nv.rope_cache_write(qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hkv], qkv[:, self.Hq + self.Hkv:], positions,
                                self.rope, slots=slots, **cache)
        o = nv.paged_attention(q, block_table=table, lengths=lengths, **cache)
        h = h + nv.gemm(o.view(-1, self.Hq * self.D), self.o)
        return nv.gemm(nv.rms_norm(h, self.norm), self.head)


def prefill(model, batch, cache, prompts, u):
    """The prompts (lists of tokens) as one batch of rows; the first token of each request (-1: no
    prompt, or no room for it)."""
    new = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    tokens = torch.tensor([t for p in prompts for t in p], device="cuda")
    t = batch.extend(new, tokens.numel(), row_tables=True)
    logits = model.logits(tokens, batch.adapters[t["request"].long()], t["positions"], t["slots"], t["row_tables"], t["row_lengths"], cache)
    last = logits[(t["starts"][1:] - 1).clamp(min=0).long()]
    return torch.where(batch.lengths > 0, nv.sample(last, u, **batch.how), -1)


def step(model, batch, cache, tokens, u, end_token):
    """One token of every request that has not ended; the next ones (-1: ended, by the end token
    or because there was no page left for it)."""
    running = tokens >= 0
    t = batch.extend(running.int(), tokens.numel())
    # rows of the requests that run come first; the rest of them store and attend to nothing
    row = t["request"].long()
    valid = row >= 0
    row = row.clamp(min=0)
    lengths = torch.where(valid, batch.lengths[row], 0)
    logits = model.logits(torch.where(valid, tokens[row], -1), torch.where(valid, batch.adapters[row], -1), t["positions"], t["slots"],
                          batch.table[row], lengths, cache)
    drawn = nv.sample(logits, u, **{k: v[row] for k, v in batch.how.items()})
    drawn = torch.where(t["slots"] >= 0, drawn, end_token)   # without room: its token went nowhere
    out = tokens.new_full((tokens.numel() + 1,), -1)         # the last: for rows behind the running requests'
    out.scatter_(0, torch.where(valid, row, tokens.numel()), drawn)
    out = torch.where(running, out[:-1], -1)
    ended = out == end_token
    batch.end(ended)
    return torch.where(ended, -1, out)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    V, H, Hq, Hkv, D, page, adapters = 32768, 2048, 16, 4, 128, 16, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    model = Model(V, H, Hq, Hkv, D, 16, adapters, 1024, g)
    n, width = a.requests, 1024 // page
    batch = Batch(n, width, n * 16, page, torch.arange(n, device="cuda", dtype=torch.int32) % (adapters + 1) - 1,
                  torch.linspace(0.0, 1.2, n, device="cuda"), torch.full((n,), 50, dtype=torch.int32, device="cuda"),
                  torch.full((n,), 0.95, device="cuda"))
    cache = {k: torch.zeros(n * 16, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for k in ("k_cache", "v_cache")}
    prompts = [torch.randint(0, V, (7 + 5 * i % 60,)).tolist() for i in range(n)]
    u = torch.rand(n, device="cuda")
    tokens = prefill(model, batch, cache, prompts, u)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        tokens = step(model, batch, cache, tokens, u, 0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            tokens.copy_(step(model, batch, cache, tokens, u, 0))
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(a.steps):
            u.uniform_()
            graph.replay()
        end.record()
    end.synchronize()
    assert nv.device_status() == 0
    held = int(((batch.lengths + page - 1) // page).sum())
    assert held + int(batch.free_count) == n * 16
    print(f"{n} requests, {int((tokens >= 0).sum())} still running with {int(batch.lengths.max())} tokens at most: "
          f"{start.elapsed_time(end) * 1e3 / a.steps:.1f} us a step")


if __name__ == "__main__":
    main()
