"""One decode step of a dense decoder layer, end to end on the library: norm with
the residual's addition, the NVFP4 projections, rotary positions with the write
into a paged cache, attention over it, and the gated MLP.

    python examples/decode_layer.py [--batch 16] [--tokens 1024] [--cache e4m3]

runs decode steps of a layer with random weights over a filled cache, replayed as
a CUDA graph while the sequences grow, and prints the time of a step.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w4a16_nvfp4_weight_gb300 as nv  # noqa: E402


class Cache:
    """A paged key-value cache and the table of each sequence's pages."""

    def __init__(self, batch, width, heads, page, head_dim, kind, dtype=torch.bfloat16):
        shape = (batch * width, heads, page, head_dim)
        dt = torch.float8_e4m3fn if kind == "e4m3" else dtype
        self.page = page
        self.rows = dict(k_cache=torch.zeros(shape, dtype=dt, device="cuda"), v_cache=torch.zeros(shape, dtype=dt, device="cuda"))
        if kind == "e4m3":
            for name in ("k_scale", "v_scale"):
                self.rows[name] = torch.ones(shape[:3], device="cuda")
        pages = torch.randperm(batch * width, device="cuda", dtype=torch.int32)
        self.table = pages.view(batch, width).contiguous()
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def slots(self, positions):
        """Slot of each sequence's token at its position."""
        page = torch.gather(self.table, 1, (positions // self.page)[:, None])[:, 0].long()
        return page * self.page + positions % self.page


class Layer:
    """Weights of one layer: qkv [(Hq + 2 Hkv) D, H], o [H, Hq D], fc1 [2I, H], fc2 [H, I]
    as NVFP4Weight, and the two norms' [H]."""

    def __init__(self, norm1, qkv, o, norm2, fc1, fc2, Hq, Hkv, D):
        self.norm1, self.qkv, self.o, self.norm2, self.fc1, self.fc2 = norm1, qkv, o, norm2, fc1, fc2
        self.Hq, self.Hkv, self.D = Hq, Hkv, D

    def step(self, h, residual, cache, table):
        """h, residual [B, H]: a new token of every sequence.  Appends its key and
        value to the cache and returns the layer's output and the residual."""
        B, Hq, Hkv = h.shape[0], self.Hq, self.Hkv
        x, residual = nv.rms_norm(h, self.norm1, residual=residual)
        qkv = nv.gemm(x, self.qkv).view(B, Hq + 2 * Hkv, self.D)
        positions = cache.lengths.long()
        cache.lengths += 1
        q = nv.rope_cache_write(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], positions, table,
                                slots=cache.slots(positions), **cache.rows)
        a = nv.paged_attention(q, block_table=cache.table, lengths=cache.lengths, **cache.rows)
        h = nv.gemm(a.view(B, Hq * self.D), self.o)
        x, residual = nv.rms_norm(h, self.norm2, residual=residual)
        return nv.mlp(x, self.fc1, self.fc2), residual


def random_weight(N, K, generator):
    """An NVFP4 weight with random codes, about N(0, 0.02)."""
    packed = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=generator)
    scales = torch.randint(0x30, 0x38, (N, K // 16), dtype=torch.uint8, device="cuda", generator=generator)   # E4M3 0.5 .. 0.94
    return nv.repack(packed, scales, 0.01, N, K, global_is_divisor=False)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--tokens", type=int, default=1024, help="tokens cached of each sequence at the start")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--cache", choices=("16", "e4m3"), default="e4m3")
    a = ap.parse_args()
    H, I, Hq, Hkv, D, page = 4096, 14336, 32, 8, 128, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    ones = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    layer = Layer(ones, random_weight((Hq + 2 * Hkv) * D, H, g), random_weight(H, Hq * D, g), ones,
                  random_weight(2 * I, H, g), random_weight(H, I, g), Hq, Hkv, D)
    most = a.tokens + a.steps + 8
    cache = Cache(a.batch, -(-most // page), Hkv, page, D, a.cache)
    table = nv.rope_table(most, D)
    # a filled cache: random keys and values of the first tokens, written as a prompt would
    for b in range(a.batch):
        t = torch.arange(a.tokens, device="cuda")
        kv = torch.randn(a.tokens, 2 * Hkv, D, device="cuda", generator=g).bfloat16()
        slots = cache.table[b].long()[t // page] * page + t % page
        nv.rope_cache_write(kv[:, :Hkv], kv[:, :Hkv], kv[:, Hkv:], t, table, slots=slots, **cache.rows)
    cache.lengths += a.tokens
    h = torch.randn(a.batch, H, device="cuda", generator=g).bfloat16()
    residual = torch.zeros_like(h)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(3):
            layer.step(h, residual, cache, table)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out, _ = layer.step(h, residual, cache, table)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(a.steps):
            graph.replay()
        end.record()
    end.synchronize()
    assert nv.device_status() == 0 and bool(out.isfinite().all())
    print(f"{a.batch} sequences, {int(cache.lengths[0])} tokens each, {a.cache} cache: "
          f"{start.elapsed_time(end) * 1e3 / a.steps:.1f} us a layer step")


if __name__ == "__main__":
    main()
