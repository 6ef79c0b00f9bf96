"""examples/decode_layer.py against the 64-bit oracle: a few decode steps of a small
layer over both cache kinds.

Each stage's output is rounded to BF16 on both sides (2^-8 relative at most, about
2^-9.2 root mean square); the eight roundings of a step, and their passage through
the next stages, stay below 2^-6 of the output's norm."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import dense, formats, layer as olayer, moe as omoe
from tests import gpu_util as gu
from w4a16_nvfp4_weight_gb300 import synth
import w4a16_nvfp4_weight_gb300 as nv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(lib):
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _bf16(x):
    return formats.bf16_to_float(formats.bf16_bits(x))


@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_decode_layer_matches_the_oracle(example, kind):
    B, H, I, Hq, Hkv, D, page, steps = 3, 256, 128, 4, 2, 64, 4, 7
    r = synth.rng(41)
    raw = {n: synth.quantize(synth.normal_weight(r, N, K)) for n, (N, K) in
           dict(qkv=((Hq + 2 * Hkv) * D, H), o=(H, Hq * D), fc1=(2 * I, H), fc2=(H, I)).items()}
    dev = {n: nv.repack(gu.u8(w[0]), gu.u8(w[1]), float(w[2]), w[0].shape[0], w[0].shape[1] * 2) for n, w in raw.items()}
    norms = [1 + 0.1 * r.standard_normal(H) for _ in range(2)]
    norm_bits = [formats.bf16_bits(n) for n in norms]
    lay = example.Layer(gu.bits_to_bf16_tensor(norm_bits[0]), dev["qkv"], dev["o"], gu.bits_to_bf16_tensor(norm_bits[1]),
                        dev["fc1"], dev["fc2"], Hq, Hkv, D)
    cache = example.Cache(B, 4, Hkv, page, D, kind)
    table = nv.rope_table(32, D)
    tn = table.cpu().numpy()
    start = torch.tensor([0, 1, 5], dtype=torch.int32, device="cuda")
    held = [[], [], []]                                       # (k, v) of each sequence's tokens, as cached

    def stored(x):
        if kind == "16":
            return _bf16(x)
        codes, s = olayer.quantise(x)
        return codes * s[..., None].astype(np.float64)

    for b, n in enumerate(start.tolist()):                    # a prefix, written by the library
        if n:
            kv = torch.from_numpy(r.standard_normal((n, 2 * Hkv, D)).astype(np.float32)).cuda().bfloat16()
            t = torch.arange(n, device="cuda")
            slots = cache.table[b].long()[t // page] * page + t % page
            nv.rope_cache_write(kv[:, :Hkv], kv[:, :Hkv], kv[:, Hkv:], t, table, slots=slots, **cache.rows)
            f = kv.float().cpu().numpy()
            k = stored(olayer.rope(f[:, :Hkv], np.arange(n)[None], tn))
            held[b] = [(k[i], stored(f[:, Hkv:])[i]) for i in range(n)]
    cache.lengths.copy_(start)

    res_dev = torch.zeros(B, H, dtype=torch.bfloat16, device="cuda")
    for _ in range(steps):
        h = _bf16(r.standard_normal((B, H)))
        out, res = lay.step(gu.bits_to_bf16_tensor(formats.bf16_bits(h)), res_dev, cache, table)
        res_ref = _bf16(h)
        x = formats.bf16_bits(olayer.rms_norm(res_ref, formats.bf16_to_float(norm_bits[0]), 1e-6))
        qkv = formats.bf16_to_float(dense.linear(x, *raw["qkv"], True)[1]).reshape(B, Hq + 2 * Hkv, D)
        pos = np.array([[len(s) for s in held]])
        q = _bf16(olayer.rope(qkv[:, :Hq].astype(np.float32), pos, tn))
        k = stored(olayer.rope(qkv[:, Hq:Hq + Hkv].astype(np.float32), pos, tn))
        v = stored(qkv[:, Hq + Hkv:].astype(np.float32))
        att = np.empty((B, Hq * D))
        for b in range(B):
            held[b].append((k[b], v[b]))
            att[b] = olayer.attend(q[b], np.stack([t[0] for t in held[b]]), np.stack([t[1] for t in held[b]]), D ** -0.5)[0].reshape(-1)
        o = formats.bf16_to_float(dense.linear(formats.bf16_bits(att), *raw["o"], True)[1])
        res_ref = _bf16(o + res_ref)
        x = formats.bf16_bits(olayer.rms_norm(res_ref, formats.bf16_to_float(norm_bits[1]), 1e-6))
        ref = formats.bf16_to_float(omoe.mlp(x, (*raw["fc1"], True), (*raw["fc2"], True))[1])
        for got, want in ((out, ref), (res, res_ref)):
            g = got.double().cpu().numpy()
            assert np.all(np.isfinite(g))
            assert np.linalg.norm(g - want) <= 2.0 ** -6 * np.linalg.norm(want)
    assert cache.lengths.tolist() == [len(s) for s in held]
    gu.check_device_status()
