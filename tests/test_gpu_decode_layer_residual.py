"""One decode step of examples/decode_layer.py from a residual that is not zero, into
an empty cache: each sequence attends to its one token, so the attention's output is
that token's value.

Bounds as in test_gpu_decode_layer.py: each stage is rounded to BF16 on both sides, and
the eight roundings of a step stay below 2^-6 of the output's norm."""

import numpy as np
import pytest
import torch

import w4a16_nvfp4_weight_gb300 as nv
from oracle import dense, formats, layer as olayer, moe as omoe
from tests import gpu_util as gu
from tests.test_gpu_decode_layer import _bf16, example  # noqa: F401 (a fixture)
from w4a16_nvfp4_weight_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_a_step_adds_its_residual(example, kind):  # noqa: F811
    B, H, I, Hq, Hkv, D = 5, 256, 128, 4, 2, 64
    r = synth.rng(43)
    raw = {n: synth.quantize(synth.normal_weight(r, N, K)) for n, (N, K) in
           dict(qkv=((Hq + 2 * Hkv) * D, H), o=(H, Hq * D), fc1=(2 * I, H), fc2=(H, I)).items()}
    dev = {n: nv.repack(gu.u8(w[0]), gu.u8(w[1]), float(w[2]), w[0].shape[0], w[0].shape[1] * 2) for n, w in raw.items()}
    norms = [formats.bf16_bits(1 + 0.1 * r.standard_normal(H)) for _ in range(2)]
    lay = example.Layer(gu.bits_to_bf16_tensor(norms[0]), dev["qkv"], dev["o"], gu.bits_to_bf16_tensor(norms[1]),
                        dev["fc1"], dev["fc2"], Hq, Hkv, D)
    h, res = _bf16(r.standard_normal((B, H))), _bf16(2 * r.standard_normal((B, H)))
    out, res_out = lay.step(gu.bits_to_bf16_tensor(formats.bf16_bits(h)), gu.bits_to_bf16_tensor(formats.bf16_bits(res)),
                            example.Cache(B, 2, Hkv, 4, D, kind), nv.rope_table(8, D))
    first = _bf16(h + res)
    x = formats.bf16_bits(olayer.rms_norm(first, formats.bf16_to_float(norms[0]), 1e-6))
    v = formats.bf16_to_float(dense.linear(x, *raw["qkv"], True)[1]).reshape(B, Hq + 2 * Hkv, D)[:, Hq + Hkv:]
    if kind == "e4m3":
        codes, s = olayer.quantise(v.astype(np.float32))
        v = codes * s[..., None].astype(np.float64)
    att = np.repeat(v, Hq // Hkv, axis=1).reshape(B, Hq * D)
    second = _bf16(formats.bf16_to_float(dense.linear(formats.bf16_bits(att), *raw["o"], True)[1]) + first)
    x = formats.bf16_bits(olayer.rms_norm(second, formats.bf16_to_float(norms[1]), 1e-6))
    want = formats.bf16_to_float(omoe.mlp(x, (*raw["fc1"], True), (*raw["fc2"], True))[1])
    for got, ref in ((out, want), (res_out, second)):
        g = got.double().cpu().numpy()
        assert np.all(np.isfinite(g)) and np.linalg.norm(g - ref) <= 2.0 ** -6 * np.linalg.norm(ref)
    gu.check_device_status()
