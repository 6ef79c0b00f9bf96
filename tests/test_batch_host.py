"""The batch operators' refusals, on the host before any launch (made-up addresses:
every call here is refused or has nothing to do)."""

import ctypes

import pytest
import torch

import w4a16_nvfp4_weight_gb300 as nv
from w4a16_nvfp4_weight_gb300 import _lib

V = ctypes.c_void_p
BASE = 1 << 40
FAR = [BASE + (i << 34) for i in range(1, 20)]


def _err(lib):
    return lib.nvfp4_last_error().decode()


def _extend(lib, n=FAR[0], m=FAR[1], B=8, table=FAR[2], stride=16, width=16, pages=FAR[3], P=64, count=FAR[4], page=16, rows=8,
            pos=FAR[5], slots=FAR[6], req=FAR[7], starts=FAR[8], n_out=FAR[9], c_out=FAR[10], tabs=None, lens=None):
    return lib.nvfp4_extend_tables(V(n), V(m), B, V(table), stride, width, V(pages), P, V(count), page, rows, V(pos), V(slots), V(req),
                                   V(starts), V(n_out), V(c_out), V(tabs), V(lens), None)


def test_extend_refusals(lib):
    e = lambda **k: _extend(lib, **k)
    assert e(B=-1) == 1 and e(width=-1) == 1 and e(P=-1) == 1 and e(stride=-1) == 1 and e(rows=-1) == 1
    assert e(B=16385) == 2 and e(page=0) == 2 and e(page=1 << 31) == 2 and e(rows=1 << 31) == 2 and e(width=1 << 31, stride=1 << 31) == 2
    assert e(stride=15) == 1 and "overlap" in _err(lib)
    for name in ("n", "m", "table", "pages", "count", "pos", "slots", "req", "starts", "n_out", "c_out"):
        assert e(**{name: None}) == 1 and "null" in _err(lib)
    assert e(tabs=FAR[11]) == 1 and "row_lengths" in _err(lib)
    for name, bad in (("n", FAR[0] + 2), ("table", FAR[2] + 1), ("pos", FAR[5] + 4), ("slots", FAR[6] + 4), ("c_out", FAR[10] + 2)):
        assert e(**{name: bad}) == 3


@pytest.mark.parametrize("over", ["m", "table", "pages"])
@pytest.mark.parametrize("out", ["pos", "slots", "req", "starts", "n_out", "c_out", "tabs", "lens"])
def test_extend_outputs_over_inputs(lib, out, over):
    at = dict(m=FAR[1], table=FAR[2], pages=FAR[3])[over]
    assert _extend(lib, **dict(dict(tabs=FAR[11], lens=FAR[12]), **{out: at})) == 1 and "overlaps" in _err(lib)


def test_extend_overlaps(lib):
    e = lambda **k: _extend(lib, **k)
    assert e(n_out=FAR[0] + 4) == 1 and "lengths itself" in _err(lib)
    assert e(req=FAR[0]) == 1 and e(starts=FAR[4]) == 1 and e(c_out=FAR[0]) == 1 and e(n_out=FAR[4]) == 1
    assert e(req=FAR[8]) == 1 and e(pos=FAR[6]) == 1 and e(slots=FAR[6], pos=FAR[6] + 8) == 1
    assert e(pages=FAR[2]) == 1 and e(n=FAR[2] + 64) == 1 and e(count=FAR[2] + 4) == 1


def test_trim_refusals(lib):
    def t(n=FAR[0], k=FAR[1], B=8, table=FAR[2], stride=16, width=16, pages=FAR[3], P=64, count=FAR[4], page=16, n_out=FAR[5], c_out=FAR[6]):
        return lib.nvfp4_trim_tables(V(n), V(k), B, V(table), stride, width, V(pages), P, V(count), page, V(n_out), V(c_out), None)
    assert t(B=-1) == 1 and t(P=-1) == 1 and t(stride=4) == 1
    assert t(B=16385) == 2 and t(page=0) == 2 and t(P=1 << 31) == 2
    for name in ("n", "k", "table", "pages", "count", "n_out", "c_out"):
        assert t(**{name: None}) == 1 and "null" in _err(lib)
    assert t(k=FAR[1] + 2) == 3 and t(pages=FAR[3] + 1) == 3
    for at in (FAR[0], FAR[1], FAR[2], FAR[4], FAR[5], FAR[6]):
        assert t(pages=at) == 1 and "free_pages" in _err(lib)
    assert t(n_out=FAR[0] + 8) == 1 and t(n_out=FAR[1]) == 1 and t(n_out=FAR[4]) == 1 and t(c_out=FAR[0] + 4) == 1 and t(c_out=FAR[5]) == 1


def test_lora_refusals(lib):
    big = 1 << 40

    def f(y=FAR[0], ys=64, x=FAR[1], xs=128, A=FAR[2], B=FAR[3], s=FAR[4], ids=FAR[5], T=4, n=3, r=16, K=128, N=64, f16=0, out=FAR[6], ws=FAR[7], wsb=big):
        return lib.nvfp4_lora_add(V(y), ys, V(x), xs, V(A), V(B), V(s), V(ids), T, n, r, K, N, f16, V(out), V(ws), wsb, None)
    assert f(T=-1) == 1 and f(N=-1) == 1 and f(n=-1) == 1 and f(f16=2) == 1 and f(xs=-1) == 1 and f(ys=-1) == 1
    assert f(r=0) == 2 and f(r=257) == 2 and f(n=4097) == 2 and f(K=0) == 2 and f(K=1 << 25) == 2 and f(T=1 << 25) == 2
    assert f(T=0, y=None, x=None, A=None, B=None, ids=None, out=None, ws=None) == 0 and f(N=0, out=None) == 0
    for name in ("y", "x", "A", "B", "ids", "out"):
        assert f(**{name: None}) == 1 and "null" in _err(lib)
    assert f(x=FAR[1] + 1) == 3 and f(ids=FAR[5] + 2) == 3 and f(s=FAR[4] + 2) == 3 and f(ws=FAR[7] + 128) == 3
    need = lib.nvfp4_lora_workspace(4, 3, 16, 128)
    assert need > 0 and f(wsb=need - 1) == 4 and "needs" in _err(lib) and f(ws=None) == 4
    assert lib.nvfp4_lora_workspace(0, 3, 16, 128) == 0 and lib.nvfp4_lora_workspace(4, 3, 300, 128) == 0
    assert f(out=FAR[0] + 2) == 1 and f(ys=72, out=FAR[0]) == 1 and "dense" in _err(lib)
    for at in (FAR[1], FAR[2], FAR[3], FAR[4], FAR[5], FAR[7]):
        assert f(out=at) == 1 and "out overlaps" in _err(lib)
    for at in (FAR[0], FAR[1], FAR[2], FAR[3], FAR[4], FAR[5]):
        assert f(ws=at) == 1 and "workspace" in _err(lib)


def test_sample_refusals(lib):
    def f(l=FAR[0], stride=100, type=0, B=4, vocab=100, u=FAR[1], how=True, tokens=FAR[2], lp=None, **arrays):
        s = _lib.Sampling(temperature_all=1.0, top_p_all=1.0, **arrays)
        return lib.nvfp4_sample(V(l), stride, type, B, vocab, V(u), ctypes.byref(s) if how else None, V(tokens), V(lp), None)
    assert f(B=-1) == 1 and f(stride=-1) == 1 and f(type=3) == 1 and f(type=-1) == 1 and f(how=False) == 1
    assert f(vocab=0) == 2 and f(vocab=(1 << 20) + 1) == 2 and f(B=1 << 25) == 2
    assert f(B=0, l=None, u=None, tokens=None) == 0
    assert f(l=None) == 1 and f(u=None) == 1 and f(tokens=None) == 1
    assert f(l=FAR[0] + 1) == 3 and f(l=FAR[0] + 2, type=2) == 3 and f(tokens=FAR[2] + 4) == 3 and f(lp=FAR[3] + 2) == 3 and f(top_p=FAR[3] + 1) == 3
    assert f(tokens=FAR[0] + 400) == 1 and "tokens overlaps logits" in _err(lib)
    assert f(tokens=FAR[1]) == 1 and f(lp=FAR[1]) == 1 and f(lp=FAR[2]) == 1
    assert f(top_k=FAR[4], tokens=FAR[4]) == 1 and "top_k" in _err(lib) and f(min_p=FAR[4], lp=FAR[4]) == 1


def test_python_refuses_cpu_tensors_and_types(lib):
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: nv.extend_tables(i, i, i[None], i, i, 16, 2), lambda: nv.trim_tables(i, i, i[None], i, i, 16),
                 lambda: nv.lora_add(torch.zeros(2, 4), torch.zeros(2, 4), None, None, i), lambda: nv.sample(torch.zeros(2, 4), torch.zeros(2)),
                 lambda: nv.sample(None, None), lambda: nv.extend_tables(3, i, i, i, i, 16, 2)):
        with pytest.raises(nv.Nvfp4Error) as e:
            call()
        assert e.value.status == 1
