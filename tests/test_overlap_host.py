"""Outputs over inputs or over each other are refused on the host, before any launch
(made-up addresses: every call here is refused)."""

import ctypes

import pytest

from w4a16_nvfp4_weight_gb300 import _lib

V = ctypes.c_void_p
BASE = 1 << 40
FAR = [BASE + (i << 32) for i in range(1, 12)]


def _refused(lib, status, names):
    text = lib.nvfp4_last_error().decode()
    assert status == 1 and "overlap" in text and all(n in text for n in names), (status, text)


@pytest.mark.parametrize("out_type", [0, 1])
def test_norm(lib, out_type):
    T, H = 8, 64
    size = T * H * (1 if out_type else 2)

    def norm(names, x=FAR[0], xs=H, res=None, rs=H, w=FAR[1], y=FAR[2], scales=FAR[3] if out_type else None, added=None):
        _refused(lib, lib.nvfp4_rms_norm(V(x), xs, V(res), rs, V(w), T, H, 1e-6, out_type, 0, 0, V(y), V(scales), V(added), None), names)

    norm(["Y", "X"], y=FAR[0] + 128)                        # a row on
    norm(["Y", "X"], y=FAR[0] - size + 2)                   # the last element over the first
    norm(["Y", "X"], xs=1024, y=FAR[0] + 7 * 2048 + 126)    # the last of rows far apart
    norm(["Y", "X"], xs=1024, y=FAR[0])                     # the same place, but not dense
    norm(["Y", "weight"], y=FAR[1] + 2 * H - 2)
    norm(["Y", "residual"], res=FAR[4], added=FAR[5], y=FAR[4] + 16)
    norm(["residual_out", "X"], res=FAR[4], added=FAR[0] + 16)
    norm(["residual_out", "residual"], res=FAR[4], rs=2 * H, added=FAR[4])
    norm(["residual_out", "weight"], res=FAR[4], added=FAR[1])
    norm(["Y", "residual_out"], res=FAR[4], added=FAR[5], y=FAR[5])
    if out_type:
        norm(["Y", "X"], y=FAR[0])                          # codes over 16-bit rows
        norm(["scales", "X"], scales=FAR[0])
        norm(["Y", "scales"], scales=FAR[2])
        norm(["residual_out", "scales"], res=FAR[4], added=FAR[5], scales=FAR[5] + 4)


def _cache(kind, pages=4, heads=2, page=16, D=64):
    c = _lib.KVCache(k=FAR[0], v=FAR[1], num_pages=pages, page_size=page, heads=heads, head_dim=D,
                     page_stride=heads * page * D, head_stride=page * D, token_stride=D, type=kind)
    if kind:
        c.k_scale, c.v_scale = FAR[2], FAR[3]
    return c


@pytest.mark.parametrize("kind", [0, 1])
def test_cache_write(lib, kind):
    T, Hq, D = 8, 4, 64
    c = _cache(kind)

    def write(names, q=FAR[4], qt=8 * D, k=FAR[5], v=FAR[6], pos=FAR[7], table=FAR[8], slots=FAR[9], to=FAR[10]):
        st = lib.nvfp4_rope_cache_write(V(q), qt, D, V(k), 2 * D, D, V(v), 2 * D, D, T, Hq, V(pos), 1, None, V(table), 100, D, 0, 0,
                                        V(slots), ctypes.byref(c), V(to), None)
        _refused(lib, st, names)

    write(["q_out", "q"], to=FAR[4])                        # q is a part of wider rows
    write(["q_out", "q"], to=FAR[4] + 7 * 16 * D + 2 * Hq * D - 16)
    write(["q_out", "q"], qt=Hq * D, to=FAR[4] + 16)
    write(["q_out", "k"], to=FAR[5] - 2 * T * Hq * D + 16)
    write(["q_out", "v"], to=FAR[6] + 16)
    write(["q_out", "positions"], to=FAR[7])
    write(["q_out", "slots"], to=FAR[9])
    write(["q_out", "table"], to=FAR[8] + 100 * D * 4 - 16)
    write(["q_out", "keys"], to=FAR[0] + (4 * 2 * 16 * 64 << (1 - kind)) - 16)
    write(["q_out", "values"], to=FAR[1])
    if kind:
        write(["q_out", "scales"], to=FAR[3] + 4 * 2 * 16 * 4 - 16)


@pytest.mark.parametrize("kind", [0, 1])
def test_cache_read(lib, kind):
    T = 8
    c = _cache(kind)

    def read(names, slots=FAR[4], k=FAR[5], v=FAR[6]):
        _refused(lib, lib.nvfp4_kv_cache_read(ctypes.byref(c), V(slots), T, 0, V(k), V(v), None), names)

    read(["k_out", "v_out"], v=FAR[5] + 2 * T * 2 * 64 - 16)
    read(["k_out", "slots"], k=FAR[4])
    read(["v_out", "keys"], v=FAR[0])
    read(["k_out", "values"], k=FAR[1])


@pytest.mark.parametrize("kind", [0, 1])
def test_attention(lib, kind):
    B, Hq, D, width = 3, 8, 64, 5
    c = _cache(kind)
    size = 1 << 31

    def attend(names, q=FAR[4], qr=Hq * D, table=FAR[5], lengths=FAR[6], out=FAR[7], lse=FAR[8], ws=FAR[9]):
        st = lib.nvfp4_paged_attention(V(q), qr, D, ctypes.byref(c), V(table), width, width, V(lengths), B, Hq, 0.1, 0, 0, V(out), V(lse),
                                       V(ws), size, None)
        _refused(lib, st, names)

    attend(["out", "q"], out=FAR[4] + 2 * D)
    attend(["out", "q"], qr=2 * Hq * D, out=FAR[4])
    attend(["lse", "q"], lse=FAR[4] + 4)
    attend(["lse", "out"], lse=FAR[7] + 2 * B * Hq * D - 4)
    attend(["lse", "lengths"], lse=FAR[6] + 8)
    attend(["out", "block_table"], out=FAR[5])
    attend(["out", "keys"], out=FAR[0] + 64)
    attend(["lse", "values"], lse=FAR[1] + 64)
    if lib.nvfp4_paged_attention_workspace(B, Hq, 2, D):
        attend(["workspace", "q"], ws=FAR[4])
        attend(["workspace", "out"], ws=FAR[7])
        attend(["workspace", "keys"], ws=FAR[0] - 256)
