"""The operators between a decoder layer's linears against the 64-bit oracle:
norm, rotary positions with the cache write, cache read, paged attention.

Tolerances.  u is the unit roundoff of a 16-bit type (BF16 2^-8, FP16 2^-11; FP16
has an absolute 2^-25 below its normals).  A 16-bit output computed in 32 bits is
within u |ref| of the 64-bit value, plus the 32-bit error (at most 2^-13 relative
here: sums of up to 2^11 terms per thread).  Attention also rounds each softmax
weight to the 16-bit type that meets the values in the MMA (BF16 for a BF16
cache, else FP16), which moves the output by at most u_p sum_j p_j |v_j|; scores in 32
bits move it by their error, at most 2^-12 relative to that sum for the
magnitudes here.  Caches and the rotation are defined step by step in 32 bits, so
their codes, scales and 16-bit values are equal bit for bit.
"""

import numpy as np
import pytest
import torch

import w4a16_nvfp4_weight_gb300 as nv
from oracle import layer
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    torch.cuda.init()
    yield
    gu.check_device_status()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, act="bf16", std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[act])


def _np(t):
    return t.detach().cpu().double().numpy()


def _close16(got, ref, act, rel=2.0 ** -13):
    got = _np(got)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    err = np.abs(got - ref)[fine]
    assert np.all(err <= (U[act] + rel) * np.abs(ref[fine]) + TINY[act]), err.max()


# ------------------------------------------------------------------- norm ---

NORM_SHAPES = [(1, 1), (3, 7), (5, 16), (2, 64), (9, 128), (33, 720), (4, 1000), (7, 2064), (1, 4096), (300, 4096),
               (3, 5120), (2, 8192), (1300, 256), (2, 16384), (3, 40000), (2, 40008)]


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("res", [False, True])
def test_norm(T, H, act, res):
    g = _gen(T * 131 + H)
    x, w, r = _randn(g, (T, H), act), _randn(g, (H,), act), _randn(g, (T, H), act, 3.0)
    if res:
        y, added = nv.rms_norm(x, w, eps=1e-5, residual=r)
        want = (x.float() + r.float()).to(DT[act])
        assert torch.equal(added, want)
        x = want
    else:
        y = nv.rms_norm(x, w, eps=1e-5)
    _close16(y, layer.rms_norm(_np(x), _np(w), 1e-5), act)


@pytest.mark.parametrize("T,H,group", [(1, 16, 16), (5, 64, 0), (3, 720, 16), (33, 2064, 0), (4, 4096, 128),
                                       (300, 4096, 0), (7, 5120, 256), (2, 8192, 32), (9, 1024, 64), (2, 33024, 128),
                                       (3, 7, 0), (2, 40008, 0), (700, 128, 64)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_norm_e4m3(T, H, group, act):
    g = _gen(T + H + group)
    x, w, r = _randn(g, (T, H), act), _randn(g, (H,), act), _randn(g, (T, H), act)
    codes, scales, added = nv.rms_norm_e4m3(x, w, group=group, residual=r)
    n = group or H
    assert codes.dtype == E4M3 and scales.shape == (T, H // n)
    ref = layer.rms_norm(_np(added), _np(w), 1e-6).reshape(T, H // n, n)
    s = np.maximum(np.abs(ref).max(-1) / 448, 2.0 ** -100)
    got_s = _np(scales)
    assert np.all(np.abs(got_s - s) <= 2.0 ** -13 * s)
    # a code is a nearest one: within half a step of y / s, allowing the 32-bit error of y / s
    q = ref / got_s[..., None]
    c = _np(codes.float()).reshape(q.shape)
    _, e = np.frexp(q)
    step = np.exp2(np.maximum(e.astype(float) - 4, -9.0))
    assert np.all(np.abs(c - q) <= step / 2 * (1 + 2.0 ** -8) + 2.0 ** -13 * np.abs(q))
    plain, added2 = nv.rms_norm(x, w, residual=r)
    assert torch.equal(added, added2)


def test_norm_strides_offsets_and_in_place():
    g = _gen(5)
    w = _randn(g, (512,))
    wide = _randn(g, (40, 1600))
    for start in (0, 8, 3):                               # aligned and odd starts, row stride above H
        x = wide[:, start:start + 512]
        _close16(nv.rms_norm(x, w), layer.rms_norm(_np(x), _np(w), 1e-6), "bf16")
        r = wide[:, 1024 + start:1536 + start]
        y, a = nv.rms_norm(x, w, residual=r)
        assert torch.equal(a, (x.float() + r.float()).to(torch.bfloat16))
        _close16(y, layer.rms_norm(_np(a), _np(w), 1e-6), "bf16")
    odd = _randn(g, (17, 1601))[:, :512]                  # odd row stride
    _close16(nv.rms_norm(odd, w), layer.rms_norm(_np(odd), _np(w), 1e-6), "bf16")
    once = _randn(g, (1, 512))                            # one row for all: stride 0
    assert torch.equal(nv.rms_norm(once.expand(6, 512), w), nv.rms_norm(once.repeat(6, 1), w))
    for H in (512, 509):
        x, r = _randn(g, (64, H)), _randn(g, (64, H))
        y, a = nv.rms_norm(x, w[:H].contiguous(), residual=r)
        r2, x2 = r.clone(), x.clone()
        y2, a2 = nv.rms_norm(x, w[:H].contiguous(), residual=r2, residual_out=r2)
        assert a2 is r2 and torch.equal(r2, a) and torch.equal(y2, y)
        y3, _ = nv.rms_norm(x2, w[:H].contiguous(), residual=r, residual_out=x2)
        assert torch.equal(x2, a) and torch.equal(y3, y)


def test_norm_special_values():
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda")
    x[1] = 1e-30
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    x[4] = 2.0 ** 55
    y = nv.rms_norm(x, w)
    assert torch.all(y[0] == 0) and torch.all(y[2].isnan())
    assert y[3, 9].isnan() and torch.all(y[3, :9] == 0)
    assert torch.all(y[4] == 1)                           # 256 squares of 2^110 sum inside 32 bits
    c, s = nv.rms_norm_e4m3(x, w, group=64)
    assert torch.all(s[0] == 2.0 ** -100) and torch.all(c[0].float() == 0)
    assert torch.all(c[2].float().isnan())
    assert torch.all(c[4].float() == 448) and nv.rms_norm(x[:0], w).shape == (0, 256)


@pytest.mark.parametrize("T,H", [(1, 3), (2, 65), (700, 33), (17, 268), (900, 268), (350, 1001), (2, 8190), (400, 4098),
                                 (3, 16383), (320, 16384), (2, 16386), (330, 12345)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_norm_widths_that_are_no_multiple_of_eight(T, H, act):
    g = _gen(T * 3 + H)
    x, w, r = _randn(g, (T, H), act), _randn(g, (H,), act), _randn(g, (T, H), act)
    y, added = nv.rms_norm(x, w, residual=r)
    assert torch.equal(added, (x.float() + r.float()).to(DT[act]))
    ref = layer.rms_norm(_np(added), _np(w), 1e-6)
    _close16(y, ref, act)
    _close16(nv.rms_norm(added, w), ref, act)
    codes, scales = nv.rms_norm_e4m3(added, w)
    s = np.maximum(np.abs(ref).max(-1, keepdims=True) / 448, 2.0 ** -100)
    assert np.all(np.abs(_np(scales) - s) <= 2.0 ** -13 * s)
    q = ref / _np(scales)
    _, e = np.frexp(q)
    step = np.exp2(np.maximum(e.astype(float) - 4, -9.0))
    assert np.all(np.abs(_np(codes.float()) - q) <= step / 2 * (1 + 2.0 ** -8) + 2.0 ** -13 * np.abs(q))
    # views whose rows start anywhere
    if H > 40:
        for cut in (1, 2):
            v = added[:, cut:H - 7]
            _close16(nv.rms_norm(v, w[:H - 7 - cut].contiguous()), layer.rms_norm(_np(v), _np(w)[:H - 7 - cut], 1e-6), act)


# ----------------------------------------------------- cache write and read ---

def _make_cache(pages, heads, page, D, act, kind, fill=float("nan"), layout="hnd"):
    dt = E4M3 if kind == "e4m3" else DT[act]

    def full(shape):
        if kind == "e4m3":
            return torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
        return torch.full(shape, fill, dtype=dt, device="cuda")
    if layout == "hnd":
        k, v = full((pages, heads, page, D)), full((pages, heads, page, D))
    elif layout == "nhd":
        k, v = (full((pages, page, heads, D)).transpose(1, 2) for _ in range(2))
    else:                                                 # one pool, keys and values of a page side by side, rows padded
        pool = full((pages, 2, heads, page, D + 16))
        k, v = pool[:, 0, :, :, :D], pool[:, 1, :, :, :D]
    c = dict(k_cache=k, v_cache=v)
    if kind == "e4m3":
        c.update({n: torch.full((pages, heads, page), float("nan"), device="cuda") for n in ("k_scale", "v_scale")})
    return c


def _cached_values(c, which, slots, page):
    """[T, heads, D] float64 of cached rows, read with torch."""
    p, a = slots // page, slots % page
    x = c[which + "_cache"]
    if x.dtype == E4M3:
        x = x.view(torch.uint8)[p, :, a].view(E4M3).double() * c[which + "_scale"][p, :, a].double()[..., None]
    else:
        x = x[p, :, a].double()
    return x.cpu().numpy()


ROPE_CASES = [
    # T, Hq, Hkv, D, rot, page, axes/sections, interleaved, act, kind, layout
    (1, 32, 8, 128, 128, 16, None, False, "bf16", "16", "hnd"),
    (16, 32, 8, 128, 128, 16, None, False, "bf16", "e4m3", "hnd"),
    (7, 4, 4, 64, 64, 1, None, True, "f16", "e4m3", "nhd"),
    (33, 5, 1, 80, 80, 24, [20, 10, 10], False, "bf16", "16", "pool"),
    (50, 6, 2, 256, 128, 64, [13, 21, 30], False, "f16", "16", "hnd"),
    (19, 8, 2, 96, 34, 8, [5, 0, 12], False, "bf16", "e4m3", "pool"),
    (19, 8, 2, 112, 38, 8, [19], True, "bf16", "e4m3", "nhd"),
    (300, 40, 8, 128, 128, 64, [16, 24, 24], False, "bf16", "16", "hnd"),
    (300, 12, 3, 192, 192, 32, [24, 24, 24, 24], True, "f16", "e4m3", "hnd"),
    (5, 2, 1, 16, 2, 4, None, False, "bf16", "e4m3", "hnd"),
    (5, 0, 1, 48, 0, 4, None, False, "bf16", "16", "hnd"),
    (2000, 16, 4, 128, 64, 16, None, False, "bf16", "e4m3", "nhd"),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page,sections,inter,act,kind,layout", ROPE_CASES)
def test_rope_cache_write_and_read(T, Hq, Hkv, D, rot, page, sections, inter, act, kind, layout):
    g, r = _gen(T + D), np.random.default_rng(T * 7 + D)
    qkv = _randn(g, (T, Hq + 2 * Hkv, D), act)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    rows, axes = 500, len(sections) if sections else 1
    table = nv.rope_table(rows, rot)
    positions = torch.from_numpy(r.integers(0, rows, (axes, T)))
    pages = -(-T // page) + 2
    slots = torch.from_numpy(r.permutation(pages * page)[:T]).cuda()
    if T > 4:
        slots[3] = -1
    c = _make_cache(pages, Hkv, page, D, act, kind, layout=layout)
    before = {n: t.clone() for n, t in c.items()}
    pos = positions.cuda() if sections else positions[0].cuda()
    out = nv.rope_cache_write(q, k, v, pos, table, slots=slots, sections=sections, interleaved=inter, **c)
    gu.check_device_status()
    tn = table.cpu().numpy()
    turn = lambda x: layer.rope(x.float().cpu().numpy(), positions.numpy(), tn, sections, inter)  # noqa: E731
    assert torch.equal(out.cpu(), torch.from_numpy(turn(q)).to(DT[act]))
    held = (slots >= 0).cpu().numpy()
    read = nv.cache_read(slots=slots, dtype=DT[act], **c)
    for which, x, back in (("k", turn(k), read[0]), ("v", v.float().cpu().numpy(), read[1])):
        if kind == "e4m3":
            codes, s = layer.quantise(x)
            want = codes * s[..., None].astype(np.float64)
            p, a = slots // page, slots % page
            assert np.array_equal(c[which + "_scale"][p, :, a].cpu().numpy()[held], s[held])
        else:
            want = torch.from_numpy(x).to(DT[act]).double().numpy()
        got = _cached_values(c, which, slots, page)
        assert np.array_equal(got[held], want[held])
        back16 = torch.from_numpy(want.astype(np.float32)).to(DT[act])
        back16[~torch.from_numpy(held)] = 0
        assert torch.equal(back.cpu(), back16)
    # nothing else was written
    free = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    free[slots[slots >= 0]] = False
    other = free.nonzero()[:, 0]
    for n, t in c.items():
        a, b = ((u.view(torch.uint8) if u.dtype == E4M3 else u)[other // page, :, other % page] for u in (t, before[n]))
        assert torch.equal(torch.nan_to_num(a.float(), nan=-5.0), torch.nan_to_num(b.float(), nan=-5.0))


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,sections,inter,kind", [
    (3, 4, 2, 80, 40, None, False, "e4m3"), (900, 6, 2, 80, 40, [8, 7, 5], False, "16"), (40, 3, 1, 256, 136, [1, 0, 67], False, "e4m3"),
    (1300, 2, 2, 112, 56, None, True, "e4m3"), (7, 8, 8, 48, 24, [12], True, "16"), (2000, 12, 4, 256, 256, None, True, "e4m3"),
    (5, 1, 1, 16, 8, None, False, "e4m3"), (600, 192, 16, 80, 40, [8, 6, 6], False, "e4m3")])
def test_rope_on_half_heads(T, Hq, Hkv, D, rot, sections, inter, kind):
    test_rope_cache_write_and_read(T, Hq, Hkv, D, rot, 16, sections, inter, "bf16", kind, "hnd")


def test_rope_in_place_and_separate_tensors():
    g = _gen(9)
    q, k, v = _randn(g, (40, 8, 128)), _randn(g, (40, 2, 128)), _randn(g, (40, 2, 128))
    table, slots = nv.rope_table(64, 128), torch.arange(40, device="cuda")
    pos = slots.clone()
    for inter in (False, True):
        a, b = (_make_cache(3, 2, 16, 128, "bf16", "16") for _ in range(2))
        want = nv.rope_cache_write(q, k, v, pos, table, slots=slots, interleaved=inter, **a)
        q2 = q.clone()
        got = nv.rope_cache_write(q2, k, v, pos, table, slots=slots, interleaved=inter, q_out=q2, **b)
        assert got is q2 and torch.equal(want, got)
        for n in a:
            assert torch.equal(a[n].view(torch.int16), b[n].view(torch.int16))


def test_rope_out_of_range_is_reported_not_followed():
    g = _gen(10)
    q, k, v = _randn(g, (4, 2, 64)), _randn(g, (4, 1, 64)), _randn(g, (4, 1, 64))
    table = nv.rope_table(10, 64)
    c = _make_cache(2, 1, 4, 64, "bf16", "16", fill=0.0)
    slots = torch.tensor([0, 8, 1 << 40, 2], device="cuda")
    pos = torch.tensor([3, 4, 5, 6], device="cuda")
    nv.rope_cache_write(q, k, v, pos, table, slots=slots, **c)
    assert nv.device_status() == 8
    assert torch.equal(c["v_cache"][0, 0, 0], v[0, 0]) and torch.equal(c["v_cache"][0, 0, 2], v[3, 0])
    assert torch.all(c["v_cache"][1] == 0)
    out = nv.rope_cache_write(q, k, v, torch.tensor([10, -1, 1 << 50, 0], device="cuda"), table,
                              slots=torch.arange(4, device="cuda"), **c)
    assert nv.device_status() == 8 and torch.equal(out, q)      # unrotated; position 0 rotates by nothing
    kk, vv = nv.cache_read(slots=torch.tensor([8, 0], device="cuda"), **c)
    assert nv.device_status() == 8 and torch.all(kk[0] == 0) and torch.equal(vv[1], v[0])


def test_cache_write_special_values():
    x = torch.zeros(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[1, 0, 5] = float("nan")
    x[1, 0, 6] = 2.0
    x[2, 0, 3] = float("inf")
    x[3] = 1e-38
    c = _make_cache(1, 1, 4, 64, "bf16", "e4m3")
    slots = torch.arange(4, device="cuda")
    nv.rope_cache_write(x, x, x, slots, nv.rope_table(4, 0), slots=slots, **c)
    k, _ = nv.cache_read(slots=slots, dtype=torch.bfloat16, **c)
    assert torch.all(k[0] == 0) and torch.all(k[3] == 0)
    assert k[1, 0, 5].isnan() and k[1, 0, 6] == 2 and k[1].isnan().sum() == 1
    assert torch.all(k[2].isnan())
    gu.check_device_status()


# -------------------------------------------------------------- attention ---

def _attention_case(lengths, Hq, Hkv, D, page, act, kind, seed, layout="hnd", std=1.0, extra=3, width=None):
    """A cache whose unused rows hold NaN and a table whose unused entries are -1."""
    g, r = _gen(seed), np.random.default_rng(seed)
    B, n = len(lengths), np.array(lengths)
    per = -(-n // page)
    pages = int(per.sum()) + extra
    c = _make_cache(pages, Hkv, page, D, act, kind, layout=layout)
    order = r.permutation(pages)
    table = np.full((B, width or max(1, per.max())), -1, dtype=np.int32)
    at, rows = 0, []
    for b in range(B):
        table[b, :per[b]] = order[at:at + per[b]]
        at += per[b]
        t = np.arange(n[b])
        rows.append(table[b, t // page].astype(np.int64) * page + t % page)
    slots = torch.from_numpy(np.concatenate(rows)).cuda() if n.sum() else torch.empty(0, dtype=torch.int64, device="cuda")
    T = slots.numel()
    k, v = _randn(g, (T, Hkv, D), act, std), _randn(g, (T, Hkv, D), act)
    if kind == "e4m3":                                    # rows of very different sizes
        v = (v.float() * torch.exp2(torch.randint(-12, 3, (T, Hkv, 1), generator=g, device="cuda").float())).to(DT[act])
    nv.rope_cache_write(k, k, v, slots, nv.rope_table(1, 0), slots=slots, **c)
    q = _randn(g, (B, Hq, D), act)
    return c, q, torch.from_numpy(table).cuda(), torch.from_numpy(n.astype(np.int32)).cuda(), slots


def _check_attention(c, q, table, lengths, slots, page, act, kind, window=0, scale=None, **kw):
    out, lse = nv.paged_attention(q, block_table=table, lengths=lengths, window=window, softmax_scale=scale,
                                  return_lse=True, **c, **kw)
    gu.check_device_status()
    k, v = _cached_values(c, "k", slots, page), _cached_values(c, "v", slots, page)
    u_p = U["bf16"] if kind == "16" and act == "bf16" else U["f16"]
    at = 0
    got, got_lse, qn = _np(out), _np(lse), _np(q)
    for b, n in enumerate(lengths.tolist()):
        first = max(0, n - window) if window else 0
        kk, vv = k[at + first:at + n], v[at + first:at + n]
        at += n
        ref, ref_lse, mag = layer.attend(qn[b], kk, vv, q.shape[2] ** -0.5 if scale is None else scale)
        if n == 0:
            assert np.all(got[b] == 0) and np.all(got_lse[b] == -np.inf)
            continue
        top = np.abs(vv).max() if vv.size else 0.0
        bound = U[act] * np.abs(ref) + TINY[act] + (u_p + 2.0 ** -11) * mag + 2.0 ** -25 * n * top
        err = np.abs(got[b] - ref)
        assert np.all(err <= bound), (b, n, (err / bound).max())
        assert np.all(np.abs(got_lse[b] - ref_lse) <= 2.0 ** -17 * (1 + np.abs(ref_lse))), (b, n)
    return out, lse


ATTN_CASES = [
    # lengths, Hq, Hkv, D, page, act, kind, layout, window
    ([1], 1, 1, 64, 16, "bf16", "16", "hnd", 0),
    ([1, 2, 15, 16, 17, 31, 33, 0, 64], 32, 8, 128, 16, "bf16", "16", "hnd", 0),
    ([0, 0, 5], 8, 1, 128, 8, "f16", "16", "nhd", 0),
    ([0], 8, 8, 128, 8, "bf16", "e4m3", "hnd", 0),
    ([1000], 32, 8, 128, 16, "bf16", "16", "hnd", 0),
    ([1000, 3], 32, 8, 128, 1, "f16", "e4m3", "nhd", 0),
    ([777, 130, 1], 5, 1, 80, 24, "bf16", "16", "pool", 0),
    ([777, 130, 1], 5, 1, 80, 24, "bf16", "e4m3", "pool", 0),
    ([300, 41], 12, 1, 128, 32, "f16", "16", "hnd", 0),
    ([300, 41], 16, 1, 128, 32, "bf16", "e4m3", "hnd", 0),
    ([257, 90], 20, 1, 128, 64, "bf16", "16", "hnd", 0),      # more heads a key head than one MMA row block
    ([257, 90], 40, 1, 64, 64, "bf16", "e4m3", "hnd", 0),
    ([400, 7], 8, 2, 256, 16, "bf16", "16", "hnd", 0),
    ([400, 7], 32, 2, 256, 16, "bf16", "e4m3", "nhd", 0),
    ([100, 7], 4, 2, 192, 16, "f16", "16", "hnd", 0),
    ([100, 7], 4, 2, 16, 16, "bf16", "16", "hnd", 0),
    ([100, 7], 4, 2, 16, 16, "f16", "e4m3", "hnd", 0),
    ([100, 7], 4, 2, 48, 40, "bf16", "e4m3", "hnd", 0),
    ([500, 100, 17, 16, 0, 33], 8, 2, 128, 16, "bf16", "16", "hnd", 17),
    ([500, 100, 17, 16, 0, 33], 8, 2, 64, 24, "f16", "e4m3", "hnd", 100),
    ([3000, 1], 8, 2, 128, 16, "bf16", "16", "hnd", 1),
    ([9000, 33, 4000], 16, 2, 128, 128, "bf16", "16", "hnd", 0),
    ([9000, 33, 4000], 16, 2, 128, 128, "bf16", "e4m3", "hnd", 0),
    ([9000, 33, 4000], 16, 16, 64, 128, "f16", "16", "hnd", 0),
    (list(range(0, 300)), 4, 2, 64, 16, "bf16", "16", "hnd", 0),
    ([20] * 700, 8, 4, 64, 16, "bf16", "e4m3", "hnd", 0),
]


@pytest.mark.parametrize("lengths,Hq,Hkv,D,page,act,kind,layout,window", ATTN_CASES)
def test_paged_attention(lengths, Hq, Hkv, D, page, act, kind, layout, window):
    case = _attention_case(lengths, Hq, Hkv, D, page, act, kind, len(lengths) * 31 + D + Hq, layout)
    out, lse = _check_attention(*case, page, act, kind, window)
    again, lse2 = nv.paged_attention(case[1], block_table=case[2], lengths=case[3], window=window, return_lse=True,
                                     **case[0])
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))


SPLIT_CASES = [
    # lengths, Hq, Hkv, D, page, act, kind, layout, window
    ([70001], 8, 1, 128, 16, "bf16", "16", "hnd", 0),            # one unit over every block
    ([70001], 12, 1, 128, 16, "bf16", "e4m3", "hnd", 0),
    ([30000, 1, 0, 257], 2, 2, 80, 24, "f16", "e4m3", "pool", 0),
    ([30000, 1, 0, 257], 20, 1, 64, 24, "bf16", "16", "nhd", 5000),
    ([20000, 300], 8, 2, 256, 64, "bf16", "16", "hnd", 0),
    ([20000, 300], 32, 2, 256, 64, "f16", "e4m3", "hnd", 0),
    ([6000, 5999], 4, 4, 48, 1, "bf16", "e4m3", "hnd", 4097),
    ([1] * 40 + [12000] + [17] * 40, 8, 4, 128, 16, "bf16", "16", "hnd", 0),
    ([(i * 37) % 90 for i in range(1500)], 2, 1, 64, 16, "bf16", "16", "hnd", 0),
    ([255, 256, 1, 0, 16, 200], 16, 4, 128, 16, "bf16", "e4m3", "hnd", 0),        # units kept whole
    ([(i * 53) % 257 for i in range(700)], 8, 2, 64, 128, "f16", "16", "hnd", 0),
    ([9000, 100, 3], 8, 2, 128, 16, "bf16", "16", "hnd", 200),   # short windows of a long cache
]


@pytest.mark.parametrize("lengths,Hq,Hkv,D,page,act,kind,layout,window", SPLIT_CASES)
def test_paged_attention_splits_and_joins(lengths, Hq, Hkv, D, page, act, kind, layout, window):
    """Units cut into many pieces, many units a block, and both in one call; the same
    bits on a second call, and with a table wider than any length needs."""
    case = _attention_case(lengths, Hq, Hkv, D, page, act, kind, len(lengths) + D + Hq, layout)
    out, lse = _check_attention(*case, page, act, kind, window)
    again = nv.paged_attention(case[1], block_table=case[2], lengths=case[3], window=window, **case[0])
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    wide = torch.full((len(lengths), case[2].shape[1] + 4000 // page), -1, dtype=torch.int32, device="cuda")
    wide[:, :case[2].shape[1]] = case[2]
    out, _ = nv.paged_attention(case[1], block_table=wide, lengths=case[3], window=window, return_lse=True, **case[0])
    gu.check_device_status()
    _check_attention(case[0], case[1], wide, *case[3:], page, act, kind, window)


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_paged_attention_scales_and_peaked_rows(kind, scale):
    """Negative and zero scales, and scores whose largest comes at any token."""
    case = _attention_case([2000, 65, 16], 8, 2, 128, 16, "bf16", kind, 77, std=2.0)
    _check_attention(*case, 16, "bf16", kind, scale=scale)


@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_paged_attention_strided_query_and_large_queries(kind):
    case = list(_attention_case([120, 3], 8, 2, 128, 16, "bf16", kind, 78))
    wide = _randn(_gen(79), (2, 12, 128), std=1e4)
    case[1] = wide[:, 2:10]                               # scores in the thousands: one token takes it all
    _check_attention(*case, 16, "bf16", kind, scale=1e-4)
    assert torch.equal(nv.paged_attention(case[1], block_table=case[2], lengths=case[3], **case[0]),
                       nv.paged_attention(case[1].contiguous(), block_table=case[2], lengths=case[3], **case[0]))


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("step", [0.02, 0.4, -0.4, 30.0])
def test_paged_attention_of_scores_that_rise_or_fall_with_the_tokens(kind, step):
    """The base of the exponentials lags behind a rising maximum, or never moves."""
    c, q, table, lengths, slots = _attention_case([1500, 400, 17], 8, 2, 64, 16, "bf16", kind, 83)
    q = torch.zeros_like(q)
    q[:, :, 0] = 1.0
    T = slots.numel()
    k = torch.zeros(T, 2, 64, dtype=torch.bfloat16, device="cuda")
    k[:, :, 0] = torch.cat([torch.arange(n) for n in lengths.tolist()]).cuda()[:, None] * step
    v = _randn(_gen(84), (T, 2, 64), "bf16")
    nv.rope_cache_write(k, k, v, slots, nv.rope_table(1, 0), slots=slots, **c)
    _check_attention(c, q, table, lengths, slots, 16, "bf16", kind, scale=1.0)


@pytest.mark.parametrize("all_zero", [True, False])
def test_paged_attention_of_values_whose_scale_is_zero(all_zero):
    """Rows of zeros (a scale of 0 is no scale the write gives) weigh as others do."""
    case = _attention_case([700, 19, 3], 8, 2, 128, 16, "bf16", "e4m3", 82)
    scales = case[0]["v_scale"]
    scales[torch.arange(scales.shape[0], device="cuda") % (1 if all_zero else 2) == 0] = 0
    _check_attention(*case, 16, "bf16", "e4m3")


def test_paged_attention_nan_and_infinity_in_held_tokens():
    c, q, table, lengths, slots = _attention_case([40, 40], 4, 2, 64, 16, "bf16", "16", 80)
    c["k_cache"][int(table[0, 1]), 0, 3, 5] = float("nan")
    c["v_cache"][int(table[1, 0]), 1, 2, 7] = float("inf")
    out = nv.paged_attention(q, block_table=table, lengths=lengths, **c)
    assert torch.all(out[0, :2].isnan()) and torch.all(out[0, 2:].isfinite())
    assert torch.all(out[1, 2:, 7] == float("inf")) and torch.all(out[1, :2].isfinite())


def test_paged_attention_bad_lengths_and_pages_are_reported():
    c, q, table, lengths, slots = _attention_case([40, 40], 4, 2, 64, 16, "bf16", "16", 81)
    good = nv.paged_attention(q, block_table=table, lengths=lengths, **c)
    gu.check_device_status()
    bad = table.clone()
    bad[1, 2] = 1 << 30
    out = nv.paged_attention(q, block_table=bad, lengths=lengths, **c)
    assert nv.device_status() == 8 and torch.equal(out[0], good[0])
    out = nv.paged_attention(q, block_table=table, lengths=torch.tensor([40, -7], dtype=torch.int32, device="cuda"), **c)
    assert nv.device_status() == 8 and torch.equal(out[0], good[0]) and torch.all(out[1] == 0)
    nv.paged_attention(q, block_table=table, lengths=torch.tensor([40, 1 << 30], dtype=torch.int32, device="cuda"), **c)
    assert nv.device_status() == 8


def test_paged_attention_shared_pages_and_drafted_tokens():
    """Two rows with one table and lengths one apart: each attends to its own tokens."""
    c, q, table, lengths, slots = _attention_case([100], 8, 2, 128, 16, "bf16", "16", 82)
    both = nv.paged_attention(q.repeat(2, 1, 1), block_table=table.repeat(2, 1),
                              lengths=torch.tensor([99, 100], dtype=torch.int32, device="cuda"), **c)
    assert torch.equal(both[1:], nv.paged_attention(q, block_table=table, lengths=lengths, **c))
    assert not torch.equal(both[0], both[1])


def test_cache_rows_past_four_gigabytes():
    """A pool whose rows lie past 2^32 bytes from its start."""
    pages, Hkv, page, D = 90000, 2, 128, 128              # 5.9 GB a tensor
    k = torch.empty((pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c, q, table, lengths, slots = _attention_case([500, 200], 8, Hkv, D, page, "bf16", "16", 83)
    small = nv.paged_attention(q, block_table=table, lengths=lengths, **c)
    high = torch.where(table >= 0, pages - 1 - table, table)
    rows = nv.cache_read(slots=slots, **c)
    far = (pages - 1 - slots // page) * page + slots % page
    nv.rope_cache_write(rows[0], rows[0], rows[1], slots, nv.rope_table(1, 0), k, v, far)
    assert torch.equal(nv.paged_attention(q, k, v, high, lengths), small)
    back = nv.cache_read(k, v, far)
    assert torch.equal(back[0], rows[0]) and torch.equal(back[1], rows[1])
    gu.check_device_status()


def test_side_stream_and_graph_replay_as_sequences_grow():
    c, q, table, lengths, slots = _attention_case([200, 64], 8, 2, 128, 16, "bf16", "e4m3", 84)
    want = {}
    for n in ((200, 64), (17, 1), (0, 63)):
        lengths.copy_(torch.tensor(n, dtype=torch.int32))
        want[n] = nv.paged_attention(q, block_table=table, lengths=lengths, **c)
    size = nv.paged_attention_workspace_size(2, 8, 2, 128)
    ws = torch.full((max(size, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        nv.paged_attention(q, block_table=table, lengths=lengths, out=out, workspace=ws, **c)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            nv.paged_attention(q, block_table=table, lengths=lengths, out=out, workspace=ws, **c)
        for n, w in want.items():
            lengths.copy_(torch.tensor(n, dtype=torch.int32))
            out.fill_(3.0)
            g.replay()
            s.synchronize()
            assert torch.equal(out, w)
    torch.cuda.current_stream().wait_stream(s)


def test_refusals():
    g = _gen(90)
    x, w = _randn(g, (4, 64)), _randn(g, (64,))
    c = _make_cache(4, 2, 16, 64, "bf16", "16")
    e = _make_cache(4, 2, 16, 64, "bf16", "e4m3")
    q, kv = _randn(g, (3, 8, 64)), _randn(g, (3, 2, 64))
    slots, table = torch.arange(3, device="cuda"), nv.rope_table(8, 64)
    bt, n = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")

    def refused(status, fn, *a, **kw):
        with pytest.raises(nv.Nvfp4Error) as err:
            fn(*a, **kw)
        assert err.value.status == status, err.value

    refused(1, nv.rms_norm, x.float(), w)
    refused(1, nv.rms_norm, x, w.half())
    refused(2, nv.rms_norm, x, w[:32])
    refused(1, nv.rms_norm, x.cpu(), w)
    refused(1, nv.rms_norm, x.t(), w[:4])
    refused(1, nv.rms_norm, x, w, eps=float("nan"))
    refused(1, nv.rms_norm, x, w, residual_out=x)
    refused(2, nv.rms_norm_e4m3, x, w, group=24)
    refused(2, nv.rms_norm_e4m3, x, w, group=8)
    refused(2, nv.rms_norm_e4m3, x, w, group=-16)
    write = lambda q=q, k=kv, v=kv, pos=slots, tab=table, slots=slots, cc=c, **kw: nv.rope_cache_write(  # noqa: E731
        q, k, v, pos, tab, slots=slots, **cc, **kw)
    refused(1, write, q=q.half())
    refused(2, write, k=kv[:2])
    refused(2, write, q=_randn(g, (3, 8, 32)))
    refused(1, write, slots=slots.int())
    refused(2, write, tab=nv.rope_table(8, 80))
    refused(2, write, pos=torch.zeros((3, 3), dtype=torch.int64, device="cuda"), sections=[8, 8, 8])
    refused(2, write, pos=torch.zeros((5, 3), dtype=torch.int64, device="cuda"), sections=[8, 8, 8, 4, 4])
    refused(1, write, pos=torch.zeros((2, 3), dtype=torch.int64, device="cuda"), sections=[40, -8])
    refused(1, write, cc=dict(e, k_scale=None))
    refused(1, write, cc=dict(c, k_scale=e["k_scale"], v_scale=e["v_scale"]))
    refused(1, write, cc=dict(c, v_cache=c["v_cache"].transpose(1, 2).contiguous().transpose(1, 2)))
    refused(3, write, q=_randn(g, (3, 8, 65))[:, :, 1:])
    attend = lambda q=q, bt=bt, n=n, cc=c, **kw: nv.paged_attention(q, block_table=bt, lengths=n, **cc, **kw)  # noqa: E731
    refused(2, attend, q=_randn(g, (3, 7, 64)))
    refused(1, attend, n=n.long())
    refused(2, attend, n=n[:2])
    refused(1, attend, window=-1)
    refused(1, attend, softmax_scale=float("inf"))
    refused(1, attend, bt=bt.t().contiguous().t())
    refused(2, attend, cc=_make_cache(4, 2, 16, 24, "bf16", "16"), q=_randn(g, (3, 8, 24)))
    if nv.paged_attention_workspace_size(3, 8, 2, 64):
        refused(4, attend, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    refused(1, nv.cache_read, slots=slots, **e)
    refused(1, nv.cache_read, slots=slots, dtype=torch.float16, **c)
    assert attend(q=q[:0], bt=bt[:0], n=n[:0]).shape == (0, 8, 64)
    assert write(q=q[:0], k=kv[:0], v=kv[:0], pos=slots[:0], slots=slots[:0]).shape == (0, 8, 64)
    assert nv.cache_read(slots=slots[:0], **c)[0].shape == (0, 2, 64)
    gu.check_device_status()


def _far_token_case(act, kind, gap, spread, at, n=40000, B=320, Hkv=8, D=64, page=64):
    """One token `gap` above the rest in score, B sequences over the same pages: with as many
    (sequence, head) units as warps, a warp has the far token and thousands of others.  The
    far token's value is zero, from an E4M3 cache zero but for its first dimension."""
    g = _gen(int(gap) * 10 + at % 7 + (kind == "e4m3"))
    c = _make_cache(-(-n // page), Hkv, page, D, act, kind)
    k = torch.zeros(n, Hkv, D, device="cuda")
    k[:, :, 0] = spread * torch.randn(n, Hkv, generator=g, device="cuda")
    k[at, :, 0] = gap
    v = 1 + 0.1 * torch.randn(n, Hkv, D, generator=g, device="cuda")
    v[at] = 0
    if kind == "e4m3":
        v[at, :, 0] = 100.0
    else:
        v *= 1e4
    slots = torch.arange(n, device="cuda")
    k, v = k.to(DT[act]), v.to(DT[act])
    nv.rope_cache_write(k, k, v, slots, nv.rope_table(1, 0), slots=slots, **c)
    q = torch.zeros(B, Hkv, D, dtype=DT[act], device="cuda")
    q[:, :, 0] = 1
    table = torch.arange(-(-n // page), dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    out, lse = nv.paged_attention(q, block_table=table, lengths=torch.full((B,), n, dtype=torch.int32, device="cuda"),
                                  softmax_scale=1.0, return_lse=True, **c)
    gu.check_device_status()
    return c, slots, q, out, lse


@pytest.mark.parametrize("at", [0, 19999])
@pytest.mark.parametrize("spread", [0, 1])
@pytest.mark.parametrize("gap", [14, 17, 20, 24, 28])
@pytest.mark.parametrize("act", ["f16", "bf16"])
def test_paged_attention_beside_a_far_token_whose_value_is_zero(act, gap, spread, at):
    """The weights of the others keep their bits: a weight that meets the values as FP16 is
    off by 2^-11 of itself, or by 2^-25 of a step whose largest is 2^-7 at least; of 16 such and values
    0.5 to 1.5 times their mean, 2^-12 of the step's sum.  In the far token's own step 2^-36 of
    its weight is where FP16 ends.  BF16 weights are off by 2^-8.  Scores and sums in 32
    bits: 2^-12."""
    n = 40000
    c, slots, q, out, lse = _far_token_case(act, "16", gap, spread, at)
    k, v = _cached_values(c, "k", slots, 64), _cached_values(c, "v", slots, 64)
    ref, ref_lse, mag = layer.attend(_np(q[0]), k, v, 1.0)
    near = np.exp(np.minimum(k[at // 16 * 16:at // 16 * 16 + 16, :, 0] - gap, 0.0))      # [16, Hkv]
    lost = np.einsum("th,thd->hd", np.minimum(near, 2.0 ** -36), np.abs(v[at // 16 * 16:at // 16 * 16 + 16]))
    bound = U[act] * np.abs(ref) + TINY[act] + (U[act] + 2.0 ** -11) * mag + (lost if act == "f16" else 0)
    err = np.abs(_np(out) - ref[None])
    assert np.all(err <= bound[None]), (err / bound[None]).max()
    assert np.all(np.abs(_np(lse) - ref_lse[None]) <= 2.0 ** -17 * (1 + np.abs(ref_lse[None])))


@pytest.mark.parametrize("gap", [8, 14, 16, 17])
@pytest.mark.parametrize("act", ["f16", "bf16"])
def test_paged_attention_beside_a_far_token_in_e4m3(act, gap):
    """A weight times its value row's scale, as FP16, is off by 2^-11 of itself or by 2^-25 where
    the largest such product is 2^10 at least (2^11 over the scale rounded up to a power of two),
    which its codes, at most 448, multiply."""
    c, slots, q, out, lse = _far_token_case(act, "e4m3", gap, 0, 0)
    k, v = _cached_values(c, "k", slots, 64), _cached_values(c, "v", slots, 64)
    ref, ref_lse, mag = layer.attend(_np(q[0]), k, v, 1.0)
    s = c["v_scale"].transpose(1, 2).reshape(-1, 8)[slots].double().cpu().numpy()        # [n, Hkv]
    w = np.exp(k[:, :, 0] - k[:, :, 0].max(0))
    under = 2.0 ** -35 * (w * s).max(0) / w.sum(0) * (np.abs(v) / s[..., None]).sum(0).max(-1)
    bound = U[act] * np.abs(ref) + TINY[act] + (U["f16"] + 2.0 ** -12) * mag + under[:, None]
    err = np.abs(_np(out) - ref[None])
    assert np.all(err <= bound[None]), (err / bound[None]).max()
    assert np.all(np.abs(_np(lse) - ref_lse[None]) <= 2.0 ** -17 * (1 + np.abs(ref_lse[None])))


@pytest.mark.parametrize("act,kind,G,D", [("f16", "16", 1, 64), ("f16", "16", 4, 128), ("f16", "16", 12, 128),
                                          ("f16", "16", 16, 256), ("f16", "e4m3", 12, 64), ("bf16", "e4m3", 3, 128)])
def test_paged_attention_of_scores_that_fall_far_and_rise_again(act, kind, G, D):
    """Scores in stretches up to 60 apart, other ones for each head, one stretch after another:
    bases that fall, rise and fall again, and pieces of different bases joined.  Weights lost
    beside the stretches far above them are below 2^-36 of the largest each."""
    n = 9000
    case = _attention_case([n, 700], G * 2, 2, D, 16, act, kind, 85)
    c, q, table, lengths, slots = case
    g = _gen(86)
    T = slots.numel()
    level = torch.tensor([-3.0, 20, -25, 30, -30, 29, 5, -20, 30, 11], device="cuda")
    k = torch.zeros(T, 2, D, device="cuda")
    t = torch.cat([torch.arange(m) for m in lengths.tolist()]).cuda()
    for j in range(8):                                     # dimension j has the levels shifted by j
        k[:, :, j] = (level[(t // 137 + j) % 10] + torch.randn(T, generator=g, device="cuda"))[:, None]
    v = _randn(g, (T, 2, D), act)
    q = torch.zeros_like(q)
    for h in range(G * 2):
        q[:, h, h % 8] = 1
    k = k.to(DT[act])
    nv.rope_cache_write(k, k, v, slots, nv.rope_table(1, 0), slots=slots, **c)
    _check_attention(c, q, table, lengths, slots, 16, act, kind, scale=1.0)


def _half_step(x, act):
    """Half the distance of neighbouring 16-bit values at x."""
    _, e = np.frexp(x)
    least, bits = (-126, 8) if act == "bf16" else (-14, 11)
    return np.exp2(np.maximum(e - 1, least).astype(float) - bits)


@pytest.mark.parametrize("gap", [0.3, 0.55, 0.8])
@pytest.mark.parametrize("G,D", [(1, 64), (12, 64), (4, 128), (16, 128), (2, 256)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_paged_attention_weights_keep_their_bits_over_16_bit_caches(act, G, D, gap):
    """One token in 16 has a higher score, all others equal weights, values of one sign: a
    rounding of the weights to 16 bits would move every output alike, by up to 2^-9
    (BF16) or 2^-12.  As two halves the weights are off by 2^-16 at most, sums in 32 bits over a few
    dozen steps and the exponentials by 2^-16: the rest is the output's one rounding."""
    c, q, table, lengths, slots = _attention_case([1500, 400, 17], G * 2, 2, D, 16, act, "16", 87)
    T = slots.numel()
    k = torch.zeros(T, 2, D, dtype=DT[act], device="cuda")
    t = torch.cat([torch.arange(m) for m in lengths.tolist()]).cuda()
    k[:, :, 0] = (t % 16 == 0)[:, None] * gap
    v = (1.5 + 0.1 * torch.randn(T, 2, D, generator=_gen(88), device="cuda")).to(DT[act])
    nv.rope_cache_write(k, k, v, slots, nv.rope_table(1, 0), slots=slots, **c)
    q = torch.zeros_like(q)
    q[:, :, 0] = 1
    out = _np(nv.paged_attention(q, block_table=table, lengths=lengths, softmax_scale=1.0, **c))
    gu.check_device_status()
    at = 0
    for b, n in enumerate(lengths.tolist()):
        ref, _, mag = layer.attend(_np(q[b]), _np(k[at:at + n]), _np(v[at:at + n]), 1.0)
        at += n
        bound = _half_step(ref, act) + 2.0 ** -15 * mag
        assert np.all(np.abs(out[b] - ref) <= bound), (b, (np.abs(out[b] - ref) / bound).max())


@pytest.mark.parametrize("G,D", [(2, 64), (10, 128), (2, 256), (16, 256)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_paged_attention_of_infinite_values_gives_infinities(act, G, D):
    """Values of plus and minus infinity beside finite ones, at weights of every rounding."""
    c, q, table, lengths, slots = _attention_case([300, 70], G * 2, 2, D, 16, act, "16", 89)
    kv = nv.cache_read(slots=slots, **c)
    v = kv[1].clone()
    v[::7, :, 3] = float("inf")
    v[5::11, :, 8] = float("-inf")
    nv.rope_cache_write(kv[0], kv[0], v, slots, nv.rope_table(1, 0), slots=slots, **c)
    out = nv.paged_attention(q, block_table=table, lengths=lengths, **c)
    assert torch.all(out[:, :, 3] == float("inf")) and torch.all(out[:, :, 8] == float("-inf"))
    rest = [d for d in range(D) if d not in (3, 8)]
    assert torch.all(out[:, :, rest].isfinite())


# (head dim, heads a key head) -> warps a block of the instance that has more of them, 8 heads a tile
WORKSPACE = [(64, 1, 16, 8), (64, 16, 16, 16), (128, 8, 16, 8), (128, 9, 12, 16), (256, 1, 8, 8), (256, 16, 8, 16), (200, 40, 8, 16)]


@pytest.mark.parametrize("D,G,warps,heads", WORKSPACE)
def test_paged_attention_workspace_is_what_the_kernels_use(D, G, warps, heads):
    """A partial result a warp and two a block of one block an SM; the bytes behind them stay."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    padded = 64 if D <= 64 else 128 if D <= 128 else 256
    size = nv.paged_attention_workspace_size(3, 2 * G, 2, D)
    assert size == sms * (2 + warps) * heads * (padded + 2) * 4
    if D % 16:
        return
    for kind in ("16", "e4m3"):
        case = _attention_case([9000, 33, 4000], 2 * G, 2, D, 16, "bf16", kind, 91)
        buf = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        _check_attention(*case, 16, "bf16", kind, workspace=buf[:size])
        assert torch.all(buf[size:] == 0xA5)
        with pytest.raises(nv.Nvfp4Error) as err:
            nv.paged_attention(case[1], block_table=case[2], lengths=case[3], workspace=buf[:size - 1], **case[0])
        assert err.value.status == 4


@pytest.mark.parametrize("T,H", [(64, 512), (700, 512), (64, 509), (3, 40008), (5, 20480), (400, 268)])
def test_norm_in_place_of_its_inputs(T, H):
    g = _gen(92)
    x, r, w = _randn(g, (T, H)), _randn(g, (T, H)), _randn(g, (H,))
    plain, (y, a) = nv.rms_norm(x, w), nv.rms_norm(x, w, residual=r)
    x1 = x.clone()
    assert nv.rms_norm(x1, w, out=x1) is x1 and torch.equal(x1, plain)
    for names in (("x", None), ("r", None), ("x", "r"), ("r", "x"), ("r", "r2"), (None, "x")):
        t = {"x": x.clone(), "r": r.clone(), None: None, "r2": torch.empty_like(r)}
        got, added = nv.rms_norm(t["x"], w, residual=t["r"], out=t[names[0]], residual_out=t[names[1]])
        assert torch.equal(got, y) and torch.equal(added, a)
        assert names[0] is None or got is t[names[0]]
        assert names[1] is None or added is t[names[1]]


@pytest.mark.parametrize("lengths,Hq,Hkv,D,act,kind", [([70001], 8, 1, 128, "bf16", "16"), ([9000, 0, 33, 4000], 40, 2, 64, "f16", "e4m3"),
                                                       ([120, 255, 1, 0], 16, 4, 128, "bf16", "e4m3"), ([30000, 5], 16, 1, 256, "f16", "16")])
def test_paged_attention_in_place_of_its_query(lengths, Hq, Hkv, D, act, kind):
    c, q, table, n, _ = _attention_case(lengths, Hq, Hkv, D, 16, act, kind, 93)
    want = nv.paged_attention(q, block_table=table, lengths=n, **c)
    got = nv.paged_attention(q, block_table=table, lengths=n, out=q, **c)
    assert got is q and torch.equal(got.view(torch.int16), want.view(torch.int16))
    gu.check_device_status()


def test_outputs_beside_and_between_inputs_are_taken_and_over_them_refused():
    g = _gen(94)
    w, T, H = _randn(g, (256,)), 6, 256
    pool = _randn(g, (4 * T * H,)).view(torch.bfloat16)

    def refused(fn, *a, **kw):
        with pytest.raises(nv.Nvfp4Error) as err:
            fn(*a, **kw)
        assert err.value.status == 1 and "overlap" in str(err.value)

    x = pool[:T * H].view(T, H)
    want = nv.rms_norm(x.clone(), w)
    assert torch.equal(nv.rms_norm(x, w, out=pool[T * H:2 * T * H].view(T, H)), want)
    refused(nv.rms_norm, x, w, out=pool[H:H + T * H].view(T, H))
    refused(nv.rms_norm, x, w, residual=_randn(g, (T, H)), residual_out=pool[8:8 + T * H].view(T, H))
    codes = pool.view(torch.uint8)[:T * H].view(E4M3).view(T, H)
    refused(nv.rms_norm_e4m3, x, w, out=codes)
    apart = pool.view(2, -1)[:, :H]                         # two rows far apart, the output between them
    want = nv.rms_norm(apart.clone(), w)
    assert torch.equal(nv.rms_norm(apart, w, out=pool[H:3 * H].view(2, H)), want)
    c = _make_cache(4, 2, 16, 64, "bf16", "16", fill=0.0)
    qkv = _randn(g, (3, 8, 64))
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    slots, table = torch.arange(3, device="cuda"), nv.rope_table(8, 64)
    refused(nv.rope_cache_write, q, k, v, slots, table, slots=slots, q_out=qkv.view(-1)[:3 * 4 * 64].view(3, 4, 64), **c)
    refused(nv.rope_cache_write, q, k, v, slots, table, slots=slots, q_out=c["v_cache"].view(-1)[:3 * 4 * 64].view(3, 4, 64), **c)
    one = [t[:1] for t in (q, k, v, slots)]                 # one token's heads are dense
    assert nv.rope_cache_write(*one, table, slots=slots[:1], q_out=one[0], **c) is one[0]
    out = torch.empty(2, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    refused(nv.cache_read, slots=slots, k_out=out[0], v_out=out[0], **c)
    refused(nv.cache_read, slots=slots, k_out=out[0], v_out=c["k_cache"].view(-1)[:3 * 2 * 64].view(3, 2, 64), **c)
    nv.cache_read(slots=slots, k_out=out[0], v_out=out[1], **c)
    bt, n = torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    refused(nv.paged_attention, q.contiguous(), block_table=bt, lengths=n, out=c["k_cache"].view(-1)[:3 * 4 * 64].view(3, 4, 64), **c)
    refused(nv.paged_attention, q, block_table=bt, lengths=n, out=qkv.view(-1)[:3 * 4 * 64].view(3, 4, 64), **c)
    gu.check_device_status()


@pytest.mark.parametrize("heads,page,pages", [(1, 16, 5), (2, 1, 30), (1, 1, 30), (2, 32, 1), (1, 32, 1)])
@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_cache_strides_of_dimensions_of_one_element_do_not_matter(heads, page, pages, kind):
    """Keys laid out [pages, heads, page, D] and values [pages, page, heads, D]: the same places
    where there is one head or one token a page, whatever strides torch gives that dimension."""
    D, n = 64, 25
    a = _make_cache(pages, heads, page, D, "bf16", kind)
    b = dict(a, k_cache=a["k_cache"].clone() if kind == "16" else a["k_cache"].view(torch.uint8).clone().view(E4M3))
    b["v_cache"] = _make_cache(pages, heads, page, D, "bf16", kind, layout="nhd")["v_cache"]
    shape = a["k_cache"].shape
    odd = [s if m > 1 else 8 * i + 3 for i, (s, m) in enumerate(zip(a["k_cache"].stride(), shape))]
    c = dict(b, v_cache=torch.as_strided(b["v_cache"], shape, b["v_cache"].stride()),
             k_cache=torch.as_strided(b["k_cache"].clone() if kind == "16" else b["k_cache"].view(torch.uint8).clone().view(E4M3), shape, odd))
    for t in (b, c):
        t.update({s: a[s].clone() for s in ("k_scale", "v_scale") if s in a})
    if heads > 1 and page > 1:
        b["v_cache"] = c["v_cache"] = torch.empty_like(a["v_cache"])
    g = _gen(95)
    q, k, v = _randn(g, (n, 4, D)), _randn(g, (n, heads, D)), _randn(g, (n, heads, D))
    slots, table = torch.arange(n, device="cuda"), nv.rope_table(n, D)
    bt = torch.arange(-(-n // page), dtype=torch.int32, device="cuda")[None]
    got = []
    for t in (a, b, c):
        turned = nv.rope_cache_write(q, k, v, slots, table, slots=slots, **t)
        rows = nv.cache_read(slots=slots, dtype=torch.bfloat16, **t)
        got.append((turned, *rows, nv.paged_attention(q[:1], block_table=bt, lengths=slots[-1:].int(), **t)))
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))
    gu.check_device_status()


@pytest.mark.parametrize("T,H,group", [(400, 5120, 128), (400, 5120, 16), (400, 16384, 256), (400, 2304, 64),       # four pieces, several warps a row
                                       (3, 16392, 0), (320, 16392, 0), (2, 20480, 32), (400, 20480, 128), (330, 32768, 0), (2, 32768, 256)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_norm_e4m3_of_many_and_of_wide_rows(T, H, group, act):
    test_norm_e4m3(T, H, group, act)


@pytest.mark.parametrize("T,H", [(1, 16392), (320, 16392), (7, 20480), (400, 20480), (310, 32768), (2, 32768)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_norm_of_wide_rows(T, H, act):
    g = _gen(T + H)
    x, w, r = _randn(g, (T, H), act), _randn(g, (H,), act), _randn(g, (T, H), act)
    _close16(nv.rms_norm(x, w, eps=1e-5), layer.rms_norm(_np(x), _np(w), 1e-5), act)
    y, added = nv.rms_norm(x, w, residual=r)
    assert torch.equal(added, (x.float() + r.float()).to(DT[act]))
    _close16(y, layer.rms_norm(_np(added), _np(w), 1e-6), act)


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,sections", [(3000, 8, 2, 80, 40, None), (2900, 9, 3, 112, 56, [10, 9, 9]), (1500, 24, 1, 256, 136, [1, 67])])
def test_rope_interleaved_in_pieces_of_four_with_many_heads_a_thread(T, Hq, Hkv, D, rot, sections, act, kind):
    test_rope_cache_write_and_read(T, Hq, Hkv, D, rot, 16, sections, True, act, kind, "hnd")


@pytest.mark.parametrize("gap", [0.3, 0.55, 0.8])
@pytest.mark.parametrize("G,D", [(1, 64), (4, 128), (8, 128), (2, 256)])
def test_paged_attention_weights_keep_their_bits_over_e4m3_caches(G, D, gap):
    """As over 16-bit caches, of an FP16 output (BF16's rounding is eight times that of the weights):
    rows of one scale, so that a rounding of weight times scale would move every output alike."""
    c, q, table, lengths, slots = _attention_case([1500, 400, 17], G * 2, 2, D, 16, "f16", "e4m3", 96)
    T = slots.numel()
    k = torch.zeros(T, 2, D, dtype=torch.float16, device="cuda")
    t = torch.cat([torch.arange(m) for m in lengths.tolist()]).cuda()
    k[:, :, 0] = (t % 16 == 0)[:, None] * gap
    v = (1.5 + 0.1 * torch.randn(T, 2, D, generator=_gen(97), device="cuda")).clamp(0, 1.9).half()
    v[:, :, 5] = 2.0
    nv.rope_cache_write(k, k, v, slots, nv.rope_table(1, 0), slots=slots, **c)
    q = torch.zeros_like(q)
    q[:, :, 0] = 1
    out = _np(nv.paged_attention(q, block_table=table, lengths=lengths, softmax_scale=1.0, **c))
    gu.check_device_status()
    kk, vv = _cached_values(c, "k", slots, 16), _cached_values(c, "v", slots, 16)
    at = 0
    for b, n in enumerate(lengths.tolist()):
        ref, _, mag = layer.attend(_np(q[b]), kk[at:at + n], vv[at:at + n], 1.0)
        at += n
        bound = _half_step(ref, "f16") + 2.0 ** -15 * mag
        assert np.all(np.abs(out[b] - ref) <= bound), (b, (np.abs(out[b] - ref) / bound).max())
