"""The operators around a decoder layer's linears, measured: RMS norm with the
residual's addition (16-bit and E4M3 outputs), rotary positions with the write
into a paged key-value cache, reading that cache back, and the attention of one
new token over it.

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, by the framework's entry points.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100
EPS = 1e-6


def listed():
    return [
        # one token's hidden state between two linears of a decode step
        dict(name="norm decode 1x4096", op="norm", T=1, H=4096, dtype="bf16"),
        # a prompt chunk ahead of a large prefill linear
        dict(name="norm prefill 8192x8192", op="norm", T=8192, H=8192, dtype="bf16"),
        # an odd batch of an odd width, one E4M3 scale a row
        dict(name="norm8 333x2064 rows", op="norm8", T=333, H=2064, dtype="f16", group=0),
        # a prompt chunk with E4M3 scales of 128 columns
        dict(name="norm8 4096x5120 g128", op="norm8", T=4096, H=5120, dtype="bf16", group=128),
        # a decode batch into an 8-bit cache
        dict(name="write decode 16 e4m3", op="write", T=16, Hq=32, Hkv=8, D=128, rot=128, page=16, axes=1,
             interleaved=False, dtype="bf16", cache="e4m3"),
        # a prompt with image tokens (time, height, width) into a 16-bit cache
        dict(name="write prompt 4096 3-axis", op="write", T=4096, Hq=40, Hkv=8, D=128, rot=128, page=64, axes=3,
             interleaved=False, dtype="bf16", cache="16"),
        # a short prefix read back
        dict(name="read 301 f16", op="read", T=301, Hkv=8, D=128, page=16, dtype="f16", cache="e4m3"),
        # a long prefix read back for the next prompt chunk
        dict(name="read 65536 e4m3", op="read", T=65536, Hkv=8, D=128, page=32, dtype="bf16", cache="e4m3"),
        # one short conversation
        dict(name="attend 1x1000", op="attend", B=1, Hq=32, Hkv=8, D=128, page=16, lo=1000, hi=1000, window=0,
             dtype="bf16", cache="16"),
        # a ragged batch, one row still empty, 8-bit cache
        dict(name="attend 16x4096 e4m3", op="attend", B=16, Hq=32, Hkv=8, D=128, page=16, lo=0, hi=4096, window=0,
             dtype="bf16", cache="e4m3"),
        # many sequences with a sliding window, as many key heads as query heads, odd page size
        dict(name="attend 48x3001 window", op="attend", B=48, Hq=16, Hkv=16, D=64, page=24, lo=17, hi=3001,
             window=1024, dtype="f16", cache="16"),
        # a full serving batch with long contexts
        dict(name="attend 64x16384", op="attend", B=64, Hq=64, Hkv=8, D=128, page=64, lo=129, hi=16384, window=0,
             dtype="bf16", cache="16"),
    ]


def _spread(rng, lo, hi):
    """Log-uniform whole number in [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "write", "read", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op in ("norm", "norm8"):
        H = rng.choice([1024, 2048, 2064, 4096, 5120, 7168, 8192, 720, 1000, _spread(rng, 64, 16384)])
        group = rng.choice([g for g in (0, 0, 16, 32, 64, 128, 256) if g == 0 or H % g == 0])
        T = _spread(rng, 1, max(1, 8192 * 8192 // H // 2))
        c = dict(op=op, T=T, H=H, dtype=dtype)
        return dict(c, group=group) if op == "norm8" else c
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    D = rng.choice([64, 80, 128, 128, 128, 256])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    cache = rng.choice(["16", "e4m3"])
    G = rng.choice([1, 2, 4, 5, 8, 12, 16])
    if op == "write":
        axes = rng.choice([1, 1, 2, 3, 4])
        rot = rng.choice([D, D, D // 2])
        T = _spread(rng, 1, max(1, 4096 * 128 * 56 // (D * Hkv * (G + 2))))
        return dict(op=op, T=min(T, 16384), Hq=G * Hkv, Hkv=Hkv, D=D, rot=rot, page=page, axes=axes,
                    interleaved=rng.random() < 0.3, dtype=dtype, cache=cache)
    if op == "read":
        T = _spread(rng, 1, min(65536, 65536 * 1024 // (Hkv * D)))
        return dict(op=op, T=T, Hkv=Hkv, D=D, page=page, dtype=dtype, cache=cache)
    hi = _spread(rng, 1, 131072)
    most = max(1, 64 * 8192 * 1024 // (hi * Hkv * D))
    B = _spread(rng, 1, min(256, most))
    if hi * Hkv * D > 64 * 8192 * 1024:
        hi = 64 * 8192 * 1024 // (Hkv * D)
    lo = rng.choice([hi, hi // 2, 0, min(hi, 1)])
    window = rng.choice([0, 0, 0, _spread(rng, 16, 8192)])
    return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, page=page, lo=lo, hi=hi, window=window, dtype=dtype,
                cache=cache)


def _lengths(case):
    """Tokens cached of each sequence: evenly spread from lo to hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi] if B == 1 else [lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _attended(case):
    w = case["window"]
    return sum(min(n, w) if w else n for n in _lengths(case))


def _sections(case):
    """Frequencies of each axis: as even as they go, the first axis the rest."""
    half, axes = case["rot"] // 2, case["axes"]
    part = half // axes
    return [half - part * (axes - 1)] + [part] * (axes - 1)


def work(case):
    op = case["op"]
    if op in ("norm", "norm8"):
        T, H = case["T"], case["H"]
        size = 2 * T * H * 3 + 2 * H                                # x, residual, its sum; the weight
        if op == "norm":
            return {"bytes": size + 2 * T * H, "flops": 6 * T * H}
        groups = H // case["group"] if case["group"] else 1
        return {"bytes": size + T * H + 4 * T * groups, "flops": 8 * T * H}
    Hkv, D = case["Hkv"], case["D"]
    row = D * (1 if case["cache"] == "e4m3" else 2) + (4 if case["cache"] == "e4m3" else 0)   # one head's key or value
    if op == "write":
        T, Hq = case["T"], case["Hq"]
        size = T * (2 * D * (Hq + 2 * Hkv) + 2 * D * Hq + 2 * Hkv * row)
        return {"bytes": size + T * (4 * case["rot"] + 8 * case["axes"] + 8), "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    if op == "read":
        T = case["T"]
        return {"bytes": T * (2 * Hkv * row + 2 * Hkv * D * 2 + 8), "flops": 2 * T * Hkv * D}
    tokens, B, Hq = _attended(case), case["B"], case["Hq"]
    return {"bytes": 2 * Hkv * row * tokens + 4 * B * Hq * D + 4 * B * Hq + 4 * (tokens // case["page"] + 2 * B),
            "flops": 4 * Hq * D * tokens}


# ------------------------------------------------------------------ inputs ---

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _cache(g, pages, case):
    """A paged cache in use: keys and values, and their scales where it is held in 8 bits."""
    Hkv, page, D, dt = case["Hkv"], case["page"], case["D"], DTYPES[case["dtype"]]
    shape = (pages, Hkv, page, D)
    k, v = _normal(g, shape, dt), _normal(g, shape, dt)
    if case["cache"] == "16":
        return dict(k_cache=k, v_cache=v, k_scale=None, v_scale=None)
    ks = (k.abs().amax(-1).float() / E4M3_MAX).clamp_min_(MIN_SCALE)
    vs = (v.abs().amax(-1).float() / E4M3_MAX).clamp_min_(MIN_SCALE)
    return dict(k_cache=(k / ks[..., None].to(dt)).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3),
                v_cache=(v / vs[..., None].to(dt)).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3), k_scale=ks, v_scale=vs)


def prepare(case, seed):
    op, dt, g = case["op"], DTYPES[case["dtype"]], _gen(seed)
    r = np.random.RandomState(int(seed) % (1 << 32))
    if op in ("norm", "norm8"):
        T, H = case["T"], case["H"]
        weight = (1 + 0.1 * _normal(g, (H,), torch.float32)).to(dt)
        return dict(case=case, x=_normal(g, (T, H), dt), residual=3 * _normal(g, (T, H), dt), weight=weight)
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    if op == "attend":
        B, Hq = case["B"], case["Hq"]
        lengths = r.permutation(np.array(_lengths(case), dtype=np.int64))
        per = -(-lengths // page)
        width = max(1, int(per.max()))
        pages = int(per.sum()) + 3
        order = r.permutation(pages).astype(np.int32)
        table = np.zeros((B, width), dtype=np.int32)
        held = np.arange(width)[None, :] < per[:, None]
        table[held] = order[:int(per.sum())]
        return dict(case=case, q=_normal(g, (B, Hq, D), dt), block_table=torch.from_numpy(table).cuda(),
                    lengths=torch.from_numpy(lengths.astype(np.int32)).cuda(), **_cache(g, pages, case))
    T = case["T"]
    pages = -(-T // page) + 3
    slots = torch.from_numpy(r.permutation(pages)[:, None].astype(np.int64) * page + np.arange(page)[None, :])
    slots = slots.reshape(-1)[:T].contiguous().cuda()               # whole pages in any order, the last one partly filled
    if op == "read":
        return dict(case=case, slots=slots, **_cache(g, pages, case))
    Hq, rot, axes = case["Hq"], case["rot"], case["axes"]
    most = 32768
    angle = np.arange(most)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))[None, :]
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
    start = int(r.randint(0, most - T))
    positions = start + np.arange(T, dtype=np.int64)
    if axes > 1:                                                    # image tokens: later axes run over a grid
        positions = np.stack([positions] + [start + (np.arange(T) // 24 ** a) % 24 for a in range(axes - 1)])
    qkv = _normal(g, (T, Hq + 2 * Hkv, D), dt)                      # one fused projection's output
    return dict(case=case, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], table=table, slots=slots,
                positions=torch.from_numpy(np.ascontiguousarray(positions)).cuda(),
                sections=_sections(case) if axes > 1 else None, **_cache(g, pages, case))


# ------------------------------------------------------------- plain forms ---

def _quantise(y):
    """Codes and scales over the last dimension."""
    s = (y.abs().amax(-1) / E4M3_MAX).clamp_min(MIN_SCALE)
    return (y / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), s


def _plain_norm(st):
    c, x = st["case"], st["x"]
    added = (x.float() + st["residual"].float()).to(x.dtype)
    r = added.float()
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * st["weight"].float()
    if c["op"] == "norm":
        return y.to(x.dtype), added
    T, H = x.shape
    codes, scales = _quantise(y.view(T, -1, c["group"] or H))
    return codes.view(T, H), scales, added


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_write(st):
    c, half = st["case"], st["case"]["rot"] // 2
    pos = st["positions"]
    if c["axes"] > 1:
        axis = torch.repeat_interleave(torch.arange(c["axes"], device="cuda"),
                                       torch.tensor(st["sections"], device="cuda"), output_size=half)
        pos = pos[axis].t()                                         # [T, half]
        f = torch.arange(half, device="cuda")
        cos, sin = st["table"][pos, f], st["table"][pos, half + f]
    else:
        rows = st["table"][pos]
        cos, sin = rows[:, :half], rows[:, half:]
    cos, sin = cos[:, None, :], sin[:, None, :]
    q = _rotate(st["q"], cos, sin, c["rot"], c["interleaved"]).to(st["q"].dtype)
    k, v = _rotate(st["k"], cos, sin, c["rot"], c["interleaved"]), st["v"].float()
    page, at = st["slots"] // c["page"], st["slots"] % c["page"]
    if c["cache"] == "16":
        st["k_cache"][page, :, at] = k.to(st["k_cache"].dtype)
        st["v_cache"][page, :, at] = v.to(st["v_cache"].dtype)
        return q, st["k_cache"], st["v_cache"]
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    st["k_cache"].view(torch.uint8)[page, :, at] = kc.view(torch.uint8)
    st["v_cache"].view(torch.uint8)[page, :, at] = vc.view(torch.uint8)
    st["k_scale"][page, :, at], st["v_scale"][page, :, at] = ks, vs
    return q, st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]


def _rows(cache, scale, page, at):
    if scale is None:
        return cache[page, :, at].float()
    codes = cache.view(torch.uint8)[page, :, at].view(E4M3)
    return codes.float() * scale[page, :, at][..., None]


def _plain_read(st):
    c, dt = st["case"], DTYPES[st["case"]["dtype"]]
    page, at = st["slots"] // c["page"], st["slots"] % c["page"]
    return (_rows(st["k_cache"], st["k_scale"], page, at).to(dt), _rows(st["v_cache"], st["v_scale"], page, at).to(dt))


def _pages(cache, scale, table):
    """[B, Hkv, tokens, D] in 32 bits of the pages in the table."""
    if scale is None:
        x = cache[table].float()
    else:
        x = cache.view(torch.uint8)[table].view(E4M3).float() * scale[table][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(st):
    c, q = st["case"], st["q"]
    B, Hq, D = q.shape
    table, n = st["block_table"].long(), st["lengths"].long()
    k = _pages(st["k_cache"], st["k_scale"], table)
    z = torch.matmul(q.float().view(B, c["Hkv"], -1, D), k.transpose(2, 3)) * D ** -0.5
    del k
    t = torch.arange(z.shape[-1], device="cuda")
    held = t[None, :] < n[:, None]
    if c["window"]:
        held = held & (t[None, :] >= n[:, None] - c["window"])
    z = z.masked_fill(~held[:, None, None, :], -math.inf)
    m = z.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, _pages(st["v_cache"], st["v_scale"], table)) / total.clamp_min(1e-38)
    lse = (m + torch.log(total)).masked_fill(total == 0, -math.inf)
    return out.view(B, Hq, D).to(q.dtype), lse.view(B, Hq)


def _own(st):
    import w4a16_nvfp4_weight_gb300 as nv
    c = st["case"]
    op = c["op"]
    if op == "norm":
        return nv.rms_norm(st["x"], st["weight"], eps=EPS, residual=st["residual"])
    if op == "norm8":
        return nv.rms_norm_e4m3(st["x"], st["weight"], eps=EPS, residual=st["residual"], group=c["group"])
    if op == "write":
        q = nv.rope_cache_write(st["q"], st["k"], st["v"], st["positions"], st["table"], st["k_cache"], st["v_cache"],
                                st["slots"], k_scale=st["k_scale"], v_scale=st["v_scale"], sections=st["sections"],
                                interleaved=c["interleaved"])
        if c["cache"] == "16":
            return q, st["k_cache"], st["v_cache"]
        return q, st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]
    if op == "read":
        return nv.cache_read(st["k_cache"], st["v_cache"], st["slots"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                             dtype=DTYPES[c["dtype"]])
    return nv.paged_attention(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["lengths"],
                              k_scale=st["k_scale"], v_scale=st["v_scale"], window=c["window"], return_lse=True)


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm8": _plain_norm, "write": _plain_write, "read": _plain_read,
            "attend": _plain_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact ---

def _exact_codes(y):
    """E4M3 values nearest to y / s in 64 bits, and s: the grid has 3 bits below the leading one, and steps of 2^-9 below 2^-6."""
    s = torch.clamp(y.abs().amax(-1) / E4M3_MAX, min=MIN_SCALE)
    x = y / s.unsqueeze(-1)
    _, e = torch.frexp(x)
    step = torch.pow(2.0, torch.clamp(e.double() - 4, min=-9.0))
    return torch.clamp(torch.round(x / step) * step, -E4M3_MAX, E4M3_MAX), s


def _exact_norm(st):
    c = st["case"]
    dt = st["x"].dtype
    added = (st["x"].double() + st["residual"].double()).to(torch.float32).to(dt)    # 16-bit sums are exact or far from ties in 32
    r = added.double()
    rms = torch.sqrt(torch.sum(r ** 2, 1) / r.shape[1] + EPS)
    y = r / rms.unsqueeze(1) * st["weight"].double()
    if c["op"] == "norm":
        return y, added.double()
    parts = y.reshape(c["T"], c["H"] // (c["group"] or c["H"]), c["group"] or c["H"])
    codes, scales = _exact_codes(parts)
    return codes.reshape(c["T"], c["H"]), scales, added.double()


def _exact_turn(x, st):
    """Rotation as a complex product."""
    c, rot = st["case"], st["case"]["rot"]
    half = rot // 2
    x = x.double()
    T = x.shape[0]
    z = torch.empty(T, 1, half, dtype=torch.complex128, device="cuda")
    sections, pos = st["sections"] or [half], st["positions"].reshape(c["axes"], T)
    at = 0
    for a, size in enumerate(sections):
        rows = st["table"][pos[a]].double()
        z[:, 0, at:at + size] = torch.complex(rows[:, at:at + size], rows[:, half + at:half + at + size])
        at += size
    out = x.clone()
    if c["interleaved"]:
        y = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * z
        out[..., 0:rot:2], out[..., 1:rot:2] = y.real, y.imag
    else:
        y = torch.complex(x[..., :half], x[..., half:rot]) * z
        out[..., :half], out[..., half:rot] = y.real, y.imag
    return out


def _exact_write(st):
    c = st["case"]
    q, new = _exact_turn(st["q"], st), (_exact_turn(st["k"], st), st["v"].double())
    where, inside = torch.div(st["slots"], c["page"], rounding_mode="floor"), torch.remainder(st["slots"], c["page"])
    caches, scales = [], []
    for x, name in zip(new, ("k", "v")):
        held = st[name + "_cache"].double()
        if c["cache"] == "e4m3":
            x, s = _exact_codes(x)
            whole = st[name + "_scale"].double()
            whole[where, :, inside] = s
            scales.append(whole)
        held[where, :, inside] = x
        caches.append(held)
    return tuple([q] + caches + scales)


def _exact_read(st):
    c = st["case"]
    out = []
    for name in ("k", "v"):
        held = st[name + "_cache"].double()
        if c["cache"] == "e4m3":
            held *= st[name + "_scale"].double().unsqueeze(-1)
        out.append(held.transpose(1, 2).reshape(-1, c["Hkv"], c["D"])[st["slots"]])
    return tuple(out)


def _exact_attend(st):
    c = st["case"]
    B, Hq, D, Hkv = c["B"], c["Hq"], c["D"], c["Hkv"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lengths"].tolist()):
        if n == 0:
            continue
        first = max(0, n - c["window"]) if c["window"] else 0
        pages = st["block_table"][b, :-(-n // c["page"])].long()
        kv = []
        for name in ("k", "v"):
            x = st[name + "_cache"][pages].double()
            if c["cache"] == "e4m3":
                x = x * st[name + "_scale"][pages].double().unsqueeze(-1)
            kv.append(x.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, first:n])
        z = torch.einsum("hgd,htd->hgt", st["q"][b].double().reshape(Hkv, Hq // Hkv, D), kv[0]) / math.sqrt(D)
        lse[b] = torch.logsumexp(z, -1).reshape(Hq)
        out[b] = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), kv[1]).reshape(Hq, D)
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm8": _exact_norm, "write": _exact_write, "read": _exact_read,
            "attend": _exact_attend}[case["op"]](st)
