"""The operators between a decoder layer's linears: RMS norm (with the residual's
addition, 16-bit or E4M3 output), rotary positions with the write into a paged
key-value cache, the read of cached rows, and the attention of one new token per
sequence over that cache.

    y, h = rms_norm(x, w, residual=h)                            # h + x, normalised
    q = rope_cache_write(q, k, v, positions, table, kc, vc, slots)   # rotate, store k and v
    o = paged_attention(q, kc, vc, block_table, lengths)         # [B, Hq, D]

A cache is a pair of tensors [pages, heads, page_size, head_dim] (any strides
with rows of head_dim contiguous and on 16-byte boundaries, the same for both:
views of one interleaved pool will do) in the activation type, or in
torch.float8_e4m3fn with ``k_scale`` and ``v_scale`` float32 [pages, heads,
page_size].  Slot s of a token is page * page_size + offset.
"""

import ctypes
import math

import torch

from . import _lib
from ._lib import KVCache, Nvfp4Error

_E4M3 = torch.float8_e4m3fn
_F16S = {torch.bfloat16: 0, torch.float16: 1}
_raw_stream = torch._C._cuda_getCurrentRawStream


def _bad(status, message):
    raise Nvfp4Error(status, message)


def _device(t, name):
    """Index of the CUDA device that holds ``t``, which has to be the current one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _bad(1, f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        _bad(1, f"{name} is on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _activation(t, name):
    f16 = _F16S.get(t.dtype)
    if f16 is None:
        _bad(1, f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype}")
    return f16


def _check(t, name, dev, dtype, shape, contiguous=True):
    """A CUDA tensor of this type and shape, contiguous or with a contiguous last dimension."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _bad(1, f"{name} must be a tensor on cuda:{dev}")
    if t.dtype != dtype:
        _bad(1, f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        _bad(2, f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous:
        if not t.is_contiguous():
            _bad(1, f"{name} must be contiguous")
    elif shape[-1] > 1 and t.stride(-1) != 1:
        _bad(1, f"{name} must be contiguous in its last dimension")
    return t


def _norm(x, weight, eps, residual, residual_out, out, e4m3, group, scales):
    dev = _device(x, "x")
    f16 = _activation(x, "x")
    if x.dim() != 2:
        _bad(2, f"x must be [T, H], got {tuple(x.shape)}")
    shape, dt = x.shape, x.dtype
    T, H = shape
    if H > 1 and x.stride(1) != 1:
        _bad(1, "x must be contiguous in its last dimension")
    _check(weight, "weight", dev, dt, (H,))
    res, res_stride, res_out = None, 0, None
    if residual is not None:
        _check(residual, "residual", dev, dt, shape, False)
        res, res_stride = residual.data_ptr(), residual.stride(0)
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=dt, device=x.device)
        else:
            _check(residual_out, "residual_out", dev, dt, shape)
        res_out = residual_out.data_ptr()
    elif residual_out is not None:
        _bad(1, "residual_out needs a residual")
    if out is None:
        out = torch.empty(shape, dtype=_E4M3 if e4m3 else dt, device=x.device)
    else:
        _check(out, "out", dev, _E4M3 if e4m3 else dt, shape)
    if e4m3:
        if group < 0 or (group and H % group):
            _bad(2, f"group={group} must be 0 or divide H={H}")
        need = (T, H // group if group else 1)
        if scales is None:
            scales = torch.empty(need, dtype=torch.float32, device=x.device)
        else:
            _check(scales, "scales", dev, torch.float32, need)
    st = _lib.load().nvfp4_rms_norm(
        x.data_ptr(), x.stride(0), res, res_stride, weight.data_ptr(), T, H, eps, 1 if e4m3 else 0, group, f16,
        out.data_ptr(), scales.data_ptr() if e4m3 else None, res_out, _raw_stream(dev))
    if st:
        _lib.check(st)
    return out, scales, residual_out


def rms_norm(x, weight, eps=1e-6, residual=None, residual_out=None, out=None):
    """y = RN(r * rsqrt(mean(r^2) + eps) * weight) over the rows of x [T, H] (any
    row stride), r = x, or RN(x + residual), which is returned too: y, or (y, r).
    ``residual_out`` may be ``residual`` (contiguous) to add in place."""
    y, _, r = _norm(x, weight, eps, residual, residual_out, out, False, 0, None)
    return y if residual is None else (y, r)


def rms_norm_e4m3(x, weight, eps=1e-6, group=0, residual=None, residual_out=None, out=None, scales=None):
    """rms_norm with an 8-bit output: (codes [T, H] torch.float8_e4m3fn, scales
    [T, H / group] float32), and r where there is a residual.  Values are code *
    scale; ``group`` columns (16, 32, 64, 128 or 256; 0: the row) share the scale
    max(amax / 448, 2^-100), taken from the unrounded 32-bit values."""
    y, s, r = _norm(x, weight, eps, residual, residual_out, out, True, group, scales)
    return (y, s) if residual is None else (y, s, r)


def _cache(k_cache, v_cache, k_scale, v_scale, dev, dt):
    """The cache's descriptor for the C ABI."""
    e4m3 = isinstance(k_cache, torch.Tensor) and k_cache.dtype == _E4M3
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        _bad(2, "k_cache must be a tensor [pages, heads, page_size, head_dim]")
    shape = k_cache.shape
    pages, heads, page, D = shape
    _check(k_cache, "k_cache", dev, _E4M3 if e4m3 else dt, shape, False)
    _check(v_cache, "v_cache", dev, k_cache.dtype, shape, False)
    strides = k_cache.stride()
    if v_cache.stride() != strides:
        _bad(1, f"k_cache and v_cache must have the same strides, got {strides} and {v_cache.stride()}")
    if e4m3:
        if k_scale is None or v_scale is None:
            _bad(1, "an E4M3 cache needs k_scale and v_scale")
        ks = _check(k_scale, "k_scale", dev, torch.float32, shape[:3]).data_ptr()
        vs = _check(v_scale, "v_scale", dev, torch.float32, shape[:3]).data_ptr()
    else:
        if k_scale is not None or v_scale is not None:
            _bad(1, "k_scale and v_scale go with an E4M3 cache")
        ks = vs = None
    return KVCache(k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, pages, page, heads, D,
                   strides[0], strides[1], strides[2], 1 if e4m3 else 0)


def _heads(t, name, dev, dt, T, heads, D):
    return _check(t, name, dev, dt, (T, heads, D), False)


def rope_table(rows, rot, base=10000.0, device="cuda"):
    """Table for rope_cache_write, built once at load: float32 [rows, rot], row p
    the rot/2 cosines, then the sines, of p * base^(-2i/rot), computed in 64 bits."""
    if rot < 0 or rot % 2 or rows < 0:
        _bad(2, f"rot={rot} must be even and rows={rows} not negative")
    half = rot // 2
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * \
        base ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))[None, :]
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).to(device)


def rope_cache_write(q, k, v, positions, table, k_cache, v_cache, slots, k_scale=None, v_scale=None, sections=None,
                     interleaved=False, q_out=None):
    """Rotate q [T, Hq, D] and k [T, Hkv, D], and store k and v [T, Hkv, D] in the
    cache rows of ``slots`` (int64 [T]; negative: not stored).  Returns the rotated
    q [T, Hq, D].  q, k and v may be views of one projection's output (16-byte
    aligned rows).  ``positions``: int64 [T], or [axes, T] with ``sections`` (a
    list with the number of frequencies of each axis, at most four) for positions
    with several axes.  ``table``: float32 [rows, rot] (rope_table); elements from
    rot on are not rotated.  Pairs are (i, i + rot/2), or (2i, 2i + 1) when
    ``interleaved``.  Two tokens must not share a slot.  A position outside the
    table leaves its elements unrotated, a slot outside the cache is not written,
    and device_status() then reports 8."""
    dev = _device(q, "q")
    f16 = _activation(q, "q")
    if q.dim() != 3:
        _bad(2, f"q must be [T, Hq, D], got {tuple(q.shape)}")
    T, Hq, D = q.shape
    dt = q.dtype
    if D > 1 and q.stride(2) != 1:
        _bad(1, "q must be contiguous in its last dimension")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, dev, dt)
    if cache.head_dim != D:
        _bad(2, f"q has head_dim {D}, the cache {cache.head_dim}")
    _heads(k, "k", dev, dt, T, cache.heads, D)
    _heads(v, "v", dev, dt, T, cache.heads, D)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        _bad(2, "table must be a tensor [rows, rot]")
    _check(table, "table", dev, torch.float32, table.shape)
    if sections is None:
        axes, sec = 1, None
        _check(positions, "positions", dev, torch.int64, (T,) if positions.dim() == 1 else (1, T))
    else:
        axes = len(sections)
        if not 1 <= axes <= 4:
            _bad(2, f"sections must name 1 to 4 axes, got {axes}")
        sec = (ctypes.c_int32 * axes)(*sections)
        _check(positions, "positions", dev, torch.int64, (axes, T))
    _check(slots, "slots", dev, torch.int64, (T,))
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
    else:
        _check(q_out, "q_out", dev, dt, (T, Hq, D))
    st = _lib.load().nvfp4_rope_cache_write(
        q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
        v.stride(1), T, Hq, positions.data_ptr(), axes, sec, table.data_ptr(), table.shape[0], table.shape[1],
        1 if interleaved else 0, f16, slots.data_ptr(), cache, q_out.data_ptr(), _raw_stream(dev))
    if st:
        _lib.check(st)
    return q_out


def cache_read(k_cache, v_cache, slots, k_scale=None, v_scale=None, dtype=None, k_out=None, v_out=None):
    """(k, v) [T, heads, D] of the cache rows of ``slots`` (int64 [T]; negative:
    zeros), in the activation type: the cache's, or ``dtype`` for an E4M3 cache
    (RN(code * scale))."""
    dev = _device(k_cache, "k_cache")
    dt = k_cache.dtype if k_cache.dtype != _E4M3 else dtype
    if dt is None or (dtype is not None and dtype != dt) or dt not in _F16S:
        _bad(1, "dtype must be torch.bfloat16 or torch.float16, and the cache's own where that is 16-bit")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, dev, dt)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        _bad(2, "slots must be a tensor [T]")
    _check(slots, "slots", dev, torch.int64, slots.shape)
    shape = (slots.shape[0], cache.heads, cache.head_dim)
    outs = []
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        outs.append(torch.empty(shape, dtype=dt, device=k_cache.device) if t is None
                    else _check(t, name, dev, dt, shape))
    st = _lib.load().nvfp4_kv_cache_read(cache, slots.data_ptr(), shape[0], _F16S[dt], outs[0].data_ptr(),
                                         outs[1].data_ptr(), _raw_stream(dev))
    if st:
        _lib.check(st)
    return outs[0], outs[1]


def paged_attention_workspace_size(B, Hq, heads, head_dim):
    return int(_lib.load().nvfp4_paged_attention_workspace(B, Hq, heads, head_dim))


def paged_attention(q, k_cache, v_cache, block_table, lengths, k_scale=None, v_scale=None, softmax_scale=None, window=0,
                    out=None, return_lse=False, lse=None, workspace=None):
    """Attention of one new token per sequence: q [B, Hq, D] over the lengths[b]
    cached tokens of each sequence (int32 [B]; the new token's own key and value are
    in the cache already), whose pages are block_table[b] (int32 [B, width]).  Hq is
    a multiple of the cache's heads.  ``softmax_scale`` defaults to D^-0.5;
    ``window`` > 0 attends to the last ``window`` tokens only.  Returns out [B, Hq, D],
    with ``return_lse`` also the log-sum-exp of the scaled scores (float32 [B, Hq],
    natural log).  A sequence of length 0 gives zeros and -inf.  A length or page
    outside the table or the cache is taken as the nearest end or as page 0, and
    device_status() then reports 8.

    Several drafted tokens of one sequence are rows of their own with the same
    block table and lengths one apart."""
    dev = _device(q, "q")
    f16 = _activation(q, "q")
    if q.dim() != 3:
        _bad(2, f"q must be [B, Hq, D], got {tuple(q.shape)}")
    shape, dt = q.shape, q.dtype
    B, Hq, D = shape
    if D > 1 and q.stride(2) != 1:
        _bad(1, "q must be contiguous in its last dimension")
    cache = _cache(k_cache, v_cache, k_scale, v_scale, dev, dt)
    if cache.head_dim != D:
        _bad(2, f"q has head_dim {D}, the cache {cache.head_dim}")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        _bad(2, "block_table must be a tensor [B, width]")
    width = block_table.shape[1]
    _check(block_table, "block_table", dev, torch.int32, (B, width), False)
    _check(lengths, "lengths", dev, torch.int32, (B,))
    if out is None:
        out = torch.empty(shape, dtype=dt, device=q.device)
    else:
        _check(out, "out", dev, dt, shape)
    if lse is not None:
        _check(lse, "lse", dev, torch.float32, shape[:2])
    elif return_lse:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=q.device)
    h = _lib.load()
    need = h.nvfp4_paged_attention_workspace(B, Hq, cache.heads, D)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    else:
        _check(workspace, "workspace", dev, torch.uint8, workspace.shape)
    st = h.nvfp4_paged_attention(
        q.data_ptr(), q.stride(0), q.stride(1), cache, block_table.data_ptr(), block_table.stride(0), width,
        lengths.data_ptr(), B, Hq, softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(D), window, f16,
        out.data_ptr(), lse.data_ptr() if lse is not None else None,
        workspace.data_ptr() if workspace is not None else None, workspace.numel() if workspace is not None else 0,
        _raw_stream(dev))
    if st:
        _lib.check(st)
    return (out, lse) if return_lse else out
