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

An output over an input or another output is refused but where a function says that
it may be that input itself.
"""

import torch

from . import _lib


class _Unloaded:
    """Stands for the compiled entry points until the first call."""

    def __getattr__(self, name):
        global _ops
        _ops = _lib.load_binding()
        return getattr(_ops, name)


_ops = _Unloaded()


def rms_norm(x, weight, eps=1e-6, residual=None, residual_out=None, out=None):
    """y = RN(r * rsqrt(mean(r^2) + eps) * weight) over the rows of x [T, H] (any
    row stride), r = x, or RN(x + residual), which is returned too: y, or (y, r).
    ``out`` and ``residual_out`` may each be ``x`` or ``residual`` (contiguous), to
    work in place."""
    return _ops.rms_norm(x, weight, eps, residual, residual_out, out, False, 0, None)


def rms_norm_e4m3(x, weight, eps=1e-6, group=0, residual=None, residual_out=None, out=None, scales=None):
    """rms_norm with an 8-bit output: (codes [T, H] torch.float8_e4m3fn, scales
    [T, H / group] float32), and r where there is a residual.  Values are code *
    scale; ``group`` columns (16, 32, 64, 128 or 256; 0: the row) share the scale
    max(amax / 448, 2^-100), taken from the unrounded 32-bit values."""
    return _ops.rms_norm(x, weight, eps, residual, residual_out, out, True, group, scales)


def rope_table(rows, rot, base=10000.0, device="cuda"):
    """Table for rope_cache_write, built once at load: float32 [rows, rot], row p
    the rot/2 cosines, then the sines, of p * base^(-2i/rot), computed in 64 bits."""
    if rot < 0 or rot % 2 or rows < 0:
        raise _lib.Nvfp4Error(2, f"rot={rot} must be even and rows={rows} not negative")
    half = rot // 2
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * \
        base ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))[None, :]
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).to(device)


def rope_cache_write(q, k, v, positions, table, k_cache, v_cache, slots, k_scale=None, v_scale=None, sections=None,
                     interleaved=False, q_out=None):
    """Rotate q [T, Hq, D] and k [T, Hkv, D], and store k and v [T, Hkv, D] in the
    cache rows of ``slots`` (int64 [T]; negative: not stored).  Returns the rotated
    q [T, Hq, D] (``q_out`` may be q where it is contiguous).  q, k and v may be views of one projection's output (16-byte
    aligned rows).  ``positions``: int64 [T], or [axes, T] with ``sections`` (a
    list with the number of frequencies of each axis, at most four) for positions
    with several axes.  ``table``: float32 [rows, rot] (rope_table); elements from
    rot on are not rotated.  Pairs are (i, i + rot/2), or (2i, 2i + 1) when
    ``interleaved``.  Two tokens must not share a slot.  A position outside the
    table turns its elements by an angle of zero, a slot outside the cache is not written,
    and device_status() then reports 8."""
    return _ops.rope_cache_write(q, k, v, positions, table, k_cache, v_cache, slots, k_scale, v_scale, sections, interleaved,
                                 q_out)


def cache_read(k_cache, v_cache, slots, k_scale=None, v_scale=None, dtype=None, k_out=None, v_out=None):
    """(k, v) [T, heads, D] of the cache rows of ``slots`` (int64 [T]; negative:
    zeros), in the activation type: the cache's, or ``dtype`` for an E4M3 cache
    (RN(code * scale))."""
    return _ops.cache_read(k_cache, v_cache, slots, k_scale, v_scale, dtype, k_out, v_out)


def paged_attention_workspace_size(B, Hq, heads, head_dim):
    return int(_lib.load().nvfp4_paged_attention_workspace(B, Hq, heads, head_dim))


def paged_attention(q, k_cache, v_cache, block_table, lengths, k_scale=None, v_scale=None, softmax_scale=None, window=0,
                    out=None, return_lse=False, lse=None, workspace=None):
    """Attention of one new token per sequence: q [B, Hq, D] over the lengths[b]
    cached tokens of each sequence (int32 [B]; the new token's own key and value are
    in the cache already), whose pages are block_table[b] (int32 [B, width]).  Hq is
    a multiple of the cache's heads.  ``softmax_scale`` defaults to D^-0.5;
    ``window`` > 0 attends to the last ``window`` tokens only.  Returns out [B, Hq, D]
    (``out`` may be q where it is contiguous),
    with ``return_lse`` also the log-sum-exp of the scaled scores (float32 [B, Hq],
    natural log).  A sequence of length 0 gives zeros and -inf.  A length or page
    outside the table or the cache is taken as the nearest end or as page 0, and
    device_status() then reports 8.

    Several drafted tokens of one sequence are rows of their own with the same
    block table and lengths one apart."""
    return _ops.paged_attention(q, k_cache, v_cache, block_table, lengths, k_scale, v_scale, softmax_scale, window, out,
                                return_lse, lse, workspace)
