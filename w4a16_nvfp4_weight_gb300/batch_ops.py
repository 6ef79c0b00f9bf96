"""What differs from request to request in a served batch: its pages, its adapter,
its next token.

    t = extend_tables(lengths, new_tokens, table, free_pages, free_count, page_size, rows)
    q = rope_cache_write(q, k, v, t["positions"], rope, kc, vc, t["slots"])
    y = lora_add(gemm(x, w), x, a, b, adapters)                      # beside a shared projection
    token = sample(gemm(h, head), u, temperature=0.8, top_p=0.95)
    lengths, free_count = trim_tables(lengths, keep, table, free_pages, free_count, page_size)

All of it stays on the device and can be captured in graphs: a decode loop needs no host.
"""

from . import _lib
from .layer_ops import _Unloaded

_ops = _Unloaded()


def extend_tables(lengths, new_tokens, block_table, free_pages, free_count, page_size, rows, row_tables=False, in_place=False):
    """Room for new_tokens[b] more tokens of each request (int32 [B], B at most 16384) that
    has lengths[b] (int32 [B]) in the pages block_table[b] (int32 [B, width]).  New pages
    come from the top of the stack free_pages[:free_count] (int32 [P] and int32 [1]), in
    the order of the requests, and are entered in ``block_table``.

    Returns a dict of
      positions, slots  int64 [rows] of the new tokens, request after request, as
                        rope_cache_write takes them; rows behind the last have 0 and -1,
      request           int32 [rows], whose token it is (-1 behind the last),
      starts            int32 [B + 1], the first row of each request,
      lengths, free_count  as they are from now on: new tensors, or with ``in_place`` the
                        given ones, updated,
      with ``row_tables`` also row_tables (int32 [rows, width]) and row_lengths (int32
                        [rows]): the block_table and lengths with which paged_attention
                        takes every row for itself (several drafted tokens of a request,
                        each over those before it).

    A request whose new length does not fit its table, whose rows do not all fit in
    ``rows``, or whose pages and those asked for before it are more than are free, is not
    served: its length stays, and its slots are -1.  A negative length or number of new
    tokens (not served), or a count outside the stack, makes device_status() report 8."""
    names = ("positions", "slots", "request", "starts", "lengths", "free_count", "row_tables", "row_lengths")
    return dict(zip(names, _ops.extend_tables(lengths, new_tokens, block_table, free_pages, free_count, page_size, rows,
                                              row_tables, in_place)))


def trim_tables(lengths, keep, block_table, free_pages, free_count, page_size, in_place=False):
    """Shorten requests to min(lengths, keep) tokens (int32 [B]; 0: ended; fewer than it
    has: drafts that were not accepted) and put the pages behind that back on the stack
    ``free_pages``, in the order of the requests and their pages.  Returns (lengths,
    free_count) as they are from now on: new tensors, or with ``in_place`` the given
    ones, updated.  The table's entries stay.  A negative length or keep (left as it is),
    or pages beyond the table's width or the stack's end (dropped), makes
    device_status() report 8."""
    return _ops.trim_tables(lengths, keep, block_table, free_pages, free_count, page_size, in_place)


def lora_workspace_size(T, adapters, r, K):
    return int(_lib.load().nvfp4_lora_workspace(T, adapters, r, K))


def lora_add(y, x, a, b, adapters, scales=None, out=None, workspace=None):
    """y + scales[i] * b[i] @ (a[i] @ x) row by row, i = adapters[t] (int32 [T]; negative: y
    alone): low-rank adapters of many requests at once, beside the projection y [T, N] of
    x [T, K] that they share (BF16 or FP16, rows with any stride; views of a fused
    projection will do).  ``a`` [adapters, r, K] and ``b`` [adapters, N, r] have their
    type, ``scales`` is float32 [adapters] or None (1); r at most 256, smaller ranks padded
    with zeros.  a @ x is held in 32 bits and meets b as two halves of the type; the sums are
    rounded once, to the type of y.  b has to be finite.  ``out`` may be y where that is
    contiguous.  An index that is not below the number of adapters counts as none, and
    device_status() then reports 8."""
    return _ops.lora_add(y, x, a, b, adapters, scales, out, workspace)


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, return_logprob=False, out=None, logprob=None):
    """The next token of each row of logits [B, V] (BF16, FP16 or float32, rows with any
    stride, V at most 2^20), drawn with the given random numbers u (float32 [B], in [0,
    1)): int64 [B], with ``return_logprob`` also the log-probability (float32 [B]) with which
    it was drawn.

    With w = exp((l - max l) / temperature), kept are the ``top_k`` largest logits (0:
    all; equal ones rank by index), of these the shortest prefix with at least ``top_p`` of
    their mass (1: all), of these those with w >= ``min_p``.  The token is the first kept
    one, by index, at which the running sum of w passes u times the sum of all kept.  A
    temperature of 0 takes the largest logit (the first of equal ones).  Each setting is a
    number or a tensor [B] (float32; top_k int32).  NaN and -infinity are never drawn; a
    row of nothing else gives -1 (and -infinity)."""
    return _ops.sample(logits, u, temperature, top_k, top_p, min_p, return_logprob, out, logprob)
