"""What differs from request to request in a batch, the plain way (test
infrastructure): page tables and slots from lengths, pages given back, adapters
beside a projection, the draw of a token.  numpy and Python loops; float64.

Parity: pinned by tests/test_oracle_batch.py (worked tables, conservation of pages,
dense matrices of single adapters, frequencies of draws and worked rows).
"""

import numpy as np


def extend(lengths, new, table, stack, count, page, rows):
    """dict(positions, slots, request, starts, lengths, free_count, table, row_lengths,
    row_tables, served); inputs are not changed."""
    table, out = np.array(table), {}
    B, width = table.shape
    out["positions"], out["slots"] = np.zeros(rows, np.int64), np.full(rows, -1, np.int64)
    out["request"], out["row_lengths"] = np.full(rows, -1, np.int32), np.zeros(rows, np.int32)
    out["row_tables"] = np.zeros((rows, width), np.int32)
    count = min(max(int(count), 0), len(stack))
    starts, after, served, row, asked, taken = [0], [], [], 0, 0, 0
    for b in range(B):
        n, m = int(lengths[b]), int(new[b])
        have, want = -(-n // page), -(-(n + m) // page)
        ok = n >= 0 and m >= 0 and n + m < 2 ** 31 and want <= width and row + m <= rows
        if ok and want > have:
            ok = asked + want - have <= count
            if ok:
                for j in range(have, want):
                    table[b, j] = stack[count - 1 - asked - (j - have)]
                taken += want - have
            asked += want - have
        served.append(ok)
        after.append(n + m if ok else n)
        for i in range(min(max(m, 0), max(0, rows - row))):
            at = max(n, 0) + i
            out["positions"][row + i], out["request"][row + i] = at, b
            if ok:
                out["slots"][row + i] = int(table[b, at // page]) * page + at % page
                out["row_lengths"][row + i] = at + 1
                out["row_tables"][row + i, :at // page + 1] = table[b, :at // page + 1]
        row += max(m, 0)
        starts.append(min(row, rows))
    return dict(out, starts=np.array(starts, np.int32), lengths=np.array(after, np.int32), free_count=count - taken,
                table=table, served=np.array(served))


def trim(lengths, keep, table, stack, count, page):
    """(lengths, count, stack) after pages behind min(lengths, keep) went back."""
    stack, top, after = np.array(stack), min(max(int(count), 0), len(stack)), []
    for b in range(len(lengths)):
        n, k = int(lengths[b]), int(keep[b])
        after.append(n if n < 0 or k < 0 else min(n, k))
        for j in range(-(-after[-1] // page), min(-(-n // page), table.shape[1])):
            if after[-1] < n and top < len(stack):
                stack[top] = table[b, j]
                top += 1
    return np.array(after, np.int32), top, stack


def lora(y, x, a, b, adapters, scales):
    """(out, magnitude) in float64: y + s B (A x), and |s| |B| (|A| |x|), with which the
    errors of 32-bit sums scale."""
    out, mag = np.array(y, np.float64), np.zeros(y.shape)
    with np.errstate(all="ignore"):
        for t, i in enumerate(adapters):
            if 0 <= i < len(a):
                out[t] += scales[i] * (b[i].astype(np.float64) @ (a[i].astype(np.float64) @ x[t]))
                mag[t] = abs(scales[i]) * (np.abs(b[i].astype(np.float64)) @ (np.abs(a[i].astype(np.float64)) @ np.abs(x[t])))
    return out, mag


def kept(logits, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """(indices, weights) of one row's tokens that may be drawn, by index."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    top = l.max(initial=-np.inf)
    if top == -np.inf:
        return np.zeros(0, int), np.zeros(0)
    if not temperature > 0:
        return np.array([int(np.argmax(l))]), np.ones(1)
    order = np.argsort(-l, kind="stable")
    order = order[l[order] > -np.inf]
    with np.errstate(all="ignore"):
        w = np.exp(np.where(l[order] == top, 0.0, (l[order] - top) / temperature))
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    if top_p < 1:
        n = int(np.searchsorted(np.cumsum(w), top_p * w.sum())) + 1      # first prefix with at least that mass
        order, w = order[:n], w[:n]
    some = (w >= min_p) | (l[order] == top)
    order, w = order[some], w[some]
    by_index = np.argsort(order)
    return order[by_index], w[by_index]


def draw(logits, u, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log-probability) of one row."""
    at, w = kept(logits, temperature, top_k, top_p, min_p)
    if len(at) == 0:
        return -1, -np.inf
    running = np.cumsum(w)
    i = min(int(np.searchsorted(running, max(u, 0.0) * running[-1], side="right")), int(np.flatnonzero(w)[-1]))
    return int(at[i]), float(np.log(w[i] / running[-1]))
