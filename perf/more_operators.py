"""What differs from request to request in a served batch, measured: page tables
and slot maps from the requests' lengths (and pages given back), low-rank adapters
beside a shared projection, and the draw of the next token from the logits.

``run`` computes them in elementary torch operations, or, where ``own`` is true, by
the framework's entry points.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # a decode step's bookkeeping: one new token a sequence
        dict(name="extend decode 64", op="extend", B=64, new="one", rows=64, hi=4096, page=16, tables=False, short=False),
        # a step that takes in ragged prompts beside running sequences, two of them without pages left, rows padded
        dict(name="extend prompts 48", op="extend", B=48, new="prompt", rows=16384, hi=9001, page=24, tables=False, short=True),
        # drafted tokens, each a row of the attention with a table of its own
        dict(name="extend drafts 256 tables", op="extend", B=256, new="draft", rows=1280, hi=8192, page=16, tables=True,
             short=False),
        # drafts that were not accepted
        dict(name="trim drafts 96", op="trim", B=96, part=0.0, hi=4096, page=16),
        # a large pool after many requests ended
        dict(name="trim ended 1000", op="trim", B=1000, part=0.6, hi=16384, page=32),
        # one request, a square projection
        dict(name="lora 1x4096x4096 r16", op="lora", T=1, K=4096, N=4096, r=16, n=4, order="random", none=0.0, dtype="bf16",
             wide=False),
        # a decode batch on many adapters, a third without one, fused gate and up projection
        dict(name="lora 64x4096x28672 r16", op="lora", T=64, K=4096, N=28672, r=16, n=32, order="random", none=0.3,
             dtype="bf16", wide=False),
        # odd widths, part of a fused projection's rows
        dict(name="lora 333x2064x1000 r24", op="lora", T=333, K=2064, N=1000, r=24, n=5, order="random", none=0.2,
             dtype="f16", wide=True),
        # prompt chunks of a few requests with large ranks
        dict(name="lora 8192x4096x4096 r64", op="lora", T=8192, K=4096, N=4096, r=64, n=8, order="runs", none=0.1,
             dtype="bf16", wide=False),
        # one conversation
        dict(name="sample 1x151936", op="sample", B=1, V=151936, dtype="bf16", params="both"),
        # a serving batch in which every request has its own settings, some greedy
        dict(name="sample 64x151936 mixed", op="sample", B=64, V=151936, dtype="bf16", params="mixed"),
        # rollouts by top-p over logits in 32 bits, an odd vocabulary
        dict(name="sample 256x100003 top-p", op="sample", B=256, V=100003, dtype="f32", params="top_p"),
    ]


def _spread(rng, lo, hi):
    """Log-uniform whole number in [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "trim", "lora", "lora", "sample", "sample"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    if op == "extend":
        new, tables = rng.choice(["one", "prompt", "draft"]), rng.random() < 0.3
        B, hi = _spread(rng, 1, 1024), _spread(rng, 16, 16384)
        if new == "prompt":
            rows = _spread(rng, B, 16384)
        else:
            rows = B if new == "one" else 5 * B
        if tables:
            rows = min(rows, max(1, (1 << 22) // (hi // page + 2)))
        return dict(op=op, B=B, new=new, rows=rows, hi=hi, page=page, tables=tables, short=rng.random() < 0.2)
    if op == "trim":
        return dict(op=op, B=_spread(rng, 1, 1024), part=rng.choice([0.0, 0.1, 0.5]), hi=_spread(rng, 16, 16384), page=page)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "lora":
        sizes = [720, 1000, 1024, 2048, 2064, 4096, 5120, 8192, _spread(rng, 256, 8192)]
        K, N, r = rng.choice(sizes), rng.choice(sizes), rng.choice([4, 8, 16, 16, 24, 32, 64, 64, 128])
        most = min(8192, 8192 * 8192 // (K + N))
        if r > 64:
            most //= 2
        return dict(op=op, T=_spread(rng, 1, most), K=K, N=N, r=r, n=_spread(rng, 1, 32), order=rng.choice(["random", "runs"]),
                    none=rng.choice([0.0, 0.2]), dtype=dtype, wide=rng.random() < 0.3)
    V = rng.choice([32768, 65536, 100003, 131072, 151936, _spread(rng, 1000, 200000)])
    return dict(op=op, B=_spread(rng, 1, max(1, 256 * 100003 // V)), V=V, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                params=rng.choice(["both", "mixed", "top_p", "top_k", "temperature"]))


def _lengths(case):
    """Tokens cached of each sequence: evenly spread over the range, none among them."""
    B, hi = case["B"], case["hi"]
    return [hi - 1] if B == 1 else [(hi - 1) * i // (B - 1) for i in range(B)]


def _news(case):
    """New tokens of each sequence, before they meet lengths in another order."""
    B, rows = case["B"], case["rows"]
    if case["new"] == "one":
        return [1] * B
    if case["new"] == "draft":
        return [1 + i % 5 for i in range(B)]
    each = max(1, rows // B)
    return [max(1, int(each * (0.02 if i % 3 else 2.0))) for i in range(B)]     # two decoding for each that prefills


def work(case):
    op = case["op"]
    if op == "extend":
        B, rows = case["B"], case["rows"]
        width = (case["hi"] + max(_news(case))) // case["page"] + 1
        fresh = sum(_news(case)) // case["page"] + 1
        size = 16 * B + 8 * fresh + rows * (8 + 8 + 4)
        return {"bytes": size + (rows * (4 * width + 4) if case["tables"] else 0), "flops": 8 * rows + 8 * B}
    if op == "trim":
        gone = int(sum(_lengths(case)) * case["part"]) // case["page"]
        return {"bytes": 12 * case["B"] + 8 * gone, "flops": 8 * case["B"] + gone}
    if op == "lora":
        T, K, N, r = case["T"], case["K"], case["N"], case["r"]
        rows = T if T == 1 else max(1, round(T * (1 - case["none"])))          # with an adapter
        used = min(case["n"], rows)
        return {"bytes": 2 * rows * K + 4 * T * N + 2 * used * r * (K + N) + 4 * T, "flops": 2 * rows * r * (K + N)}
    B, V = case["B"], case["V"]
    return {"bytes": B * V * (4 if case["dtype"] == "f32" else 2) + 32 * B, "flops": 6 * B * V}


# ------------------------------------------------------------------ inputs ---

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _tables(r, lengths, page, width, spare):
    """Block table of the cached tokens, and the stack of free pages above used entries."""
    per = -(-lengths // page)
    used = int(per.sum())
    order = r.permutation(used + spare).astype(np.int32)
    table = np.zeros((len(lengths), width), dtype=np.int32)
    table[np.arange(width)[None, :] < per[:, None]] = order[:used]
    stack = np.zeros(used + spare, dtype=np.int32)
    stack[:spare] = order[used:]
    return table, stack


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    r = np.random.RandomState(int(seed) % (1 << 32))
    if op in ("extend", "trim"):
        page, B = case["page"], case["B"]
        lengths = r.permutation(np.array(_lengths(case), dtype=np.int64))
        if op == "extend":
            new = r.permutation(np.array(_news(case), dtype=np.int64))
            need = int((-(-(lengths + new) // page) - -(-lengths // page)).sum())
            width = (case["hi"] + int(new.max())) // page + 1
            spare = max(1, need - need // 20 - 1) if case["short"] else need + 7
            table, stack = _tables(r, lengths, page, width, spare)
            return dict(case=case, lengths=_i32(lengths), new=_i32(new), table=_i32(table), pages=_i32(stack),
                        count=_i32([spare]))
        table, stack = _tables(r, lengths, page, case["hi"] // page + 1, 5)
        keep = np.maximum(lengths - r.randint(0, 5, B), 0)
        keep[r.random_sample(B) < case["part"]] = 0
        return dict(case=case, lengths=_i32(lengths), keep=_i32(keep), table=_i32(table), pages=_i32(stack), count=_i32([5]))
    dt = DTYPES[case["dtype"]]
    if op == "lora":
        T, K, N, rank, n = (case[k] for k in ("T", "K", "N", "r", "n"))
        if case["order"] == "runs":                                     # rows of one request side by side
            each = -(-T // (2 * n))
            adapters = np.repeat(r.randint(0, n, 2 * n), each)[:T]
            adapters[np.repeat(r.random_sample(2 * n) < case["none"], each)[:T]] = -1
        else:
            adapters = r.randint(0, n, T)
            adapters[r.random_sample(T) < case["none"]] = -1
        if T == 1:
            adapters[:] = n - 1
        x = torch.randn(T, K + (64 if case["wide"] else 0), generator=g, device="cuda", dtype=dt)[:, :K]
        y = torch.randn(T, N + (72 if case["wide"] else 0), generator=g, device="cuda", dtype=dt)[:, :N]
        a = (torch.randn(n, rank, K, generator=g, device="cuda") * K ** -0.5).to(dt)
        b = (torch.randn(n, N, rank, generator=g, device="cuda") * (0.3 * rank ** -0.5)).to(dt)
        scales = torch.rand(n, generator=g, device="cuda") + 0.5
        return dict(case=case, x=x, y=y, a=a, b=b, scales=scales, adapters=_i32(adapters))
    B, V = case["B"], case["V"]
    logits = torch.randn(B, V, generator=g, device="cuda") * 2.2         # a bulk, and a few tokens that the model means
    likely = torch.randint(0, V, (B, 24), generator=g, device="cuda")
    logits.scatter_add_(1, likely, 14 * torch.rand(B, 24, generator=g, device="cuda"))
    logits[:, V - V // 500:] = -math.inf                                 # padding of the vocabulary
    params = case["params"]
    temperature, top_k = np.full(B, 0.8), np.zeros(B)
    top_p, min_p = np.ones(B), np.zeros(B)
    if params in ("both", "top_k"):
        top_k[:] = 50
    if params in ("both", "top_p"):
        top_p[:] = 0.95
    if params == "mixed":
        temperature = r.choice([0.0, 0.6, 0.8, 1.0, 1.3], B)
        top_k, top_p, min_p = r.choice([0, 1, 20, 50, 400], B), r.choice([1.0, 0.8, 0.95, 0.99], B), r.choice([0.0, 0.0, 0.02, 0.1], B)

    def f32(v):
        return torch.from_numpy(np.asarray(v, dtype=np.float32)).cuda()
    return dict(case=case, logits=logits.to(dt), u=torch.rand(B, generator=g, device="cuda"), temperature=f32(temperature),
                top_k=_i32(top_k), top_p=f32(top_p), min_p=f32(min_p))


# ------------------------------------------------------------- plain forms ---

def _plain_extend(st):
    c, page, rows = st["case"], st["case"]["page"], st["case"]["rows"]
    n, new, table = st["lengths"].long(), st["new"].long(), st["table"]
    B, width = table.shape
    ends = new.cumsum(0)
    starts = torch.cat([ends.new_zeros(1), ends]).clamp(max=rows)
    first, last = (n + page - 1) // page, (n + new + page - 1) // page   # pages held, and held afterwards
    fits = (last <= width) & (ends <= rows)
    need = torch.where(fits, last - first, 0)
    count, upto = st["count"].long(), need.cumsum(0)
    served = fits & ((need == 0) | (upto <= count))
    e = torch.arange(width, device="cuda")[None, :]
    at = count - 1 - (upto - need)[:, None] - (e - first[:, None])
    fresh = served[:, None] & (e >= first[:, None]) & (e < last[:, None])
    table.copy_(torch.where(fresh, st["pages"][at.clamp(0, st["pages"].numel() - 1)], table))
    left = count - torch.where(served, need, 0).sum()
    lengths = torch.where(served, n + new, n)
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(ends, t, right=True)
    inside = (b < B) & (t < starts[-1])
    b = b.clamp(max=B - 1)
    position = torch.where(inside, n[b] + t - starts[b], 0)
    stored = inside & served[b]
    page_of = table[b, (position // page).clamp(max=width - 1)].long()
    out = dict(positions=position, slots=torch.where(stored, page_of * page + position % page, -1),
               request=torch.where(inside, b, -1).int(), starts=starts.int(), lengths=lengths.int(), free_count=left.int(), table=table)
    if c["tables"]:
        out["row_lengths"] = torch.where(stored, position + 1, 0).int()
        held = e < ((out["row_lengths"].long() + page - 1) // page)[:, None]
        out["row_tables"] = torch.where(held, table[b], 0)
    return out


def _plain_trim(st):
    page, stack = st["case"]["page"], st["pages"]
    n, keep, table = st["lengths"].long(), st["keep"].long(), st["table"]
    after = torch.minimum(n, keep)
    first, last = (after + page - 1) // page, (n + page - 1) // page
    gone = last - first
    upto = gone.cumsum(0)
    e = torch.arange(table.shape[1], device="cuda")[None, :]
    back = (e >= first[:, None]) & (e < last[:, None])
    at = torch.where(back, st["count"].long() + (upto - gone)[:, None] + e - first[:, None], stack.numel())
    room = torch.cat([stack, stack.new_zeros(1)])                        # entries that stay go to the last place
    room.scatter_(0, at.reshape(-1), table.reshape(-1))
    stack.copy_(room[:-1])
    return dict(lengths=after.int(), free_count=(st["count"].long() + upto[-1]).int(), pages=stack)


def _plain_lora(st):
    x, y, a, b, adapters = st["x"], st["y"], st["a"], st["b"], st["adapters"]
    n, rank, K = a.shape
    v = torch.matmul(x.float(), a.view(n * rank, K).float().t())         # every adapter of every row
    mine = adapters[:, None] == torch.arange(n, device="cuda", dtype=torch.int32)
    v = torch.where(mine[:, :, None], v.view(-1, n, rank) * st["scales"][:, None], 0.0)
    delta = torch.matmul(v.view(-1, n * rank), b.float().transpose(1, 2).reshape(n * rank, -1))
    return (y.float() + delta).to(y.dtype)


def _plain_sample(st):
    x = st["logits"].double()
    B, V = x.shape
    greedy = ~(st["temperature"] > 0)
    temperature = torch.where(greedy, 1.0, st["temperature"]).double()
    s, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((s - s[:, :1]) / temperature[:, None])
    place = torch.arange(V, device="cuda")
    k = torch.where(greedy, 1, st["top_k"].long())
    w = torch.where((place < k[:, None]) | (k <= 0)[:, None], w, 0.0)
    upto = w.cumsum(1)
    top_p = st["top_p"].double()[:, None]
    before = upto - w
    w = torch.where((before < top_p * upto[:, -1:]) | (top_p >= 1) | (place == 0), w, 0.0)
    w = torch.where((w >= st["min_p"].double()[:, None]) | (place == 0), w, 0.0)
    kept = torch.zeros_like(w).scatter_(1, order, w)
    running = kept.cumsum(1)
    total = running[:, -1:]
    token = torch.searchsorted(running, st["u"].double()[:, None] * total, right=True)
    logprob = torch.log(kept.gather(1, token) / total)
    return token[:, 0], logprob[:, 0].float()


def _own(st):
    import w4a16_nvfp4_weight_gb300 as nv
    c = st["case"]
    op = c["op"]
    if op == "extend":
        out = nv.extend_tables(st["lengths"], st["new"], st["table"], st["pages"], st["count"], c["page"], c["rows"],
                               row_tables=c["tables"])
        return dict(out, table=st["table"])
    if op == "trim":
        lengths, count = nv.trim_tables(st["lengths"], st["keep"], st["table"], st["pages"], st["count"], c["page"])
        return dict(lengths=lengths, free_count=count, pages=st["pages"])
    if op == "lora":
        return nv.lora_add(st["y"], st["x"], st["a"], st["b"], st["adapters"], scales=st["scales"])
    return nv.sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                     min_p=st["min_p"], return_logprob=True)


def run(state):
    if own:
        return _own(state)
    return {"extend": _plain_extend, "trim": _plain_trim, "lora": _plain_lora, "sample": _plain_sample}[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact ---

def _exact_extend(st):
    """Request by request, on the host."""
    c, page, rows = st["case"], st["case"]["page"], st["case"]["rows"]
    n, new, count = st["lengths"].tolist(), st["new"].tolist(), int(st["count"][0])
    table, stack = st["table"].cpu().numpy().copy(), st["pages"].cpu().numpy()
    B, width = table.shape
    position, slot = np.zeros(rows, np.int64), np.full(rows, -1, np.int64)
    request, row_lengths = np.full(rows, -1, np.int32), np.zeros(rows, np.int32)
    row_tables = np.zeros((rows if c["tables"] else 0, width), np.int32)
    starts, lengths, row, asked, taken = [0], list(n), 0, 0, 0
    for b in range(B):
        held, then = math.ceil(n[b] / page), math.ceil((n[b] + new[b]) / page)
        ok = then <= width and row + new[b] <= rows
        if ok and then > held:
            ok = asked + then - held <= count
            for j in range(held, then if ok else held):
                table[b, j] = stack[count - 1 - asked - (j - held)]
            asked += then - held
            taken += then - held if ok else 0
        if ok:
            lengths[b] = n[b] + new[b]
        for i in range(min(new[b], max(0, rows - row))):
            p = n[b] + i
            position[row + i], request[row + i] = p, b
            if ok:
                slot[row + i], row_lengths[row + i] = int(table[b, p // page]) * page + p % page, p + 1
                if c["tables"]:
                    row_tables[row + i, :p // page + 1] = table[b, :p // page + 1]
        row += new[b]
        starts.append(min(row, rows))
    out = dict(positions=torch.from_numpy(position), slots=torch.from_numpy(slot), request=torch.from_numpy(request),
               starts=torch.tensor(starts, dtype=torch.int32), lengths=torch.tensor(lengths, dtype=torch.int32),
               free_count=torch.tensor([count - taken], dtype=torch.int32), table=torch.from_numpy(table))
    if c["tables"]:
        out.update(row_lengths=torch.from_numpy(row_lengths), row_tables=torch.from_numpy(row_tables))
    return {k: v.cuda() for k, v in out.items()}


def _exact_trim(st):
    page = st["case"]["page"]
    stack, top, lengths = st["pages"].tolist(), int(st["count"][0]), []
    for n, keep, row in zip(st["lengths"].tolist(), st["keep"].tolist(), st["table"].tolist()):
        lengths.append(min(n, keep))
        for j in range(math.ceil(lengths[-1] / page), math.ceil(n / page)):
            stack[top] = row[j]
            top += 1
    return dict(lengths=_i32(lengths), free_count=_i32([top]), pages=_i32(stack))


def _exact_lora(st):
    out = st["y"].double().clone()
    for i in range(st["a"].shape[0]):
        rows = torch.nonzero(st["adapters"] == i)[:, 0]
        low = st["x"][rows].double() @ st["a"][i].double().T
        out[rows] += float(st["scales"][i]) * (low @ st["b"][i].double().T)
    return out


def _exact_sample(st):
    """Row by row, over lists of the tokens that are kept."""
    tokens, logprobs = [], []
    for i in range(st["logits"].shape[0]):
        x = st["logits"][i].double()
        t, k, p, low = float(st["temperature"][i]), int(st["top_k"][i]), float(st["top_p"][i]), float(st["min_p"][i])
        best = int(torch.nonzero(x == x.max())[0])
        if not t > 0:
            tokens.append(best)
            logprobs.append(0.0)
            continue
        order = torch.argsort(-x, stable=True)
        order = order[:int(torch.isfinite(x).sum())]
        if k > 0:
            order = order[:k]
        z = x[order] / t
        mass = torch.exp(z - z[0])
        if p < 1:
            reached = torch.cumsum(mass, 0) >= p * mass.sum()
            m = int(torch.nonzero(reached)[0]) + 1
            order, mass = order[:m], mass[:m]
        enough = mass >= low
        enough[0] = True
        kept, back = torch.sort(order[enough])
        running = torch.cumsum(mass[enough][back], 0)
        at = min(int((running <= float(st["u"][i]) * running[-1]).sum()), kept.numel() - 1)
        tokens.append(int(kept[at]))
        logprobs.append(float(torch.log(mass[enough][back][at] / running[-1])))
    return torch.tensor(tokens, device="cuda"), torch.tensor(logprobs, dtype=torch.float64, device="cuda")


def exact(case, seed):
    st = prepare(case, seed)
    return {"extend": _exact_extend, "trim": _exact_trim, "lora": _exact_lora, "sample": _exact_sample}[case["op"]](st)
