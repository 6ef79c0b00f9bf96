"""Page tables, adapters and the draw of tokens against the 64-bit oracle.

Tolerances.  Tables, slots and tokens are whole numbers: equal.  (A token could differ
where a random number lies within the error of a running sum of n weights, 2^-31.7 / sqrt(n)
of it, of one of its n borders: for all rows here together a chance of about 10^-4.)  A log-probability takes four
roundings of numbers up to its own size plus log V, each at most 2^-23 of them: 2^-21.
An adapter's output is rounded once, u |ref| (u: BF16 2^-8, FP16 2^-11, with 2^-25
below FP16's normals); before it, two sums of at most K and 256 products in 32 bits
move it by at most (K + 256) 2^-24 of |s| |B| (|A| |x|), and A x as two 16-bit halves by
2^-16 of that.
"""

import ctypes
import threading

import numpy as np
import pytest
import torch

import w4a16_nvfp4_weight_gb300 as nv
from w4a16_nvfp4_weight_gb300 import _lib as _lib_module
from oracle import batch
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _lib(lib):
    torch.cuda.init()
    yield
    gu.check_device_status()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ------------------------------------------------------------------ tables ---

def _pool(r, lengths, page, width, spare, extra=0):
    per = -(-np.maximum(lengths, 0) // page)
    used = int(per.sum())
    order = r.permutation(used + spare + extra).astype(np.int32)
    table = r.integers(0, 99, (len(lengths), width)).astype(np.int32)        # entries past the end do not matter
    table[np.arange(width)[None, :] < per[:, None]] = order[:used]
    stack = np.full(used + spare + extra, -7, np.int32)
    stack[:spare] = order[used:used + spare]
    return table, stack


def _check_extend(lengths, new, table, stack, count, page, rows, tables=True, strided=False):
    want = batch.extend(lengths, new, table, stack, count, page, rows)
    wide = torch.full((table.shape[0], table.shape[1] + 5), -3, dtype=torch.int32, device="cuda")
    dev = wide[:, :table.shape[1]] if strided else _i32(table)
    dev.copy_(_i32(table))
    n, pages, c = _i32(lengths), _i32(stack), _i32([count])
    for in_place in (False, True):
        got = nv.extend_tables(n, _i32(new), dev, pages, c, page, rows, row_tables=tables, in_place=in_place)
        for k in ("positions", "slots", "request", "starts", "lengths") + (("row_lengths", "row_tables") if tables else ()):
            assert np.array_equal(got[k].cpu().numpy(), want[k]), k
        assert got["free_count"].tolist() == [want["free_count"]]
        assert np.array_equal(dev.cpu().numpy(), want["table"]) and np.array_equal(pages.cpu().numpy(), stack)
        assert (got["lengths"] is n) == in_place or got["lengths"].data_ptr() == n.data_ptr()
    assert n.tolist() == want["lengths"].tolist() and c.tolist() == [want["free_count"]]
    assert bool((wide[:, table.shape[1]:] == -3).all())
    return want


@pytest.mark.parametrize("B", [1, 2, 31, 64, 1000, 1025, 5000])
@pytest.mark.parametrize("page", [1, 7, 16])
@pytest.mark.parametrize("kind", ["one", "drafts", "prompts"])
def test_extend(B, page, kind):
    r = np.random.default_rng(B * 100 + page)
    lengths = r.integers(0, 60, B)
    new = np.ones(B, int) if kind == "one" else r.integers(0, 6, B) if kind == "drafts" else np.where(r.random(B) < 0.3, r.integers(0, 150, B), 1)
    width = int(-(-(lengths + new).max() // page)) or 1
    need = int((-(-(lengths + new) // page) - -(-lengths // page)).sum())
    table, stack = _pool(r, lengths, page, width, need + 3)
    rows = int(new.sum()) + int(r.integers(0, 9))
    want = _check_extend(lengths, new, table, stack, need + 3, page, rows, strided=B % 2 == 0)
    assert want["served"].all() and want["free_count"] == 3


@pytest.mark.parametrize("B", [1, 40, 1500])
def test_extend_short_of_pages_rows_or_table(B):
    r = np.random.default_rng(B)
    lengths, new = r.integers(0, 50, B), r.integers(0, 40, B)
    need = int((-(-(lengths + new) // 8) - -(-lengths // 8)).sum())
    for spare, rows, width in ((need // 2, int(new.sum()), 12), (0, int(new.sum()) + 5, 12), (need, int(new.sum()) * 2 // 3, 12),
                               (need, int(new.sum()), 9), (need // 3, int(new.sum()) // 2 + 1, 10), (need, 0, 12)):
        lens = np.minimum(lengths, width * 8)
        table, stack = _pool(r, lens, 8, width, spare, extra=2)
        _check_extend(lens, new, table, stack, spare, 8, rows)


def test_extend_most_requests_and_rows():
    B, page = 16384, 4
    r = np.random.default_rng(3)
    lengths, new = r.integers(0, 40, B), r.integers(0, 12, B)
    need = int((-(-(lengths + new) // page) - -(-lengths // page)).sum())
    table, stack = _pool(r, lengths, page, 13, need)
    _check_extend(lengths, new, table, stack, need, page, int(new.sum()) + 77)


def test_extend_nothing():
    got = nv.extend_tables(_i32([]), _i32([]), torch.zeros(0, 4, dtype=torch.int32, device="cuda"), _i32([5]), _i32([1]), 16, 3, row_tables=True)
    assert got["slots"].tolist() == [-1] * 3 and got["request"].tolist() == [-1] * 3 and got["starts"].tolist() == [0]
    assert got["free_count"].tolist() == [1] and got["row_tables"].tolist() == [[0] * 4] * 3
    r = np.random.default_rng(0)
    table, stack = _pool(r, np.array([3, 0]), 16, 2, 1)
    _check_extend(np.array([3, 0]), np.array([0, 0]), table, stack, 1, 16, 0)        # no new tokens, no rows
    _check_extend(np.array([0, 0]), np.array([0, 0]), np.zeros((2, 0), np.int32), stack, 1, 16, 2)     # no table at all
    _check_extend(np.array([0, 0]), np.array([1, 0]), np.zeros((2, 0), np.int32), stack, 1, 16, 2)


@pytest.mark.parametrize("case", ["length", "new", "count above", "count below"])
def test_extend_bad_values_are_reported(case):
    r = np.random.default_rng(4)
    lengths, new, count = np.array([5, 20, 9]), np.array([3, 1, 30]), 6
    table, stack = _pool(r, lengths, 8, 6, 6)
    if case == "length":
        lengths[1] = -4
    elif case == "new":
        new[0] = -2
    else:
        count = 100 if "above" in case else -1
    want = batch.extend(lengths, new, table, stack, count, 8, 40)
    got = nv.extend_tables(_i32(lengths), _i32(new), _i32(table), _i32(stack), _i32([count]), 8, 40)
    for k in ("positions", "slots", "request", "starts", "lengths"):
        assert np.array_equal(got[k].cpu().numpy(), want[k]), k
    assert got["free_count"].tolist() == [want["free_count"]]
    assert nv.device_status() == 8


def test_extend_lengths_near_the_end_of_32_bits():
    n, m = _i32([2 ** 31 - 4, 2 ** 31 - 4]), _i32([3, 5])            # the second would pass 2^31 - 1
    page = 2 ** 30
    table = torch.tensor([[11, 12, 0], [13, 14, 0]], dtype=torch.int32, device="cuda")
    got = nv.extend_tables(n, m, table, _i32([1, 2]), _i32([2]), page, 8)
    assert got["lengths"].tolist() == [2 ** 31 - 1, 2 ** 31 - 4]
    assert got["positions"].tolist()[:3] == [2 ** 31 - 4, 2 ** 31 - 3, 2 ** 31 - 2]
    assert got["slots"].tolist() == [12 * page + page - 4 + i for i in range(3)] + [-1] * 5     # past 32 bits


@pytest.mark.parametrize("B,page,hi", [(1, 1, 5), (3, 16, 100), (96, 16, 4096), (1000, 32, 900), (1100, 1, 300), (64, 1, 9000)])
@pytest.mark.parametrize("part", [0.0, 0.5, 1.0])
def test_trim(B, page, hi, part):
    r = np.random.default_rng(B + page)
    lengths = r.integers(0, hi, B)
    keep = np.maximum(lengths - r.integers(-2, 6, B), 0)
    keep[r.random(B) < part] = 0
    table, stack = _pool(r, lengths, page, -(-hi // page), 4)
    after, count, back = batch.trim(lengths, keep, table, stack, 4, page)
    n, c = _i32(lengths), _i32([4])
    for in_place in (False, True):
        pages = _i32(stack)
        got = nv.trim_tables(n, _i32(keep), _i32(table), pages, c, page, in_place=in_place)
        assert np.array_equal(got[0].cpu().numpy(), after) and got[1].tolist() == [count]
        assert np.array_equal(pages.cpu().numpy(), back)
        assert (got[0].data_ptr() == n.data_ptr()) == in_place
    assert n.tolist() == after.tolist() and c.tolist() == [count]


def test_trim_bad_values_and_a_full_stack():
    table, stack = np.arange(12, dtype=np.int32).reshape(3, 4), np.full(5, 50, np.int32)
    for lengths, keep, count in (([8, -3, 5], [2, 1, 5], 0), ([8, 3, 5], [2, -1, 0], 0), ([16, 16, 16], [0, 0, 0], 1), ([99, 4, 4], [0, 4, 4], 0),
                                 ([8, 3, 5], [0, 0, 0], 9), ([8, 3, 5], [0, 3, 5], -2)):
        after, top, back = batch.trim(lengths, keep, table, stack, count, 4)
        pages = _i32(stack)
        got = nv.trim_tables(_i32(lengths), _i32(keep), _i32(table), pages, _i32([count]), 4)
        assert got[0].tolist() == after.tolist() and got[1].tolist() == [top] and pages.tolist() == back.tolist()
        assert nv.device_status() == 8
    got = nv.trim_tables(_i32([]), _i32([]), torch.zeros(0, 4, dtype=torch.int32, device="cuda"), _i32([5]), _i32([1]), 16)
    assert got[0].numel() == 0 and got[1].tolist() == [1]


def test_a_loop_of_steps_in_a_graph_keeps_every_page():
    """Requests grow, drafts are taken back, some end: after each replay the pages held and the
    pages free are all pages, and tables and slots are the oracle's."""
    B, page, width, P, rows = 20, 4, 12, 300, 80
    r = np.random.default_rng(8)
    lengths = np.zeros(B, int)
    table, stack = np.zeros((B, width), np.int32), r.permutation(P).astype(np.int32)
    count = P
    dn, dt, dp, dc = _i32(lengths), _i32(table), _i32(stack), _i32([count])
    dm, dk = _i32(np.zeros(B)), _i32(np.zeros(B))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            out = nv.extend_tables(dn, dm, dt, dp, dc, page, rows, in_place=True)
            nv.trim_tables(dn, dk, dt, dp, dc, page, in_place=True)
    stream.synchronize()
    for step in range(25):
        new, keep = r.integers(0, 6, B), None
        want = batch.extend(lengths, new, table, stack, count, page, rows)
        keep = np.where(r.random(B) < 0.1, 0, np.maximum(want["lengths"] - r.integers(0, 4, B), 0))
        after, count, stack = batch.trim(want["lengths"], keep, want["table"], stack, want["free_count"], page)
        dm.copy_(_i32(new))
        dk.copy_(_i32(keep))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out["slots"].cpu().numpy(), want["slots"]) and np.array_equal(out["positions"].cpu().numpy(), want["positions"])
        assert dn.tolist() == after.tolist() and dc.tolist() == [count] and dp.tolist() == stack.tolist()
        table, lengths = want["table"], after
        assert np.array_equal(dt.cpu().numpy(), table)
        held = [int(p) for b in range(B) for p in table[b, :-(-int(lengths[b]) // page)]]
        assert sorted(held + stack[:count].tolist()) == list(range(P))


def test_drafted_tokens_attend_through_their_own_tables():
    """extend_tables -> rope_cache_write -> paged_attention over the rows, against one token at a time."""
    B, Hq, Hkv, D, page, width = 5, 8, 2, 64, 4, 8
    r, g = np.random.default_rng(5), _gen(5)
    lengths, new = np.array([0, 3, 9, 16, 7]), np.array([4, 1, 0, 3, 6])
    table, stack = _pool(r, lengths, page, width, 12)
    kc = torch.randn(60, Hkv, page, D, generator=g, device="cuda").bfloat16()
    vc = torch.randn(60, Hkv, page, D, generator=g, device="cuda").bfloat16()
    rows = int(new.sum()) + 2
    q = torch.randn(rows, Hq, D, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(rows, Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    rope = nv.rope_table(64, D)
    dt = _i32(table)
    t = nv.extend_tables(_i32(lengths), _i32(new), dt, _i32(stack), _i32([12]), page, rows, row_tables=True)
    qr = nv.rope_cache_write(q, k, v, t["positions"], rope, kc, vc, t["slots"])
    out = nv.paged_attention(qr, kc, vc, t["row_tables"], t["row_lengths"])
    request = t["request"].tolist()
    for i in range(rows):
        b = request[i]
        if b < 0:
            assert bool((out[i] == 0).all())
            continue
        one = nv.paged_attention(qr[i:i + 1], kc, vc, dt[b:b + 1], t["positions"][i:i + 1].int() + 1)
        assert (out[i] - one[0]).abs().max() <= 2.0 ** -6 * one.abs().max()      # cut at other places, rounded to BF16 twice


# ------------------------------------------------------------------- adapters ---

def _lora_case(T, K, N, rank, n, act, seed, none=0.2, runs=False, wide=0):
    g, r = _gen(seed), np.random.default_rng(seed)
    ids = r.integers(0, max(n, 1), T)
    if runs:
        ids = np.sort(ids)
    ids[r.random(T) < none] = -1
    if n == 0:
        ids[:] = -1
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").to(DT[act])
    x, y = randn(T, K + wide)[:, :K], randn(T, N + wide)[:, :N]
    a, b = (randn(n, rank, K) * K ** -0.5).to(DT[act]), randn(n, N, rank)
    s = torch.rand(n, generator=g, device="cuda") + 0.5
    return y, x, a, b, _i32(ids), s


def _close_lora(got, y, x, a, b, ids, s, act):
    f = lambda t: t.double().cpu().numpy()
    s = np.ones(a.shape[0]) if s is None else f(s)
    ref, mag = batch.lora(f(y), f(x), f(a), f(b), ids.tolist(), s)
    err = np.abs(f(got) - ref)
    lim = U[act] * np.abs(ref) + ((x.shape[1] + 256) * 2.0 ** -24 + 2.0 ** -16) * mag + TINY[act]
    assert np.all(err <= lim), (err - lim).max()
    none = np.array([not 0 <= i < a.shape[0] for i in ids.tolist()], bool)
    assert torch.equal(got[torch.from_numpy(none).cuda()], y[torch.from_numpy(none).cuda()])


LORA_SHAPES = [(1, 64, 64, 16, 1), (1, 4096, 512, 16, 4), (3, 16, 8, 1, 2), (7, 2064, 1000, 24, 3), (16, 720, 300, 8, 16), (64, 1024, 2048, 64, 32),
               (65, 512, 512, 4, 1), (130, 1000, 264, 128, 2), (200, 96, 40, 256, 3), (300, 4096, 96, 20, 5), (5, 33, 17, 3, 2),
               (90, 40, 31, 5, 1), (600, 256, 256, 16, 4), (333, 2064, 1000, 24, 5), (1000, 128, 72, 32, 7)]


@pytest.mark.parametrize("T,K,N,rank,n", LORA_SHAPES)
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("runs", [False, True])
def test_lora(T, K, N, rank, n, act, runs):
    y, x, a, b, ids, s = _lora_case(T, K, N, rank, n, act, T + K + N + rank, runs=runs, none=0.0 if T == 1 else 0.2)
    got = nv.lora_add(y, x, a, b, ids, scales=s)
    _close_lora(got, y, x, a, b, ids, s, act)
    assert torch.equal(got, nv.lora_add(y, x, a, b, ids, scales=s))          # the same bits again
    z = y.clone()
    assert nv.lora_add(z, x, a, b, ids, scales=s, out=z) is not None and torch.equal(z, got)


# T >= 64 (n + 1): items of 64 rows, here with remainders.  K and N with and without vector loads, ranks below, between
# and at the tiles' sizes, up to beyond the room of the ring.
@pytest.mark.parametrize("rank", [1, 3, 8, 12, 20, 32, 64, 72, 100, 128, 192, 200, 256])
@pytest.mark.parametrize("T,K,N,n", [(129, 64, 72, 1), (200, 300, 264, 2), (333, 520, 33, 3), (450, 33, 128, 1), (260, 1032, 257, 1)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_lora_items_of_64_rows(T, K, N, n, rank, act):
    for wide, runs in ((0, True), (1, False), (8, False)):
        y, x, a, b, ids, s = _lora_case(T, K, N, rank, n, act, T + rank + wide, runs=runs, wide=wide)
        got = nv.lora_add(y, x, a, b, ids, scales=s)
        _close_lora(got, y, x, a, b, ids, s, act)
        z = torch.full((T + 1, N), 7.0, dtype=DT[act], device="cuda")
        nv.lora_add(y, x, a, b, ids, scales=s, out=z[:T])
        assert torch.equal(z[:T], got) and bool((z[T] == 7).all())


@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("T,rank", [(40, 16), (200, 16), (200, 24), (200, 128)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_lora_tensors_off_16_byte_boundaries(act, T, rank, off):
    """x, y, A and B, each by itself, begin 2, 4 or 8 bytes past a boundary."""
    y, x, a, b, ids, s = _lora_case(T, 128, 64, rank, 1, act, off)
    want = nv.lora_add(y, x, a, b, ids, scales=s)
    _close_lora(want, y, x, a, b, ids, s, act)

    def moved(t):
        room = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
        room[off:].copy_(t.reshape(-1))
        return room[off:].view(t.shape)

    for k in range(4):
        args = [y, x, a, b]
        args[k] = moved(args[k])
        _close_lora(nv.lora_add(*args, ids, scales=s), y, x, a, b, ids, s, act)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("wide", [1, 8, 72])
def test_lora_strided_rows_and_no_scales(act, wide):
    for T, K, N, rank in ((9, 256, 128, 16), (150, 256, 128, 24)):
        y, x, a, b, ids, _ = _lora_case(T, K, N, rank, 2, act, wide, wide=wide)
        got = nv.lora_add(y, x, a, b, ids)
        _close_lora(got, y, x, a, b, ids, None, act)
    once = x[:1].expand(150, K)                                              # one row for all: stride 0
    assert torch.equal(nv.lora_add(y, once, a, b, ids), nv.lora_add(y, once.contiguous(), a, b, ids))


def test_lora_without_rows_columns_or_adapters():
    y, x, a, b, ids, s = _lora_case(4, 32, 16, 8, 2, "bf16", 1)
    assert nv.lora_add(y[:0], x[:0], a, b, ids[:0], scales=s).shape == (0, 16)
    assert nv.lora_add(y[:, :0], x, a, b[:, :0], ids, scales=s).shape == (4, 0)
    y, x, a, b, ids, s = _lora_case(70, 32, 16, 8, 0, "bf16", 1)
    assert torch.equal(nv.lora_add(y, x, a, b, ids, scales=s), y)
    y, x, a, b, ids, s = _lora_case(70, 32, 16, 8, 3, "bf16", 1, none=1.0)
    assert torch.equal(nv.lora_add(y, x, a, b, ids, scales=s), y)


def test_lora_index_out_of_range_is_reported():
    y, x, a, b, ids, s = _lora_case(6, 32, 16, 8, 2, "bf16", 2, none=0.0)
    ids[2] = 2
    ids[4] = 2 ** 31 - 1
    got = nv.lora_add(y, x, a, b, ids, scales=s)
    _close_lora(got, y, x, a, b, ids, s, "bf16")
    assert nv.device_status() == 8


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T", [20, 200])
def test_lora_infinite_and_large_values_stay_in_their_rows(act, T):
    y, x, a, b, ids, s = _lora_case(T, 64, 40, 16, 2, act, 3, none=0.0)
    clean = nv.lora_add(y, x, a, b, ids, scales=s)
    x2 = x.clone()
    x2[3, 5], x2[7, 6], x2[11] = float("inf"), float("nan"), 0
    got = nv.lora_add(y, x2, a, b, ids, scales=s)
    rest = [t for t in range(T) if t not in (3, 7, 11)]
    assert torch.equal(got[rest], clean[rest]) and torch.equal(got[11], y[11])
    assert not bool(got[3].isfinite().any()) and bool(got[7].isnan().all())
    a2 = a.clone()
    a2[1] = float("nan")                                                     # an adapter that is not these rows'
    got = nv.lora_add(y, x, a2, b, ids, scales=s)
    mine = ids == 0
    assert torch.equal(got[mine], clean[mine]) and bool(got[~mine].isnan().all())
    # A x beyond FP16's range, brought back by the scale
    big = (x.float() * 64).to(DT[act])
    a3, s3 = (a.float() * 4096).to(DT[act]), s * 2.0 ** -18
    assert float((big.float() @ a3[0].float().t()).abs().max()) > 65504
    _close_lora(nv.lora_add(y, big, a3, b, ids, scales=s3), y, big, a3, b, ids, s3, act)


@pytest.mark.parametrize("rank", [1, 3, 8, 16, 20, 24, 40, 64, 72, 130])
@pytest.mark.parametrize("T,N,K", [(1, 64, 64), (40, 33, 40), (200, 72, 300), (200, 31, 33)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_lora_infinities_are_those_of_the_formula(act, T, N, K, rank):
    """An infinite x meets the rank's own columns alone: infinite of the product's sign, NaN where
    signs meet, and finite in the other rows."""
    y, x, a, b, ids, s = _lora_case(T, K, N, rank, 1, act, rank, none=0.0)
    a, b = a.abs() + 0.25, b.abs() + 0.25                                    # one sign, none zero
    b[0, 1::3] *= -1
    if rank > 1:
        b[0, 2::3, rank - 1] *= -1                                           # both
    x[0, K // 2] = float("inf")
    if T > 1:
        x[T // 2, 0], x[T - 1, K - 1] = float("-inf"), float("inf")
        x[T - 1, 0], x[T - 2] = float("-inf"), 0                             # NaN; nothing
    f = lambda t: t.double().cpu().numpy()
    got = nv.lora_add(y, x, a, b, ids, scales=s)
    with np.errstate(all="ignore"):
        ref = f(y) + f(s)[0] * (f(x) @ f(a)[0].T @ f(b)[0].T)
    got = f(got)
    assert np.isinf(ref[0, :2]).all() and np.isnan(ref[0, 2::3]).all() == (rank > 1) and np.isfinite(ref[1:T // 2]).all()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isinf(got), np.isinf(ref))
    assert np.array_equal(np.sign(got[np.isinf(ref)]), np.sign(ref[np.isinf(ref)]))


# Halves of FP16 leave a component off by 2^-22 of it or 2^-39 of its row's largest (11 bits each: 2^-11 of 2^-11; the last
# bit is 2^-24 and the largest at least 2^14, rounded by half of that bit), those of BF16 by 2^-16; then as above.  y goes
# through the accumulators of at most 12 products (two for each 16 of a rank of up to 96), each off by at most 2^-23 of it.
@pytest.mark.parametrize("apart", [3, 14, 20, 24, 30])
@pytest.mark.parametrize("T,N,rank", [(1, 64, 16), (20, 33, 2), (150, 64, 8), (150, 31, 24), (200, 40, 72), (200, 64, 64)])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_lora_small_components_beside_large_ones(apart, T, N, rank, act):
    """Every second column of B is zero at the row's largest component, as where the adapters of q, k
    and v are one block-diagonal matrix: the output there is that of components far smaller."""
    K, g, half = 64, _gen(apart), apart // 2
    x, a, b = (torch.zeros(s, device="cuda") for s in ((T, K), (1, rank, K), (1, N, rank)))
    uniform = lambda *s: 1 + torch.rand(s, generator=g, device="cuda")
    x[:, 0], x[:, 1] = 2.0 ** (half // 2) * uniform(T), 2.0 ** -((apart - half) // 2) * uniform(T)
    a[0, 0, 0], a[0, 1:, 1] = 2.0 ** (half - half // 2) * 1.5, 2.0 ** -(apart - half - (apart - half) // 2) * uniform(rank - 1)
    b[0] = torch.randn(N, rank, generator=g, device="cuda")
    b[0, ::2, 0] = 0
    y = torch.randn(T, N, generator=g, device="cuda") * 2.0 ** -9
    x, a, b, y = (t.to(DT[act]) for t in (x, a, b, y))
    ids, s = _i32(np.zeros(T)), torch.full((1,), 2.0 ** -half, device="cuda")
    for scale in (s, s * 2.0 ** half):
        got = nv.lora_add(y, x, a, b, ids, scales=scale).double().cpu().numpy()
        f = lambda t: t.double().cpu().numpy()
        ref, mag = batch.lora(f(y), f(x), f(a), f(b), ids.tolist(), f(scale))
        low = np.abs(f(x) @ f(a)[0].T) * f(scale)[0]
        halves = 2.0 ** -16 * mag if act == "bf16" else 2.0 ** -22 * mag + 2.0 ** -39 * low.max(1)[:, None] * np.abs(f(b)[0]).sum(1)
        ref[np.abs(ref) > float(torch.finfo(DT[act]).max)] = np.inf
        lim = U[act] * np.abs(ref) + (K + 256) * 2.0 ** -24 * mag + halves + 12 * 2.0 ** -23 * np.abs(f(y)) + TINY[act]
        near = np.abs(got[:, ::2] - ref[:, ::2]) <= lim[:, ::2]
        assert near.all(), np.abs(got[:, ::2] - ref[:, ::2]).max()
        finite = np.isfinite(ref)
        assert np.all(np.abs(got[finite] - ref[finite]) <= lim[finite])


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T,N,rank", [(3, 64, 16), (20, 33, 2), (200, 64, 64), (200, 31, 24)])
def test_lora_keeps_y_beside_the_largest_and_smallest_products(act, T, N, rank):
    """s A x next to either end of 32 bits: where B is zero the output is y itself."""
    g = _gen(2)
    x, a = torch.zeros(T, 32, device="cuda"), torch.zeros(1, rank, 32, device="cuda")
    x[:, 3], a[0, :, 3] = 1, torch.rand(rank, generator=g, device="cuda") * 0.5
    a[0, 0, 3] = 1
    b = torch.randn(1, N, rank, generator=g, device="cuda")
    b[0, ::3] = 0
    y = torch.randn(T, N, generator=g, device="cuda")
    x, a, b, y = (t.to(DT[act]) for t in (x, a, b, y))
    for s in (1.5 * 2.0 ** 127, 2.0 ** 127, 2.0 ** 126, 2.0 ** 100, 2.0 ** -59, 2.0 ** -60, 2.0 ** -61, 2.0 ** -100, 2.0 ** -126, 0.0):
        got = nv.lora_add(y, x, a, b, _i32(np.zeros(T)), scales=torch.full((1,), s, device="cuda"))
        assert torch.equal(got[:, ::3], y[:, ::3]), s
        if s < 2.0 ** -50:
            assert torch.equal(got, y), s
        elif act == "f16":
            assert bool((got.isinf() | (torch.arange(N, device="cuda") % 3 == 0)).all()), s


def test_lora_zero_padded_ranks_and_adapters_of_one_matrix():
    y, x, a, b, ids, s = _lora_case(40, 128, 64, 32, 3, "bf16", 4)
    a[:, 20:] = 0
    b[:, :, 20:] = 0
    # Ranks of 20 and 32 sum their products in groups of 16 and 32, so the same real number is rounded after
    # 32-bit sums of another order: each lies within the bound above of it, and two such are two bounds apart.
    small = nv.lora_add(y, x, a[:, :20].contiguous(), b[:, :, :20].contiguous(), ids, scales=s)
    _close_lora(small, y, x, a, b, ids, s, "bf16")
    _close_lora(nv.lora_add(y, x, a, b, ids, scales=s), y, x, a, b, ids, s, "bf16")


def test_lora_workspace_stream_and_graph():
    T, n = 100, 6
    y, x, a, b, ids, s = _lora_case(T, 512, 256, 16, n, "bf16", 6)
    need = nv.lora_workspace_size(T, n, 16, 512)
    room = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    want = nv.lora_add(y, x, a, b, ids, scales=s)
    got = nv.lora_add(y, x, a, b, ids, scales=s, workspace=room[:need])
    assert torch.equal(got, want) and bool((room[need:] == 77).all())
    room[:need] = 255                                                        # whatever it holds
    assert torch.equal(nv.lora_add(y, x, a, b, ids, scales=s, workspace=room[:need]), want)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            out = nv.lora_add(y, x, a, b, ids, scales=s)
    for seed in range(3):
        ids.copy_(_i32(np.random.default_rng(seed).integers(-1, n, T)))
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        _close_lora(out, y, x, a, b, ids, s, "bf16")


@pytest.mark.parametrize("rank", [1, 4, 7, 8, 9, 17, 33, 65])
@pytest.mark.parametrize("T,N", [(3, 40), (200, 33), (200, 64)])
def test_lora_reads_no_sums_that_it_has_not_made(T, N, rank):
    """Whatever lies in the columns behind the rank, which nothing is multiplied for."""
    y, x, a, b, ids, s = _lora_case(T, 264, N, rank, 1, "f16", rank)
    room = torch.full((nv.lora_workspace_size(T, 1, rank, 264),), 255, dtype=torch.uint8, device="cuda")     # NaN
    got = nv.lora_add(y, x, a, b, ids, scales=s, workspace=room)
    _close_lora(got, y, x, a, b, ids, s, "f16")
    room.zero_()
    assert torch.equal(nv.lora_add(y, x, a, b, ids, scales=s, workspace=room), got)


@pytest.mark.parametrize("T", [5, 128, 129, 3000])
@pytest.mark.parametrize("n", [1, 9])
def test_lora_in_place_without_an_adapter_keeps_the_order_of_calls(T, n):
    """In place and with no row on an adapter there is nothing to add: the call still ends behind its
    own kernels, so its indexes may be rewritten, and its workspace used again, by what follows."""
    y, x, a, b, ids, s = _lora_case(T, 256, 128, 16, n, "bf16", T + n, none=0.0)
    room = torch.empty(nv.lora_workspace_size(T, n, 16, 256), dtype=torch.uint8, device="cuda")
    none, want = torch.full_like(ids, -1), nv.lora_add(y, x, a, b, ids, scales=s)
    _close_lora(want, y, x, a, b, ids, s, "bf16")
    now = none.clone()
    for _ in range(50):
        z = y.clone()
        now.copy_(none)
        nv.lora_add(z, x, a, b, now, scales=s, out=z, workspace=room)
        now.copy_(ids)
        nv.lora_add(z, x, a, b, now, scales=s, out=z, workspace=room)
        assert torch.equal(z, want)
        nv.lora_add(z, x, a, b, none, scales=s, out=z, workspace=room)       # two such calls in a row, and a third kind behind them
        nv.lora_add(z, x, a, b, none, scales=s, out=z, workspace=room)
        nv.lora_add(y, x, a, b, ids, scales=s, out=z, workspace=room)
        assert torch.equal(z, want)


def test_lora_beside_an_nvfp4_projection():
    """gemm and lora_add as a layer would use them, against the dense product of both."""
    from w4a16_nvfp4_weight_gb300 import synth
    c = synth.gaussian_case(24, 256, 128, seed=9)
    w = gu.repack_case(c)
    x = gu.bits_to_bf16_tensor(c.x_bits)
    _, _, a, b, ids, s = _lora_case(24, 256, 128, 8, 3, "bf16", 9)
    y = nv.gemm(x, w)
    got = nv.lora_add(y, x, a, b, ids, scales=s)
    _close_lora(got, y, x, a, b, ids, s, "bf16")
    full = nv.dequant(w).double()
    for i in range(3):
        rows = ids == i
        ref = x[rows].double() @ (full + s[i].double() * b[i].double() @ a[i].double()).t()
        assert (got[rows].double() - ref).norm() <= 2 * gu.REL_FRO * ref.norm()


# --------------------------------------------------------------------- draws ---

def _check_draws(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, **kw):
    B, V = logits.shape
    dev = lambda v, f: v if not isinstance(v, np.ndarray) else f(v)
    f32 = lambda v: torch.from_numpy(v.astype(np.float32)).cuda()
    tokens, logprob = nv.sample(logits, u, dev(temperature, f32), dev(top_k, _i32), dev(top_p, f32), dev(min_p, f32), return_logprob=True, **kw)
    l, un = logits.double().cpu().numpy(), u.double().cpu().numpy()
    at = lambda v, i: float(np.float32(v[i] if isinstance(v, np.ndarray) else v))
    for i in range(B):
        t, lp = batch.draw(l[i], un[i], at(temperature, i), int(at(top_k, i)), at(top_p, i), at(min_p, i))
        assert int(tokens[i]) == t, (i, int(tokens[i]), t, at(temperature, i), at(top_k, i), at(top_p, i), at(min_p, i))
        got = float(logprob[i])
        assert got == lp or abs(got - lp) <= 2.0 ** -21 * (1 + abs(lp) + np.log(V)), (got, lp)
    return tokens, logprob


def _logits(B, V, kind, act, seed):
    g = _gen(seed)
    l = torch.randn(B, V, generator=g, device="cuda")
    if kind == "peaked":
        l = l * 2 + 0.0
        l.scatter_add_(1, torch.randint(0, V, (B, 12), generator=g, device="cuda"), 15 * torch.rand(B, 12, generator=g, device="cuda"))
    elif kind == "flat":
        l = l * 0.05
    elif kind == "ties":
        l = (l * 2).round()
    elif kind == "masked":
        l = l * 3
        l[:, torch.randperm(V, generator=g, device="cuda")[:V * 9 // 10]] = float("-inf")
    elif kind == "lowest":
        l = l * 3
        l[:, torch.randperm(V, generator=g, device="cuda")[:V * 9 // 10]] = torch.finfo(DT[act]).min
    elif kind == "far":                                                      # all of the rest beyond the histogram
        l = l - 60
        l[:, V // 2] = 0
    return l.to(DT[act])


SETTINGS = [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=7), dict(top_k=50, temperature=0.8), dict(top_p=0.9), dict(top_p=0.5, temperature=1.5),
            dict(min_p=0.05), dict(top_k=40, top_p=0.95, min_p=0.01), dict(top_k=2000, top_p=0.99), dict(temperature=0.0), dict(top_p=0.0), dict(min_p=1.0),
            dict(top_p=0.999999), dict(top_k=10 ** 6)]


@pytest.mark.parametrize("kind", ["normal", "peaked", "flat", "ties", "masked", "lowest", "far"])
@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [1, 17, 1000, 32768, 50001])
def test_sample(kind, act, V):
    for i, how in enumerate(SETTINGS):
        B = 3
        l = _logits(B, V, kind, act, V + i)
        _check_draws(l, torch.rand(B, generator=_gen(i), device="cuda"), **how)


@pytest.mark.parametrize("B,V,act", [(1, 151936, "bf16"), (70, 20011, "f16"), (200, 5003, "f32"), (2, 1 << 20, "bf16"), (40, 100003, "f32")])
def test_sample_settings_of_each_row(B, V, act):
    r = np.random.default_rng(B)
    l = _logits(B, V, "peaked", act, B)
    _check_draws(l, torch.rand(B, generator=_gen(B), device="cuda"), r.choice([0.0, 0.5, 0.8, 1.0, 1.7], B), r.choice([0, 1, 3, 40, 500], B),
                 r.choice([1.0, 0.3, 0.9, 0.97], B), r.choice([0.0, 0.0, 0.03, 0.2], B))


@pytest.mark.parametrize("B,V,act", [(2, 1 << 20, "bf16"), (1, 1 << 20, "f32"), (2, 400003, "f32"), (1, 300001, "f16"), (160, 70001, "f32")])
def test_sample_large_rows(B, V, act):
    """Rows that do not stay in shared memory, blocks of more than 2^16 logits, many rows of several blocks."""
    for i, (kind, how) in enumerate([("flat", dict(top_p=0.9)), ("normal", dict(top_k=3000, top_p=0.5)), ("ties", dict(top_p=0.7)),
                                     ("peaked", dict(top_k=50, top_p=0.9)), ("flat", dict()), ("flat", dict(top_k=V // 2))]):
        _check_draws(_logits(B, V, kind, act, i)[:3 if B > 3 else B], torch.rand(min(B, 3), generator=_gen(i), device="cuda"), **how)
        if B > 3:
            l, u = _logits(B, V, kind, act, i), torch.rand(B, generator=_gen(i), device="cuda")
            many = nv.sample(l, u, **how)
            _check_draws(l[B - 2:], u[B - 2:], **how)
            assert torch.equal(many[B - 2:], nv.sample(l[B - 2:], u[B - 2:], **how))


def test_sample_ends_of_the_random_numbers():
    l = _logits(6, 3001, "peaked", "bf16", 1)
    l[:, 0] = float("-inf")
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 2.0 ** -24, 2.0 ** -149, 0.5, 1e-30], device="cuda")
    for how in (dict(), dict(top_k=5), dict(top_p=0.8), dict(min_p=0.1)):
        _check_draws(l, u, **how)
    outside = torch.tensor([-1.0, 1.0, 7.0, float("nan"), float("inf"), float("-inf")], device="cuda")
    low, _ = nv.sample(l, torch.zeros(6, device="cuda"), top_k=9, return_logprob=True)
    high, _ = nv.sample(l, torch.full((6,), 1 - 2.0 ** -24, device="cuda"), top_k=9, return_logprob=True)
    got = nv.sample(l, outside, top_k=9)
    assert got[0] == low[0] and got[5] == low[5]
    assert torch.equal(got[1:5], high[1:5])                                  # the last kept token


def test_sample_exact_borders():
    """Equal logits: masses are whole numbers of one weight, so borders are exact."""
    V = 1000
    l = torch.zeros(8, V, device="cuda")
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.125, 0.875, 0.5 - 2.0 ** -25, 1 - 2.0 ** -24], device="cuda")
    assert nv.sample(l, u).tolist() == [0, 250, 500, 750, 125, 875, 499, 999]
    assert nv.sample(l, u, top_p=0.5).tolist() == [0, 125, 250, 375, 62, 437, 249, 499]
    assert nv.sample(l, u, top_p=0.5, top_k=100).tolist() == [0, 12, 25, 37, 6, 43, 24, 49]
    assert nv.sample(l, u, top_k=8).tolist() == [0, 2, 4, 6, 1, 7, 3, 7]
    assert nv.sample(l - 77.25, u, 0.3, top_k=8, min_p=1.0).tolist() == [0, 2, 4, 6, 1, 7, 3, 7]
    big = torch.zeros(1, 1 << 20, device="cuda")
    assert nv.sample(big, u[2:3]).tolist() == [1 << 19] and nv.sample(big, u[2:3], top_p=0.5).tolist() == [1 << 18]
    assert nv.sample(big, u[7:8], top_k=70000).tolist() == [69999]


@pytest.mark.parametrize("act", ["bf16", "f16", "f32"])
def test_sample_special_values(act):
    inf, nan = float("inf"), float("nan")
    V = 5000
    l = torch.full((9, V), -inf, device="cuda")
    l[1] = nan
    l[2, 77] = -3.0
    l[3] = 1.0
    l[3, 40] = nan
    l[4, 10], l[4, 4000], l[4, 60] = inf, inf, 5.0
    l[5] = torch.finfo(DT[act]).min
    l[6, 4999], l[6, 0] = 0.0, -0.0
    l[7], l[7, 5] = -torch.finfo(DT[act]).max, torch.finfo(DT[act]).max
    l[8, :50] = nan
    l[8, 50:70] = torch.linspace(-2, 2, 20, device="cuda")
    l = l.to(DT[act])
    u = torch.full((9,), 0.75, device="cuda")
    for how in (dict(), dict(top_k=3), dict(top_p=0.7), dict(temperature=0.0), dict(min_p=0.5), dict(temperature=1e-30), dict(temperature=1e-45),
                dict(temperature=inf), dict(temperature=1e38, top_p=0.5), dict(top_k=3000, top_p=0.9)):
        tokens, logprob = nv.sample(l, u, return_logprob=True, **how)
        assert tokens[:2].tolist() == [-1, -1] and torch.all(logprob[:2] == -inf)
        for i in range(2, 9):
            if i == 4 and how.get("temperature") == inf:
                continue                                                     # infinity over infinity
            t, lp = batch.draw(l[i].double().cpu().numpy(), 0.75, how.get("temperature", 1.0), how.get("top_k", 0),
                               float(np.float32(how.get("top_p", 1.0))), how.get("min_p", 0.0))
            assert int(tokens[i]) == t and abs(float(logprob[i]) - lp) <= 2.0 ** -21 * (1 + abs(lp) + np.log(V)), (how, i)
    assert nv.sample(l[4:5], u[:1], temperature=-1.0).tolist() == [10] and nv.sample(l[4:5], u[:1], temperature=nan).tolist() == [10]
    assert nv.sample(l[3:4], u[:1], top_p=nan, min_p=nan).tolist() == nv.sample(l[3:4], u[:1]).tolist()


def test_sample_close_logits_and_extremes():
    """Values a bit apart in one bin, far more than are sorted; rows whose products leave 32 bits."""
    V = 40000
    base = torch.arange(V, device="cuda", dtype=torch.float32)
    close = 1 + base[torch.randperm(V, generator=_gen(1), device="cuda")] * 2.0 ** -23
    steep = base.flip(0) * 1e30
    wide = torch.randn(V, generator=_gen(2), device="cuda") * 5 + 30000.0
    l = torch.stack([close, -close, steep, wide, close * 0 + 3])
    u = torch.rand(5, generator=_gen(3), device="cuda")
    for how in (dict(), dict(top_k=1500), dict(top_k=5000, top_p=0.5), dict(top_p=0.3), dict(temperature=1e-3, top_k=20000), dict(temperature=1e-6),
                dict(temperature=1e-4, top_p=0.9), dict(temperature=0.02, min_p=0.5)):
        _check_draws(l, u, **how)


def test_sample_strides_offsets_and_streams():
    V = 3001
    wide = _logits(30, V + 9, "peaked", "bf16", 4)
    u = torch.rand(30, generator=_gen(4), device="cuda")
    for start in (0, 1, 3, 8):
        part = wide[:, start:start + V]
        a, la = nv.sample(part, u, 0.9, 30, 0.9, return_logprob=True)
        b, lb = nv.sample(part.contiguous(), u, 0.9, 30, 0.9, return_logprob=True)
        assert torch.equal(a, b) and torch.equal(la, lb)
    _check_draws(wide[:, 5:5 + V], u, 0.9, 30, 0.9)
    once = wide[:1].expand(30, V + 9)
    assert torch.equal(nv.sample(once, u), nv.sample(once.contiguous(), u))
    out, lp = torch.full((30,), 9, device="cuda"), torch.empty(30, device="cuda")
    got = nv.sample(wide, u, out=out, logprob=lp)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, nv.sample(wide, u))
    assert nv.sample(wide[:0], u[:0]).shape == (0,)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            token = nv.sample(wide, u, temperature=0.9, top_p=0.9)
    for seed in range(3):
        wide.copy_(_logits(30, V + 9, "normal", "bf16", seed))
        u.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(token, nv.sample(wide, u, temperature=0.9, top_p=0.9))


def test_sample_does_not_depend_on_the_split():
    """The same row alone (several blocks) and among many (one block)."""
    V = 60000
    l = _logits(200, V, "flat", "bf16", 7)
    u = torch.rand(200, generator=_gen(7), device="cuda")
    many, lp = nv.sample(l, u, 1.1, 20000, 0.8, return_logprob=True)
    for i in (0, 63, 199):
        one, lp1 = nv.sample(l[i:i + 1], u[i:i + 1], 1.1, 20000, 0.8, return_logprob=True)
        assert one[0] == many[i] and lp1[0] == lp[i]


# The logarithm has one unit in the last place, the sum behind it half of one: 1.5 * 2^-23 of the result, whose weights
# are right to 2^-29.9 each.  Shares below 2^-19 or so may come from places instead: two fused products and one by ln 2
# (2^-24 of at most the result each, 2^-25 ln 2's own), a logarithm and a conversion (2^-23 of it, 2^-24), the difference.
@pytest.mark.parametrize("kind", ["normal", "peaked", "flat"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("how", [dict(), dict(temperature=0.6, top_k=20), dict(top_p=0.9), dict(temperature=1.5, top_k=50, top_p=0.95)])
def test_sample_log_probabilities_to_their_last_bits(kind, act, how):
    B, V = 400, 1500
    l, u = _logits(B, V, kind, act, 5), torch.rand(B, generator=_gen(5), device="cuda")
    tokens, logprob = nv.sample(l, u, return_logprob=True, **how)
    l, u, tokens, logprob = l.double().cpu().numpy(), u.double().cpu().numpy(), tokens.tolist(), logprob.double().tolist()
    f32 = {k: float(np.float32(v)) if isinstance(v, float) else v for k, v in how.items()}
    for i in range(B):
        t, lp = batch.draw(l[i], u[i], f32.get("temperature", 1.0), f32.get("top_k", 0), f32.get("top_p", 1.0))
        lim = 1.5 * 2.0 ** -23 * abs(lp) + 2.0 ** -28 if lp > -13 else 4.5 * 2.0 ** -24 * abs(lp) + 2.0 ** -24
        assert tokens[i] == t and abs(logprob[i] - lp) <= lim, (i, lp, logprob[i] - lp)


def test_sample_frequencies():
    l = torch.log(torch.tensor([0.1, 0.4, 0.2, 0.3], device="cuda")).expand(2000, 4)
    u = (torch.arange(2000, device="cuda") + 0.5) / 2000
    assert torch.bincount(nv.sample(l, u)).tolist() == [200, 800, 400, 600]


def test_calls_on_two_streams_at_once():
    """The same calls on two streams, whose kernels may run side by side, give what one stream gives."""
    l = _logits(20, 50001, "normal", "bf16", 3)
    u = torch.rand(20, generator=_gen(3), device="cuda")
    y, x, a, b, ids, s = _lora_case(300, 512, 264, 24, 5, "bf16", 8)
    r = np.random.default_rng(2)
    lengths, new = r.integers(0, 60, 300), r.integers(0, 9, 300)
    table, stack = _pool(r, lengths, 8, 12, 400)
    args = [_i32(v) for v in (lengths, new, table, stack, [400])]

    def all_of_it():
        t = nv.extend_tables(args[0], args[1], args[2].clone(), args[3], args[4], 8, 3000, row_tables=True)
        return [nv.sample(l, u, 0.9, 0, 0.9), nv.sample(l, u, 0.9, 40), nv.lora_add(y, x, a, b, ids, scales=s), t["slots"], t["row_tables"]]

    want = all_of_it()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for k, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[k].append(all_of_it())
    torch.cuda.synchronize()
    for outs in got:
        for out in outs:
            assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_calls_of_other_sizes_from_other_threads(lib):
    """The C ABI from four host threads at once (ctypes holds no lock over a call), each with sizes for which
    the same kernels take another amount of shared memory: no launch fails, and all give what one thread gives."""
    P = lambda t: ctypes.c_void_p(t.data_ptr())
    how = _lib_module.Sampling(temperature_all=1.0, top_p_all=0.9)

    def draws(V):
        l, u = _logits(2, V, "normal", "f32", V), torch.rand(2, generator=_gen(V), device="cuda")
        return nv.sample(l, u, top_p=float(np.float32(0.9))), lambda out, stream: lib.nvfp4_sample(
            P(l), V, 2, 2, V, P(u), ctypes.byref(how), P(out), None, stream)

    def adapters(n, rank):
        y, x, a, b, ids, s = _lora_case(2000, 64, 64, rank, n, "bf16", n)
        room = torch.empty(nv.lora_workspace_size(2000, n, rank, 64), dtype=torch.uint8, device="cuda")
        return nv.lora_add(y, x, a, b, ids, scales=s), lambda out, stream: lib.nvfp4_lora_add(
            P(y), 64, P(x), 64, P(a), P(b), P(s), P(ids), 2000, n, rank, 64, 64, 0, P(out), P(room), room.numel(), stream)

    calls = [draws(9000), draws(100003), adapters(1100, 4), adapters(4000, 4)]
    torch.cuda.synchronize()
    failed, wrong = [0] * 4, [0] * 4

    def run(k):
        want, call = calls[k]
        stream, out = torch.cuda.Stream(), torch.empty_like(want)
        for _ in range(1500):
            failed[k] += call(out, ctypes.c_void_p(stream.cuda_stream)) != 0
        stream.synchronize()
        wrong[k] = not torch.equal(out, want)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert failed == [0] * 4 and not any(wrong), (failed, wrong)


def test_a_batch_step_runs_together():
    """Logits of an NVFP4 head with adapters, a token of each request, its pages: twice, in a graph."""
    from w4a16_nvfp4_weight_gb300 import synth
    B, H, V, page = 12, 256, 512, 4
    c = synth.gaussian_case(B, H, V, seed=11)
    head, x = gu.repack_case(c), gu.bits_to_bf16_tensor(c.x_bits)
    _, _, a, b, ids, s = _lora_case(B, H, V, 8, 3, "bf16", 12)
    u = torch.rand(B, generator=_gen(1), device="cuda")
    lengths, table, pages, count = _i32(np.zeros(B)), _i32(np.zeros((B, 4))), _i32(np.arange(40)), _i32([40])
    ones = _i32(np.ones(B))

    def step():
        t = nv.extend_tables(lengths, ones, table, pages, count, page, B, in_place=True)
        return nv.sample(nv.lora_add(nv.gemm(x, head), x, a, b, ids, scales=s), u, 0.8, 20, 0.95), t

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            tokens, t = step()
    for i in range(9):
        u.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        l = nv.lora_add(nv.gemm(x, head), x, a, b, ids, scales=s).double().cpu().numpy()
        assert tokens.tolist() == [batch.draw(l[k], float(u[k]), float(np.float32(0.8)), 20, float(np.float32(0.95)))[0] for k in range(B)]
        assert lengths.tolist() == [i + 1] * B and t["positions"].tolist() == [i] * B
        assert count.tolist() == [40 - B * (i // page + 1)]
        assert t["slots"].tolist() == [int(table[k, i // page]) * page + i % page for k in range(B)]
