"""examples/serve_batch.py: it runs, and every page is held by a request or free."""

import importlib.util
import os

import pytest
import torch

import w4a16_nvfp4_weight_gb300 as nv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(lib):
    spec = importlib.util.spec_from_file_location("serve_batch", os.path.join(ROOT, "examples", "serve_batch.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_prompts_and_steps(example):
    n, V, page, width, pages = 5, 64, 4, 16, 60
    g = torch.Generator(device="cuda").manual_seed(3)
    model = example.Model(V, 128, 4, 2, 64, 8, 3, 64, g)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = example.Batch(n, width, pages, page, torch.tensor([-1, 0, 1, 2, 0], **i32), torch.tensor([0.0, 0.7, 1.0, 1.3, 1.0], device="cuda"),
                          torch.tensor([0, 5, 0, 20, 64], **i32), torch.tensor([1.0, 0.9, 0.8, 1.0, 0.95], device="cuda"))
    cache = {k: torch.zeros(pages, 2, page, 64, dtype=torch.bfloat16, device="cuda") for k in ("k_cache", "v_cache")}
    prompts = [[1 + i] * (1 + 3 * i) for i in range(n)]
    u = torch.rand(n, device="cuda", generator=g)
    tokens = example.prefill(model, batch, cache, prompts, u)
    assert bool(((tokens >= 0) & (tokens < V)).all()) and batch.lengths.tolist() == [len(p) for p in prompts]
    end_token, lengths = int(tokens[2]), batch.lengths.tolist()
    ended = [False] * n
    for _ in range(12):
        u.uniform_(generator=g)
        running = tokens >= 0
        tokens = example.step(model, batch, cache, tokens, u, end_token)
        for i in range(n):
            if not running[i]:
                assert tokens[i] == -1 and batch.lengths[i] == 0
            elif tokens[i] == -1:
                ended[i] = True
                assert batch.lengths[i] == 0
            else:
                assert 0 <= tokens[i] < V and tokens[i] != end_token
                lengths[i] += 1
                assert batch.lengths[i] == lengths[i]
        held = [int(p) for b in range(n) for p in batch.table[b, :-(-int(batch.lengths[b]) // page)]]
        free = batch.free_pages[:int(batch.free_count)].tolist()
        assert sorted(held + free) == list(range(pages))
    assert nv.device_status() == 0


def test_requests_without_room_end(example):
    """Six pages: two of the prompts do not fit, one is empty, and the others grow until one of them has no page left."""
    n, V, page, width, pages = 5, 64, 4, 16, 6
    g = torch.Generator(device="cuda").manual_seed(4)
    model = example.Model(V, 128, 4, 2, 64, 8, 3, 64, g)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = example.Batch(n, width, pages, page, torch.tensor([-1, 0, 1, 2, 0], **i32), torch.ones(n, device="cuda"),
                          torch.zeros(n, **i32), torch.ones(n, device="cuda"))
    cache = {k: torch.zeros(pages, 2, page, 64, dtype=torch.bfloat16, device="cuda") for k in ("k_cache", "v_cache")}
    u = torch.rand(n, device="cuda", generator=g)
    tokens = example.prefill(model, batch, cache, [[], [1] * 4, [2] * 5, [3] * 17, [4] * 3], u)
    assert (tokens >= 0).tolist() == [False, True, True, False, False] and batch.lengths.tolist() == [0, 4, 5, 0, 0]
    for _ in range(25):
        before, running = batch.lengths.tolist(), (tokens >= 0).tolist()
        u.uniform_(generator=g)
        tokens = example.step(model, batch, cache, tokens, u, V)             # no token ends a request
        for i in range(n):
            if tokens[i] >= 0:
                assert running[i] and batch.lengths[i] == before[i] + 1
            else:
                assert batch.lengths[i] == 0
                if running[i]:                                               # only where its next token needed a page too many
                    assert before[i] % page == 0 and sum(-(-b // page) for b in before) == pages
        held = [int(p) for b in range(n) for p in batch.table[b, :-(-int(batch.lengths[b]) // page)]]
        assert sorted(held + batch.free_pages[:int(batch.free_count)].tolist()) == list(range(pages))
    assert not bool((tokens >= 0).any()) and nv.device_status() == 0
