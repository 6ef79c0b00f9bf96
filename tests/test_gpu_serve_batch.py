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
