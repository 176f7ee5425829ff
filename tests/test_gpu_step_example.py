"""The operators around a step's attention in one decoding loop with the
attention block, the selector and the accept checks: pages, matrix products and
adjusted logits, with penalties, and by rejection sampling."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from speculative_decoding_draft_tcgen05_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_block.py")
    spec = importlib.util.spec_from_file_location("verify_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_blocks_emit_what_single_tokens_do_under_penalties(example):
    blocks, single = example.main(steps=12, repetition=1.5)
    plain, _ = example.main(steps=12, check=False)
    for x, y in zip(blocks, single):
        assert len(x) >= 13 and x == y[:len(x)]
    assert blocks != plain  # (the penalties do count)


def test_sampled_blocks(example):
    blocks, _ = example.main(steps=8, sample=True, repetition=1.2)
    for x in blocks:
        assert len(x) >= 9 and all(0 <= t < 2048 for t in x)


def test_pages_return(example):
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 2048, (n,), generator=g, dtype=torch.int32).cuda() for n in (20, 3, 64)]
    model = example.Model()
    blocks, _ = example.decode(model, prompts, 5, 7)
    # a prompt and what was emitted, but for the last token, which has not been through the model
    assert model.pool.lens.tolist() == [len(p) + len(x) - 1 for p, x in zip(prompts, blocks)]
    held = sum(-(-n // 16) for n in model.pool.lens.tolist())
    assert model.pool.counters.tolist() == [model.pool.free_pages.shape[0] - held, 0]
    model.pool.trim(batch=3)
    assert sorted(model.pool.free_pages.tolist()) == list(range(model.pool.free_pages.shape[0]))
