"""The attention block's operators with the selector and the accept check in
one decoding loop: blocks of drafts emit what one token at a time does."""
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


@pytest.mark.parametrize("fp8", [False, True])
def test_blocks_emit_what_single_tokens_do(example, fp8):
    blocks, single = example.main(steps=12, fp8=fp8)
    for x, y in zip(blocks, single):
        assert len(x) >= 13  # a token per step at least, and the prompt's
        # (logits of unit-variance embeddings differ by far more than the rounding of the two attention tilings)
        assert x == y[:len(x)]
