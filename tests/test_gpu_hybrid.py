"""The operators of prompts and attention together with the tree verify, as examples/hybrid_round.py uses them.

The rounds' logits and the single steps' go through different kernels.  A layer rounds its activations to bf16 about eight
times in a row (relative error 2^-9 / sqrt(3) rms each), so over the four layers of two such passes the logits are
sqrt(2 * 8 * 4) * 2^-9 / sqrt(3) = 0.9 % of their deviation apart (rms); 4.5 times that over some 10^4 logits is 0.04, and
the bar leaves a factor 2.5 for the norms.  A stale state, a lost row or a wrong path is a difference of order one."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from speculative_decoding_mamba2_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "hybrid_round.py")
    spec = importlib.util.spec_from_file_location("hybrid_round", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kw", [dict(S=2, prompt_len=150, tokens=20), dict(S=5, prompt_len=63, tokens=10, nodes=31, page=8),
                                dict(S=1, prompt_len=1, tokens=6, Hkv=4, page=128)], ids=str)
def test_rounds_equal_single_steps(example, kw):
    per_round, worst = example.run(seed=3, **kw)
    assert per_round > 1.0
    assert worst < 0.1
