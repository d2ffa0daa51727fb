"""The attention calls where something is wrong: waits that run out, and invalid requests whose items are cut."""
import time

import numpy as np
import pytest
import torch

import test_gpu_attn as ta
from speculative_decoding_verification_09_gb300 import binding

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.lib()


def calls():
    """Every layout, with items that are cut (and joined) and left whole."""
    lens = [3000, 100, 0, 777]
    return {
        "16 rows, cut": (ta.tree_call, ta.tree_inputs(1, 4, 4, 8, 2, 64, 16, lens, BF)),
        "16 rows, whole": (ta.tree_call, ta.tree_inputs(2, 4, 4, 8, 2, 128, 16, [100, 90, 0, 3], HF)),
        "32 rows, cut": (ta.tree_call, ta.tree_inputs(3, 4, 7, 8, 2, 128, 128, lens, HF)),
        "128 rows, cut": (ta.tree_call, ta.tree_inputs(4, 4, 22, 8, 2, 128, 16, lens, BF)),
        "256 rows, cut": (ta.tree_call, ta.tree_inputs(5, 4, 61, 28, 4, 64, 16, lens, HF)),
        "256 rows, whole": (ta.tree_call, ta.tree_inputs(6, 4, 61, 8, 2, 128, 64, [100, 90, 0, 3], BF)),
        "ring": (ta.ring_call, ta.ring_inputs(7, 4, 5, 8, 2, 128, 4, 2000, lens, BF)),
        "prompts, one tile": (ta.prompt_call, ta.prompt_inputs(8, [300, 5, 0, 700], 8, 2, 64, 4, 100, HF)),
        "prompt, pairs": (ta.prompt_call, ta.prompt_inputs(9, [5100], 16, 8, 128, 4, 300, BF)),
    }


def test_bounded_waits_report_timeout_and_context_recovers():
    """With one copy left out, the waits for it run out after their one-second limit: the call reports SV_ST_TIMEOUT and
    returns, and the same call afterwards gives the bits that it gave before."""
    for name, (call, c) in calls().items():
        want, st = call(c)
        assert int(st.item()) == 0, name
        binding.sv_attn_test_withhold(True)
        try:
            t0 = time.perf_counter()
            _, st = call(c)
            torch.cuda.synchronize()
            waited = time.perf_counter() - t0
        finally:
            binding.sv_attn_test_withhold(False)
        assert int(st.item()) & binding.SV_ST_TIMEOUT, name
        assert 0.5 < waited < 30.0, name
        for _ in range(2):
            again, st = call(c)
            assert int(st.item()) == 0 and torch.equal(again, want), name
