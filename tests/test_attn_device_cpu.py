"""The binding's check of the attention and cache calls' device (no GPU needed)."""
import pytest
import torch

from speculative_decoding_verification_09_gb300 import binding


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The library launches on the current device: with another one's tensors and its default stream (a null handle) the
    kernels would read that device's addresses from this one."""
    class Tensor:
        is_cuda, device = True, "cuda:1"

        def get_device(self):
            return 1

    monkeypatch.setattr(binding, "_several_devices", lambda: True, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(binding.SpecVerifyError, match="current device"):
        binding._cuda_device(Tensor(), "q")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert binding._cuda_device(Tensor(), "q") == 1
    text = open(binding.__file__).read()
    for call in ("sv_tree_attn", "sv_ring_attn", "sv_prompt_attn", "sv_kv_fill", "sv_page_commit"):
        body = text[text.index(f"def {call}("):]
        assert "_cuda_device(" in body[:body.index("_check(")], call
