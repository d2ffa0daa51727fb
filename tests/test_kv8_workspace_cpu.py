"""The workspace of the attention over 8-bit pages: bounded, whatever the batch, so that callers who only read 16-bit
pages get little that they do not use from a workspace for both."""
import pytest

from speculative_decoding_verification_09_gb300 import binding

MIB = 1 << 20
# nodes, heads, KV heads, dimensions
SIZES = [(1, 1, 1, 16), (1, 32, 8, 128), (22, 32, 8, 128), (64, 32, 32, 128), (256, 128, 8, 128), (5, 8, 1, 64),
         (130, 4, 4, 32)]


def one(N, Hq, Hkv, D):
    """What one request needs: three terms of queries and staged keys, their powers of two."""
    return 3 * N * (Hq + Hkv) * D + 4 * N * Hq + Hkv * (-(-N // 128)) * 64


@pytest.mark.parametrize("size", SIZES)
def test_workspace_is_bounded(size):
    base = binding.sv_attn_workspace_bytes(*size)
    last = 0
    for B in (1, 2, 3, 64, 500, 1024, 5000, 30000, 65535):
        n = binding.sv_attn8_workspace_bytes(B, *size)
        assert n >= last, "grows with the batch"
        assert n <= base + max(256 * MIB, one(*size)) + 5 * 256, B
        if B * one(*size) <= 256 * MIB:
            assert n >= base + B * one(*size), "holds small batches whole"
        last = n


def test_default_workspace_of_large_batches():
    """1024 requests of 64 nodes, 32 heads of 128: 0.8 GB of terms."""
    size = (64, 32, 8, 128)
    both = binding.make_attn_workspace(1024, *size, "cpu").numel()
    assert both <= binding.sv_attn_workspace_bytes(*size) + 257 * MIB
    assert binding.make_attn_workspace(1024, *size, "cpu", 16).numel() == binding.sv_attn_workspace_bytes(*size)
