"""Rates of rotation that 64-bit floats do not hold are refused, on the host before any CUDA call; those that they do
are not, however extreme."""
import pytest
import torch

import __graft_entry__
from speculative_decoding_verification_09_gb300 import binding

FAKE = 0x10000000  # never dereferenced: without a GPU no launch succeeds


@pytest.fixture(scope="module")
def table():
    __graft_entry__.build()
    L = binding.lib()

    def call(scaling, base=1e4, factor=1.0, original=4096, low=1.0, high=32.0, rot=64):
        return L.sv_rope_table(scaling, base, factor, original, low, high, 1.0, rot, 0, 8, FAKE, None)
    return call


LINEAR, BASE, RAMP, WAVE = (binding.SV_ROPE_LINEAR, binding.SV_ROPE_BASE, binding.SV_ROPE_RAMP, binding.SV_ROPE_WAVE)


@pytest.mark.parametrize("kw", [
    dict(scaling=LINEAR, factor=1e-310),                 # 1 / factor
    dict(scaling=RAMP, factor=1e-310, original=10**6),   # the last pairs' share of it
    dict(scaling=WAVE, factor=1e-310),
    dict(scaling=BASE, base=1e300, factor=1e10),         # the base itself
    dict(scaling=BASE, base=1e10, factor=1e-170, rot=4), # 0: every rate but the first infinite
    dict(scaling=BASE, base=1e300, factor=1e300),
])
def test_rates_that_no_float_holds_are_refused(table, kw):
    assert table(**kw) == binding.SV_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the call would go on to launch")
@pytest.mark.parametrize("kw", [
    dict(scaling=LINEAR, factor=1e300), dict(scaling=LINEAR, factor=1e-300), dict(scaling=BASE, base=1e4, factor=32.0),
    dict(scaling=BASE, base=1e300, factor=1e-10), dict(scaling=RAMP, factor=32.0), dict(scaling=WAVE, factor=1e300),
    dict(scaling=RAMP, factor=2.0, original=1), dict(scaling=binding.SV_ROPE_NONE, base=1.0 + 2.0 ** -52),
])
def test_others_go_on(table, kw):
    assert table(**kw) == binding.SV_ERR_CUDA
