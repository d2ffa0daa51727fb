"""The attention kernels' plan of prompt items by itself: which query tiles an item's number stands for, whatever the order
in which the numbers come (blocks take over items of blocks not yet launched, in an order that nothing promises)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from speculative_decoding_verification_09_gb300 import _build_lib

pytestmark = pytest.mark.gpu
TILE = 128


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    out = str(tmp_path_factory.mktemp("plan") / "probe.so")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([_build_lib._nvcc(), *_build_lib.NVCC_FLAGS, "-shared", "-I", os.path.join(_build_lib.ROOT, "include"),
                    "-I", os.path.join(_build_lib.PKG, "csrc"), os.path.join(here, "attn_plan_probe.cu"), "-o", out],
                   check=True)
    lib = ctypes.CDLL(out)
    P, I = ctypes.c_void_p, ctypes.c_int
    lib.plan_items.argtypes = [P, I, I, I, I, I, I, I, P, I, P, P]
    return lib


def items(lens, Hkv, tokens, sink, window):
    """[(sequence, head, query tile, key tiles)] in the order of the numbers: a sequence's last tokens first."""
    out = []
    for b, n in enumerate(lens):
        for mt in range(-(-n // tokens) - 1, -1, -1):
            q0, q1 = mt * tokens, min((mt + 1) * tokens, n) - 1
            first = max(0, q0 - window + 1)
            near = -(-sink // TILE) if first > sink else 0
            first = first if near or first > sink else 0
            out += [(b, h, mt, near + -(-(q1 + 1 - first) // TILE)) for h in range(Hkv)]
    return out


@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("pair", [0, 1])
@pytest.mark.parametrize("count,Hkv,tpt,sink,window", [(1, 3, 16, 4, 100), (31, 1, 128, 0, 1 << 30), (100, 4, 32, 200, 300),
                                                       (1000, 2, 8, 4, 64)])
def test_items_in_any_order(probe, count, Hkv, tpt, sink, window, pair, order):
    rng = np.random.default_rng(count)
    lens = [int(x) for x in rng.choice([0, 1, 30, 700], count)]
    lens[-1] = 900
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
    want = items(lens, Hkv, (2 if pair else 1) * tpt, sink, window)
    ids = np.arange(len(want) + 5)[:: max(1, len(want) // 3000)]  # some past the last item
    ids = {"up": ids, "down": ids[::-1], "mixed": rng.permutation(ids)}[order].astype(np.int64)
    out = torch.full((len(ids), 5), -7, dtype=torch.int32, device="cuda")
    d = torch.from_numpy(ids.copy()).cuda()
    assert probe.plan_items(cu.data_ptr(), count, sum(lens), Hkv, tpt, pair, sink, window, d.data_ptr(), len(ids),
                            out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    for i, got in zip(ids.tolist(), out.tolist()):
        if i < len(want):
            assert tuple(got) == (1, *want[i]), i
        else:
            assert got[0] == 0, i
