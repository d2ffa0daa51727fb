"""Packed tokens as many as an int counts: the last ones are rotated and appended like the others.  Against the 32-bit
steps of kv8_util, bit for bit."""
import numpy as np
import pytest
import torch

import kv8_util as ku
from speculative_decoding_verification_09_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def _room():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 90 GB")
    yield
    torch.cuda.empty_cache()


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def tokens(D, n):
    """MOST tokens of one head, of which the first and the last n have values."""
    g = torch.Generator().manual_seed(3)
    x = torch.empty(MOST, 1, D, dtype=BF, device=DEV)
    x[:n] = torch.randn(n, 1, D, generator=g).to(BF).to(DEV)
    x[-n:] = torch.randn(n, 1, D, generator=g).to(BF).to(DEV)
    return x


@pytest.mark.parametrize("T", [MOST, MOST - 1, MOST - 40])
def test_rotation_of_the_last_tokens(T):
    n, D, rows = 100, 8, 200
    q = tokens(D, n)[:T]
    at = torch.zeros(T, dtype=torch.int32, device=DEV)
    at[:n] = i32(np.arange(n))
    at[-n:] = i32(np.arange(n) + 100)
    angles = torch.empty(rows, 2, D // 2, device=DEV)
    binding.sv_rope_table(angles)
    want = [ku.rotate32(q[s], angles[at[s].long()], False).to(BF) for s in (slice(0, n), slice(T - n, T))]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.sv_rope(q, None, at, angles, q, dev_status=st)
    assert int(st.item()) == 0
    assert torch.equal(q[:n], want[0]) and torch.equal(q[T - n:], want[1])


def test_append_of_the_last_tokens():
    n, D, page = 300, 8, 16
    k = tokens(D, n)
    P = 20
    kp, vp = (torch.zeros(P, 1, page, D, dtype=BF, device=DEV) for _ in "kv")
    table, out, st = i32(np.arange(P)[None, ::-1].copy()), i32([0]), i32([0])
    binding.sv_page_append(k, k, kp, vp, table, i32([5]), i32([MOST - n, MOST]), out_seq_lens=out, dev_status=st)
    assert int(st.item()) == 0 and out.tolist() == [5 + n]
    for pool in (kp, vp):
        got = pool[table[0].long()].transpose(1, 2).reshape(-1, 1, D)[5:5 + n]
        assert torch.equal(got, k[-n:])


@pytest.mark.parametrize("block", [8, 128])
def test_append8_of_the_last_tokens(block):
    n, D, page, start = 300, 16, 128, 3
    k = tokens(D, n)
    P = 4
    kp, vp = (torch.zeros(P, 1, page, D, dtype=torch.uint8, device=DEV).view(ku.E4M3) for _ in "kv")
    ks, vs = (torch.zeros(P, 1, page // block, dtype=torch.uint8, device=DEV).view(ku.E8M0) for _ in "kv")
    table, out, st = i32([[2, 0, 3]]), i32([0]), i32([0])
    want = ku.split(kp.cpu(), ks.cpu())
    ku.write(*want, k[-n:].transpose(0, 1).double().cpu(), [2, 0, 3], start, BF)
    binding.sv_page_append8(k, k, kp, vp, ks, vs, table, i32([start]), i32([MOST - n, MOST]), out_seq_lens=out,
                            dev_status=st)
    assert int(st.item()) == 0 and out.tolist() == [start + n]
    for pages, scales in ((kp, ks), (vp, vs)):
        values, exps = ku.split(pages.cpu(), scales.cpu())
        for t in range(start, start + n):  # (before them: entries of zero, whatever the scale)
            pg, row = (2, 0, 3)[t // page], t % page
            assert torch.equal(values[pg, 0, row], want[0][pg, 0, row]), t
            assert int(exps[pg, 0, row // block]) == int(want[1][pg, 0, row // block]), t
