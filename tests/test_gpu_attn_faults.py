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
    """With a slot that never fills, the waits for it run out after their one-second limit: the call reports SV_ST_TIMEOUT and
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


def test_a_long_item_before_others_is_no_timeout():
    """An item that takes longer than a wait may: the CTA's plan waits for it to end before it plans the fifth after it.
    No queries, so every weight is 1, and ones in one value row of the page that all tables name: the output is exact."""
    page, groups, cols = 65536, 152, 9216
    lens = []
    for _ in range(groups):
        lens += [cols * page, 8, 8, 8, 8, 8]
    B = len(lens)
    dev = ta.DEV
    q = torch.zeros(B, 1, 1, 8, dtype=BF, device=dev)
    kp, vp = torch.randn(1, 1, page, 8, device=dev).to(BF), torch.zeros(1, 1, page, 8, dtype=BF, device=dev)
    vp[0, 0, 5] = 1.0
    kn, vn = torch.randn(B, 1, 1, 8, device=dev).to(BF), torch.zeros(B, 1, 1, 8, dtype=BF, device=dev)
    table, out, st = torch.zeros(B, cols, dtype=torch.int32, device=dev), torch.empty_like(q), ta.status()
    ws = binding.make_attn_workspace(B, 1, 1, 1, 8, dev)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in "be")
    begin.record()
    binding.sv_tree_attn(q, kp, vp, table, ta.i32(lens), kn, vn, None, out, ws, dev_status=st)
    end.record()
    torch.cuda.synchronize()
    assert begin.elapsed_time(end) > 1200.0  # the long item alone outlasts the limit
    assert int(st.item()) == 0
    n = torch.tensor(lens, device=dev, dtype=torch.float64)
    seen = torch.where(n == 8, 1.0, n / page)
    assert torch.equal(out[:, 0, 0], (seen / (n + 1)).to(BF)[:, None].expand(B, 8))


@pytest.mark.parametrize("N,G", [(1, 4), (4, 6), (20, 4), (60, 4)])
def test_many_small_weights_in_16_bits(N, G):
    """A million keys whose weights are 2^-25.5 of one key's, in 16-bit floats: together 2 % of the sum, and all of the
    output.  With 2^20 keys (and no more than 2^21 in all) the kernel's 16-bit weights are at least 2^7 for a row's largest,
    in steps of 2^-24 at the least: a weight is off by at most 2^-32 of the largest, beside half a step of its own (2^-11),
    which also bounds the output's rounding; 32-bit sums and scores add 2^-23 of the sum for each of the L / 16 products' terms, and 2 (D + 8) E 2^-23 as
    in attn_util.  A request for every SM, so that none is cut: a part of its own would have a maximum of its own."""
    page, cols, D, Hkv, B = 4096, 256, 8, 1, 152
    L = page * cols
    dev = ta.DEV
    kp, vp = torch.zeros(cols, Hkv, page, D, dtype=HF, device=dev), torch.ones(cols, Hkv, page, D, dtype=HF, device=dev)
    kp[:, :, :, 0] = -25.5
    kn, vn = torch.zeros(B, Hkv, N, D, dtype=HF, device=dev), torch.zeros(B, Hkv, N, D, dtype=HF, device=dev)
    q = torch.zeros(B, N, Hkv * G, D, dtype=HF, device=dev)
    q[..., 0] = 1.0
    kp[0, 0, 7, 0], vp[0, 0, 7] = 0.0, 0.0  # the one key, early: the others never raise the maximum
    kn[..., 0] = -60.0  # the staged entries weigh nothing
    parent = ta.i32([[-1] + [0] * (N - 1)] * B)
    out, st = torch.empty_like(q), ta.status()
    ws = binding.make_attn_workspace(B, N, Hkv * G, Hkv, D, dev)
    binding.sv_tree_attn(q, kp, vp, ta.i32([range(cols)] * B), ta.i32([L] * B), kn, vn, parent, out, ws,
                         scale=float(np.log(2.0)), dev_status=st)
    assert int(st.item()) == 0
    small = (L - 1) * 2.0 ** -25.5
    want = small / (1.0 + small)
    tol = 2.0 ** -32 * L + want * (2 * 2.0 ** -11 + (L / 16 + 2 * (D + 8) * 25.5) * 2.0 ** -23)
    assert float((out.double() - want).abs().max()) <= tol
    assert tol < want / 40


# ------------------------------------------------------------------ invalid requests whose items are cut

LAYOUTS = [(3, 4, 64), (5, 5, 128), (22, 4, 128), (61, 4, 64), (200, 2, 128)]  # 12, 25, 88, 244 and 400 rows


@pytest.mark.parametrize("N,G,D", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_cut_invalid_trees(N, G, D, dtype):
    """Items cut over many blocks, of which one or a few see what is wrong: the whole request is zeros."""
    lens, page = [4100, 3000, 5000], 16
    good = ta.tree_inputs(21, 3, N, 2 * G, 2, D, page, lens, dtype)
    want, st = ta.tree_call(good)
    assert int(st.item()) == 0
    for b in range(3):
        ta.au.check(want[b], *ta.tree_reference(good, b), f"request {b}")
    cases = [("page", at, binding.SV_ST_BAD_PAGE) for at in (0, 94, 187)]  # the first, a middle and the last part
    cases += [("parent", at, binding.SV_ST_BAD_TOKEN) for at in (0, N - 1)]
    cases += [("length", n, binding.SV_ST_BAD_LENGTH) for n in (-1, 1 << 30)]
    for what, at, bit in cases:
        c = dict(good, lens=list(lens), table=good["table"].copy(), parent=good["parent"].copy())
        if what == "page":
            c["table"][1, at] = c["kp"].shape[0] if at else -1
        elif what == "parent":
            c["parent"][1, at] = at
        else:
            c["lens"][1] = at
        out, st = ta.tree_call(c)
        assert int(st.item()) == bit, (what, at)
        assert torch.count_nonzero(out[1]) == 0, (what, at)
        for b in (0, 2):
            if what == "length":  # (the others' items are cut elsewhere)
                ta.au.check(out[b], *ta.tree_reference(good, b), f"{what} {at}, request {b}")
            else:
                assert torch.equal(out[b], want[b]), (what, at, b)


@pytest.mark.parametrize("N,G,D", [(3, 4, 64), (5, 5, 128), (22, 4, 128), (61, 4, 64)])
def test_cut_invalid_positions(N, G, D):
    good = ta.ring_inputs(22, 3, N, 2 * G, 2, D, 4, 5000, [9000, 4321, 5004], BF)
    for p in (-1, 2147483647, 2147483647 - N + 1):
        c = dict(good, pos=[9000, p, 5004])
        out, st = ta.ring_call(c)
        assert int(st.item()) == binding.SV_ST_BAD_LENGTH and torch.count_nonzero(out[1]) == 0, p
        for b in (0, 2):
            ta.au.check(out[b], *ta.ring_reference(good, b), f"position {p}, request {b}")


@pytest.mark.parametrize("N,G,D", LAYOUTS)
def test_whole_invalid_trees(N, G, D):
    """The same with items left whole (short tables)."""
    good = ta.tree_inputs(23, 3, N, 2 * G, 2, D, 16, [100, 60, 120], BF)
    want, _ = ta.tree_call(good)
    for what, bit in (("page", binding.SV_ST_BAD_PAGE), ("parent", binding.SV_ST_BAD_TOKEN)):
        c = dict(good, table=good["table"].copy(), parent=good["parent"].copy())
        c["table" if what == "page" else "parent"][1, 1] = 1 << 20
        out, st = ta.tree_call(c)
        assert int(st.item()) == bit and torch.count_nonzero(out[1]) == 0, what
        assert torch.equal(out[[0, 2]], want[[0, 2]]), what


# ------------------------------------------------------------------ wide tables

@pytest.mark.parametrize("B,N,G,D,n", [(160, 1, 4, 64, 500), (90, 20, 2, 64, 1300), (80, 50, 4, 64, 900), (5, 6, 4, 64, 330)])
def test_a_tables_width_changes_nothing(B, N, G, D, n):
    """Whether items are cut goes by the requests' lengths: the columns that no length reaches change no bit."""
    lens = [n - 7 * (b % 11) for b in range(B)]
    c = ta.tree_inputs(31, B, N, 2 * G, 2, D, 16, lens, BF)
    out, st = ta.tree_call(c)
    wide = dict(c, table=np.concatenate([c["table"], np.full((B, 2000), -1, np.int32)], 1))
    again, st2 = ta.tree_call(wide)
    assert int(st.item()) == 0 and int(st2.item()) == 0
    assert torch.equal(out, again)
    for b in (0, 7 % B, B - 1):
        ta.au.check(out[b], *ta.tree_reference(c, b), f"request {b}")
