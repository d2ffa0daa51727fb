"""Attention over 8-bit pages whose value blocks differ in size, and staged entries that do: against 64-bit attention
with the elementwise bound of attn_util.

The size of a value that a row gives no weight must not reach the row's output.  So the large blocks' keys are made such
that their weights are below 2^-149 of the largest, and the definition leaves them out: their values are below 2^120, so
what they add is below 2^-29, and the bound allows 2^-9 (bf16) of outputs of about 2^-3; in fp16 they are below 2^16,
which adds less than 2^-133.  Then neither the definition's sums nor the bound, which counts the sizes of what it sees,
knows of them.
"""
import numpy as np
import pytest
import torch

import attn_util as au
import kv8_util as ku
from speculative_decoding_verification_09_gb300 import binding
from test_gpu_kv8 import BF, DEV, HF, entries, tree_call, tree_check, tree_inputs, tree_reference, u8

pytestmark = pytest.mark.gpu

# nodes and query heads (of two KV heads): 1 and 27 rows of a KV head, 64, 180
LAYOUTS = [(1, 2), (9, 6), (64, 2), (90, 4)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.lib()


def place(c, b, t):
    """(page, block of the page) of request b's position t."""
    return int(c["table"][b, t // c["page"]]), t % c["page"] // c["block"]


def hide(c, b, t):
    """Keys of the block that holds position t at which every score is below the others by 150 and more (base 2)."""
    pg, blk = place(c, b, t)
    rows = slice(blk * c["block"], (blk + 1) * c["block"])
    u8(c["kp"])[pg, :, rows] = 0
    u8(c["kp"])[pg, :, rows, 0] = 0xfe  # -448
    u8(c["ks"])[pg, :, blk] = 127 + 2
    c["q"][b, :, :, 0] = 2.0
    n = t // c["block"] * c["block"]
    return range(n, min(n + c["block"], c["lens"][b]))


def check_without(c, hidden):
    out, st = tree_call(c)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for b in range(c["B"]):
        k, v = entries(c, b)
        h = slice(c["head0"], c["head0"] + c["Hkv"])
        k, v = (torch.cat([x, c[y][b, h].transpose(0, 1).double()]) for x, y in ((k, "kn"), (v, "vn")))
        seen = au.tree_visible(c["lens"][b], c["parent"][b]).to(DEV)
        for t in hidden[b]:
            seen[:, t] = False
        want, tol = au.attend(c["q"][b], k, v, seen, c["D"] ** -0.5, c["dtype"])
        au.check(out[b], want, tol, f"request {b}")


@pytest.mark.parametrize("N,Hq", LAYOUTS)
@pytest.mark.parametrize("dtype,by", [(BF, 12), (BF, 22), (BF, 26), (BF, 40), (BF, 110), (HF, 12), (HF, 20), (HF, 22)])
def test_values_without_weight_leave_the_others_alone(dtype, by, N, Hq):
    """One block's values 2^by times the others', its keys such that no row gives it weight."""
    for D, lens in ((64, [300, 45, 17]), (128, [130, 700, 2])):
        c = tree_inputs(700 + by, 3, N, Hq, 2, D, 32, 16, lens, dtype, spread=0)
        hidden = []
        if dtype == HF:  # (all of the type's exponents: from -15 to 7)
            u8(c["vs"])[:] = 127 - 15
        for b, t in ((0, 50), (1, 0), (2, 16)):
            if t >= lens[b]:
                hidden.append(())
                continue
            hidden.append(hide(c, b, t))
            pg, blk = place(c, b, t)
            u8(c["vs"])[pg, :, blk] += by
        check_without(c, hidden)


@pytest.mark.parametrize("N,Hq", LAYOUTS)
@pytest.mark.parametrize("dtype,by", [(BF, 26), (BF, 100), (HF, 22)])
def test_large_values_far_from_the_others(dtype, by, N, Hq):
    """The same in long contexts, whose tiles several CTAs share: large blocks at the start, in the middle, at the end."""
    lens = [9000]
    c = tree_inputs(720 + by, 1, N, Hq, 2, 64, 64, 32, lens, dtype, spread=0)
    if dtype == HF:
        u8(c["vs"])[:] = 127 - 15
    hidden = []
    for t in (0, 3000, 4500, 8999):
        hidden += hide(c, 0, t)
        pg, blk = place(c, 0, t)
        u8(c["vs"])[pg, :, blk] += by
    check_without(c, [hidden])


@pytest.mark.parametrize("N,Hq", LAYOUTS)
@pytest.mark.parametrize("dtype,spread", [(BF, 40), (BF, 100), (HF, 11)])
def test_values_of_all_sizes(dtype, spread, N, Hq):
    """Values' blocks anywhere in the type's range, keys of one size: every row weighs them all."""
    c = tree_inputs(740, 2, N, Hq, 2, 64, 32, 16, [300, 45], dtype, spread=0)
    rng = np.random.default_rng(741)
    c["vp"], c["vs"] = ku.used_cache(rng, c["vp"].shape[0], c["vp"].shape[1], 32, 64, 16, dtype, DEV, spread)
    tree_check(c)


@pytest.mark.parametrize("N,Hq", [(5, 2), (9, 6), (64, 2), (90, 4)])
@pytest.mark.parametrize("dtype,by", [(BF, 12), (BF, 20), (BF, 26), (BF, 60), (HF, 12), (HF, 21)])
def test_staged_values_of_another_branch(dtype, by, N, Hq):
    """Two branches whose nodes alternate, one with values 2^by times the other's: neighbours, and of the cache."""
    for lens in ([0], [100]):
        c = tree_inputs(760 + by, 1, N, Hq, 2, 64, 32, 16, lens, dtype, spread=0)
        c["parent"] = np.array([[-1, 0, 0] + list(range(1, N - 2))], np.int32)
        if dtype == HF:
            c["vn"] *= 2.0 ** -8
            u8(c["vs"])[:] -= 8
        c["vn"][:, :, 2::2] *= 2.0 ** by
        tree_check(c)


@pytest.mark.parametrize("N,Hq", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_the_largest_and_the_smallest_values(dtype, N, Hq):
    """All blocks at the largest exponent (sums of weights times values stay finite), and at one whose values are
    the smallest that the bound can tell from nothing."""
    lo, hi = ku.LIMITS[dtype]
    for e in (hi, max(lo, -90)):
        c = tree_inputs(780, 2, N, Hq, 2, 64, 32, 16, [300, 2000], dtype, spread=0)
        u8(c["vs"])[:] = 127 + e
        c["vn"].zero_()
        # (up to 12 binades between the first entries' weights and the later ones')
        c["q"] *= 2.0
        tree_check(c)


def test_blocks_of_zeros_beside_others():
    """A block without a value has the least exponent; the others' weights do not depend on it."""
    for N, Hq in LAYOUTS:
        c = tree_inputs(790, 1, N, Hq, 2, 64, 32, 16, [200], BF, spread=0)
        for t in (0, 64, 199):
            pg, blk = place(c, 0, t)
            u8(c["vp"])[pg, :, blk * 16:(blk + 1) * 16] = 0
            u8(c["vs"])[pg, :, blk] = 127 - 117
        tree_check(c)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("N,Hq", [(5, 2), (9, 6), (64, 2), (90, 4)])
def test_staged_entries_that_are_not_finite(dtype, N, Hq):
    """They show in the rows that see them, and in their own request only."""
    for what in ("kn", "vn", "q"):
        for bad in (float("nan"), float("inf"), -float("inf")):
            c = tree_inputs(800, 3, N, Hq, 2, 64, 32, 16, [50, 200, 31], dtype, kind="chain")
            at = 3
            if what == "q":
                c["q"][1, at, 0, 5] = bad
            else:
                c[what][1, 0, at, 5] = bad
            out, st = tree_call(c)
            assert int(st.item()) == 0
            for b in (0, 2):
                want, tol = tree_reference(c, b)
                au.check(out[b], want, tol, what)
            G = Hq // 2
            assert bool((~out[1][at:, :G].isfinite()).any(-1).all()) if what != "q" else not bool(out[1][at, 0].isfinite().any())
            assert bool(out[1][:, G:].isfinite().all())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_batches_beyond_the_workspace(dtype):
    """A batch that is taken in parts: requests around their borders and elsewhere, with a parent array and without; a
    bad page in one part is reported and its request alone gets zeros."""
    N, Hq, Hkv, D, B = 256, 32, 8, 128, 150
    one = 3 * N * (Hq + Hkv) * D + 4 * N * Hq + Hkv * 2 * 64
    parts = -(-B // (2 ** 28 // one))
    assert parts == 3 and binding.sv_attn8_workspace_bytes(B, N, Hq, Hkv, D) < B * one
    c = tree_inputs(820, B, N, Hq, Hkv, D, 32, 16, [(37 * i) % 90 + 20 for i in range(B)], dtype, LH=Hkv + 1)
    ws = binding.make_attn_workspace(B, N, Hq, Hkv, D, DEV, 8)
    for parent in (True, False):
        out, st = tree_call(c, parent=parent, ws=ws)
        assert int(st.item()) == 0
        for b in (0, 1, 48, 49, 50, 51, 77, 98, 99, 100, 101, 148, 149):
            want, tol = tree_reference(c, b, parent=parent)
            au.check(out[b], want, tol, f"request {b}")
    again, _ = tree_call(c, parent=False, ws=ws)
    assert torch.equal(out, again)
    c["table"][70, 0] = -1
    out, st = tree_call(c, parent=False, ws=ws)
    assert int(st.item()) == binding.SV_ST_BAD_PAGE and bool((out[70] == 0).all())
    rest = torch.arange(B, device=DEV) != 70
    assert torch.equal(out[rest], again[rest])
