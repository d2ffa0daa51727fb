"""The attention and cache calls at the limits that their headers state, and with arguments that the other tests leave at
their defaults."""
import numpy as np
import pytest
import torch

import test_gpu_attn as ta
from attn_util import attend, check, slot, tensor, window_visible
from speculative_decoding_verification_09_gb300 import binding

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.lib()


def some(B):
    return [0, 1, 31, 32, 33, 383, 384, 12345, 40000, B - 2, B - 1]


def test_largest_batches():
    """65535 requests: trees, rings, prompts, a fill and a commit in place."""
    rng = np.random.default_rng(1)
    B = 65535
    lens = [int(x) for x in rng.choice([0, 1, 5, 40], B)]
    lens[12345], lens[B - 1] = 300, 77
    c = ta.tree_inputs(2, B, 1, 1, 1, 8, 8, lens, BF)
    out, st = ta.tree_call(c)
    r = ta.ring_inputs(3, B, 2, 1, 1, 8, 1, 6, lens, HF)
    rout, rst = ta.ring_call(r)
    p = ta.prompt_inputs(4, lens, 2, 1, 8, 1, 6, HF, tail=3)
    pout, pst = ta.prompt_call(p)
    kp, vp = (torch.zeros(B, 1, 7, 8, dtype=HF, device=ta.DEV) for _ in "kv")
    pos, fst = ta.i32([-1] * B), ta.status()
    binding.sv_kv_fill(p["k"], p["v"], ta.i32(p["cu"]), kp, vp, pos, 1, 6, dev_status=fst)
    assert int(st.item()) == int(rst.item()) == int(pst.item()) == int(fst.item()) == 0
    assert pos.tolist() == lens and (pout[p["cu"][-1]:] == 7.0).all()
    for b in some(B):
        check(out[b], *ta.tree_reference(c, b), f"tree {b}")
        check(rout[b], *ta.ring_reference(r, b), f"ring {b}")
        a, e = int(p["cu"][b]), int(p["cu"][b + 1])
        at = range(e - a)
        if e > a:
            check(pout[a:e], *attend(p["q"][a:e], p["k"][a:e], p["v"][a:e], window_visible(at, at, 1, 6).to(ta.DEV),
                                     8 ** -0.5, HF), f"prompt {b}")
        for t in set(range(min(1, e - a))) | set(range(max(0, e - a - 6), e - a)):
            assert torch.equal(kp[b, 0, slot(t, 1, 6)], p["k"][a + t, 0])
    table = torch.arange(B, dtype=torch.int32, device=ta.DEV)[:, None].contiguous()
    pages = [torch.zeros(B, 1, 4, 8, dtype=BF, device=ta.DEV) for _ in "kv"]
    new = [tensor(rng, (B, 1, 2, 8), BF) for _ in "kv"]
    seq, cst = ta.i32([1] * B), ta.status()
    binding.sv_page_commit(*pages, *new, table, seq, None, ta.i32([1] * B), seq, dev_status=cst)
    assert int(cst.item()) == 0 and (seq == 3).all()
    assert all(torch.equal(x[:, :, 1:3], y) and not x[:, :, 3].any() for x, y in zip(pages, new))


@pytest.mark.parametrize("N,Hq,D,lens", [(256, 128, 128, [300]), (256, 128, 8, [0, 129]), (129, 65, 64, [130, 5])])
def test_most_rows_of_a_head(N, Hq, D, lens):
    """Up to 256 nodes of up to 128 query heads on one KV head."""
    ta.tree_check(ta.tree_inputs(5, len(lens), N, Hq, 1, D, 16, lens, BF))


def test_heads_in_the_middle_of_a_pool():
    """One layer's heads with others before and behind them, which hold anything; default scale, no status."""
    c = ta.tree_inputs(6, 2, 5, 8, 2, 64, 16, [200, 33], HF, LH=7)  # heads 5 and 6
    want, _ = ta.tree_call(c)
    moved = {x: c[x].clone().fill_(float("nan")) for x in ("kp", "vp", "kn", "vn")}
    for x in moved:
        moved[x][:, 2:4] = c[x][:, 5:7]
    out = torch.empty_like(want)
    ws = binding.make_attn_workspace(2, 5, 8, 2, 64, ta.DEV)
    binding.sv_tree_attn(c["q"], moved["kp"], moved["vp"], ta.i32(c["table"]), ta.i32(c["lens"]), moved["kn"], moved["vn"],
                         ta.i32(c["parent"]), out, ws, head0=2, kv_heads=2)
    assert torch.equal(out, want)
    r = ta.ring_inputs(7, 3, 4, 8, 2, 64, 4, 90, [20, 94, 400], BF, LH=5)  # heads 3 and 4
    want, _ = ta.ring_call(r)
    moved = {x: r[x].clone().fill_(float("nan")) for x in ("kp", "vp", "kn", "vn")}
    for x in moved:
        moved[x][:, 1:3] = r[x][:, 3:5]
    out = torch.empty_like(want)
    binding.sv_ring_attn(r["q"], moved["kp"], moved["vp"], ta.i32(r["pos"]), moved["kn"], moved["vn"], 4, 90, out, ws,
                         head0=1, kv_heads=2)
    assert torch.equal(out, want)


def test_rows_before_the_first_sequence():
    """Bounds that begin behind the first rows: those, too, are left as they were and hold anything."""
    c = ta.prompt_inputs(8, [130, 40], 8, 2, 128, 4, 50, BF, tail=2)
    want, _ = ta.prompt_call(c)
    lead = {x: torch.cat([torch.full_like(c[x][:37], float("nan")), c[x]]) for x in ("q", "k", "v")}
    out, st = ta.prompt_call(dict(c, **lead, cu=c["cu"] + 37))
    assert int(st.item()) == 0 and torch.equal(out[37:], want) and (out[:37] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_windows_and_sinks_past_the_prompt(dtype):
    """Sinks and windows up to the largest int: plain causal attention."""
    c = ta.prompt_inputs(9, [700, 3], 4, 2, 64, 0, 1 << 30, dtype)
    want, _ = ta.prompt_call(c)
    for S, W in ((2147483647, 1), (2147483647, 2147483647), (0, 2147483647), (700, 5)):
        out, st = ta.prompt_call(dict(c, S=S, W=W))
        assert int(st.item()) == 0
        for a, e in ((0, 700), (700, 703)):
            at = range(e - a)
            check(out[a:e], *attend(c["q"][a:e], c["k"][a:e], c["v"][a:e],
                                    torch.ones(e - a, e - a, dtype=torch.bool).tril().to(ta.DEV), 64 ** -0.5, dtype),
                  f"sinks {S}, window {W}")
    assert torch.equal(want, ta.prompt_call(c)[0])


def test_long_fp16_rings_and_prompts():
    """More keys than 2^14, where fp16 weights get a lift."""
    r = ta.ring_inputs(10, 2, 3, 4, 2, 64, 4, 70000, [200000, 50001], HF)
    ta.ring_check(r)
    c = ta.prompt_inputs(11, [20000], 1, 1, 64, 3, 40000, HF)
    out, st = ta.prompt_call(c)
    assert int(st.item()) == 0
    at = [*range(0, 300), *range(19700, 20000)]
    check(out[at], *attend(c["q"][at], c["k"], c["v"], window_visible(at, range(20000), 3, 40000).to(ta.DEV),
                           64 ** -0.5, HF))
