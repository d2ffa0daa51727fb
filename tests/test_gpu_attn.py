"""Attention over the caches (sv_tree_attn, sv_ring_attn, sv_prompt_attn) and the cache steps beside it (sv_kv_fill,
sv_page_commit) on the GPU against plain implementations: 64-bit attention with the elementwise bound of attn_util, and
bit-exact copies."""
import os

import numpy as np
import pytest
import torch

import attn_util as au
import oracle
from speculative_decoding_verification_09_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.lib()


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ trees over pages

def tree_inputs(seed, B, N, Hq, Hkv, D, page, lens, dtype, kind="random", LH=None, qs=2.0, dead=None):
    """`dead` fills what no request may use: rows past a length, unused pages, other layers' heads."""
    rng = np.random.default_rng(seed)
    LH = LH or Hkv
    head0 = LH - Hkv
    need = [-(-n // page) for n in lens]
    cols, P = max(1, max(need)) + 1, sum(need) + 2
    order = rng.permutation(P)
    table = np.zeros((B, cols), np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        table[b, need[b]:] = rng.choice([-1, 0, P + 5])  # past the length: never looked at
        at += need[b]
    kp, vp = (au.tensor(rng, (P, LH, page, D), dtype) for _ in "kv")
    kn, vn = (au.tensor(rng, (B, LH, N, D), dtype) for _ in "kv")
    if dead is not None:
        used = torch.zeros(P, page, dtype=torch.bool)
        for b in range(B):
            for t in range(lens[b]):
                used[table[b, t // page], t % page] = True
        for x in (kp, vp):
            x.permute(0, 2, 1, 3)[~used.to(DEV)] = dead
            x[:, :head0] = dead
        for x in (kn, vn):
            x[:, :head0] = dead
    q = au.tensor(rng, (B, N, Hq, D), dtype, qs)
    parent = np.array([au.random_parents(N, rng, kind) for _ in range(B)], np.int32)
    return dict(q=q, kp=kp, vp=vp, kn=kn, vn=vn, table=table, lens=lens, parent=parent, page=page,
                head0=head0, Hkv=Hkv, N=N, B=B, Hq=Hq, D=D, dtype=dtype)


def tree_call(c, parent=True, ws=None, out=None, **kw):
    out = torch.full_like(c["q"], 7.0) if out is None else out
    ws = binding.make_attn_workspace(c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], DEV) if ws is None else ws
    st = status()
    binding.sv_tree_attn(c["q"], c["kp"], c["vp"], i32(c["table"]), i32(c["lens"]), c["kn"], c["vn"],
                         i32(c["parent"]) if parent else None, out, ws, head0=c["head0"], kv_heads=c["Hkv"],
                         dev_status=st, **kw)
    return out, st


def tree_reference(c, b, scale=None):
    n, page, h0, H = c["lens"][b], c["page"], c["head0"], c["Hkv"]
    ids = torch.as_tensor(c["table"][b, :-(-n // page)].astype(np.int64)).to(DEV)
    k, v = (x[ids][:, h0:h0 + H].transpose(1, 2).reshape(-1, H, c["D"])[:n] for x in (c["kp"], c["vp"]))
    k = torch.cat([k, c["kn"][b, h0:h0 + H].transpose(0, 1)])
    v = torch.cat([v, c["vn"][b, h0:h0 + H].transpose(0, 1)])
    return au.attend(c["q"][b], k, v, au.tree_visible(n, c["parent"][b]).to(DEV),
                     scale or c["D"] ** -0.5, c["dtype"])


def tree_check(c, **kw):
    out, st = tree_call(c, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for b in range(c["B"]):
        want, tol = tree_reference(c, b, kw.get("scale"))
        au.check(out[b], want, tol, f"request {b}, length {c['lens'][b]}")
    return out


TREES = [
    # B, N, Hq, Hkv, D, page, lens, dtype, kind
    (1, 1, 1, 1, 8, 8, [0], BF, "chain"),
    (1, 1, 4, 4, 128, 16, [1], BF, "chain"),
    (1, 1, 16, 16, 128, 16, [500], BF, "chain"),
    (3, 5, 8, 2, 64, 16, [0, 127, 128], HF, "chain"),
    (4, 22, 32, 8, 128, 128, [129, 1000, 0, 4097], BF, "random"),
    (2, 61, 28, 4, 64, 16, [2000, 777], HF, "random"),
    (2, 256, 2, 1, 128, 64, [300, 1], BF, "random"),
    (1, 256, 8, 1, 40, 24, [511], HF, "star"),
    (2, 128, 3, 3, 80, 24, [640, 383], BF, "random"),
    (2, 129, 5, 1, 96, 8, [255, 256], HF, "chain"),
    (1, 3, 128, 1, 72, 256, [3000], BF, "random"),
    (2, 7, 100, 1, 16, 72, [300, 71], HF, "random"),
    (70, 4, 4, 2, 64, 32, [(37 * i) % 300 for i in range(70)], BF, "random"),
    (1, 22, 32, 1, 128, 128, [20000], BF, "random"),
]


@pytest.mark.parametrize("i", range(len(TREES)))
def test_tree(i):
    tree_check(tree_inputs(50 + i, *TREES[i]))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dead", [float("nan"), float("inf"), float("-inf"), "lowest"])
def test_tree_dead_places(dead, dtype):
    """Rows past a length, unused pages and other layers' heads hold anything."""
    dead = torch.finfo(dtype).min if dead == "lowest" else dead
    tree_check(tree_inputs(5, 4, 9, 8, 2, 64, 16, [0, 5, 130, 1021], dtype, dead=dead, LH=5))
    tree_check(tree_inputs(6, 2, 40, 8, 1, 128, 128, [100, 700], dtype, dead=dead, LH=2))


@pytest.mark.parametrize("N,D", [(6, 128), (30, 64), (50, 128), (140, 64), (256, 128)])
def test_tree_chain_without_parent(N, D):
    c = tree_inputs(8, 3, N, 8, 4, D, 16, [100, 0, 513], BF, "chain")
    a = tree_check(c)
    b, _ = tree_call(c, parent=False)
    assert torch.equal(a, b)


@pytest.mark.parametrize("page", [8, 40, 192, 1024, 65536])
def test_tree_page_sizes(page):
    tree_check(tree_inputs(17, 2, 4, 4, 2, 64, page, [1500, 77], BF))


def test_tree_scales():
    c = tree_inputs(9, 2, 6, 8, 4, 128, 16, [300, 65], BF)
    for scale in (1e-4, 0.5, 3.0):
        tree_check(c, scale=scale)


def test_tree_rising_scores():
    """Scores that grow along the cache: the running maximum rises with every tile, by far more than a rounding."""
    c = tree_inputs(10, 1, 4, 4, 2, 64, 16, [2000], HF)
    P, LH, page, D = c["kp"].shape
    for t in range(2000):
        c["kp"][c["table"][0, t // page], :, t % page] = 0
        c["kp"][c["table"][0, t // page], :, t % page, 0] = t / 8.0
    c["q"][:] = 0
    c["q"][..., 0] = torch.tensor([1.0, -1.0, 0.25, 0.0], dtype=HF, device=DEV)[None, :, None]
    tree_check(c, scale=1.0)


def test_tree_far_scores():
    """One key far above all others, and rows far below their own maximum."""
    c = tree_inputs(11, 2, 5, 4, 2, 128, 16, [900, 130], BF, qs=40.0)
    tree_check(c)


def test_tree_invalid_requests():
    """Bad lengths, pages and parents give zeros and a status bit; the others are untouched by them."""
    good = tree_inputs(12, 6, 5, 8, 2, 64, 16, [100, 90, 80, 70, 60, 50], BF)
    want, _ = tree_call(good)
    for what, bit in (("len", binding.SV_ST_BAD_LENGTH), ("low", binding.SV_ST_BAD_LENGTH),
                      ("page", binding.SV_ST_BAD_PAGE), ("negative page", binding.SV_ST_BAD_PAGE),
                      ("parent", binding.SV_ST_BAD_TOKEN), ("root", binding.SV_ST_BAD_TOKEN)):
        c = dict(good, lens=list(good["lens"]), table=good["table"].copy(), parent=good["parent"].copy())
        if what == "len":
            c["lens"][2] = c["table"].shape[1] * 16 + 1
        if what == "low":
            c["lens"][2] = -1
        if what == "page":
            c["table"][2, 3] = c["kp"].shape[0]
        if what == "negative page":
            c["table"][2, 0] = -1
        if what == "parent":
            c["parent"][2, 3] = 3
        if what == "root":
            c["parent"][2, 0] = 0
        out, st = tree_call(c)
        assert int(st.item()) == bit, what
        assert torch.count_nonzero(out[2]) == 0, what
        assert torch.equal(out[[0, 1, 3, 4, 5]], want[[0, 1, 3, 4, 5]]), what


def test_tree_non_finite_stays_in_its_request():
    c = tree_inputs(13, 3, 5, 8, 2, 64, 16, [300, 290, 280], BF)
    want, _ = tree_call(c)
    c["vp"][c["table"][1, 3], 0, 2, 5] = float("inf")
    c["kn"][1, 1, 2, 7] = float("nan")
    out, _ = tree_call(c)
    assert torch.equal(out[[0, 2]], want[[0, 2]])
    assert not torch.isfinite(out[1].float()).all()


def test_tree_same_page_twice():
    """Requests that share pages, and one page at two places of a table."""
    c = tree_inputs(14, 3, 4, 4, 2, 64, 16, [64, 64, 64], BF)
    c["table"][1] = c["table"][0]
    c["table"][2, 1] = c["table"][2, 0]
    tree_check(c)


def test_tree_over_a_windowed_table():
    """The draft model's window: sv_window_block_table's outputs are the table and lengths."""
    c = tree_inputs(15, 3, 4, 4, 2, 64, 16, [40, 400, 1000], BF)
    W, page, K = 128, 16, 3
    cols = binding.sv_window_cols(W, page)
    seq, table = i32([0] * 3), torch.empty(3, cols, dtype=torch.int32, device=DEV)
    full = i32(np.maximum(c["table"], 0))
    binding.sv_window_block_table(i32(c["lens"]), full, W, page, K, seq, table)
    c.update(table=table.cpu().numpy(), lens=[int(x) for x in seq.cpu()])
    assert max(c["lens"]) < 1000
    tree_check(c)


def test_tree_far_pages():
    """A pool of more than 2^31 elements: pages far behind it."""
    P, H, page, D = 9000, 16, 128, 128
    kp, vp = (torch.zeros(P, H, page, D, dtype=BF, device=DEV) for _ in "kv")
    assert kp.numel() > 1 << 31
    c = tree_inputs(16, 2, 3, 16, 16, 128, 128, [400, 250], BF)
    far = {int(p): P - 1 - i for i, p in enumerate(np.unique(c["table"][c["table"] >= 0])) if p < c["kp"].shape[0]}
    for old, new in far.items():
        kp[new], vp[new] = c["kp"][old], c["vp"][old]
    c.update(kp=kp, vp=vp, table=np.vectorize(lambda p: far.get(int(p), 0))(c["table"]).astype(np.int32))
    tree_check(c)


# ------------------------------------------------------------------ the ring

def ring_inputs(seed, B, R, Hq, Hkv, D, S, W, pos, dtype, LH=None, dead=None):
    rng = np.random.default_rng(seed)
    LH = LH or Hkv
    head0 = LH - Hkv
    kp, vp = (au.tensor(rng, (B, LH, S + W, D), dtype) for _ in "kv")
    kn, vn = (au.tensor(rng, (B, LH, R, D), dtype) for _ in "kv")
    if dead is not None:
        for b in range(B):
            live = torch.zeros(S + W, dtype=torch.bool)
            # token 0 sees positions above pos - W: the slot that holds pos - W is seen by none
            for t in au.ring_positions(pos[b], S, W):
                if t < S or t > pos[b] - W:
                    live[au.slot(t, S, W)] = True
            for x in (kp, vp):
                x[b, :, ~live] = dead
                x[b, :head0] = dead
    return dict(q=au.tensor(rng, (B, R, Hq, D), dtype, 2.0), kp=kp, vp=vp, kn=kn, vn=vn, pos=list(pos), S=S, W=W,
                head0=head0, Hkv=Hkv, N=R, B=B, Hq=Hq, D=D, dtype=dtype)


def ring_call(c, ws=None, out=None, **kw):
    out = torch.full_like(c["q"], 7.0) if out is None else out
    ws = binding.make_attn_workspace(c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], DEV) if ws is None else ws
    st = status()
    binding.sv_ring_attn(c["q"], c["kp"], c["vp"], i32(c["pos"]), c["kn"], c["vn"], c["S"], c["W"], out, ws,
                         head0=c["head0"], kv_heads=c["Hkv"], dev_status=st, **kw)
    return out, st


def ring_reference(c, b):
    p, S, W, h0, H = c["pos"][b], c["S"], c["W"], c["head0"], c["Hkv"]
    held = au.ring_positions(p, S, W)
    slots = torch.tensor([au.slot(t, S, W) for t in held], dtype=torch.long, device=DEV)
    k, v = (torch.cat([x[b, h0:h0 + H][:, slots].transpose(0, 1), y[b, h0:h0 + H].transpose(0, 1)])
            for x, y in ((c["kp"], c["kn"]), (c["vp"], c["vn"])))
    at = [p + j for j in range(c["N"])]
    return au.attend(c["q"][b], k, v, au.window_visible(at, held + at, S, W).to(DEV), c["D"] ** -0.5, c["dtype"])


def ring_check(c):
    out, st = ring_call(c)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for b in range(c["B"]):
        want, tol = ring_reference(c, b)
        au.check(out[b], want, tol, f"request {b}, position {c['pos'][b]}")
    return out


RINGS = [
    # B, R, Hq, Hkv, D, S, W, pos, dtype
    (1, 1, 1, 1, 8, 0, 1, [0], BF),
    (6, 1, 4, 4, 128, 0, 1, [0, 1, 2, 3, 100, 101], BF),
    (8, 1, 16, 16, 128, 4, 64, [0, 1, 3, 4, 67, 68, 69, 300], BF),
    (9, 5, 8, 2, 64, 4, 6, [0, 2, 4, 5, 9, 10, 11, 33, 1000], HF),
    (6, 8, 32, 8, 128, 4, 2048, [100, 2052, 2053, 2051, 9000, 0], BF),
    (5, 4, 12, 4, 80, 3, 509, [509, 512, 513, 1021, 77], HF),
    (4, 64, 6, 1, 128, 7, 64, [0, 30, 71, 500], BF),
    (4, 64, 20, 5, 96, 130, 250, [100, 130, 380, 4000], HF),
    (3, 33, 16, 2, 40, 0, 129, [128, 129, 555], BF),
    (3, 3, 128, 1, 128, 1, 1000, [5, 1001, 123456], BF),
    (2, 2, 3, 3, 24, 0, 300, [2147483000, 2147483640], HF),
    (120, 4, 4, 2, 64, 4, 130, [(7 * i) % 400 for i in range(120)], HF),
]


@pytest.mark.parametrize("i", range(len(RINGS)))
def test_ring(i):
    ring_check(ring_inputs(150 + i, *RINGS[i]))


@pytest.mark.parametrize("dead", [float("nan"), float("-inf"), "lowest"])
@pytest.mark.parametrize("S,W", [(0, 9), (4, 124), (3, 300)])
def test_ring_dead_places(dead, S, W):
    dead = torch.finfo(BF).min if dead == "lowest" else dead
    pos = [0, 1, S, S + 1, W, S + W - 1, S + W, S + W + 1, 5 * W + 3]
    ring_check(ring_inputs(7, len(pos), 5, 8, 2, 64, S, W, pos, BF, dead=dead, LH=3))


def test_ring_invalid_positions():
    good = ring_inputs(3, 4, 3, 4, 2, 64, 4, 60, [10, 20, 100, 300], BF)
    want, _ = ring_call(good)
    for p in (-1, 2147483647, 2147483645):
        out, st = ring_call(dict(good, pos=[10, p, 100, 300]))
        assert int(st.item()) == binding.SV_ST_BAD_LENGTH
        assert torch.count_nonzero(out[1]) == 0 and torch.equal(out[[0, 2, 3]], want[[0, 2, 3]])


def test_ring_steps():
    """A prompt and then twelve steps as they are used: prompt attention, the ring filled, then attention of the
    staged tokens and a commit of some of them; every step against attention over the whole history."""
    rng = np.random.default_rng(21)
    B, R, Hq, Hkv, D, S, W, LH = 3, 4, 8, 2, 64, 4, 40, 4
    head0 = 2
    lens = [3, 0, 97]
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    q, k, v = au.tensor(rng, (T, Hq, D), BF, 2.0), au.tensor(rng, (T, Hkv, D), BF), au.tensor(rng, (T, Hkv, D), BF)
    out = torch.empty_like(q)
    binding.sv_prompt_attn(q, k, v, i32(cu), S, W, out)
    kp, vp = (torch.full((B, LH, S + W, D), float("nan"), dtype=BF, device=DEV) for _ in "kv")
    pos = i32([-9] * B)
    binding.sv_kv_fill(k, v, i32(cu), kp, vp, pos, S, W, head0=head0)
    assert pos.tolist() == lens
    hist = [(k[a:e], v[a:e]) for a, e in zip(cu[:-1], cu[1:])]
    for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        if e > a:
            at = range(e - a)
            want, tol = au.attend(q[a:e], *hist[b], au.window_visible(at, at, S, W).to(DEV), D ** -0.5, BF)
            au.check(out[a:e], want, tol, f"prompt {b}")
    ws = binding.make_attn_workspace(B, R, Hq, Hkv, D, DEV)
    for step in range(12):
        qs = au.tensor(rng, (B, R, Hq, D), BF, 2.0)
        kn, vn = (au.tensor(rng, (B, LH, R, D), BF) for _ in "kv")
        got = torch.empty_like(qs)
        binding.sv_ring_attn(qs, kp, vp, pos, kn, vn, S, W, got, ws, head0=head0, kv_heads=Hkv)
        acc = rng.integers(-1, R, B)
        for b in range(B):
            hk, hv = (torch.cat([h, x[b, head0:].transpose(0, 1)]) for h, x in zip(hist[b], (kn, vn)))
            n = hk.shape[0]
            want, tol = au.attend(qs[b], hk, hv, au.window_visible(range(n - R, n), range(n), S, W).to(DEV),
                                  D ** -0.5, BF)
            au.check(got[b], want, tol, f"step {step}, request {b}")
            hist[b] = tuple(h[:n - R + acc[b] + 1] for h in (hk, hv))
        binding.sv_kv_commit(kp, vp, kn, vn, i32(acc), pos, S, W)


# ------------------------------------------------------------------ prompts

def prompt_inputs(seed, lens, Hq, Hkv, D, S, W, dtype, tail=0):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1]) + tail
    return dict(q=au.tensor(rng, (T, Hq, D), dtype, 2.0), k=au.tensor(rng, (T, Hkv, D), dtype),
                v=au.tensor(rng, (T, Hkv, D), dtype), cu=cu, S=S, W=W, D=D, dtype=dtype)


def prompt_call(c, out=None, **kw):
    out = torch.full_like(c["q"], 7.0) if out is None else out
    st = status()
    binding.sv_prompt_attn(c["q"], c["k"], c["v"], i32(c["cu"]), c["S"], c["W"], out, dev_status=st, **kw)
    return out, st


def prompt_check(c):
    out, st = prompt_call(c)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for b, (a, e) in enumerate(zip(c["cu"][:-1], c["cu"][1:])):
        if e > a:
            at = range(e - a)
            want, tol = au.attend(c["q"][a:e], c["k"][a:e], c["v"][a:e],
                                  au.window_visible(at, at, c["S"], c["W"]).to(DEV), c["D"] ** -0.5, c["dtype"])
            au.check(out[a:e], want, tol, f"sequence {b} of {e - a}")
    assert (out[c["cu"][-1]:] == 7.0).all()  # rows behind the last sequence
    return out


PROMPTS = [
    # lens, Hq, Hkv, D, S, W, dtype
    ([1], 1, 1, 8, 0, 1, BF),
    ([5, 0, 1, 0, 0, 3], 4, 2, 64, 0, 2, HF),
    ([127, 128, 129], 4, 4, 128, 4, 64, BF),
    ([255, 256, 257, 64], 2, 1, 128, 0, 1 << 30, BF),
    ([1000], 8, 1, 64, 4, 128, HF),
    ([1500, 3, 700], 16, 4, 64, 4, 512, HF),
    ([900], 3, 3, 80, 130, 127, BF),
    ([800, 411], 5, 1, 96, 300, 129, HF),
    ([700], 7, 1, 40, 1, 1, BF),
    ([600], 128, 1, 128, 4, 100, BF),
    ([333, 100], 100, 2, 72, 0, 100, BF),
    ([2500], 4, 2, 128, 4, 1000, BF),
    ([1300], 2, 2, 128, 200, 600, HF),
    ([17] * 90, 4, 2, 64, 2, 9, BF),
    ([4100], 8, 8, 128, 0, 5000, BF),
]


@pytest.mark.parametrize("i", range(len(PROMPTS)))
def test_prompt(i):
    prompt_check(prompt_inputs(250 + i, *PROMPTS[i], tail=i % 4))


def test_prompt_many_small_and_one_long():
    prompt_check(prompt_inputs(4, [3] * 40 + [3001] + [50] * 20, 8, 2, 64, 4, 700, BF, tail=9))


def test_prompt_other_sequences_hold_anything():
    """A sequence of NaN between two others, and NaN in rows of no sequence."""
    c = prompt_inputs(6, [200, 77, 300], 8, 2, 128, 4, 100, BF, tail=60)
    want, _ = prompt_call(c)
    for x in ("q", "k", "v"):
        c[x][200:277] = float("nan")
        c[x][577:] = float("nan")
    out, _ = prompt_call(c)
    keep = [*range(200), *range(277, 577)]
    assert torch.equal(out[keep], want[keep])
    assert (out[577:] == 7.0).all()


def test_ring_and_prompt_scales():
    r, p = ring_inputs(18, 3, 5, 8, 2, 64, 4, 90, [20, 94, 400], BF), prompt_inputs(19, [150, 40], 8, 2, 64, 4, 90, BF)
    for scale in (1e-3, 0.7):
        out, _ = ring_call(r, scale=scale)
        for b in range(3):
            q = dict(r, q=r["q"])
            pp, S, W, H = q["pos"][b], 4, 90, 2
            held = au.ring_positions(pp, S, W)
            slots = torch.tensor([au.slot(t, S, W) for t in held], dtype=torch.long, device=DEV)
            k, v = (torch.cat([x[b][:, slots].transpose(0, 1), y[b].transpose(0, 1)])
                    for x, y in ((r["kp"], r["kn"]), (r["vp"], r["vn"])))
            at = [pp + j for j in range(5)]
            au.check(out[b], *au.attend(r["q"][b], k, v, au.window_visible(at, held + at, S, W).to(DEV), scale, BF))
        out, _ = prompt_call(p, scale=scale)
        for a, e in ((0, 150), (150, 190)):
            at = range(e - a)
            au.check(out[a:e], *au.attend(p["q"][a:e], p["k"][a:e], p["v"][a:e],
                                          au.window_visible(at, at, 4, 90).to(DEV), scale, BF))


def test_prompt_far_rows():
    """More than 2^31 query elements: the last tokens of a long prompt, and of the sequence before it."""
    T0, T, Hq, D, S, W = 500, 140000, 128, 128, 3, 40
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    q = torch.empty(T0 + T, Hq, D, dtype=BF, device=DEV).normal_(generator=gen)
    assert q.numel() > 1 << 31
    k, v = (torch.empty(T0 + T, 1, D, dtype=BF, device=DEV).normal_(generator=gen) for _ in "kv")
    out, st = torch.empty_like(q), status()
    binding.sv_prompt_attn(q, k, v, i32([0, T0, T0 + T]), S, W, out, dev_status=st)
    assert int(st.item()) == 0
    for a, e in ((0, T0), (T0, T0 + T)):
        n = e - a
        at = [n - 3, n - 2, n - 1]
        seen = sorted(set(range(S)) | set(range(n - 3 - W, n)))
        rows = torch.tensor(seen, device=DEV) + a
        au.check(out[e - 3:e], *au.attend(q[e - 3:e], k[rows], v[rows], au.window_visible(at, seen, S, W).to(DEV),
                                          D ** -0.5, BF))


def test_empty_batches_and_strides():
    c = tree_inputs(20, 2, 3, 4, 2, 64, 16, [40, 50], BF)
    e = dict(c, B=0, q=c["q"][:0], kn=c["kn"][:0], vn=c["vn"][:0], table=c["table"][:0], lens=[], parent=c["parent"][:0])
    assert tree_call(e)[0].numel() == 0
    p = prompt_inputs(21, [0], 4, 2, 64, 0, 8, BF)
    assert prompt_call(p)[0].numel() == 0 and prompt_call(dict(p, cu=np.zeros(1, np.int32)))[0].numel() == 0
    with pytest.raises(binding.SpecVerifyError):
        tree_call(dict(c, kp=c["kp"].transpose(1, 2).contiguous().transpose(1, 2)))
    with pytest.raises(binding.SpecVerifyError):
        tree_call(c, ws=torch.empty(64, dtype=torch.uint8, device=DEV))


def test_prompt_invalid_bounds():
    """A sequence whose bounds decrease or leave the rows is skipped, the others are not."""
    c = prompt_inputs(7, [50, 60, 70], 4, 2, 64, 4, 30, BF)
    want, _ = prompt_call(c)
    out, st = prompt_call(dict(c, cu=np.array([0, 50, 110, 181], np.int32)))
    assert int(st.item()) == binding.SV_ST_BAD_LENGTH
    assert torch.equal(out[:110], want[:110]) and (out[110:] == 7.0).all()
    out, st = prompt_call(dict(c, cu=np.array([-1, 50, 110, 180], np.int32)))
    assert int(st.item()) == binding.SV_ST_BAD_LENGTH
    assert torch.equal(out[50:], want[50:]) and (out[:50] == 7.0).all()
    out, st = prompt_call(dict(c, cu=np.array([0, 50, 40, 180], np.int32)))
    assert int(st.item()) == binding.SV_ST_BAD_LENGTH and torch.equal(out[:40], want[:40])


# ------------------------------------------------------------------ cache steps

@pytest.mark.parametrize("S,W,dtype,D,LH,head0", [(0, 5, np.int16, 8, 3, 0), (4, 6, np.int16, 64, 5, 2),
                                                  (3, 200, np.float32, 4, 3, 0), (7, 64, np.int16, 4096, 4, 1)])
def test_fill(S, W, dtype, D, LH, head0):
    """Pools, positions and untouched slots are those of the oracle's commits of one token after another."""
    rng = np.random.default_rng(S + W)
    Hkv = 3
    lens = [0, 1, S, S + 1, S + W - 1, S + W, S + W + 1, 3 * W + 2]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T, B = int(cu[-1]) + 3, len(lens)
    k, v = (rng.integers(0, 1 << 14, (T, Hkv, D)).astype(dtype) for _ in "kv")
    kp, vp = (rng.integers(0, 1 << 14, (B, LH, S + W, D)).astype(dtype) for _ in "kv")
    wk, wv = kp.copy(), vp.copy()
    for b in range(B):
        for t in range(lens[b]):
            wk[b, head0:head0 + Hkv, au.slot(t, S, W)] = k[cu[b] + t]
            wv[b, head0:head0 + Hkv, au.slot(t, S, W)] = v[cu[b] + t]
    d = [torch.from_numpy(x).to(DEV) for x in (k, v, kp, vp)]
    pos, st = i32([-5] * B), status()
    binding.sv_kv_fill(d[0], d[1], i32(cu), d[2], d[3], pos, S, W, head0=head0, dev_status=st)
    assert int(st.item()) == 0 and pos.tolist() == lens
    assert np.array_equal(d[2].cpu().numpy(), wk) and np.array_equal(d[3].cpu().numpy(), wv)
    # and the oracle's own commits agree on one request (all rows staged one by one)
    b = B - 1
    o = dict(k_pool=kp[b:b + 1, head0:head0 + Hkv].copy(), v_pool=vp[b:b + 1, head0:head0 + Hkv].copy(),
             pos=np.zeros(1, np.int32))
    for t in range(lens[b]):
        r = oracle.kv_commit(o["k_pool"], o["v_pool"], k[cu[b] + t][None, :, None], v[cu[b] + t][None, :, None],
                             np.zeros(1, np.int32), o["pos"], S, W)
        o = {n: r[n] for n in ("k_pool", "v_pool", "pos")}
    assert np.array_equal(o["k_pool"][0], wk[b, head0:head0 + Hkv]) and o["pos"][0] == lens[b]


def test_fill_invalid_bounds():
    k = torch.ones(10, 1, 8, dtype=BF, device=DEV)
    kp, vp = (torch.zeros(3, 1, 6, 8, dtype=BF, device=DEV) for _ in "kv")
    pos, st = i32([-5] * 3), status()
    binding.sv_kv_fill(k, k, i32([0, 4, 2, 11]), kp, vp, pos, 1, 5, dev_status=st)
    assert int(st.item()) == binding.SV_ST_BAD_LENGTH and pos.tolist() == [4, -5, -5]
    assert int(kp[0].sum()) == 32 and int(kp[1:].sum()) == 0


def commit_case(seed, B, LH, N, D, page, lens, chain, dtype=np.int16):
    rng = np.random.default_rng(seed)
    room = [-(-(n + N) // page) for n in lens]
    cols, P = max(room), sum(room) + 2
    order = rng.permutation(P)
    table, at = np.full((B, cols), -3, np.int32), 0
    for b in range(B):
        table[b, :room[b]] = order[at:at + room[b]]
        at += room[b]
    kp, vp = (rng.integers(0, 1 << 14, (P, LH, page, D)).astype(dtype) for _ in "kv")
    kn, vn = (rng.integers(0, 1 << 14, (B, LH, N, D)).astype(dtype) for _ in "kv")
    acc = rng.integers(-1, N, B).astype(np.int32)
    nodes = None
    if not chain:
        nodes = np.full((B, N), -1, np.int32)
        for b in range(B):
            k = max(0, int(acc[b]))
            nodes[b, :k] = np.sort(rng.choice(np.arange(1, N), k, replace=False)) if k else []
    return kp, vp, kn, vn, table, np.array(lens, np.int32), nodes, acc


def commit_plain(kp, vp, kn, vn, table, lens, nodes, acc):
    kp, vp, out, page = kp.copy(), vp.copy(), lens.copy(), kp.shape[2]
    for b in range(len(lens)):
        for j in range(acc[b] + 1):
            e = j if nodes is None or j == 0 else nodes[b, j - 1]
            t = lens[b] + j
            kp[table[b, t // page], :, t % page] = kn[b, :, e]
            vp[table[b, t // page], :, t % page] = vn[b, :, e]
        out[b] += max(0, acc[b] + 1)
    return kp, vp, out


def commit_gpu(case, in_place):
    d = [torch.from_numpy(x.copy()).to(DEV) for x in case[:4]]
    lens = i32(case[5])
    out, st = (lens if in_place else i32(np.full(len(case[5]), -7))), status()
    binding.sv_page_commit(d[0], d[1], d[2], d[3], i32(case[4]), lens, None if case[6] is None else i32(case[6]),
                           i32(case[7]), out, dev_status=st)
    torch.cuda.synchronize()
    return d[0].cpu().numpy(), d[1].cpu().numpy(), out.cpu().numpy(), int(st.item())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,LH,N,D,page,lens,chain", [
    (1, 1, 1, 8, 1, [0], True),
    (3, 5, 7, 64, 16, [0, 15, 16], False),
    (4, 17, 22, 128, 16, [1, 700, 33, 5], False),
    (2, 16, 256, 8, 24, [100, 23], False),
    (2, 3, 1000, 16, 24, [7, 0], True),
    (2, 2, 9000, 8, 40, [3, 100], True),
    (40, 33, 5, 8, 3, list(range(40)), True),
    (2, 2, 4, 4096, 8, [3, 9], False),
])
def test_page_commit(B, LH, N, D, page, lens, chain, in_place):
    case = commit_case(B + N, B, LH, N, D, page, lens, chain)
    k, v, out, st = commit_gpu(case, in_place)
    wk, wv, wout = commit_plain(*case)
    assert st == 0 and np.array_equal(out, wout)
    assert np.array_equal(k, wk) and np.array_equal(v, wv)


@pytest.mark.parametrize("in_place", [False, True])
def test_page_commit_invalid_requests(in_place):
    good = commit_case(3, 4, 3, 6, 16, 8, [5, 6, 7, 8], False)
    good[7][:] = [2, 3, 1, 0]
    for b in range(4):
        good[6][b] = [1, 2, 3, 4, 5, -1]
    for what, bit in (("node", binding.SV_ST_BAD_TOKEN), ("low node", binding.SV_ST_BAD_TOKEN),
                      ("page", binding.SV_ST_BAD_PAGE), ("count", binding.SV_ST_BAD_LENGTH),
                      ("length", binding.SV_ST_BAD_LENGTH), ("full", binding.SV_ST_BAD_LENGTH)):
        case = [None if x is None else x.copy() for x in good]
        if what == "node":
            case[6][1, 2] = 6
        if what == "low node":
            case[6][1, 0] = -1
        if what == "page":
            case[4][1, 1] = case[0].shape[0]
        if what == "count":
            case[7][1] = 6
        if what == "length":
            case[5][1] = -1
        if what == "full":
            case[5][1] = case[4].shape[1] * 8 - 3
        k, v, out, st = commit_gpu(case, in_place)
        assert st == bit, what
        left = [None if x is None else x.copy() for x in case]
        left[7][1] = -1
        wk, wv, wout = commit_plain(*left)
        assert np.array_equal(k, wk) and np.array_equal(v, wv) and np.array_equal(out, wout), what


def test_copies_far_rows():
    """Pools of more than 2^31 elements: a commit and a fill behind it."""
    P, LH, page, D = 9000, 16, 128, 128
    kp, vp = (torch.zeros(P, LH, page, D, dtype=BF, device=DEV) for _ in "kv")
    assert kp.numel() > 1 << 31
    kn, vn = (torch.randn(1, LH, 3, D, device=DEV).to(BF) for _ in "kv")
    lens = i32([126])
    binding.sv_page_commit(kp, vp, kn, vn, i32([[P - 1, P - 2]]), lens, None, i32([2]), lens)
    assert lens.tolist() == [129]
    for pool, new in ((kp, kn), (vp, vn)):
        assert torch.equal(pool[P - 1, :, 126:], new[0, :, :2]) and torch.equal(pool[P - 2, :, 0], new[0, :, 2])
        assert torch.count_nonzero(pool) == torch.count_nonzero(new)
    kp, vp = kp.view(P, LH, page, D), vp.view(P, LH, page, D)  # as rings of 126 behind 2 sinks
    kp.zero_(), vp.zero_()
    k, v = (torch.randn(200, 2, D, device=DEV).to(BF) for _ in "kv")
    cu = torch.zeros(P + 1, dtype=torch.int32, device=DEV)
    cu[P] = 200  # the last sequence holds all
    pos = torch.empty(P, dtype=torch.int32, device=DEV)
    binding.sv_kv_fill(k, v, cu, kp, vp, pos, 2, 126, head0=14)
    assert pos[P - 1] == 200 and torch.count_nonzero(pos) == 1
    for pool, new in ((kp, k), (vp, v)):
        for t in (0, 1, 74, 100, 199):
            assert torch.equal(pool[P - 1, 14:, au.slot(t, 2, 126)], new[t])
        assert torch.count_nonzero(pool[:P - 1]) == 0 and torch.count_nonzero(pool[P - 1, :14]) == 0


def test_tree_steps():
    """Pages as they are used: a prompt committed as a chain, then steps of tree attention, tree verification and the
    commit of the verified path; every step's attention against the whole history."""
    from speculative_decoding_verification_09_gb300 import synth
    rng = np.random.default_rng(31)
    B, Hq, Hkv, D, page, LH, head0 = 3, 8, 2, 64, 8, 3, 1
    parent = np.asarray(synth.tree_parents((3, 2, 1)), np.int32)
    N = parent.shape[-1]
    parents = np.broadcast_to(parent.reshape(-1, N)[0], (B, N)).copy()
    cols, P = 12, 40
    table = i32(rng.permutation(P)[:B * cols].reshape(B, cols))
    kp, vp = (torch.full((P, LH, page, D), float("nan"), dtype=BF, device=DEV) for _ in "kv")
    lens, zero = i32([0] * B), i32([0] * B)
    kn, vn = (au.tensor(rng, (B, LH, 20, D), BF) for _ in "kv")
    count = np.array([19, -1, 6])
    binding.sv_page_commit(kp, vp, kn, vn, table, lens, None, i32(count), lens)
    hist = [tuple(x[b, head0:, :count[b] + 1].transpose(0, 1) for x in (kn, vn)) for b in range(B)]
    ws = binding.make_attn_workspace(B, N, Hq, Hkv, D, DEV)
    for step in range(6):
        q = au.tensor(rng, (B, N, Hq, D), BF, 2.0)
        kn, vn = (au.tensor(rng, (B, LH, N, D), BF) for _ in "kv")
        got = torch.empty_like(q)
        binding.sv_tree_attn(q, kp, vp, table, lens, kn, vn, i32(parents), got, ws, head0=head0, kv_heads=Hkv)
        V = 300
        inp = synth.make_tree_inputs(synth.custom_config(B, 0, V, "bf16", "mix", temp=1.0),
                                     synth.tree_parents((3, 2, 1)), seed=step)
        t = {n: torch.from_numpy(np.ascontiguousarray(getattr(inp, n))).to(DEV)
             for n in ("Lt", "Ld", "parent", "tokens", "u_acc", "u_res", "temp")}
        tok, nodes = (torch.empty(B, N, dtype=torch.int32, device=DEV) for _ in "tn")
        acc = torch.empty(B, dtype=torch.int32, device=DEV)
        binding.sv_tree_verify(t["Lt"].view(BF), t["Ld"].view(BF), t["parent"], t["tokens"], t["u_acc"], t["u_res"],
                               t["temp"], tok, acc, nodes)
        before = lens.clone()
        binding.sv_page_commit(kp, vp, kn, vn, table, lens, nodes, acc, lens)
        for b in range(B):
            hk, hv = (torch.cat([h, x[b, head0:].transpose(0, 1)]) for h, x in zip(hist[b], (kn, vn)))
            n = hist[b][0].shape[0]
            assert n == int(before[b])
            want, tol = au.attend(q[b], hk, hv, au.tree_visible(n, parents[b]).to(DEV), D ** -0.5, BF)
            au.check(got[b], want, tol, f"step {step}, request {b}")
            path = [0] + nodes[b, :int(acc[b])].tolist()
            hist[b] = tuple(torch.cat([h, x[b, head0:][:, path].transpose(0, 1)])
                            for h, x in zip(hist[b], (kn, vn)))
            assert int(lens[b]) == n + len(path)


# ------------------------------------------------------------------ streams, graphs, repeats

def test_same_bits_every_time():
    c = tree_inputs(70, 5, 22, 8, 2, 128, 16, [3000, 100, 1, 0, 777], BF)
    ws = binding.make_attn_workspace(5, 22, 8, 2, 128, DEV)
    first, _ = tree_call(c, ws=ws)
    ws.fill_(255)  # a workspace needs no preparation
    for _ in range(3):
        again, _ = tree_call(c, ws=ws)
        assert torch.equal(first, again)


def test_long_runs():
    """Batches large enough that every SM walks tens of key tiles of several items: right, and the same bits again."""
    r = ring_inputs(74, 32, 8, 32, 8, 128, 4, 2048, [(911 * i + 100) % 9000 for i in range(32)], BF)
    c = tree_inputs(75, 48, 12, 32, 8, 128, 64, [(677 * i + 30) % 3500 for i in range(48)], BF)
    d = tree_inputs(76, 24, 70, 16, 4, 64, 32, [(677 * i + 30) % 3500 for i in range(24)], HF)
    for check, call, x in ((ring_check, ring_call, r), (tree_check, tree_call, c), (tree_check, tree_call, d)):
        first = check(x)
        for _ in range(4):
            assert torch.equal(first, call(x)[0])


def test_many_requests():
    """More requests than a block has threads, most of them short or empty; more sequences than a warp plans at once."""
    rng = np.random.default_rng(77)
    B = 1500
    lens = [int(x) for x in rng.choice([0, 1, 5, 130], B, p=[0.5, 0.3, 0.15, 0.05])]
    lens[-1] = 700
    c = tree_inputs(78, B, 2, 2, 1, 64, 16, lens, BF)
    out, st = tree_call(c)
    r = ring_inputs(79, B, 2, 2, 1, 64, 2, 300, lens, BF)
    rout, rst = ring_call(r)
    p = prompt_inputs(80, lens, 2, 1, 64, 2, 50, BF)
    pout, pst = prompt_call(p)
    assert int(st.item()) == int(rst.item()) == int(pst.item()) == 0
    for b in [*range(0, B, 97), *np.flatnonzero(np.array(lens) == 130)[:3].tolist(), B - 1]:
        au.check(out[b], *tree_reference(c, b), f"tree {b}")
        au.check(rout[b], *ring_reference(r, b), f"ring {b}")
        a, e = int(p["cu"][b]), int(p["cu"][b + 1])
        if e > a:
            at = range(e - a)
            au.check(pout[a:e], *au.attend(p["q"][a:e], p["k"][a:e], p["v"][a:e],
                                           au.window_visible(at, at, 2, 50).to(DEV), 64 ** -0.5, BF), f"prompt {b}")


def test_prompt_all_empty():
    p = prompt_inputs(81, [0] * 70, 4, 2, 64, 2, 50, BF, tail=5)
    out, st = prompt_call(p)
    assert int(st.item()) == 0 and (out == 7.0).all()


def test_two_calls_at_once():
    """Two streams, each with its own workspace and outputs, many calls in flight on both."""
    c = tree_inputs(82, 6, 9, 8, 2, 128, 16, [300, 100, 1200, 5, 0, 2000], BF)
    r = ring_inputs(83, 6, 3, 8, 2, 128, 4, 500, [300, 100, 1200, 5, 0, 2000], BF)
    want = tree_call(c)[0], ring_call(r)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(w) for w in want]
    ws = [binding.make_attn_workspace(6, n, 8, 2, 128, DEV) for n in (9, 3)]
    d = [i32(c["table"]), i32(c["lens"]), i32(c["parent"]), i32(r["pos"])]
    torch.cuda.synchronize()
    for _ in range(20):
        binding.sv_tree_attn(c["q"], c["kp"], c["vp"], d[0], d[1], c["kn"], c["vn"], d[2], outs[0], ws[0],
                             stream=streams[0])
        binding.sv_ring_attn(r["q"], r["kp"], r["vp"], d[3], r["kn"], r["vn"], 4, 500, outs[1], ws[1],
                             stream=streams[1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_other_stream_and_graph():
    """Calls on a side stream, and captured ones replayed on new data, two graphs sharing a workspace in turn."""
    c = tree_inputs(71, 3, 9, 8, 2, 64, 16, [300, 100, 1200], HF)
    r = ring_inputs(72, 3, 9, 8, 2, 64, 4, 500, [300, 100, 1200], HF)
    p = prompt_inputs(73, [300, 20], 8, 2, 64, 4, 100, HF)
    side = torch.cuda.Stream()
    ws = binding.make_attn_workspace(3, 9, 8, 2, 64, DEV)
    want = [tree_call(c, ws=ws)[0], ring_call(r, ws=ws)[0], prompt_call(p)[0]]
    torch.cuda.synchronize()
    outs = [torch.zeros_like(w) for w in want]
    d = [i32(c["table"]), i32(c["lens"]), i32(c["parent"]), i32(r["pos"]), i32(p["cu"])]
    torch.cuda.synchronize()

    def calls(stream=None):
        binding.sv_tree_attn(c["q"], c["kp"], c["vp"], d[0], d[1], c["kn"], c["vn"], d[2], outs[0], ws, stream=stream)
        binding.sv_ring_attn(r["q"], r["kp"], r["vp"], d[3], r["kn"], r["vn"], 4, 500, outs[1], ws, stream=stream)
        binding.sv_prompt_attn(p["q"], p["k"], p["v"], d[4], 4, 100, outs[2], stream=stream)

    calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        graphs.append(g)
    for rep in range(3):
        for g in graphs:
            for o in outs:
                o.fill_(5.0)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
    c["lens"] = [17, 0, 1300]
    d[1].copy_(i32(c["lens"]))
    graphs[0].replay()
    assert torch.equal(outs[0], tree_call(c)[0])


@pytest.mark.parametrize("seed", range(int(os.environ.get("SV_ATTN_FUZZ_SEEDS", "20"))))
def test_fuzz(seed):
    """Random shapes of all three calls."""
    rng = np.random.default_rng(9000 + seed)
    dtype = [BF, HF][seed % 2]
    Hkv, G, D = int(rng.choice([1, 2, 3, 8])), int(rng.choice([1, 2, 3, 4, 7, 16])), 8 * int(rng.integers(1, 17))
    B, N, page = int(rng.integers(1, 7)), int(rng.integers(1, 90)), 8 * int(rng.integers(1, 20))
    lens = [int(x) for x in rng.integers(0, 1500, B)]
    tree_check(tree_inputs(seed, B, N, Hkv * G, Hkv, D, page, lens, dtype, LH=Hkv + int(rng.integers(0, 3)),
                           dead=float("nan")))
    R, S = int(rng.integers(1, 65)), int(rng.integers(0, 150))
    W = R + int(rng.integers(0, 600))
    pos = [int(x) for x in rng.integers(0, 2 * (S + W) + 2, B)]
    ring_check(ring_inputs(seed, B, R, Hkv * G, Hkv, D, S, W, pos, dtype, dead=float("nan")))
    prompt_check(prompt_inputs(seed, lens, Hkv * G, Hkv, D, S, int(rng.integers(1, 900)), dtype, tail=seed % 3))
