"""The 8-bit paged cache on the GPU: writing it (sv_page_append8, sv_page_commit8) against the definition of kv8_util,
byte for byte where the inputs are exact and within its bounds where keys are rotated; the attention over it
(sv_tree_attn8) against 64-bit attention with the elementwise bound of attn_util; and a decoding run of them together."""
import numpy as np
import pytest
import torch

import attn_util as au
import kv8_util as ku
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


def u8(t):
    return t.view(torch.uint8)


def pages_for(rng, lens, more, page, spare=2):
    room = [-(-(n + m) // page) for n, m in zip(lens, more)]
    cols, P = max(1, max(room)) + 1, sum(room) + spare
    order = list(rng.permutation(P))
    table = np.full((len(lens), cols), -1, np.int32)
    for b, r in enumerate(room):
        table[b, :r] = [order.pop() for _ in range(r)]
    return table, P


def same(got, want):
    """Equal bytes, but for the sign of a NaN."""
    a, b = u8(got), u8(want)
    both = (a & 0x7f == 0x7f) & (b & 0x7f == 0x7f)
    return bool(((a == b) | both).all())


def joined(values, exps):
    """The tensors of a cache whose e4m3 values and exponents these are."""
    return values.float().to(ku.E4M3), (exps + 127).to(torch.uint8).view(ku.E8M0)


# ------------------------------------------------------------------ packed tokens

def append_case(seed, lens, more, Hkv, D, rot, inter, page, block, dtype, LH=None, gap=0, by=1.0):
    rng = np.random.default_rng(seed)
    LH = LH or Hkv
    table, P = pages_for(rng, lens, more, page)
    cu = gap + np.concatenate([[0], np.cumsum(more)])
    T = int(cu[-1]) + gap
    c = dict(lens=lens, more=more, table=table, cu=cu, T=T, page=page, block=block, head0=LH - Hkv, Hkv=Hkv,
             inter=inter, B=len(lens), P=P, LH=LH)
    # tokens whose sizes differ, so that scales rise inside a block and across calls
    size = torch.from_numpy(2.0 ** rng.integers(-3, 4, (T, 1, 1))).to(DEV).float()
    for x in "kv":
        c[x] = (au.tensor(rng, (T, Hkv, D), torch.float32, by) * size).to(dtype)
        c[x + "p"], c[x + "s"] = ku.used_cache(rng, P, LH, page, D, block, dtype, DEV)
    c["angles"] = ku.angles(max(1, max(a + b for a, b in zip(lens, more))), rot).float().to(DEV) if rot else None
    return c


def append_call(c, pools=None, positions=None, **kw):
    kp, vp, ks, vs = pools or [c[x].clone() for x in ("kp", "vp", "ks", "vs")]
    out, st = i32([-5] * c["B"]), status()
    binding.sv_page_append8(c["k"], c["v"], kp, vp, ks, vs, i32(c["table"]), i32(c["lens"]), i32(c["cu"]),
                            c["angles"], positions, out, head0=c["head0"], interleaved=c["inter"], dev_status=st, **kw)
    return kp, vp, ks, vs, out, st


def append_want(c, positions=None):
    """The cache by the definition, from the rotation in 32 bits (exact from there on), on the CPU."""
    got, angles = [], None if c["angles"] is None else c["angles"].cpu()
    for x in "kv":
        vals, exps = ku.split(c[x + "p"].cpu(), c[x + "s"].cpu())
        rows = slice(c["head0"], c["head0"] + c["Hkv"])
        for b, n in enumerate(c["lens"]):
            a, e = int(c["cu"][b]), int(c["cu"][b + 1])
            new = c[x][a:e].cpu()
            if x == "k" and angles is not None:
                at = torch.arange(n, n + e - a) if positions is None else positions[a:e].long().cpu()
                new = ku.rotate32(new, angles[at], c["inter"])
            part_v, part_e = vals[:, rows].clone(), exps[:, rows].clone()
            ku.write(part_v, part_e, new.double().cpu().transpose(0, 1), c["table"][b], n, c[x].dtype)
            vals[:, rows], exps[:, rows] = part_v, part_e
        got.append(joined(vals, exps))
    return got


APPENDS = [  # lens, more, Hkv, D, rot, interleaved, page, block, dtype, LH, gap
    ([0], [1], 1, 16, 16, False, 8, 8, BF, None, 0),
    ([5], [1], 2, 128, 128, False, 16, 16, BF, None, 0),
    ([0, 15, 16, 17], [3, 1, 0, 40], 2, 64, 32, False, 16, 8, BF, 5, 0),
    ([7, 0, 100], [0, 0, 0], 4, 128, 128, False, 16, 16, BF, None, 0),
    ([i * 5 for i in range(70)], [(7 * i) % 4 for i in range(70)], 3, 80, 20, True, 24, 8, HF, 3, 2),
    ([0, 3], [700, 130], 4, 128, 128, False, 64, 32, BF, 8, 3),
    ([9], [150], 1, 112, 0, False, 128, 64, HF, 2, 1),
    ([1] * 40, [1] * 40, 8, 128, 64, True, 32, 32, BF, 16, 0),
    ([100, 0], [900, 300], 2, 96, 48, False, 256, 128, BF, None, 0),
    ([130], [140], 1, 128, 128, True, 128, 128, HF, None, 0),
    ([3], [20], 2, 128, 18, False, 128, 128, BF, None, 0),
    ([0, 11], [2000, 1], 16, 64, 64, False, 16, 16, BF, None, 0),
]


@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append8(i):
    c = append_case(i, *APPENDS[i])
    kp, vp, ks, vs, out, st = append_call(c)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and out.tolist() == [a + b for a, b in zip(c["lens"], c["more"])]
    (wk, wks), (wv, wvs) = append_want(c)
    assert torch.equal(u8(ks.cpu()), u8(wks)) and torch.equal(u8(vs.cpu()), u8(wvs))
    assert same(kp.cpu(), wk) and same(vp.cpu(), wv)


@pytest.mark.parametrize("i", [1, 4, 5, 8])
def test_appended_values_are_near_the_tokens(i):
    """What the pages hold against the rotation in 64 bits: half a step of e4m3, and the rotation's own error."""
    c = append_case(i, *APPENDS[i])
    kp, vp, ks, vs, _, _ = append_call(c)
    held = {"k": ku.values(kp, ks), "v": ku.values(vp, vs)}
    scale = {"k": ks, "v": vs}
    for b, n in enumerate(c["lens"]):
        a, e = int(c["cu"][b]), int(c["cu"][b + 1])
        at = np.arange(n, n + e - a)
        pg, row = torch.from_numpy(c["table"][b, at // c["page"]].astype(np.int64)).to(DEV), torch.from_numpy(at % c["page"]).to(DEV)
        for x in "kv":
            rows = slice(c["head0"], c["head0"] + c["Hkv"])
            got = held[x][:, rows].transpose(1, 2)[pg, row]
            want, size = c[x][a:e].double(), c[x][a:e].double().abs()
            if x == "k" and c["angles"] is not None:
                want, size = ku.rotate(c[x][a:e], c["angles"][torch.from_numpy(at).to(DEV)], c["inter"])
            f = ku.power(u8(scale[x])[:, rows].transpose(1, 2)[pg, row // c["block"]].long() - 127)[..., None]
            tol = torch.maximum(want.abs() * 2.0 ** -4, f * 2.0 ** -10) + ku.ROT * size * 1.1
            assert bool(((got - want).abs() <= tol).all())


def test_append8_at_given_positions_and_from_slices():
    c = append_case(20, [3, 20], [30, 5], 2, 64, 64, False, 32, 16, BF)
    pos = i32(np.random.default_rng(1).integers(0, c["angles"].shape[0], c["T"]))
    (wk, wks), (wv, wvs) = append_want(c, pos)
    wide = torch.cat([c["k"], torch.zeros_like(c["k"]), c["v"]], 1).contiguous()
    c["k"], c["v"] = wide[:, :2], wide[:, 4:]
    kp, vp, ks, vs, _, st = append_call(c, positions=pos)
    assert int(st.item()) == 0
    assert same(kp.cpu(), wk) and same(vp.cpu(), wv) and torch.equal(u8(ks.cpu()), u8(wks))


def test_a_scale_rises_token_by_token():
    """A block filled one token at a time with ever larger ones: older entries are rounded again at each rise."""
    D, block = 32, 16
    rng = np.random.default_rng(2)
    c = append_case(21, [0], [1], 1, D, 0, False, block, block, BF)
    c["table"] = np.array([[1, -1]], np.int32)
    pools = [c[x].clone() for x in ("kp", "vp", "ks", "vs")]
    vals, exps = ku.split(c["kp"].cpu(), c["ks"].cpu())
    for n in range(block):
        c["lens"], c["k"] = [n], (au.tensor(rng, (1, 1, D), torch.float32) * 2.0 ** (3 * n - 20)).to(BF)
        append_call(c, pools)
        ku.write(vals, exps, c["k"].double().cpu().transpose(0, 1), c["table"][0], n, BF)
        want, scale = joined(vals, exps)
        assert same(pools[0].cpu(), want) and torch.equal(u8(pools[2].cpu()), u8(scale)), n


@pytest.mark.parametrize("dtype", [BF, HF])
def test_values_that_are_not_finite_extreme_or_zero(dtype):
    """NaN for what is not finite, the scale from the rest; the type's largest and smallest values; blocks of zeros."""
    D, page = 16, 8
    c = append_case(22, [0], [40], 1, D, 0, False, page, 8, dtype)
    big = torch.finfo(dtype).max
    k = c["k"]
    k[0:8] = 0
    k[8:16] = torch.finfo(dtype).tiny
    k[16:24, 0, ::2] = big
    k[24, 0, 3], k[25, 0, 4], k[26, 0, 5] = float("nan"), float("inf"), -float("inf")
    k[32:40] = float("nan")
    kp, vp, ks, vs, _, st = append_call(c)
    (wk, wks), _ = append_want(c)
    assert same(kp.cpu(), wk) and torch.equal(u8(ks.cpu()), u8(wks)) and int(st.item()) == 0
    held = ku.values(kp, ks)
    lo, hi = ku.LIMITS[dtype]
    pg = [int(x) for x in c["table"][0, :5]]
    assert bool((held[pg[0]] == 0).all()) and int(u8(ks)[pg[0], 0, 0]) == lo + 127
    assert bool((held[pg[2], 0, :, ::2] == 448 * 2.0 ** hi).all())
    assert bool(held[pg[4]].isnan().all()) and int(held[pg[3]].isnan().sum()) == 3


@pytest.mark.parametrize("fault", ["page", "page high", "length", "room", "table", "positions", "bounds"])
def test_append8_faults_stay_with_their_request(fault):
    c = append_case(30, [10, 33, 7], [20, 30, 5], 2, 64, 64, False, 16, 16, BF)
    lens, table, cu, pos = list(c["lens"]), c["table"].copy(), c["cu"].copy(), None
    want = binding.SV_ST_BAD_LENGTH
    full = c["angles"]
    if fault == "page":
        table[1, 3], want = -1, binding.SV_ST_BAD_PAGE
    elif fault == "page high":
        table[1, 3], want = c["P"], binding.SV_ST_BAD_PAGE
    elif fault == "length":
        lens[1] = -4
    elif fault == "room":
        lens[1] = c["table"].shape[1] * 16 - 29
    elif fault == "table":
        full = full[:60]
    elif fault == "positions":
        pos = i32(np.zeros(c["T"]))
        pos[int(cu[1]) + 7] = full.shape[0]
    else:
        cu[2] = c["T"] + 9
    d = dict(c, lens=lens, table=table, cu=cu, angles=full)
    kp, vp, ks, vs, out, st = append_call(d, positions=pos)
    assert int(st.item()) == want
    bad = [1, 2] if fault == "bounds" else [1]
    assert out.tolist() == [lens[b] if b in bad else lens[b] + c["more"][b] for b in range(3)]
    before, after = ku.values(c["kp"], c["ks"]), ku.values(kp, ks)
    for b in bad:  # the cached entries keep their values, the block of the last one among them
        for p in range(c["lens"][b]):
            at = (int(c["table"][b, p // 16]), slice(None), p % 16)
            assert torch.equal(before[at], after[at]), (b, p)
    (wk, wks), _ = append_want(c, pos if pos is None else torch.zeros_like(pos))
    for b in range(3):
        if b not in bad:
            for p in range(c["lens"][b] + c["more"][b]):
                pg = int(c["table"][b, p // 16])
                assert same(kp[pg, :, p % 16].cpu(), wk[pg, :, p % 16])


# ------------------------------------------------------------------ verified paths

COMMITS = [  # lens, accepted, N, LH, D, page, block, dtype, path
    ([0], [0], 1, 1, 16, 8, 8, BF, False),
    ([5, 0, 31], [3, 0, 6], 7, 4, 128, 16, 16, BF, True),
    ([16, 15, 17, 9], [-1, 21, 2, 0], 22, 6, 64, 32, 16, HF, True),
    ([100, 3], [127, 60], 128, 2, 80, 24, 8, BF, False),
    ([250, 128], [30, 5], 64, 3, 96, 256, 128, HF, True),
    ([i for i in range(50)], [i % 4 for i in range(50)], 5, 2, 112, 64, 32, BF, True),
    ([7], [999], 1000, 1, 32, 16, 8, BF, False),
]


def commit_case(seed, lens, acc, N, LH, D, page, block, dtype, path):
    rng = np.random.default_rng(100 + seed)
    table, P = pages_for(rng, lens, [max(0, k + 1) for k in acc], page)
    c = dict(lens=lens, acc=acc, table=table, P=P, page=page, N=N)
    size = torch.from_numpy(2.0 ** rng.integers(-3, 4, (len(lens), 1, N, 1))).to(DEV).float()
    for x in "kv":
        c[x + "n"] = (au.tensor(rng, (len(lens), LH, N, D), torch.float32) * size).to(dtype)
        c[x + "p"], c[x + "s"] = ku.used_cache(rng, P, LH, page, D, block, dtype, DEV)
    nodes = np.full((len(lens), N), -1, np.int32)
    for b, k in enumerate(acc):
        if k > 0:
            nodes[b, :k] = np.sort(rng.choice(np.arange(1, N), k, replace=False))
    c["nodes"] = nodes if path else None
    return c


def commit_call(c, in_place=False):
    pools = [c[x].clone() for x in ("kp", "vp", "ks", "vs")]
    lens, st = i32(c["lens"]), status()
    out = lens if in_place else i32([-5] * len(c["lens"]))
    binding.sv_page_commit8(*pools, c["kn"], c["vn"], i32(c["table"]), lens,
                            None if c["nodes"] is None else i32(c["nodes"]), i32(c["acc"]), out, st)
    return (*pools, out, st)


def commit_want(c, keep=()):
    got = []
    for x in "kv":
        vals, exps = ku.split(c[x + "p"].cpu(), c[x + "s"].cpu())
        for b, (n, k) in enumerate(zip(c["lens"], c["acc"])):
            if k >= 0 and b not in keep:
                path = [0] + (list(range(1, k + 1)) if c["nodes"] is None else [int(i) for i in c["nodes"][b, :k]])
                ku.write(vals, exps, c[x + "n"][b][:, path].double().cpu(), c["table"][b], n, c[x + "n"].dtype)
        got.append(joined(vals, exps))
    return got


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("i", range(len(COMMITS)))
def test_commit8(i, in_place):
    c = commit_case(i, *COMMITS[i])
    kp, vp, ks, vs, out, st = commit_call(c, in_place)
    assert int(st.item()) == 0 and out.tolist() == [n + k + 1 if k >= 0 else n for n, k in zip(c["lens"], c["acc"])]
    (wk, wks), (wv, wvs) = commit_want(c)
    assert same(kp.cpu(), wk) and same(vp.cpu(), wv)
    assert torch.equal(u8(ks.cpu()), u8(wks)) and torch.equal(u8(vs.cpu()), u8(wvs))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fault", ["accepted", "length", "room", "node", "page"])
def test_commit8_faults_commit_nothing(fault, in_place):
    c = commit_case(1, *COMMITS[1])
    want = binding.SV_ST_BAD_LENGTH
    if fault == "accepted":
        c["acc"] = [3, 7, 6]
    elif fault == "length":
        c["lens"] = [5, -1, 31]
    elif fault == "room":
        c["lens"] = [5, c["table"].shape[1] * 16, 31]
    elif fault == "node":
        c["acc"][1], c["nodes"][1, 0], want = 1, 7, binding.SV_ST_BAD_TOKEN
        c["table"][1, 0] = 1
    else:
        c["table"][1, 0], want = -1, binding.SV_ST_BAD_PAGE
    kp, vp, ks, vs, out, st = commit_call(c, in_place)
    assert int(st.item()) == want
    assert out.tolist() == [n if b == 1 else n + c["acc"][b] + 1 for b, n in enumerate(c["lens"])]
    (wk, wks), (wv, wvs) = commit_want(c, keep=(1,))
    assert same(kp.cpu(), wk) and same(vp.cpu(), wv) and torch.equal(u8(ks.cpu()), u8(wks))


# ------------------------------------------------------------------ attention

def tree_inputs(seed, B, N, Hq, Hkv, D, page, block, lens, dtype, kind="random", LH=None, qs=2.0, dead=False, spread=2):
    """`dead`: NaN in what no request may use: rows past a length, unused pages, other layers' heads."""
    rng = np.random.default_rng(seed)
    LH = LH or Hkv
    c = dict(B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, page=page, block=block, lens=lens, dtype=dtype, head0=LH - Hkv)
    table, P = pages_for(rng, lens, [0] * B, page)
    for b in range(B):  # past the length: never looked at
        table[b, -(-lens[b] // page):] = rng.choice([-1, 0, P + 5])
    c["table"] = table
    used = torch.zeros(P, page, dtype=torch.bool)
    for b in range(B):
        for t in range(lens[b]):
            used[table[b, t // page], t % page] = True
    for x in "kv":
        c[x + "p"], c[x + "s"] = ku.used_cache(rng, P, LH, page, D, block, dtype, DEV, spread)
        c[x + "n"] = au.tensor(rng, (B, LH, N, D), dtype)
        if dead:
            u8(c[x + "p"]).permute(0, 2, 1, 3)[~used.to(DEV)] = 0x7f
            u8(c[x + "p"])[:, :c["head0"]] = 0xff
            blocks = used.view(P, page // block, block).any(2).to(DEV)
            u8(c[x + "s"]).transpose(1, 2)[~blocks] = 255
            u8(c[x + "s"])[:, :c["head0"]] = 255
            c[x + "n"][:, :c["head0"]] = float("nan")
    c["q"] = au.tensor(rng, (B, N, Hq, D), dtype, qs)
    c["parent"] = np.array([au.random_parents(N, rng, kind) for _ in range(B)], np.int32)
    return c


def tree_call(c, parent=True, ws=None, out=None, **kw):
    out = torch.full_like(c["q"], 7.0) if out is None else out
    ws = binding.make_attn_workspace(c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], DEV) if ws is None else ws
    st = status()
    binding.sv_tree_attn8(c["q"], c["kp"], c["vp"], c["ks"], c["vs"], i32(c["table"]), i32(c["lens"]), c["kn"], c["vn"],
                          i32(c["parent"]) if parent else None, out, ws, head0=c["head0"], kv_heads=c["Hkv"],
                          dev_status=st, **kw)
    return out, st


def entries(c, b):
    """Request b's cached keys and values in 64 bits, [n][Hkv][D]."""
    n, page, h0 = c["lens"][b], c["page"], c["head0"]
    ids = torch.as_tensor(c["table"][b, :-(-n // page)].astype(np.int64)).to(DEV)
    got = []
    for x in "kv":
        held = ku.values(u8(c[x + "p"])[ids].view(ku.E4M3), u8(c[x + "s"])[ids].view(ku.E8M0))
        got.append(held[:, h0:h0 + c["Hkv"]].transpose(1, 2).reshape(-1, c["Hkv"], c["D"])[:n])
    return got


def tree_reference(c, b, scale=None, parent=True):
    k, v = entries(c, b)
    h = slice(c["head0"], c["head0"] + c["Hkv"])
    k, v = (torch.cat([x, c[y][b, h].transpose(0, 1).double()]) for x, y in ((k, "kn"), (v, "vn")))
    own = c["parent"][b] if parent else [-1] + list(range(c["N"] - 1))
    return au.attend(c["q"][b], k, v, au.tree_visible(c["lens"][b], own).to(DEV), scale or c["D"] ** -0.5, c["dtype"])


def tree_check(c, **kw):
    out, st = tree_call(c, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for b in range(c["B"]):
        want, tol = tree_reference(c, b, kw.get("scale"), kw.get("parent", True))
        au.check(out[b], want, tol, f"request {b}, length {c['lens'][b]}")
    return out


TREES = [
    # B, N, Hq, Hkv, D, page, block, lens, dtype, kind
    (1, 1, 1, 1, 16, 8, 8, [0], BF, "chain"),
    (1, 1, 4, 4, 128, 16, 16, [1], BF, "chain"),
    (1, 1, 16, 16, 128, 16, 16, [500], BF, "chain"),
    (3, 5, 8, 2, 64, 16, 8, [0, 127, 128], HF, "chain"),
    (4, 22, 32, 8, 128, 128, 32, [129, 1000, 0, 4097], BF, "random"),
    (2, 61, 28, 4, 64, 16, 16, [2000, 777], HF, "random"),
    (2, 256, 2, 1, 128, 64, 64, [300, 1], BF, "random"),
    (1, 256, 8, 1, 48, 24, 8, [511], HF, "star"),
    (2, 128, 3, 3, 80, 24, 8, [640, 383], BF, "random"),
    (2, 129, 5, 1, 96, 8, 8, [255, 256], HF, "chain"),
    (1, 3, 128, 1, 112, 256, 128, [3000], BF, "random"),
    (2, 7, 100, 1, 16, 64, 16, [300, 71], HF, "random"),
    (70, 4, 4, 2, 64, 32, 16, [(37 * i) % 300 for i in range(70)], BF, "random"),
    (1, 22, 32, 1, 128, 128, 128, [20000], BF, "random"),
    (2, 9, 12, 3, 128, 32, 32, [1000, 33], HF, "random"),
    (3, 30, 4, 1, 128, 64, 32, [200, 0, 1500], HF, "random"),
    (2, 40, 8, 1, 128, 64, 32, [700, 90], HF, "random"),
    (40, 6, 2, 2, 128, 16, 16, [(61 * i) % 700 for i in range(40)], HF, "chain"),
]


@pytest.mark.parametrize("i", range(len(TREES)))
def test_tree8(i):
    tree_check(tree_inputs(50 + i, *TREES[i]))


@pytest.mark.parametrize("i", [2, 4, 5, 6, 8, 11, 14, 16])
def test_tree8_never_uses_what_no_row_sees(i):
    """NaN entries and NaN scales past the lengths, in unused pages and in other layers' rows."""
    a = list(TREES[i])
    tree_check(tree_inputs(150 + i, *a, LH=a[3] + 3, dead=True))


@pytest.mark.parametrize("i", [2, 3, 4, 9, 15])
def test_tree8_chain_without_a_parent_array(i):
    tree_check(tree_inputs(250 + i, *TREES[i]), parent=False)


@pytest.mark.parametrize("dtype,spread", [(BF, 40), (HF, 6)])
@pytest.mark.parametrize("N,Hq", [(1, 2), (9, 6), (64, 2), (90, 4)])
def test_tree8_blocks_of_very_different_sizes(dtype, spread, N, Hq):
    """Scales across a wide range, up to scores whose differences leave one key; a small scale of the softmax."""
    c = tree_inputs(300, 2, N, Hq, 2, 64, 32, 16, [300, 45], dtype, spread=spread)
    for scale in (1e-4, 0.125):
        if dtype == BF and scale == 0.125:
            continue  # (scores past 2^40 differ by more than 64 bits against 32 can say; covered by the small scale)
        tree_check(c, scale=scale * 2.0 ** -spread if dtype == BF else scale)


def test_tree8_every_byte_and_every_exact_scale():
    """One key per byte of e4m3 and per scale: v = 1 elsewhere, a single key visible beside the node's own, whose score
    is far below.  The output is the entry itself, exactly."""
    D, block = 16, 8
    for dtype in (BF, HF):
        lo, hi = ku.LIMITS[dtype]
        exps = list(range(lo, hi + 1))
        P = len(exps)
        fin = [x for x in range(256) if x & 0x7f != 0x7f]
        vp = torch.zeros(P, 1, block, D, dtype=torch.uint8, device=DEV)
        vp.view(P, -1)[:, :] = torch.tensor([fin[i % len(fin)] for i in range(block * D)], dtype=torch.uint8, device=DEV)
        # (a page's 8 x 16 entries are the first 128 bytes; a second pool takes the others)
        for shift in (0, 127):
            vp.view(P, -1)[:, :] = torch.tensor([fin[(i + shift) % len(fin)] for i in range(block * D)], dtype=torch.uint8,
                                                device=DEV)
            sc = torch.tensor(exps, device=DEV).add(127).to(torch.uint8).view(P, 1, 1)
            kp = torch.zeros_like(vp)
            B = P * block  # request (page, row): only that row's key is large
            one = torch.full((P, 1, 1), 127, dtype=torch.uint8, device=DEV)
            for row in range(block):
                kp.zero_()
                kp[:, 0, row] = 0x7e  # 448
                q = torch.full((P, 1, 1, D), 1.0, dtype=dtype, device=DEV)
                kn = torch.zeros(P, 1, 1, D, dtype=dtype, device=DEV)
                out = torch.empty_like(q)
                ws = binding.make_attn_workspace(P, 1, 1, 1, D, DEV)
                binding.sv_tree_attn8(q, kp.view(ku.E4M3), vp.view(ku.E4M3), one.view(ku.E8M0), sc.view(ku.E8M0),
                                      i32(np.arange(P)[:, None]), i32([block] * P), kn, kn, None, out, ws, scale=1.0)
                want = ku.values(vp.view(ku.E4M3), sc.view(ku.E8M0))[:, 0, row]
                assert torch.equal(out[:, 0, 0].double(), want), (dtype, row)


def test_tree8_nan_entries_and_scales_spoil_their_request_only():
    for what in ("k", "v", "ks", "vs"):
        for N, Hq in ((1, 2), (22, 8), (64, 2), (140, 4)):
            c = tree_inputs(400, 3, N, Hq, 2, 64, 16, 16, [50, 200, 31], BF)
            at = int(c["table"][1, 150 // 16])
            if what in ("ks", "vs"):
                u8(c[what])[at, 1, 0] = 255
            else:
                u8(c[what + "p"])[at, 1, 150 % 16, 5] = 0xff
            out, st = tree_call(c)
            for b in (0, 2):
                want, tol = tree_reference(c, b)
                au.check(out[b], want, tol, what)
            G = Hq // 2
            assert bool(out[1][:, G:].isnan().any()) and not bool(out[1][:, :G].isnan().any())


def test_tree8_scales_outside_the_exact_range_are_nan():
    c = tree_inputs(410, 1, 3, 4, 2, 64, 16, 16, [40], HF)
    for byte in (0, 111, 135, 200, 254):
        d = dict(c, vs=c["vs"].clone())
        u8(d["vs"])[int(c["table"][0, 1]), 0, 0] = byte
        out, _ = tree_call(d)
        assert bool(out[0][:, :2].isnan().all()) and not bool(out[0][:, 2:].isnan().any())


def test_tree8_invalid_requests_get_zeros():
    c = tree_inputs(420, 5, 6, 8, 2, 128, 16, 16, [100, 300, 40, 0, 500], BF)
    c["table"][1, 3] = -1
    c["table"][4, 20] = 10**6
    c["lens"] = [100, 300, -1, 0, 500]
    c["parent"][3, 2] = 4
    out, st = tree_call(c)
    assert int(st.item()) == binding.SV_ST_BAD_PAGE | binding.SV_ST_BAD_LENGTH | binding.SV_ST_BAD_TOKEN
    assert all(bool((out[b] == 0).all()) for b in (1, 2, 3, 4))
    want, tol = tree_reference(c, 0)
    au.check(out[0], want, tol)


def test_tree8_is_deterministic_and_leaves_its_workspace_free():
    c = tree_inputs(430, 6, 22, 32, 8, 128, 128, 32, [129, 1000, 0, 4097, 7, 2000], BF)
    ws = binding.make_attn_workspace(6, 22, 32, 8, 128, DEV)
    a, _ = tree_call(c, ws=ws)
    ws.fill_(255)
    b, _ = tree_call(c, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d, _ = tree_call(c)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, d)


def test_tree8_graph_serves_other_lengths():
    c = tree_inputs(440, 3, 5, 8, 2, 128, 32, 16, [700, 320, 64], HF)
    lens, par, table = i32(c["lens"]), i32(c["parent"]), i32(c["table"])
    ws = binding.make_attn_workspace(3, 5, 8, 2, 128, DEV)
    out = torch.empty_like(c["q"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.sv_tree_attn8(c["q"], c["kp"], c["vp"], c["ks"], c["vs"], table, lens, c["kn"], c["vn"], par, out, ws)
    for new in ([700, 320, 64], [1, 0, 63], [699, 13, 17]):
        lens.copy_(i32(new))
        c["lens"] = new
        g.replay()
        torch.cuda.synchronize()
        for b in range(3):
            want, tol = tree_reference(c, b)
            au.check(out[b], want, tol, f"{new} {b}")


def test_tree8_timeout_is_reported_and_ends():
    """A stage that never counts as filled: the bounded waits run out and say so; the next call is right."""
    for N, Hq in ((1, 2), (40, 4), (100, 4)):
        c = tree_inputs(450, 2, N, Hq, 2, 128, 32, 16, [700, 320], BF)
        binding.sv_attn_test_withhold(True)
        try:
            _, st = tree_call(c)
            torch.cuda.synchronize()
        finally:
            binding.sv_attn_test_withhold(False)
        assert int(st.item()) & binding.SV_ST_TIMEOUT
        tree_check(c)


def test_tree8_pages_past_32_bit_offsets():
    """A pool of more than 2^32 bytes: pages at both ends."""
    P, LH, page, D, block = 9000, 4, 1024, 128, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB")
    rng = np.random.default_rng(11)
    small, sc = ku.used_cache(rng, 3, LH, page, D, block, BF, DEV)
    kp = torch.zeros(P, LH, page, D, dtype=torch.uint8, device=DEV)
    vp = torch.zeros(P, LH, page, D, dtype=torch.uint8, device=DEV)
    ks, vs = (torch.full((P, LH, page // block), 127, dtype=torch.uint8, device=DEV) for _ in "kv")
    for x in (kp, vp):
        for i, pg in enumerate((P - 1, 0, P - 3)):
            x[pg] = u8(small)[i]
    for x in (ks, vs):
        for i, pg in enumerate((P - 1, 0, P - 3)):
            x[pg] = u8(sc)[i]
    c = dict(B=1, N=3, Hq=4, Hkv=2, D=D, page=page, block=block, lens=[2500], dtype=BF, head0=2,
             table=np.array([[P - 1, 0, P - 3]], np.int32), kp=kp.view(ku.E4M3), vp=vp.view(ku.E4M3),
             ks=ks.view(ku.E8M0), vs=vs.view(ku.E8M0), q=au.tensor(rng, (1, 3, 4, D), BF, 2.0),
             kn=au.tensor(rng, (1, LH, 3, D), BF), vn=au.tensor(rng, (1, LH, 3, D), BF),
             parent=np.array([[-1, 0, 0]], np.int32))
    tree_check(c)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [BF, HF])
def test_decoding_run(dtype):
    """Prompts appended, then steps of rotation into the staged layout, tree attention, a verified path and its commit;
    against 64-bit attention over the cache's values after every step, and those against the tokens at the end."""
    rng = np.random.default_rng(12)
    B, N, Hq, Hkv, D, page, block = 3, 6, 8, 2, 64, 32, 16
    prompts, steps = [37, 5, 64], 7
    cols = -(-(max(prompts) + steps * N) // page) + 1
    P = B * cols
    table = rng.permutation(P).reshape(B, cols).astype(np.int32)
    angles = torch.empty(512, 2, D // 2, device=DEV)
    binding.sv_rope_table(angles)
    kp, vp = (torch.zeros(P, Hkv, page, D, dtype=torch.uint8, device=DEV).view(ku.E4M3) for _ in "kv")
    ks, vs = (torch.zeros(P, Hkv, page // block, dtype=torch.uint8, device=DEV).view(ku.E8M0) for _ in "kv")
    lens = i32([0] * B)
    cu = i32(np.concatenate([[0], np.cumsum(prompts)]))
    T = sum(prompts)
    k, v = au.tensor(rng, (T, Hkv, D), dtype), au.tensor(rng, (T, Hkv, D), dtype)
    bt, new = i32(table), torch.empty_like(lens)
    binding.sv_page_append8(k, v, kp, vp, ks, vs, bt, lens, cu, angles, out_seq_lens=new)
    lens = new
    assert lens.tolist() == prompts
    history = [[(k[int(cu[b]) + j], v[int(cu[b]) + j], j) for j in range(prompts[b])] for b in range(B)]
    ws = binding.make_attn_workspace(B, N, Hq, Hkv, D, DEV)
    for step in range(steps):
        at = lens.tolist()
        parent = np.array([au.random_parents(N, rng) for _ in range(B)], np.int32)
        depth = np.zeros((B, N), np.int64)
        for b in range(B):
            for n in range(1, N):
                depth[b, n] = depth[b, parent[b, n]] + 1
        pos = i32((np.array(at)[:, None] + depth).reshape(-1))
        q, k, v = (au.tensor(rng, (B * N, h, D), dtype, s) for h, s in ((Hq, 2.0), (Hkv, 1.0), (Hkv, 1.0)))
        kn, vn = torch.empty(B, Hkv, N, D, dtype=dtype, device=DEV), torch.empty(B, Hkv, N, D, dtype=dtype, device=DEV)
        binding.sv_page_append(k, v, kn, vn, i32([[b] for b in range(B)]), i32([0] * B), i32(np.arange(B + 1) * N), angles,
                               pos, q, q)
        c = dict(B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, page=page, block=block, lens=at, dtype=dtype, head0=0, table=table, kp=kp,
                 vp=vp, ks=ks, vs=vs, kn=kn, vn=vn, q=q.view(B, N, Hq, D), parent=parent)
        out, st = tree_call(c, ws=ws)
        assert int(st.item()) == 0
        for b in range(B):
            want, tol = tree_reference(c, b)
            au.check(out[b], want, tol, f"step {step} request {b}")
        nodes, acc = np.full((B, N), -1, np.int32), []
        for b in range(B):
            path, node = [], 0
            while True:
                below = [n for n in range(N) if parent[b, n] == node]
                if not below or rng.random() < 0.3:
                    break
                node = int(rng.choice(below))
                path.append(node)
            nodes[b, :len(path)] = path
            acc.append(len(path))
            for n in [0] + path:
                history[b].append((k[b * N + n], v[b * N + n], at[b] + int(depth[b, n])))
        binding.sv_page_commit8(kp, vp, ks, vs, kn, vn, bt, lens, i32(nodes), i32(acc), lens)
        assert lens.tolist() == [len(h) for h in history]
    c = dict(c, lens=lens.tolist())
    for b in range(B):
        held_k, held_v = entries(c, b)
        x = torch.stack([h[0] for h in history[b]])
        turned, size = ku.rotate(x, angles[torch.tensor([h[2] for h in history[b]], device=DEV)], False)
        u = torch.finfo(dtype).eps / 2
        for got, want in ((held_k, turned), (held_v, torch.stack([h[1] for h in history[b]]).double())):
            # twice half a step (a block's scale may rise once between near sizes), the staged rounding, the smallest step
            tol = want.abs() * (2.0 ** -3 + 2 * u) + size * 2 * ku.ROT + 2.0 ** -9 * want.abs().max() / 100
            assert bool(((got - want).abs() <= tol).all())


# ------------------------------------------------------------------ several rows of a CTA, several at a time

@pytest.mark.parametrize("i,case", list(enumerate([
    ([0, 9], [3000, 2000], 24, 128, 128, False, 64, 32, BF, 30, 0),
    ([0, 5, 40], [1500, 700, 900], 40, 32, 32, True, 32, 16, HF, 41, 1),
    ([3], [2500], 24, 48, 18, True, 32, 16, HF, None, 0),
    ([0, 120], [2000, 1900], 20, 128, 64, False, 128, 128, BF, None, 0),
    ([7 * i % 90 for i in range(350)], [(1, 1, 2, 1, 0, 1)[i % 6] for i in range(350)], 12, 64, 64, False, 32, 16, BF, 13, 1),
    ([i % 60 for i in range(150)], [1 + 11 * i % 23 for i in range(150)], 6, 80, 48, True, 64, 64, HF, None, 0),
])))
def test_append8_of_many_heads(i, case):
    c = append_case(60 + i, *case)
    for x, bad in (("k", float("inf")), ("v", float("nan")), ("v", -float("inf"))):
        for t in (7, 8, c["T"] // 2, c["T"] - 2):
            c[x][t, t % c["Hkv"], t % c["k"].shape[2]] = bad
    kp, vp, ks, vs, out, st = append_call(c)
    assert int(st.item()) == 0 and out.tolist() == [a + b for a, b in zip(c["lens"], c["more"])]
    (wk, wks), (wv, wvs) = append_want(c)
    assert torch.equal(u8(ks.cpu()), u8(wks)) and torch.equal(u8(vs.cpu()), u8(wvs))
    assert same(kp.cpu(), wk) and same(vp.cpu(), wv)


@pytest.mark.parametrize("i,case", list(enumerate([
    ([(3 * i) % 50 for i in range(60)], [(7 * i) % 22 for i in range(60)], 22, 70, 128, 16, 16, BF, True),
    ([i % 8 for i in range(152)], [i % 3 - 1 for i in range(152)], 2, 2100, 16, 8, 8, BF, True),
    ([100] * 30, [5, 127, -1] * 10, 128, 90, 32, 128, 128, HF, False),
])))
def test_commit8_of_many_rows(i, case):
    c = commit_case(60 + i, *case)
    kp, vp, ks, vs, out, st = commit_call(c, in_place=i == 1)
    assert int(st.item()) == 0 and out.tolist() == [n + k + 1 if k >= 0 else n for n, k in zip(c["lens"], c["acc"])]
    (wk, wks), (wv, wvs) = commit_want(c)
    assert same(kp.cpu(), wk) and same(vp.cpu(), wv)
    assert torch.equal(u8(ks.cpu()), u8(wks)) and torch.equal(u8(vs.cpu()), u8(wvs))
