"""Rotary positions (sv_rope_table, sv_rope) and appending rotated keys to pages (sv_page_append) on the GPU against the
definitions of kv8_util: 64-bit bounds for the rotation, bit-exact copies for the rest."""
import numpy as np
import pytest
import torch

import kv8_util as ku
from speculative_decoding_verification_09_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16
FILL = 7.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.lib()


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def normal(rng, *shape, dtype=BF, by=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * by).astype(np.float32)).to(DEV).to(dtype)


# ------------------------------------------------------------------ the table

TABLES = [dict(rows=1, rot=2), dict(rows=4097, rot=64), dict(rows=33, rot=256, first=1 << 20), dict(rows=5, rot=6, base=5e5),
          dict(rows=70, rot=128, first=2**31 - 71), dict(rows=64, rot=64, scaling="linear", factor=4.0, first=100000),
          dict(rows=64, rot=64, scaling="base", factor=8.0, first=30000),
          dict(rows=64, rot=128, base=1e6, scaling="ramp", factor=32.0, original=4096, first=131000),
          dict(rows=9, rot=20, scaling="ramp", factor=2.0, original=1, first=3, gain=0.5),
          dict(rows=64, rot=128, base=5e5, scaling="wave", factor=8.0, original=8192, low=1.0, high=4.0, first=131000),
          dict(rows=20, rot=32, scaling="linear", factor=0.25, first=1000, gain=1.25)]


@pytest.mark.parametrize("i", range(len(TABLES)))
def test_table(i):
    c = dict(TABLES[i])
    rows, rot = c.pop("rows"), c.pop("rot")
    want = ku.angles(rows, rot, **c)
    out = torch.full((rows + 1, 2, rot // 2), FILL, device=DEV)
    kw = dict(c, scaling=getattr(binding, "SV_ROPE_" + c.get("scaling", "none").upper()))
    binding.sv_rope_table(out[:rows], **kw)
    # 2^-22 of the gain for the functions; both sides' rates are off by some 2^-50 of an angle
    far = (c.get("first", 0) + rows) * ku.rates(rot, c.get("base", 1e4), **{k: v for k, v in c.items() if k in (
        "scaling", "factor", "original", "low", "high")}).max() * 2.0 ** -49
    off = (out[:rows].double().cpu() - want).abs().max()
    assert off <= (2.0 ** -22 + far) * c.get("gain", 1.0)
    assert bool((out[rows] == FILL).all())


def test_table_rows_do_not_depend_on_the_window():
    whole, part = torch.empty(900, 2, 40, device=DEV), torch.empty(7, 2, 40, device=DEV)
    binding.sv_rope_table(whole)
    binding.sv_rope_table(part, first=333)
    assert torch.equal(whole[333:340], part)


# ------------------------------------------------------------------ rotation

ROPES = [  # T, Hq, Hk, D, rot, interleaved, dtype
    (1, 1, 1, 8, 2, False, BF), (1, 32, 8, 128, 128, False, BF), (22, 32, 8, 128, 128, True, HF),
    (300, 28, 4, 64, 64, False, HF), (77, 4, 2, 80, 20, False, BF), (77, 4, 2, 80, 20, True, BF),
    (1000, 6, 3, 96, 48, True, BF), (513, 3, 0, 40, 40, False, HF), (64, 5, 1, 256, 64, False, BF),
    (2049, 16, 16, 128, 32, False, BF), (9, 2, 1, 24, 18, True, HF), (1, 65, 1, 72, 72, False, BF),
]


@pytest.mark.parametrize("i", range(len(ROPES)))
@pytest.mark.parametrize("mode", ["apart", "in place", "slices"])
def test_rope(i, mode):
    T, Hq, Hk, D, rot, inter, dtype = ROPES[i]
    rng = np.random.default_rng(i)
    table = ku.angles(500, rot).float().to(DEV)
    pos = i32(rng.integers(0, 500, T))
    pos[0] = 499
    cs = table[pos.long()]
    if mode == "slices":  # a fused projection's rows: queries, keys, values side by side
        wide = normal(rng, T, Hq + 2 * Hk + 1, D, dtype=dtype)
        q, k = wide[:, :Hq], wide[:, Hq:Hq + Hk] if Hk else None
    else:
        q, k = normal(rng, T, Hq, D, dtype=dtype), normal(rng, T, Hk, D, dtype=dtype) if Hk else None
    q0, k0 = q.clone(), k.clone() if Hk else None
    before = wide.clone() if mode == "slices" else None
    qo, ko = (q, k) if mode != "apart" else (torch.full_like(q, FILL), torch.full_like(k, FILL) if Hk else None)
    st = status()
    binding.sv_rope(q, k, pos, table, qo, ko, interleaved=inter, dev_status=st)
    assert int(st.item()) == 0
    ku.check_rotated(qo, q0, cs, inter)
    assert torch.equal(qo, ku.rotate32(q0, cs, inter).to(dtype))
    if Hk:
        ku.check_rotated(ko, k0, cs, inter)
    if mode == "slices":
        assert torch.equal(wide[:, Hq + Hk:], before[:, Hq + Hk:])
    if mode == "apart":
        assert torch.equal(q, q0)


def test_rope_leaves_out_bad_positions():
    rng = np.random.default_rng(3)
    table = ku.angles(10, 64).float().to(DEV)
    q, k = normal(rng, 6, 4, 64), normal(rng, 6, 2, 64)
    pos = i32([0, 9, 10, -1, 2**31 - 1, 3])
    qo, ko, st = torch.full_like(q, FILL), torch.full_like(k, FILL), status()
    binding.sv_rope(q, k, pos, table, qo, ko, dev_status=st)
    assert int(st.item()) == binding.SV_ST_BAD_LENGTH
    good = torch.tensor([0, 1, 5], device=DEV)
    ku.check_rotated(qo[good], q[good], table[pos[good].long()], False)
    ku.check_rotated(ko[good], k[good], table[pos[good].long()], False)
    assert bool((qo[2:5] == FILL).all()) and bool((ko[2:5] == FILL).all())


def test_rope_of_no_tokens_and_of_what_is_not_finite():
    table = ku.angles(4, 8).float().to(DEV)
    e = torch.empty(0, 2, 8, dtype=BF, device=DEV)
    binding.sv_rope(e, e, i32([]), table, e, e)
    x = torch.ones(3, 1, 8, dtype=BF, device=DEV)
    x[1, 0, 2] = float("nan")
    x[2, 0, 5] = float("inf")
    y = torch.empty_like(x)
    binding.sv_rope(x, None, i32([1, 1, 1]), table, y)
    bad = (~y.isfinite()).tolist()
    assert bad[0] == [[False] * 8]
    assert bad[1] == [[i in (2, 6) for i in range(8)]] and bad[2] == [[i in (1, 5) for i in range(8)]]


# ------------------------------------------------------------------ appending to pages

def append_case(seed, lens, more, Hq, Hkv, D, rot, inter, page, dtype, LH=None, gap=0):
    """Requests of `lens` entries and `more` tokens; `gap` packed rows before the first and behind the last request."""
    rng = np.random.default_rng(seed)
    B, LH = len(lens), LH or Hkv
    room = [-(-(n + m) // page) for n, m in zip(lens, more)]
    cols, P = max(1, max(room)) + 1, sum(room) + 2
    order = list(rng.permutation(P))
    table = np.full((B, cols), -1, np.int32)  # columns past a request's need are never looked at
    for b in range(B):
        table[b, :room[b]] = [order.pop() for _ in range(room[b])]
    cu = gap + np.concatenate([[0], np.cumsum(more)])
    T = int(cu[-1]) + gap
    c = dict(lens=lens, more=more, table=table, cu=cu, T=T, page=page, head0=LH - Hkv, Hkv=Hkv, inter=inter, B=B, P=P)
    c["k"], c["v"] = normal(rng, T, Hkv, D, dtype=dtype), normal(rng, T, Hkv, D, dtype=dtype)
    c["q"] = normal(rng, T, Hq, D, dtype=dtype, by=2.0) if Hq else None
    c["kp"], c["vp"] = normal(rng, P, LH, page, D, dtype=dtype), normal(rng, P, LH, page, D, dtype=dtype)
    c["angles"] = ku.angles(max(1, max(a + b for a, b in zip(lens, more))), rot).float().to(DEV) if rot else None
    return c


def places(c):
    """[(request, packed token, cache position)]"""
    return [(b, int(c["cu"][b]) + j, n + j) for b, n in enumerate(c["lens"]) for j in range(c["more"][b])]


APPENDS = [  # lens, more, Hq, Hkv, D, rot, interleaved, page, dtype, LH, gap
    ([5], [1], 4, 2, 128, 128, False, 16, BF, None, 0),
    ([0], [1], 1, 1, 8, 8, True, 1, HF, None, 0),
    ([0, 15, 16, 17], [3, 1, 0, 40], 8, 2, 64, 32, False, 16, BF, 5, 0),
    ([7, 0, 100], [0, 0, 0], 4, 4, 128, 128, False, 8, BF, None, 0),
    ([i * 5 for i in range(70)], [(7 * i) % 4 for i in range(70)], 0, 3, 80, 20, True, 24, HF, 3, 2),
    ([0, 3], [700, 130], 16, 4, 128, 128, False, 64, BF, 8, 3),
    ([9], [50], 6, 1, 256, 0, False, 7, HF, 2, 1),
    ([1] * 40, [1] * 40, 32, 8, 128, 64, True, 16, BF, 16, 0),
    ([0], [3000], 2, 2, 96, 96, True, 128, BF, None, 0),
]


@pytest.mark.parametrize("positions", [False, True])
@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append(i, positions):
    c = append_case(i, *APPENDS[i])
    dtype, rot = c["k"].dtype, 0 if c["angles"] is None else 2 * c["angles"].shape[2]
    where = places(c)
    t = torch.tensor([x[1] for x in where], dtype=torch.long, device=DEV)
    at = torch.tensor([x[2] for x in where], dtype=torch.long, device=DEV)
    pos = None
    if positions:
        rng = np.random.default_rng(i)
        rows = 1 if c["angles"] is None else c["angles"].shape[0]
        pos = i32(rng.integers(0, rows, c["T"]))
        at_turn = pos[t].long()
    else:
        at_turn = at
    q, k = c["q"] if rot else None, c["k"]
    qo, ko = None if q is None else torch.full_like(q, FILL), torch.full_like(k, FILL)
    kp, vp, out, st = c["kp"].clone(), c["vp"].clone(), i32([-5] * c["B"]), status()
    binding.sv_page_append(k, c["v"], kp, vp, i32(c["table"]), i32(c["lens"]), i32(c["cu"]), c["angles"], pos, q, qo, ko,
                           out, head0=c["head0"], interleaved=c["inter"], dev_status=st)
    assert int(st.item()) == 0
    assert out.tolist() == [a + b for a, b in zip(c["lens"], c["more"])]
    want_k, want_v = c["kp"].clone(), c["vp"].clone()
    turned = k[t].clone()
    if rot:
        cs = c["angles"][at_turn]
        turned = ku.rotate32(k[t], cs, c["inter"]).to(dtype)
        ku.check_rotated(ko[t], k[t], cs, c["inter"])
        if q is not None:
            ku.check_rotated(qo[t], q[t], cs, c["inter"])
    b = torch.tensor([x[0] for x in where], dtype=torch.long)
    if len(where):
        pg = torch.from_numpy(c["table"].astype(np.int64))[b, at.cpu() // c["page"]].to(DEV)
        rows = slice(c["head0"], c["head0"] + c["Hkv"])
        want_k[:, rows].transpose(1, 2)[pg, at % c["page"]] = turned
        want_v[:, rows].transpose(1, 2)[pg, at % c["page"]] = c["v"][t]
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    assert torch.equal(ko[t], turned)
    rest = torch.ones(c["T"], dtype=torch.bool, device=DEV)
    rest[t] = False
    assert bool((ko[rest] == FILL).all()) and (qo is None or bool((qo[rest] == FILL).all()))


def test_append_in_place_of_a_fused_projection():
    c = append_case(40, [3, 20], [30, 5], 6, 2, 64, 64, False, 16, BF)
    wide = torch.cat([c["q"], c["k"], c["v"]], 1).contiguous()
    q, k, v = wide[:, :6], wide[:, 6:8], wide[:, 8:]
    kp, vp, kp2, vp2 = (c[x].clone() for x in ("kp", "vp", "kp", "vp"))
    qo, ko = torch.empty_like(c["q"]), torch.empty_like(c["k"])
    args = (i32(c["table"]), i32(c["lens"]), i32(c["cu"]), c["angles"])
    binding.sv_page_append(c["k"], c["v"], kp2, vp2, *args, q=c["q"], q_out=qo, k_out=ko)
    binding.sv_page_append(k, v, kp, vp, *args, q=q, q_out=q, k_out=k)
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2)
    assert torch.equal(wide, torch.cat([qo, ko, c["v"]], 1))



@pytest.mark.parametrize("fault", ["page", "page high", "length", "room", "table", "positions", "bounds"])
def test_append_faults_stay_with_their_request(fault):
    """A request that cannot be appended keeps its length and its cached entries; the others are appended."""
    c = append_case(50, [10, 33, 7], [20, 30, 5], 4, 2, 64, 64, False, 16, BF)
    lens, table, cu, angles, pos = list(c["lens"]), c["table"].copy(), c["cu"].copy(), c["angles"], None
    want = binding.SV_ST_BAD_LENGTH
    if fault == "page":
        table[1, 3], want = -1, binding.SV_ST_BAD_PAGE
    elif fault == "page high":
        table[1, 2], want = c["P"], binding.SV_ST_BAD_PAGE
    elif fault == "length":
        lens[1] = -4
    elif fault == "room":
        lens[1] = c["table"].shape[1] * 16 - 29
    elif fault == "table":
        angles = angles[:60]  # request 1 reaches position 62
    elif fault == "positions":
        pos = i32([0] * c["T"])
        pos[int(cu[1]) + 7] = angles.shape[0]
    else:
        cu[2] = c["T"] + 9  # requests 1 and 2 have bounds outside the packed rows
    kp, vp, out, st = c["kp"].clone(), c["vp"].clone(), i32([-5] * 3), status()
    qo = torch.empty_like(c["q"])
    binding.sv_page_append(c["k"], c["v"], kp, vp, i32(table), i32(lens), i32(cu), angles, pos, c["q"], qo, None, out,
                           dev_status=st)
    assert int(st.item()) == want
    bad = [1, 2] if fault == "bounds" else [1]
    assert out.tolist() == [lens[b] if b in bad else lens[b] + c["more"][b] for b in range(3)]
    for b in range(3):
        n = c["lens"][b] if fault in ("length", "room") else lens[b]
        for p in range(n):
            at = (int(c["table"][b, p // 16]), slice(None), p % 16)
            if 0 <= table[b, p // 16] < c["P"]:
                assert torch.equal(kp[at], c["kp"][at]) and torch.equal(vp[at], c["vp"][at])
        if b not in bad:
            for j in range(c["more"][b]):
                p, t = n + j, int(c["cu"][b]) + j
                at = (int(table[b, p // 16]), slice(None), p % 16)
                turn = p if pos is None else 0
                assert torch.equal(kp[at], ku.rotate32(c["k"][t:t + 1], angles[turn:turn + 1], False)[0].to(BF))
                assert torch.equal(vp[at], c["v"][t])


def test_staged_entries_of_a_tree():
    """The staged layout [B][LH][N][D] as pages of N rows: nodes rotated to their depths' positions."""
    rng = np.random.default_rng(8)
    B, N, Hq, Hkv, D, LH = 3, 7, 8, 2, 64, 6
    lens, depth = [40, 3, 0], rng.integers(0, 4, (B, N))
    pos = i32((np.array(lens)[:, None] + depth).reshape(-1))
    q, k, v = (normal(rng, B * N, h, D) for h in (Hq, Hkv, Hkv))
    kn, vn = (torch.full((B, LH, N, D), FILL, dtype=BF, device=DEV) for _ in "kv")
    table = ku.angles(64, D).float().to(DEV)
    qo = torch.empty_like(q)
    binding.sv_page_append(k, v, kn, vn, i32([[b] for b in range(B)]), i32([0] * B), i32(np.arange(B + 1) * N), table, pos,
                           q, qo, head0=4)
    cs = table[pos.long()]
    want = ku.rotate32(k, cs, False).to(BF).view(B, N, Hkv, D).transpose(1, 2)
    assert torch.equal(kn[:, 4:], want) and torch.equal(vn[:, 4:], v.view(B, N, Hkv, D).transpose(1, 2))
    assert bool((kn[:, :4] == FILL).all())
    ku.check_rotated(qo, q, cs, False)


def test_graph_replays_with_new_lengths_and_on_another_stream():
    """One captured append serves other lengths, bounds and tokens: nothing of the call is kept from the capture."""
    c = append_case(60, [0, 0, 0], [40, 40, 40], 4, 2, 64, 64, False, 16, BF)
    lens, cu = i32([0, 0, 0]), i32([0, 40, 80, 120])
    kp, vp, out, qo = c["kp"].clone(), c["vp"].clone(), i32([0] * 3), torch.empty_like(c["q"])
    args = (c["k"], c["v"], kp, vp, i32(c["table"]), lens, cu, c["angles"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.sv_page_append(*args, q=c["q"], q_out=qo, out_seq_lens=out)
    for new_lens, new_cu in (([0, 0, 0], [0, 40, 80, 120]), ([5, 17, 0], [0, 1, 20, 60])):
        lens.copy_(i32(new_lens))
        cu.copy_(i32(new_cu))
        kp.copy_(c["kp"])
        g.replay()
        kp2, vp2, out2, qo2 = c["kp"].clone(), vp.clone(), torch.empty_like(out), torch.empty_like(qo)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            binding.sv_page_append(*args[:2], kp2, vp2, *args[4:], q=c["q"], q_out=qo2, out_seq_lens=out2)
        torch.cuda.synchronize()
        assert torch.equal(kp, kp2) and out.tolist() == out2.tolist()
        n = new_cu[-1]
        assert torch.equal(qo[:n], qo2[:n])


def test_pages_past_32_bit_offsets():
    """A pool of more than 2^32 elements: pages at both ends."""
    P, LH, page, D = 9000, 4, 1024, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB")
    kp = torch.empty(P, LH, page, D, dtype=BF, device=DEV)
    vp = torch.empty_like(kp)
    assert kp.numel() > 1 << 32
    rng = np.random.default_rng(9)
    k, v = normal(rng, 4, LH, D), normal(rng, 4, LH, D)
    table = ku.angles(1100, D).float().to(DEV)
    binding.sv_page_append(k, v, kp, vp, i32([[P - 1, 0], [5, P - 2]]), i32([1022, 1024]), i32([0, 3, 4]), table)
    want = ku.rotate32(k, table[torch.tensor([1022, 1023, 1024, 1024], device=DEV)], False).to(BF)
    for t, (pg, row) in enumerate([(P - 1, 1022), (P - 1, 1023), (0, 0), (P - 2, 0)]):
        assert torch.equal(kp[pg, :, row], want[t]) and torch.equal(vp[pg, :, row], v[t])


@pytest.mark.parametrize("T,H,D,rot,inter,dtype", [(700, 3, 24, 16, True, BF), (3000, 3, 40, 32, True, HF), (1500, 7, 40, 16, False, BF),
                                                   (700, 2, 72, 16, True, HF), (5000, 1, 16, 6, True, BF), (40, 5, 256, 240, True, BF)])
def test_dimensions_behind_the_rotated_ones_keep_their_bits(T, H, D, rot, inter, dtype):
    """Whatever they hold (any bits: infinities and NaN too), whole and in vectors of which only a part is rotated."""
    rng = np.random.default_rng(D + rot)
    q = normal(rng, T, H, D, dtype=dtype)
    q.view(torch.int16)[..., rot:] = torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, (T, H, D - rot)).astype(np.int16)).to(DEV)
    table, pos = ku.angles(300, rot).float().to(DEV), i32(rng.integers(0, 300, T))
    out = torch.full_like(q, FILL)
    binding.sv_rope(q, None, pos, table, out, interleaved=inter)
    assert torch.equal(out.view(torch.int16)[..., rot:], q.view(torch.int16)[..., rot:])
    assert torch.equal(out[..., :rot], ku.rotate32(q, table[pos.long()], inter).to(dtype)[..., :rot])


@pytest.mark.parametrize("rot,rows", [(2, 70000), (6, 5000), (254, 3000), (256, 20000), (128, 40000)])
def test_table_rows_of_a_thread(rot, rows):
    """Several rows per thread, and threads that have no pair: the rows of two halves are those of the whole."""
    whole = torch.full((rows + 1, 2, rot // 2), FILL, device=DEV)
    binding.sv_rope_table(whole[:rows], base=5e5)
    part = torch.empty(rows - rows // 2, 2, rot // 2, device=DEV)
    binding.sv_rope_table(part, base=5e5, first=rows // 2)
    assert torch.equal(whole[rows // 2:rows], part) and bool((whole[rows] == FILL).all())
    # as in test_table: 2^-22 for the functions, and some 2^-50 of an angle on either side
    off = (whole[:rows].double().cpu() - ku.angles(rows, rot, base=5e5)).abs().max()
    assert off <= 2.0 ** -22 + rows * 2.0 ** -49


def test_queries_and_keys_of_other_ranks_are_refused():
    x = torch.zeros(4, 1, 8, dtype=BF, device=DEV)
    flat, table, pages = torch.zeros(32, dtype=BF, device=DEV), ku.angles(4, 8).float().to(DEV), torch.zeros(1, 1, 8, 8, dtype=BF, device=DEV)
    for bad in (flat, x[0], x[None], x[:, :, :0], x[:3]):
        with pytest.raises(binding.SpecVerifyError):
            binding.sv_rope(x, bad, i32([0] * 4), table, x, bad)
        with pytest.raises(binding.SpecVerifyError):
            binding.sv_page_append(x, x, pages, pages.clone(), i32([[0]]), i32([0]), i32([0, 4]), table, q=bad, q_out=bad)
        with pytest.raises(binding.SpecVerifyError):
            binding.sv_page_append(x, bad, pages, pages.clone(), i32([[0]]), i32([0]), i32([0, 4]), table)
