"""Rotary positions and the 8-bit paged cache: what is measured of them.

Five operators: the table of rotation angles, scaled for long contexts (`table`), rotating queries and keys (`rope`),
appending keys and values to a paged cache with the rotation on the way (`append`), writing into a cache held in 8 bits
with a scale for each block of tokens and head (`write8`: packed tokens, or a verified path of staged ones) and the
attention of drafted trees over it (`attn8`).  A case is a dict of sizes; `prepare` makes its inputs on the GPU, `run`
makes one pass: in plain torch operations, or through the library where `own` is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LIMITS = {"bf16": (-117, 119), "fp16": (-15, 7)}  # a block's exponent: what the type holds exactly
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def listed():
    return [
        # the angles of a small draft model's context, part of its heads rotated
        dict(name="table_short", op="table", count=4096, rot=32, base=10000.0, scaling="none", factor=1.0, original=0),
        # those of a long context, stretched 32 times over the trained one, low frequencies interpolated
        dict(name="table_long", op="table", count=131072, rot=128, base=500000.0, scaling="ramp", factor=32.0,
             original=4096),
        # one user's tree of 22 nodes before its attention
        dict(name="rope_tree", op="rope", T=22, Hq=32, Hk=8, D=128, rot=128, inter=False, span=9000, dtype="bf16"),
        # a long prompt, the layout with neighbours as pairs, half of the head rotated
        dict(name="rope_prompt", op="rope", T=8192, Hq=32, Hk=8, D=128, rot=64, inter=True, span=8192, dtype="fp16"),
        # a decoding step of a serving batch: one token each, queries rotated in the same call
        dict(name="append_step", op="append", B=64, n_lo=1, n_hi=1, lo=1, hi=900, Hq=32, Hkv=8, D=128, rot=128,
             inter=False, page=16, dtype="bf16"),
        # ragged prompts into empty pages, queries and keys rotated for the attention that follows
        dict(name="append_prompts", op="append", B=24, n_lo=1, n_hi=1500, lo=0, hi=0, Hq=32, Hkv=8, D=128, rot=128,
             inter=False, page=64, dtype="bf16"),
        # one token each of a batch into 8-bit pages, most of them inside a block that has entries
        dict(name="append8_step", op="write8", path=False, B=64, n_lo=1, n_hi=1, lo=1, hi=900, Hkv=8, D=128, rot=128,
             inter=False, page=32, block=16, dtype="bf16"),
        # ragged prompts into 8-bit pages, some behind a cached prefix
        dict(name="append8_prompts", op="write8", path=False, B=32, n_lo=0, n_hi=5000, lo=0, hi=100, Hkv=8, D=128,
             rot=128, inter=False, page=64, block=32, dtype="bf16"),
        # a batch's verified paths for every layer and head of a 24-layer, 16-head target
        dict(name="commit8_batch", op="write8", path=True, B=64, N=22, LH=384, lo=1, hi=47, D=128, page=16, block=16,
             dtype="bf16"),
        # one token of one user after a short prompt: the latency of a decoding step
        dict(name="attn8_one_token", op="attn8", B=1, N=1, Hq=16, Hkv=16, D=128, page=16, block=16, lo=500, hi=500,
             dtype="bf16"),
        # a serving batch verifying trees of 22 nodes, ragged contexts, grouped heads
        dict(name="attn8_batch", op="attn8", B=64, N=22, Hq=32, Hkv=8, D=128, page=128, block=32, lo=2000, hi=9000,
             dtype="bf16"),
        # long contexts, a wide tree of odd size, small pages and 16-bit IEEE floats
        dict(name="attn8_long", op="attn8", B=4, N=61, Hq=28, Hkv=4, D=64, page=16, block=16, lo=20000, hi=32768,
             dtype="fp16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["table", "rope", "append", "write8", "write8", "write8", "attn8", "attn8", "attn8"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "table":
        scaling = rng.choice(["none", "linear", "base", "ramp", "wave"])
        return dict(op=op, count=_spread(rng, 1, 131072), rot=2 * rng.randint(2, 64),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                    original=rng.choice([2048, 4096, 8192]))
    Hkv, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    while Hkv * G > 32:
        G = rng.choice([1, 2, 3, 4])
        Hkv = min(Hkv, 8)
    if op == "rope":
        D = rng.choice([64, 128, 80, 96, 40])
        return dict(op=op, T=_spread(rng, 1, 8192), Hq=Hkv * G, Hk=Hkv, D=D, rot=rng.choice([D, D // 2, D // 4 * 2 - 2]),
                    inter=rng.random() < 0.5, span=_spread(rng, 1, 32768), dtype=dtype)
    if op == "append":
        D = rng.choice([64, 128, 80, 96, 40])
        B = _spread(rng, 1, 64)
        return dict(op=op, B=B, n_lo=rng.choice([0, 1]), n_hi=_spread(rng, 1, 16000 // B), lo=0,
                    hi=rng.choice([0, 50, 1000]), Hq=Hkv * G, Hkv=Hkv, D=D, rot=rng.choice([D, D // 2]),
                    inter=rng.random() < 0.5, page=rng.choice([1, 8, 16, 24, 64]), dtype=dtype)
    D = rng.choice([64, 128, 128, 80, 96, 32])
    page, block = rng.choice([(8, 8), (16, 8), (16, 16), (24, 8), (32, 16), (64, 32), (64, 64), (128, 16), (128, 128),
                              (256, 64)])
    if op == "write8":
        if rng.random() < 0.4:
            return dict(op=op, path=True, B=_spread(rng, 1, 64), N=_spread(rng, 1, 128), LH=_spread(rng, 1, 256), lo=0,
                        hi=_spread(rng, 1, 100), D=D, page=page, block=block, dtype=dtype)
        B = _spread(rng, 1, 64)
        return dict(op=op, path=False, B=B, n_lo=rng.choice([0, 1]), n_hi=_spread(rng, 1, 60000 // B), lo=0,
                    hi=rng.choice([0, 50, 1000]), Hkv=Hkv, D=D, rot=rng.choice([D, D // 2, 0]),
                    inter=rng.random() < 0.5, page=page, block=block, dtype=dtype)
    N = _spread(rng, 1, 256)
    B = _spread(rng, 1, 64)
    hi = _spread(rng, 1, max(1, min(32768, (1 << 17) // B, (1 << 23) // (B * N))))
    return dict(op=op, B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, block=block, lo=rng.choice([0, hi // 3, hi]),
                hi=hi, dtype=dtype)


# ------------------------------------------------------------------ inputs

def _lens(lo, hi, count, what):
    """Ragged lengths, the same for every seed's sizes: the first the longest, so that a case's work is known."""
    rng = random.Random("%s %d %d %d" % (what, lo, hi, count))
    out = [rng.randint(lo, hi) for _ in range(count)]
    out[0] = hi
    return out


def _parents(N, rng):
    """A tree of N nodes in index order: each node hangs below one of the last few before it."""
    return [-1] + [rng.randint(max(0, n - 1 - rng.choice([0, 2, 5])), n - 1) for n in range(1, N)]


def _path(parent, rng):
    """Nodes accepted below the root: a walk down from it that ends early half of the time."""
    path, at = [], 0
    while rng.random() < 0.8:
        below = [n for n in range(at + 1, len(parent)) if parent[n] == at]
        if not below:
            break
        at = rng.choice(below)
        path.append(at)
    return path


def _angles(count, rot, base=10000.0):
    """The table that such a program keeps: [count][2][rot / 2], cosines and sines."""
    w = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(1, rot))
    a = torch.arange(count, dtype=torch.float64, device="cuda")[:, None] * w[None]
    return torch.stack([a.cos(), a.sin()], 1).float()


def _power(e):
    """2^e in 32 bits, exactly (0 and below: 2^-126 at the least)."""
    return ((e.int().clamp(min=-126) + 127) << 23).view(torch.float32)


def _pages(rows, total, page, D, block, gen, limits):
    """A used 8-bit cache: entries of blocks whose sizes differ, at the exponents that these ask for."""
    nb = page // block
    x = torch.empty(total, rows, nb, block, D, dtype=torch.bfloat16, device="cuda").normal_(0.0, 1.0, generator=gen)
    by = torch.randint(-2, 3, (total, rows, nb, 1, 1), device="cuda", generator=gen)
    x *= _power(by).to(x.dtype)
    e = _exponent(x.abs().amax((-1, -2)).float(), *limits)
    # (bf16 times a power of two is exact; the type's conversion rounds once)
    x *= _power(-e)[..., None, None].to(x.dtype)
    return x.to(E4M3).reshape(total, rows, page, D), (e + 127).to(torch.uint8).view(E8M0)


def _inputs(case, seed):
    """The case's inputs as a dict of tensors on the GPU, from the seed alone."""
    op, dev = case["op"], "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    if op == "table":  # (a window of positions: another seed, other positions)
        return dict(first=rng.randrange(0, 1000))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, by=1.0):
        return torch.empty(*shape, dtype=dt, device=dev).normal_(0.0, by, generator=gen)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def tables(lens, more, page):
        """A block table with room for `more` tokens behind the cached ones, the pages in no order; and their number."""
        room = [-(-(n + m) // page) for n, m in zip(lens, more)]
        cols, pages = max(1, max(room)), sum(room) + 3
        free = list(range(pages))
        rng.shuffle(free)
        return ints([[free.pop() for _ in range(r)] + [0] * (cols - r) for r in room]), pages

    D = case["D"]
    if op == "rope":
        T = case["T"]
        pos = torch.randint(0, case["span"], (T,), device=dev, generator=gen, dtype=torch.int32)
        return dict(q=normal(T, case["Hq"], D, by=2.0), k=normal(T, case["Hk"], D), positions=pos,
                    table=_angles(case["span"], case["rot"]))
    B = case["B"]
    lens = _lens(case["lo"], case["hi"], B, "cached")
    page = case["page"]
    if op == "attn8":
        N, Hkv, block = case["N"], case["Hkv"], case["block"]
        table, total = tables(lens, [0] * B, page)
        s = dict(q=normal(B, N, case["Hq"], D, by=2.0), k_new=normal(B, Hkv, N, D), v_new=normal(B, Hkv, N, D),
                 block_table=table, seq_lens=ints(lens), parent=ints([_parents(N, rng) for _ in range(B)]))
        for x in "kv":
            s[x + "_pages"], s[x + "_scales"] = _pages(Hkv, total, page, D, block, gen, LIMITS[case["dtype"]])
        return s
    if op == "write8" and case["path"]:
        N, LH = case["N"], case["LH"]
        table, total = tables(lens, [N] * B, page)
        paths = [_path(_parents(N, rng), rng) for _ in range(B)]
        s = dict(k_new=normal(B, LH, N, D), v_new=normal(B, LH, N, D), block_table=table, seq_lens=ints(lens),
                 nodes=ints([p + [-1] * (N - len(p)) for p in paths]), num_accepted=ints([len(p) for p in paths]))
    else:
        more, LH = _lens(case["n_lo"], case["n_hi"], B, "new"), case["Hkv"]
        ends = [0]
        for n in more:
            ends.append(ends[-1] + n)
        table, total = tables(lens, more, page)
        s = dict(k=normal(ends[-1], LH, D), v=normal(ends[-1], LH, D), block_table=table, seq_lens=ints(lens),
                 cu_seqlens=ints(ends), table=_angles(max(a + b for a, b in zip(lens, more)), case["rot"]))
        if op == "append":
            s["q"] = normal(ends[-1], case["Hq"], D, by=2.0)
            for x in "kv":
                s[x + "_pages"] = normal(total, LH, page, D)
            return s
    for x in "kv":
        s[x + "_pages"], s[x + "_scales"] = _pages(LH, total, page, D, case["block"], gen, LIMITS[case["dtype"]])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "table":
        s["out"] = torch.empty(case["count"], 2, case["rot"] // 2, device="cuda")
    elif case["op"] == "attn8":
        s["out"] = torch.empty_like(s["q"])
    else:
        for x in "qk":
            if x in s and case["op"] != "write8":
                s[x + "_out"] = torch.empty_like(s[x])
        if "seq_lens" in s:
            s["out_seq_lens"] = torch.empty_like(s["seq_lens"])
    return s


# ------------------------------------------------------------------ the library's calls

def _run_own(s):
    from speculative_decoding_verification_09_gb300 import binding
    c = s["case"]
    op = c["op"]
    if op == "table":
        low, high = (1.0, 32.0) if c["scaling"] == "ramp" else (1.0, 4.0)
        binding.sv_rope_table(s["out"], c["base"], getattr(binding, "SV_ROPE_" + c["scaling"].upper()), c["factor"],
                              c["original"], low, high, first=s["first"])
        return s["out"]
    if op == "rope":
        binding.sv_rope(s["q"], s["k"], s["positions"], s["table"], s["q_out"], s["k_out"], interleaved=c["inter"])
        return s["q_out"], s["k_out"]
    if op == "append":
        binding.sv_page_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"],
                               s["cu_seqlens"], s["table"], q=s["q"], q_out=s["q_out"], k_out=s["k_out"],
                               out_seq_lens=s["out_seq_lens"], interleaved=c["inter"])
        return s["q_out"], s["k_out"], s["k_pages"], s["v_pages"], s["out_seq_lens"]
    if op == "write8":
        if c["path"]:
            binding.sv_page_commit8(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["k_new"], s["v_new"],
                                    s["block_table"], s["seq_lens"], s["nodes"], s["num_accepted"], s["out_seq_lens"])
        else:
            binding.sv_page_append8(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                                    s["block_table"], s["seq_lens"], s["cu_seqlens"],
                                    s["table"] if c["rot"] else None, out_seq_lens=s["out_seq_lens"],
                                    interleaved=c["inter"])
        return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["out_seq_lens"]
    if "workspace" not in s:
        s["workspace"] = binding.make_attn_workspace(c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], s["q"].device)
    binding.sv_tree_attn8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["block_table"],
                          s["seq_lens"], s["k_new"], s["v_new"], s["parent"], s["out"], s["workspace"])
    return s["out"]


# ------------------------------------------------------------------ the plain form

def _frequencies(c):
    """The angles' rates, one for each pair, in 64 bits."""
    rot, base, factor = c["rot"], c["base"], c["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    w = base ** (-2 * i / rot)
    if c["scaling"] == "linear":
        return w / factor
    if c["scaling"] == "base":
        return (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
    if c["scaling"] == "ramp":  # pairs that turn more than 32 times over the original context stay, below once: all / factor
        at = [rot * math.log(c["original"] / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        part = ((i - lo) / (hi - lo if hi != lo else 0.001)).clamp(0, 1)
        return w / factor * part + w * (1 - part)
    if c["scaling"] == "wave":  # by the wavelength against the original context: kept below 1/4 of it, / factor above it
        turns = c["original"] * w / (2 * math.pi)
        part = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return w / factor * (1 - part) + w * part
    return w


def _rotate(x, cs, inter):
    """x [T][H][D] in 32 bits, cs [T][2][rot / 2]: its first rot dimensions turned."""
    half = cs.shape[2]
    if not half:
        return x
    cos, sin = cs[:, None, 0], cs[:, None, 1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if inter else (x[..., :half], x[..., half:2 * half])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([lo, hi], -1).flatten(-2) if inter else torch.cat([lo, hi], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _exponent(amax, least, most):
    """The smallest e with amax <= 448 * 2^e, within the type's range."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).int()
    return torch.where(amax > 0, e, torch.full_like(e, least)).clamp(least, most)


def _places(s, page):
    """(request, position) of every packed token."""
    cu = s["cu_seqlens"].long()
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    at = s["seq_lens"].long()[b] + t - cu[b]
    return b, at


def _write8(pages, scales, x, b, at, table, lens, block, limits):
    """Entries x [n][rows][D] (32 bits) of requests b at positions `at` into 8-bit pages, block scales raised on the way."""
    P, rows, page, D = pages.shape
    nb = page // block
    # bytes [blocks of all pages][rows][block][D] would need a copy: blocks stay addressed as (page, row, block)
    bytes_ = pages.view(torch.uint8).view(P, rows, nb, block, D)
    held = scales.view(torch.uint8)
    pg, blk, row = table[b, at // page], at % page // block, at % block
    flat = pg * nb + blk
    most = torch.zeros(P * nb, rows, device="cuda")
    most.scatter_reduce_(0, flat[:, None].expand(-1, rows), x.abs().amax(-1), "amax")
    e = _exponent(most, *limits).view(P, nb, rows).transpose(1, 2)
    # blocks that hold entries already: those of each request's first new position, when it is not a block's first
    count = torch.zeros(lens.shape[0], dtype=torch.long, device="cuda").scatter_add_(0, b, torch.ones_like(b))
    first = (lens % block != 0) & (count > 0)
    q, n = first.nonzero(as_tuple=True)[0], lens[first]
    fp, fb = table[q, n // page], n % page // block
    old = held[fp, :, fb].int() - 127
    now = torch.maximum(old, e[fp, :, fb])
    e[fp, :, fb] = now
    entries = bytes_[fp, :, fb]
    again = (entries.view(E4M3).float() * _power(old - now)[..., None, None]).to(E4M3).view(torch.uint8)
    keep = torch.arange(block, device="cuda")[None] < (n % block)[:, None]
    bytes_[fp, :, fb] = torch.where(keep[:, None, :, None], again, entries)
    new = (x * _power(-e[pg, :, blk])[..., None]).clamp(-448, 448)
    bytes_[pg, :, blk, row] = new.to(E4M3).view(torch.uint8)
    held[pg, :, blk] = (e[pg, :, blk] + 127).to(torch.uint8)


def _ancestors(parent):
    """[B][N][N] truth values: whether m is n or above it in n's tree (the reach of the parent edge, doubled each step)."""
    B, N = parent.shape
    reach = torch.eye(N, dtype=torch.float32, device=parent.device).repeat(B, 1, 1)
    step = torch.zeros_like(reach)
    step.scatter_(2, parent.clamp(min=0).long()[:, :, None], (parent >= 0).float()[:, :, None])
    step = ((step + reach) > 0).float()
    for _ in range(max(1, (N - 1).bit_length())):
        step = ((step @ step) > 0).float()
    return step > 0


def _values(pages, scales, table):
    """What the 8-bit pages of a table hold, [B][rows][cols * page][D] in 32 bits."""
    B, cols = table.shape
    P, rows, page, D = pages.shape
    x = pages.view(torch.uint8)[table].view(E4M3).float()
    by = _power(scales.view(torch.uint8)[table].int() - 127)
    x = x.view(B, cols, rows, by.shape[-1], -1, D) * by[..., None, None]
    return x.view(B, cols, rows, page, D).transpose(1, 2).reshape(B, rows, cols * page, D)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "table":
        at = torch.arange(s["first"], s["first"] + c["count"], dtype=torch.float64, device="cuda")
        a = at[:, None] * _frequencies(c)[None]
        return torch.stack([a.cos(), a.sin()], 1).float()
    if op == "rope":
        cs = s["table"][s["positions"].long()]
        return tuple(_rotate(s[x].float(), cs, c["inter"]).to(s[x].dtype) for x in "qk")
    if op == "append":
        b, at = _places(s, c["page"])
        cs, where, row = s["table"][at], s["block_table"].long()[b, at // c["page"]], at % c["page"]
        q, k = (_rotate(s[x].float(), cs, c["inter"]).to(s[x].dtype) for x in "qk")
        s["k_pages"][where, :, row] = k
        s["v_pages"][where, :, row] = s["v"]
        s["out_seq_lens"].copy_(s["seq_lens"] + s["cu_seqlens"][1:] - s["cu_seqlens"][:-1])
        return q, k, s["k_pages"], s["v_pages"], s["out_seq_lens"]
    if op == "write8":
        table, lens, limits = s["block_table"].long(), s["seq_lens"].long(), LIMITS[c["dtype"]]
        if c["path"]:
            N = c["N"]
            j = torch.arange(N, device="cuda")
            # entry 0 is the root, entry j the j-th accepted node
            node = torch.cat([torch.zeros_like(s["nodes"][:, :1]), s["nodes"][:, :-1]], 1).long()
            b, j = (j[None] <= s["num_accepted"][:, None]).nonzero(as_tuple=True)
            at, node = lens[b] + j, node[b, j]
            k, v = s["k_new"][b, :, node].float(), s["v_new"][b, :, node].float()
            s["out_seq_lens"].copy_(s["seq_lens"] + s["num_accepted"] + 1)
        else:
            b, at = _places(s, c["page"])
            k, v = _rotate(s["k"].float(), s["table"][at], c["inter"]), s["v"].float()
            s["out_seq_lens"].copy_(s["seq_lens"] + s["cu_seqlens"][1:] - s["cu_seqlens"][:-1])
        _write8(s["k_pages"], s["k_scales"], k, b, at, table, lens, c["block"], limits)
        _write8(s["v_pages"], s["v_scales"], v, b, at, table, lens, c["block"], limits)
        return s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["out_seq_lens"]
    B, N, Hq, Hkv, D = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"]
    table = s["block_table"].long()
    k = torch.cat([_values(s["k_pages"], s["k_scales"], table), s["k_new"].float()], 2)
    v = torch.cat([_values(s["v_pages"], s["v_scales"], table), s["v_new"].float()], 2)
    L = k.shape[2]
    inside = (torch.arange(L - N, device="cuda")[None] < s["seq_lens"][:, None])[:, None].expand(B, N, L - N)
    seen = torch.cat([inside, _ancestors(s["parent"])], 2)
    G = Hq // Hkv
    rows = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    scores = (rows * D ** -0.5) @ k.transpose(-1, -2)
    scores.masked_fill_(~seen[:, None, :, None, :].expand(B, 1, N, G, L).reshape(B, 1, N * G, L), float("-inf"))
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    out = (scores @ v) / scores.sum(-1, keepdim=True)
    return out.view(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(s["q"].dtype)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work, and the definition in 64 bits

def work(case):
    op = case["op"]
    if op == "table":
        n = case["count"] * case["rot"]
        return {"bytes": 4 * n, "flops": 40 * n}
    D = case["D"]
    if op == "rope":
        rows = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 4 * rows * D + 4 * case["T"] + 4 * case["rot"] * min(case["T"], case["span"]),
                "flops": 3 * rows * case["rot"]}
    B = case["B"]
    if op == "attn8":
        N, Hq, Hkv = case["N"], case["Hq"], case["Hkv"]
        total = sum(_lens(case["lo"], case["hi"], B, "cached"))
        return {"bytes": 2 * Hkv * total * D + 2 * Hkv * total // case["block"] + 4 * Hkv * D * B * N
                + 4 * B * N * Hq * D + 4 * B * (N + 1),
                "flops": 4 * Hq * D * N * (total + B * (N + 1) // 2)}
    if op == "write8" and case["path"]:
        kept = B * min(case["N"], 4)
        return {"bytes": 6 * kept * case["LH"] * D + 16 * B, "flops": 4 * kept * case["LH"] * D}
    T = sum(_lens(case["n_lo"], case["n_hi"], B, "new"))
    if op == "append":  # keys to two places
        return {"bytes": T * D * (10 * case["Hkv"] + 4 * case["Hq"]) + 4 * case["rot"] * T + 16 * B,
                "flops": 3 * T * (case["Hkv"] + case["Hq"]) * case["rot"]}
    return {"bytes": 6 * T * case["Hkv"] * D + 4 * case["rot"] * T + 16 * B,
            "flops": 3 * T * case["Hkv"] * case["rot"] + 4 * T * case["Hkv"] * D}


def _exact_turn(x, cs, inter):
    """x [n][H][D], cs [n][2][half]: the rotation in 64 bits, dimension by dimension as complex products."""
    half = cs.shape[2]
    y = x.double().clone()
    lo = torch.arange(half, device="cuda") * (2 if inter else 1)
    hi = lo + (1 if inter else half)
    z = torch.complex(y[..., lo], y[..., hi]) * torch.complex(cs[:, None, 0].double(), cs[:, None, 1].double())
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _wide_power(e):
    """2^e in 64 bits, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _to_e4m3(x):
    """64-bit values to the nearest ones of the 8-bit format, ties to even: steps of 2^-3 of the binade, 2^-9 at least."""
    step = _wide_power(torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 4)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits, request by request."""
    s, op = _inputs(case, seed), case["op"]
    if op == "table":
        rot, base, f, n0 = case["rot"], case["base"], case["factor"], case["original"]
        rates = []
        for i in range(rot // 2):
            w = math.exp(-2 * i / rot * math.log(base))
            if case["scaling"] == "linear":
                w /= f
            elif case["scaling"] == "base":
                w = math.exp(-2 * i / rot * (math.log(base) + rot / (rot - 2) * math.log(f)))
            elif case["scaling"] == "ramp":
                dim = [rot * math.log(n0 / (2 * math.pi * t)) / (2 * math.log(base)) for t in (32, 1)]
                lo, hi = max(math.floor(dim[0]), 0), min(math.ceil(dim[1]), rot - 1)
                far = min(1.0, max(0.0, (i - lo) / ((hi - lo) or 0.001)))
                w = (1 - far) * w + far * w / f
            elif case["scaling"] == "wave":
                length = 2 * math.pi / w
                if length > n0:
                    w /= f
                elif length > n0 / 4:
                    near = (n0 / length - 1) / 3
                    w = (1 - near) * w / f + near * w
            rates.append(w)
        a = torch.outer(torch.arange(case["count"], dtype=torch.float64, device="cuda") + s["first"],
                        torch.tensor(rates, dtype=torch.float64, device="cuda"))
        return torch.stack([torch.cos(a), torch.sin(a)], 1)
    lists = {n: s[n].tolist() for n in ("block_table", "seq_lens", "parent", "cu_seqlens", "nodes", "num_accepted") if n in s}
    if op == "rope":
        cs = s["table"].index_select(0, s["positions"])
        return _exact_turn(s["q"], cs, case["inter"]), _exact_turn(s["k"], cs, case["inter"])
    page = case["page"]
    if op == "append":
        q, k, v = torch.empty_like(s["q"], dtype=torch.float64), torch.empty_like(s["k"], dtype=torch.float64), s["v"].double()
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        for b, n in enumerate(lists["seq_lens"]):
            a, e = lists["cu_seqlens"][b:b + 2]
            cs = s["table"][n:n + e - a]
            q[a:e], k[a:e] = _exact_turn(s["q"][a:e], cs, case["inter"]), _exact_turn(s["k"][a:e], cs, case["inter"])
            done = 0
            while done < e - a:  # page by page
                p, r = divmod(n + done, page)
                m = min(page - r, e - a - done)
                for pool, x in ((kp, k), (vp, v)):
                    pool[lists["block_table"][b][p], :, r:r + m] = x[a + done:a + done + m].transpose(0, 1)
                done += m
        return q, k, kp, vp, None
    if op == "write8":
        block, (least, most) = case["block"], LIMITS[case["dtype"]]
        if not case["path"] and s["k"].shape[0] // block > 8000:
            return None  # block by block it would take long
        got = []
        for x in "kv":
            pool = s[x + "_pages"].double()
            by = s[x + "_scales"].view(torch.uint8).long() - 127
            for b, n in enumerate(lists["seq_lens"]):
                if case["path"]:
                    path = [0] + lists["nodes"][b][:lists["num_accepted"][b]]
                    new = s[x + "_new"][b][:, path].double()
                else:
                    a, e = lists["cu_seqlens"][b:b + 2]
                    new = s[x][a:e]
                    new = _exact_turn(new, s["table"][n:n + e - a], case["inter"]) if x == "k" else new.double()
                    new = new.transpose(0, 1)
                done = 0
                while done < new.shape[1]:
                    p, r = divmod(n + done, page)
                    j, first = divmod(r, block)
                    part = new[:, done:done + block - first]
                    where = lists["block_table"][b][p]
                    peak = part.abs().amax((1, 2))
                    above = torch.frexp(peak / 448)
                    e2 = above.exponent.long() - (above.mantissa == 0.5).long()
                    e2 = torch.where(peak > 0, e2, least).clamp(least, most)
                    rows = pool[where, :, j * block:(j + 1) * block]
                    if first:
                        was = by[where, :, j]
                        e2 = torch.maximum(e2, was)
                        rows[:, :first] = _to_e4m3(rows[:, :first] * _wide_power(was - e2)[:, None, None])
                    rows[:, first:first + part.shape[1]] = _to_e4m3(part * _wide_power(-e2)[:, None, None])
                    by[where, :, j] = e2
                    done += part.shape[1]
            got.append((pool, _wide_power(by)))
        return got[0][0], got[1][0], got[0][1], got[1][1], None
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    N, G, block = case["N"], case["Hq"] // case["Hkv"], case["block"]
    for b, n in enumerate(lists["seq_lens"]):
        ids = torch.tensor(lists["block_table"][b][:-(-n // page)], dtype=torch.long, device="cuda")
        tree = torch.zeros(N, N, dtype=torch.bool)
        for m in range(N):
            at = m
            while at >= 0:
                tree[m, at] = True
                at = lists["parent"][b][at]
        visible = torch.cat([torch.ones(N, n, dtype=torch.bool), tree], 1).cuda()
        for h in range(case["Hkv"]):
            both = []
            for x in "kv":
                cached = s[x + "_pages"].view(torch.uint8)[ids, h].view(E4M3).double().reshape(-1, case["D"])
                e = s[x + "_scales"].view(torch.uint8)[ids, h].reshape(-1).long() - 127
                cached = cached * _wide_power(e).repeat_interleave(block)[:, None]
                both.append(torch.cat([cached[:n], s[x + "_new"][b, h].double()]))
            for g in range(h * G, (h + 1) * G):
                w = s["q"][b, :, g].double() @ both[0].T / math.sqrt(case["D"])
                w = torch.where(visible, w, torch.full_like(w, -math.inf))
                out[b, :, g] = torch.softmax(w, dim=1) @ both[1]
    return out
