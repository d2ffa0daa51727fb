"""Attention over the caches of speculative decoding, and the cache steps beside it: what is measured of them.

Five operators: attention of a drafted token tree over a paged cache (`tree`), attention of the newest tokens over a
sink + ring cache (`ring`), attention of whole prompts with a sliding window and sinks (`prompt`), writing a verified
path into the pages (`commit`) and loading prompts into the ring (`fill`).  A case is a dict of sizes; `prepare` makes
its inputs on the GPU, `run` makes one pass: in plain torch operations, or through the library where `own` is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one token of one user after a short prompt: the latency of a plain decoding step over pages of 16
        dict(name="tree_one_token", op="tree", B=1, N=1, Hq=16, Hkv=16, D=128, page=16, lo=500, hi=500, dtype="bf16"),
        # a serving batch verifying trees of 22 nodes (branching 3-2-2 below the root), ragged contexts, grouped heads
        dict(name="tree_batch", op="tree", B=64, N=22, Hq=32, Hkv=8, D=128, page=128, lo=2000, hi=9000, dtype="bf16"),
        # long contexts, a wide tree of odd size, small pages and 16-bit floats
        dict(name="tree_long", op="tree", B=4, N=61, Hq=28, Hkv=4, D=64, page=16, lo=20000, hi=32768, dtype="fp16"),
        # one stream on an edge cache: 4 sinks and a ring of 64
        dict(name="ring_one_token", op="ring", B=1, R=1, Hq=16, Hkv=16, D=128, S=4, W=64, lo=300, hi=300, dtype="bf16"),
        # verification of 7 drafts for 32 requests over rings of 2048
        dict(name="ring_batch", op="ring", B=32, R=8, Hq=32, Hkv=8, D=128, S=4, W=2048, lo=100, hi=9000, dtype="bf16"),
        # the largest batch: 1024 requests, 3 drafts, an odd ring and head size
        dict(name="ring_wide", op="ring", B=1024, R=4, Hq=12, Hkv=4, D=80, S=3, W=509, lo=0, hi=3000, dtype="fp16"),
        # a batch of ragged prompts, some of a few tokens, grouped heads of 64
        dict(name="prompt_ragged", op="prompt", n=24, lo=1, hi=1500, Hq=16, Hkv=4, D=64, S=4, W=512, dtype="fp16"),
        # one long prompt under a window of half its length
        dict(name="prompt_long", op="prompt", n=1, lo=8192, hi=8192, Hq=32, Hkv=8, D=128, S=4, W=4096, dtype="bf16"),
        # one user's tree path into the pages, a small draft model's rows
        dict(name="commit_one", op="commit", B=1, N=22, LH=32, D=128, page=16, lo=700, hi=700, chain=False, dtype="bf16"),
        # a batch's paths for every layer and head of a 24-layer, 16-head target
        dict(name="commit_batch", op="commit", B=64, N=22, LH=384, D=128, page=16, lo=1, hi=47, chain=False, dtype="bf16"),
        # one short prompt into an edge cache
        dict(name="fill_one", op="fill", n=1, lo=300, hi=300, Hkv=16, D=128, S=4, W=64, dtype="bf16"),
        # ragged prompts into rings of 2048, longer and shorter than the ring
        dict(name="fill_batch", op="fill", n=32, lo=0, hi=5000, Hkv=8, D=128, S=4, W=2048, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "ring", "ring", "prompt", "prompt", "commit", "fill"])
    dtype = rng.choice(["bf16", "fp16"])
    Hkv, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    while Hkv * G > 32:
        G = rng.choice([1, 2, 3, 4])
        Hkv = min(Hkv, 8)
    D = rng.choice([64, 128, 128, 80, 96, 40])
    if op == "tree":
        N = _spread(rng, 1, 256)
        B = _spread(rng, 1, 64)
        hi = _spread(rng, 1, max(1, min(32768, (1 << 17) // B, (1 << 23) // (B * N))))
        return dict(op=op, B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([8, 16, 24, 32, 64, 128, 256]),
                    lo=rng.choice([0, hi // 3, hi]), hi=hi, dtype=dtype)
    if op == "ring":
        B, R, S = _spread(rng, 1, 1024), _spread(rng, 1, 64), rng.choice([0, 1, 4, 7, 64])
        W = max(R, _spread(rng, 16, max(16, min(8192, (1 << 17) // B))))
        while B * R * W > 1 << 24:
            R = (R + 1) // 2
            B = (B + 1) // 2
        return dict(op=op, B=B, R=R, Hq=Hkv * G, Hkv=Hkv, D=D, S=S, W=W, lo=0, hi=rng.choice([W // 2, W + S, 3 * W]),
                    dtype=dtype)
    if op == "prompt":
        n = _spread(rng, 1, 48)
        hi = _spread(rng, 1, 6000 // n)
        return dict(op=op, n=n, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D,
                    S=rng.choice([0, 1, 4, 30, 130]), W=_spread(rng, 1, 8192), dtype=dtype)
    if op == "commit":
        page = rng.choice([1, 8, 16, 24, 64])
        return dict(op=op, B=_spread(rng, 1, 64), N=_spread(rng, 1, 128), LH=_spread(rng, 1, 256), D=D, page=page,
                    lo=0, hi=_spread(rng, 1, 100), chain=rng.random() < 0.4, dtype=dtype)
    n = _spread(rng, 1, 64)
    return dict(op=op, n=n, lo=0, hi=_spread(rng, 1, 60000 // n), Hkv=Hkv, D=D, S=rng.choice([0, 1, 4, 33]),
                W=_spread(rng, 8, 4096), dtype=dtype)


# ------------------------------------------------------------------ inputs

def _lens(case, count, seed):
    """Ragged lengths, the same for every seed's sizes: the first the longest, so that a case's work is known."""
    rng = random.Random("%d %d %d" % (case["lo"], case["hi"], count))
    out = [rng.randint(case["lo"], case["hi"]) for _ in range(count)]
    out[0] = case["hi"]
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


def _inputs(case, seed):
    """The case's inputs as a dict of tensors on the GPU, from the seed alone."""
    dev, dt, op = "cuda", DTYPES[case["dtype"]], case["op"]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape, by=1.0):
        return torch.empty(*shape, dtype=dt, device=dev).normal_(0.0, by, generator=gen)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    if op in ("tree", "commit"):
        B, N, D, page = case["B"], case["N"], case["D"], case["page"]
        rows = case["Hkv"] if op == "tree" else case["LH"]
        lens = _lens(case, B, seed)
        room = [-(-(n + (N if op == "commit" else 0)) // page) for n in lens]  # a commit's pages are there before it
        cols, pages = max(1, max(room)), sum(room) + 3
        free = list(range(pages))
        rng.shuffle(free)
        table = [[free.pop() for _ in range(r)] + [0] * (cols - r) for r in room]
        s = dict(k_pages=normal(pages, rows, page, D), v_pages=normal(pages, rows, page, D),
                 k_new=normal(B, rows, N, D), v_new=normal(B, rows, N, D), block_table=ints(table), seq_lens=ints(lens))
        parents = [_parents(N, rng) for _ in range(B)]
        if op == "tree":
            s["q"] = normal(B, N, case["Hq"], D, by=2.0)
            s["parent"] = ints(parents)
        elif case["chain"]:
            s["num_accepted"] = ints([rng.randint(0, N - 1) for _ in range(B)])
        else:
            paths = [_path(p, rng) for p in parents]
            s["num_accepted"] = ints([len(p) for p in paths])
            s["nodes"] = ints([p + [-1] * (N - len(p)) for p in paths])
        return s
    if op == "ring":
        B, R, Hkv, D, C = case["B"], case["R"], case["Hkv"], case["D"], case["S"] + case["W"]
        return dict(q=normal(B, R, case["Hq"], D, by=2.0), k_pool=normal(B, Hkv, C, D), v_pool=normal(B, Hkv, C, D),
                    k_new=normal(B, Hkv, R, D), v_new=normal(B, Hkv, R, D), pos=ints(_lens(case, B, seed)))
    lens = _lens(case, case["n"], seed)
    T, D, Hkv = sum(lens), case["D"], case["Hkv"]
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    s = dict(k=normal(T, Hkv, D), v=normal(T, Hkv, D), cu_seqlens=ints(ends))
    if op == "prompt":
        s["q"] = normal(T, case["Hq"], D, by=2.0)
    else:
        C = case["S"] + case["W"]
        s["k_pool"], s["v_pool"] = normal(case["n"], Hkv, C, D), normal(case["n"], Hkv, C, D)
        s["pos"] = ints([0] * case["n"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if "q" in s:
        s["out"] = torch.empty_like(s["q"])
    if case["op"] == "commit":
        s["out_seq_lens"] = torch.empty_like(s["seq_lens"])
    return s


# ------------------------------------------------------------------ the library's calls

def _run_own(s):
    from speculative_decoding_verification_09_gb300 import binding
    c = s["case"]
    op = c["op"]
    if op in ("tree", "ring") and "workspace" not in s:
        s["workspace"] = binding.make_attn_workspace(c["B"], c["N" if op == "tree" else "R"], c["Hq"], c["Hkv"], c["D"],
                                                     s["q"].device)
    if op == "tree":
        binding.sv_tree_attn(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], s["k_new"], s["v_new"],
                             s["parent"], s["out"], s["workspace"])
        return s["out"]
    if op == "ring":
        binding.sv_ring_attn(s["q"], s["k_pool"], s["v_pool"], s["pos"], s["k_new"], s["v_new"], c["S"], c["W"], s["out"],
                             s["workspace"])
        return s["out"]
    if op == "prompt":
        binding.sv_prompt_attn(s["q"], s["k"], s["v"], s["cu_seqlens"], c["S"], c["W"], s["out"])
        return s["out"]
    if op == "commit":
        binding.sv_page_commit(s["k_pages"], s["v_pages"], s["k_new"], s["v_new"], s["block_table"], s["seq_lens"],
                               s.get("nodes"), s["num_accepted"], s["out_seq_lens"])
        return s["k_pages"], s["v_pages"], s["out_seq_lens"]
    binding.sv_kv_fill(s["k"], s["v"], s["cu_seqlens"], s["k_pool"], s["v_pool"], s["pos"], c["S"], c["W"])
    return s["k_pool"], s["v_pool"], s["pos"]


# ------------------------------------------------------------------ the plain form

def _softmax_product(scores, seen, v):
    """softmax of the scores where `seen`, times v; the scores are overwritten."""
    scores.masked_fill_(~seen, float("-inf"))
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    return (scores @ v) / scores.sum(-1, keepdim=True)


def _attend(q, k, v, seen, scale, kind):
    """q [B][R][Hq][D], k/v [B][Hkv][L][D], seen [B][R][L]: the attention [B][R][Hq][D], computed in `kind`."""
    B, R, Hq, D = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    G = Hq // Hkv
    rows = q.to(kind).reshape(B, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, D)
    scores = (rows * scale) @ k.to(kind).transpose(-1, -2)
    mask = seen[:, None, :, None, :].expand(B, 1, R, G, L).reshape(B, 1, R * G, L)
    out = _softmax_product(scores, mask, v.to(kind))
    return out.reshape(B, Hkv, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D)


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


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    scale = 1.0 / math.sqrt(c["D"])
    if op == "tree":
        B, N = c["B"], c["N"]
        P, H, page, D = s["k_pages"].shape
        table = s["block_table"].long()
        cols = table.shape[1]
        k = s["k_pages"][table].permute(0, 2, 1, 3, 4).reshape(B, H, cols * page, D)
        v = s["v_pages"][table].permute(0, 2, 1, 3, 4).reshape(B, H, cols * page, D)
        k, v = torch.cat([k, s["k_new"]], 2), torch.cat([v, s["v_new"]], 2)
        t = torch.arange(cols * page, device=k.device)
        inside = (t[None] < s["seq_lens"][:, None])[:, None].expand(B, N, cols * page)
        seen = torch.cat([inside, _ancestors(s["parent"])], 2)
        return _attend(s["q"], k, v, seen, scale, torch.float32).to(s["q"].dtype)
    if op == "ring":
        B, R, S, W = c["B"], c["R"], c["S"], c["W"]
        k, v = torch.cat([s["k_pool"], s["k_new"]], 2), torch.cat([s["v_pool"], s["v_new"]], 2)
        slot = torch.arange(S + W, device=k.device)
        pos = s["pos"].long()[:, None]
        # the position a slot holds: its own below the sinks, else the newest one before pos that falls on it
        held = torch.where(slot[None] < S, slot[None], slot[None] + torch.div(pos - 1 - slot[None], W,
                                                                              rounding_mode="floor") * W)
        filled = (slot[None] < pos) & (held >= 0)
        j = torch.arange(R, device=k.device)
        at = pos + j[None]
        recent = held[:, None, :] > at[:, :, None] - W
        cache = filled[:, None, :] & (recent | (slot[None, None] < S))
        new = (j[:, None] >= j[None, :])[None].expand(B, R, R)
        return _attend(s["q"], k, v, torch.cat([cache, new], 2), scale, torch.float32).to(s["q"].dtype)
    if op == "prompt":
        return _prompt(s["q"], s["k"], s["v"], s["cu_seqlens"], c, scale, torch.float32).to(s["q"].dtype)
    if op == "commit":
        B, N, page = c["B"], c["N"], c["page"]
        j = torch.arange(N, device="cuda")
        node = j[None].expand(B, N)
        if "nodes" in s:  # entry 0 is the root, entry j the j-th accepted node
            node = torch.cat([torch.zeros_like(s["nodes"][:, :1]), s["nodes"][:, :-1]], 1).clamp(min=0).long()
        at = s["seq_lens"].long()[:, None] + j[None]
        col = torch.div(at, page, rounding_mode="floor").clamp(max=s["block_table"].shape[1] - 1)
        where = torch.gather(s["block_table"].long(), 1, col)
        b = torch.arange(B, device="cuda")[:, None].expand(B, N)
        keep = (j[None] <= s["num_accepted"][:, None]).nonzero(as_tuple=True)
        b, node, where, at = b[keep], node[keep], where[keep], at[keep] % page
        s["k_pages"][where, :, at] = s["k_new"][b, :, node]
        s["v_pages"][where, :, at] = s["v_new"][b, :, node]
        s["out_seq_lens"].copy_(s["seq_lens"] + s["num_accepted"] + 1)
        return s["k_pages"], s["v_pages"], s["out_seq_lens"]
    S, W, n = c["S"], c["W"], c["n"]
    start, length = s["cu_seqlens"][:-1].long(), (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long()
    slot = torch.arange(S + W, device="cuda")[None]
    last = length[:, None] - 1
    held = torch.where(slot < S, slot, slot + torch.div(last - slot, W, rounding_mode="floor") * W)
    b, at = ((slot <= last) & (held >= 0)).nonzero(as_tuple=True)
    row = start[b] + held[b, at]
    s["k_pool"][b, :, at] = s["k"][row]
    s["v_pool"][b, :, at] = s["v"][row]
    s["pos"].copy_(length)
    return s["k_pool"], s["v_pool"], s["pos"]


def _prompt(q, k, v, cu, case, scale, kind):
    """The sequences side by side, padded to the longest; a token sees those of its own sequence, by their places in it."""
    T, n, most = q.shape[0], case["n"], case["hi"]
    start, length = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    i = torch.arange(most, device=q.device)
    row = (start[:, None] + i[None]).clamp(max=T - 1)
    near = i[:, None] - i[None, :] < case["W"]
    seen = ((i[:, None] >= i[None, :]) & (near | (i[None, :] < case["S"])))[None].expand(n, most, most)
    wide = _attend(q[row], k[row].transpose(1, 2), v[row].transpose(1, 2), seen, scale, kind)
    t = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(cu.dtype), right=True)
    return wide[seq, t - start[seq]]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work, and the definition in 64 bits

def work(case):
    op, D = case["op"], case["D"]
    if op == "tree":
        B, N, Hq, Hkv = case["B"], case["N"], case["Hq"], case["Hkv"]
        total = sum(_lens(case, B, 0))
        return {"bytes": 4 * Hkv * D * (total + B * N) + 4 * B * N * Hq * D + 4 * B * (N + 1),
                "flops": 4 * Hq * D * N * (total + B * (N + 1) // 2)}
    if op == "ring":
        B, R, S, W = case["B"], case["R"], case["S"], case["W"]
        total = sum(min(p, S + W) for p in _lens(case, B, 0))
        return {"bytes": 4 * case["Hkv"] * D * (total + B * R) + 4 * B * R * case["Hq"] * D + 4 * B,
                "flops": 4 * case["Hq"] * D * R * (total + B * (R + 1) // 2)}
    if op == "commit":
        kept = case["B"] * (case["N"] // 2 + 1 if case["chain"] else min(case["N"], 4))
        return {"bytes": 8 * kept * case["LH"] * D + 8 * case["B"], "flops": 0}
    lens = _lens(case, case["n"], 0)
    if op == "fill":
        return {"bytes": 8 * case["Hkv"] * D * sum(min(n, case["S"] + case["W"]) for n in lens) + 8 * case["n"],
                "flops": 0}
    pairs = 0
    for n in lens:
        S, W = min(case["S"], n), case["W"]
        near = n * (n + 1) // 2 if n <= W else W * (W + 1) // 2 + (n - W) * W
        first = max(0, n - W)  # queries that have lost position 0 from their window; sink t is lost t queries later
        pairs += near + sum(max(0, first - t) for t in range(S))
    return {"bytes": 4 * sum(lens) * D * (case["Hq"] + case["Hkv"]), "flops": 4 * case["Hq"] * D * pairs}


def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits, request by request."""
    s, op = _inputs(case, seed), case["op"]
    lists = {n: s[n].tolist() for n in ("block_table", "seq_lens", "parent", "pos", "cu_seqlens", "nodes", "num_accepted") if n in s}
    if op == "commit":
        pools, page = [s["k_pages"].double(), s["v_pages"].double()], case["page"]
        for b in range(case["B"]):
            path = [0] + (lists["nodes"][b] if "nodes" in s else list(range(1, case["N"])))
            for j in range(lists["num_accepted"][b] + 1):
                at = lists["seq_lens"][b] + j
                for pool, new in zip(pools, (s["k_new"], s["v_new"])):
                    pool[lists["block_table"][b][at // page], :, at % page] = new[b, :, path[j]].double()
        return pools[0], pools[1], None
    if op == "fill":
        pools, S, W = [s["k_pool"].double(), s["v_pool"].double()], case["S"], case["W"]
        for b, (a, e) in enumerate(zip(lists["cu_seqlens"][:-1], lists["cu_seqlens"][1:])):
            kept = sorted({t for t in range(min(S, e - a))} | {t for t in range(max(0, e - a - W), e - a)})
            slots = torch.tensor([t if t < S else S + (t - S) % W for t in kept], dtype=torch.long, device="cuda")
            rows = torch.tensor([a + t for t in kept], dtype=torch.long, device="cuda")
            for pool, new in zip(pools, (s["k"], s["v"])):
                pool[b][:, slots] = new[rows].transpose(0, 1).double()
        return pools[0], pools[1], None
    scale = case["D"] ** -0.5
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    G = case["Hq"] // case["Hkv"]

    def one(q, k, v, visible):
        """q [R][Hq][D], k/v [L][Hkv][D], visible [R][L]; head by head."""
        got = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        for h in range(case["Hq"]):
            w = q[:, h].double() @ k[:, h // G].double().T * scale
            w = torch.where(visible, w, torch.full_like(w, -math.inf))
            got[:, h] = torch.softmax(w, dim=1) @ v[:, h // G].double()
        return got

    if op == "prompt":
        for a, e in zip(lists["cu_seqlens"][:-1], lists["cu_seqlens"][1:]):
            if e > a:
                i = torch.arange(e - a, device="cuda")
                behind = i[:, None] - i[None, :]
                visible = (behind >= 0) & ((behind < case["W"]) | (i[None, :] < case["S"]))
                out[a:e] = one(s["q"][a:e], s["k"][a:e], s["v"][a:e], visible)
        return out
    for b in range(case["B"]):
        if op == "tree":
            n, page, N = lists["seq_lens"][b], case["page"], case["N"]
            ids = torch.tensor(lists["block_table"][b][:-(-n // page)], dtype=torch.long, device="cuda")
            cache = [s[x][ids].transpose(1, 2).reshape(-1, case["Hkv"], case["D"])[:n] for x in ("k_pages", "v_pages")]
            tree = torch.zeros(N, N, dtype=torch.bool)
            for m in range(N):
                at = m
                while at >= 0:
                    tree[m, at] = True
                    at = lists["parent"][b][at]
            visible = torch.cat([torch.ones(N, n, dtype=torch.bool), tree], 1).cuda()
        else:
            p, S, W, R = lists["pos"][b], case["S"], case["W"], case["R"]
            held = sorted({t for t in range(min(S, p))} | {t for t in range(max(0, p - W), p)})
            slots = torch.tensor([t if t < S else S + (t - S) % W for t in held], dtype=torch.long, device="cuda")
            cache = [s[x][b][:, slots].transpose(0, 1) for x in ("k_pool", "v_pool")]
            t = torch.tensor(held + [p + j for j in range(R)], device="cuda")
            at = p + torch.arange(R, device="cuda")
            visible = (t[None] <= at[:, None]) & ((t[None] > at[:, None] - W) | (t[None] < S))
        k = torch.cat([cache[0], s["k_new"][b].transpose(0, 1)], 0)
        v = torch.cat([cache[1], s["v_new"][b].transpose(0, 1)], 0)
        out[b] = one(s["q"][b], k, v, visible)
    return out
