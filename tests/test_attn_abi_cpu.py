"""The attention calls and the cache steps beside them on the host (no GPU needed): exported symbols, workspace sizes,
and bad arguments refused before any CUDA call."""
import os
import re

import pytest
import torch

import __graft_entry__
from speculative_decoding_verification_09_gb300 import binding
from speculative_decoding_verification_09_gb300._build_lib import ROOT

FAKE = 0x10000000  # never dereferenced: every call below fails validation first
BAD = binding.SV_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return binding.lib()


def test_header_symbols_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "svattn.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+([a-z_][a-z0-9_]*)\s*\(", text, flags=re.M))
    assert names == set(binding.EXPORTED_ATTN)
    assert all(hasattr(L, n) for n in names)


def test_workspace_bytes(L):
    ws = binding.sv_attn_workspace_bytes
    assert ws(1, 16, 16, 128) > 0 and ws(256, 128, 1, 8) > 0
    assert ws(256, 32, 1, 128) >= ws(1, 32, 32, 64)
    for bad in ((0, 4, 4, 64), (257, 4, 4, 64), (1, 4, 3, 64), (1, 129, 1, 64), (1, 4, 4, 12), (1, 4, 4, 136),
                (1, 0, 1, 64), (1, 4, 0, 64), (1, 4, 4, 0)):
        assert ws(*bad) == 0, bad


def tree(L, **kw):
    a = dict(dt=binding.SV_BF16, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, kn=FAKE, vn=FAKE, par=FAKE, scale=0.1, B=2,
             N=5, Hq=8, Hkv=4, D=64, P=10, LH=4, h0=0, page=16, cols=3, out=FAKE, ws=FAKE, wsb=1 << 40, st=None)
    a.update(kw)
    return L.sv_tree_attn(*a.values(), None)


def test_tree_refusals(L):
    assert tree(L, dt=binding.SV_F32) == binding.SV_ERR_DTYPE
    assert tree(L, dt=3) == binding.SV_ERR_DTYPE
    for bad in (dict(B=-1), dict(B=65536), dict(N=0), dict(N=257), dict(Hq=6), dict(Hq=0), dict(Hkv=0), dict(D=0),
                dict(D=60), dict(D=136), dict(P=0), dict(LH=3), dict(h0=1), dict(h0=-1), dict(page=0), dict(page=12),
                dict(page=65544), dict(cols=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(scale=3e38), dict(Hq=1032, Hkv=8, LH=8),
                dict(B=65535, LH=1 << 16)):
        assert tree(L, **bad) == BAD, bad
    for p in ("q", "k", "v", "bt", "sl", "kn", "vn", "out"):
        assert tree(L, **{p: None}) == BAD, p
        assert tree(L, **{p: FAKE + 2}) == BAD, p
    for p in ("q", "k", "v", "kn", "vn", "out"):
        assert tree(L, **{p: FAKE + 8}) == BAD, p
    assert tree(L, par=FAKE + 1) == BAD and tree(L, st=FAKE + 2) == BAD
    for w in (dict(ws=None), dict(ws=FAKE + 16), dict(wsb=64)):
        assert tree(L, **w) == binding.SV_ERR_WORKSPACE, w
    assert tree(L, B=0, q=None) == binding.SV_OK  # an empty batch
    if not torch.cuda.is_available():
        assert tree(L) == binding.SV_ERR_CUDA and tree(L, par=None) == binding.SV_ERR_CUDA


def ring(L, **kw):
    a = dict(dt=binding.SV_F16, q=FAKE, k=FAKE, v=FAKE, pos=FAKE, kn=FAKE, vn=FAKE, scale=0.1, B=2, R=5, Hq=8, Hkv=4,
             D=64, LH=4, h0=0, S=4, W=60, out=FAKE, ws=FAKE, wsb=1 << 40, st=None)
    a.update(kw)
    return L.sv_ring_attn(*a.values(), None)


def test_ring_refusals(L):
    assert ring(L, dt=binding.SV_F32) == binding.SV_ERR_DTYPE
    for bad in (dict(B=-1), dict(B=65536), dict(R=0), dict(R=65, W=100), dict(W=4), dict(S=-1), dict(S=1 << 30, W=(1 << 30) + 5),
                dict(Hq=7), dict(D=4), dict(D=144), dict(LH=2), dict(h0=2), dict(scale=0.0), dict(B=65535, LH=1 << 16)):
        assert ring(L, **bad) == BAD, bad
    for p in ("q", "k", "v", "pos", "kn", "vn", "out"):
        assert ring(L, **{p: None}) == BAD, p
        assert ring(L, **{p: FAKE + 2}) == BAD, p
    for w in (dict(ws=None), dict(ws=FAKE + 16), dict(wsb=64)):
        assert ring(L, **w) == binding.SV_ERR_WORKSPACE, w
    assert ring(L, B=0, pos=None) == binding.SV_OK
    if not torch.cuda.is_available():
        assert ring(L) == binding.SV_ERR_CUDA


def prompt(L, **kw):
    a = dict(dt=binding.SV_BF16, q=FAKE, k=FAKE, v=FAKE, cu=FAKE, scale=0.1, B=2, T=50, Hq=8, Hkv=4, D=64, S=4, W=60,
             out=FAKE, st=None)
    a.update(kw)
    return L.sv_prompt_attn(*a.values(), None)


def test_prompt_refusals(L):
    assert prompt(L, dt=binding.SV_F32) == binding.SV_ERR_DTYPE
    for bad in (dict(B=-1), dict(B=65536), dict(T=-1), dict(T=0x7fffffff), dict(Hq=9), dict(D=20), dict(D=256), dict(S=-1),
                dict(W=0), dict(scale=float("nan"))):
        assert prompt(L, **bad) == BAD, bad
    for p in ("q", "k", "v", "cu", "out"):
        assert prompt(L, **{p: None}) == BAD, p
        assert prompt(L, **{p: FAKE + 2}) == BAD, p
    assert prompt(L, T=0, q=None) == binding.SV_OK and prompt(L, B=0) == binding.SV_OK
    if not torch.cuda.is_available():
        assert prompt(L) == binding.SV_ERR_CUDA


def test_fill_refusals(L):
    def fill(**kw):
        a = dict(k=FAKE, v=FAKE, cu=FAKE, kp=FAKE, vp=FAKE, pos=FAKE, B=2, T=50, Hkv=2, LH=4, h0=1, rb=256, S=4, W=60,
                 st=None)
        a.update(kw)
        return L.sv_kv_fill(*a.values(), None)
    for bad in (dict(B=-1), dict(B=65536), dict(T=-1), dict(Hkv=0), dict(LH=2), dict(h0=3), dict(h0=-1), dict(rb=24),
                dict(rb=8208), dict(S=-1), dict(W=0), dict(T=1 << 30, W=1 << 30), dict(k=FAKE + 8), dict(kp=None),
                dict(pos=None), dict(cu=FAKE + 2), dict(k=None)):
        assert fill(**bad) == BAD, bad
    assert fill(B=0) == binding.SV_OK
    if not torch.cuda.is_available():
        assert fill() == binding.SV_ERR_CUDA
        assert fill(T=0, k=None, v=None) == binding.SV_ERR_CUDA


def test_page_commit_refusals(L):
    def commit(**kw):
        a = dict(kp=FAKE, vp=FAKE, kn=FAKE, vn=FAKE, bt=FAKE, sl=FAKE, nodes=FAKE, acc=FAKE, B=2, LH=3, N=5, rb=256,
                 P=9, page=16, cols=4, out=FAKE, st=None)
        a.update(kw)
        return L.sv_page_commit(*a.values(), None)
    for bad in (dict(B=-1), dict(B=65536), dict(LH=0), dict(N=0), dict(N=(1 << 20) + 1), dict(rb=8), dict(rb=8208), dict(P=0),
                dict(page=0), dict(cols=0), dict(kp=None), dict(vn=FAKE + 8), dict(bt=None), dict(sl=FAKE + 1),
                dict(nodes=FAKE + 2), dict(acc=None), dict(out=None), dict(out=FAKE + 4)):
        assert commit(**bad) == BAD, bad
    assert commit(B=0) == binding.SV_OK
    if not torch.cuda.is_available():
        assert commit() == binding.SV_ERR_CUDA and commit(out=FAKE + 64, nodes=None) == binding.SV_ERR_CUDA


def test_binding_refuses_wrong_shapes():
    """The binding's own checks raise before the library is asked."""
    z = torch.zeros
    q, kp, kn = z(2, 3, 4, 64, dtype=torch.bfloat16), z(5, 2, 16, 64, dtype=torch.bfloat16), z(2, 2, 3, 64, dtype=torch.bfloat16)
    bt, sl, par, ws = z(2, 3, dtype=torch.int32), z(2, dtype=torch.int32), z(2, 3, dtype=torch.int32), z(8, dtype=torch.uint8)

    def call(q=q, kp=kp, vp=kp, bt=bt, sl=sl, kn=kn, vn=kn, par=par, out=None):
        binding.sv_tree_attn(q, kp, vp, bt, sl, kn, vn, par, torch.empty_like(q) if out is None else out, ws)
    for bad in (dict(q=q[0]), dict(kp=kp[:, :1]), dict(kn=kn[:1]), dict(bt=bt[:1]), dict(sl=sl[:1]), dict(par=par[:, :2]),
                dict(out=z(2, 3, 4, 32, dtype=torch.bfloat16)), dict(q=q.half()), dict(vn=kn[..., :32]), dict(),
                dict(q=q.float(), kp=kp.float(), vp=kp.float(), kn=kn.float(), vn=kn.float())):
        with pytest.raises(binding.SpecVerifyError):  # dict(): CPU tensors are refused last
            call(**bad)
