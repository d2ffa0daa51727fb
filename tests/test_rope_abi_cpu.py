"""Rotary positions and the 8-bit cache on the host (no GPU needed): exported symbols, and bad arguments refused before
any CUDA call."""
import os
import re

import pytest
import torch

import __graft_entry__
import kv8_util as ku
from speculative_decoding_verification_09_gb300 import binding
from speculative_decoding_verification_09_gb300._build_lib import ROOT

FAKE = 0x10000000  # never dereferenced: every call below fails validation first
BAD = binding.SV_ERR_INVALID_ARG
HERE = not torch.cuda.is_available()


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    return binding.lib()


@pytest.mark.parametrize("header,names", [("svrope.h", binding.EXPORTED_ROPE), ("svkv8.h", binding.EXPORTED_KV8)])
def test_header_symbols_exported(L, header, names):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    assert set(re.findall(r"^\s*(?:int|size_t)\s+([a-z_][a-z0-9_]*)\s*\(", text, flags=re.M)) == set(names)
    assert all(hasattr(L, n) for n in names)


def refuses(call, bad, result=BAD):
    for kw in bad:
        assert call(**kw) == result, kw


def test_table_refusals(L):
    def table(**kw):
        a = dict(scaling=0, base=1e4, factor=1.0, original=0, low=1.0, high=32.0, gain=1.0, rot=64, first=0, rows=8,
                 table=FAKE)
        a.update(kw)
        return L.sv_rope_table(*a.values(), None)
    nan, inf = float("nan"), float("inf")
    refuses(table, [dict(scaling=-1), dict(scaling=5), dict(base=1.0), dict(base=nan), dict(base=inf), dict(factor=0.0),
                    dict(factor=-1.0), dict(factor=nan), dict(factor=inf), dict(gain=nan), dict(gain=1e300), dict(rot=0),
                    dict(rot=7), dict(rot=258), dict(first=-1), dict(rows=-1), dict(first=1 << 30, rows=1 << 30),
                    dict(scaling=2, rot=2), dict(table=None), dict(table=FAKE + 4)])
    for scaling in (3, 4):
        refuses(table, [dict(scaling=scaling, original=4096, **x) for x in (
            dict(low=0.0), dict(low=-1.0), dict(low=32.0), dict(low=40.0), dict(high=inf), dict(high=nan))] +
            [dict(scaling=scaling)])
    assert table(rows=0, table=None) == binding.SV_OK
    if HERE:
        assert table() == binding.SV_ERR_CUDA


def test_rope_refusals(L):
    def rope(**kw):
        a = dict(dt=binding.SV_BF16, q=FAKE, qs=512, k=FAKE, ks=256, pos=FAKE, table=FAKE, rows=10, rot=64, inter=0, T=4,
                 Hq=8, Hk=4, D=64, qo=FAKE, qos=512, ko=FAKE, kos=256, st=None)
        a.update(kw)
        return L.sv_rope(*a.values(), None)
    refuses(rope, [dict(dt=binding.SV_F32), dict(dt=7)], binding.SV_ERR_DTYPE)
    refuses(rope, [dict(T=-1), dict(Hq=0), dict(Hq=65536), dict(Hk=-1), dict(Hk=65536), dict(D=0), dict(D=60), dict(D=264),
                   dict(rows=0), dict(rot=0), dict(rot=63), dict(rot=66), dict(qs=504), dict(qs=516), dict(ks=255),
                   dict(qos=8), dict(kos=0), dict(q=None), dict(k=None), dict(pos=None), dict(table=None), dict(qo=None),
                   dict(ko=None), dict(q=FAKE + 8), dict(k=FAKE + 2), dict(qo=FAKE + 8), dict(ko=FAKE + 4),
                   dict(pos=FAKE + 2), dict(table=FAKE + 4), dict(st=FAKE + 1), dict(qs=520), dict(kos=264)])
    assert rope(T=0, q=None, k=None) == binding.SV_OK
    if HERE:
        assert rope() == binding.SV_ERR_CUDA
        assert rope(k=None, ko=None, Hk=0, ks=0, kos=0) == binding.SV_ERR_CUDA


def test_append_refusals(L):
    def append(**kw):
        a = dict(dt=binding.SV_F16, k=FAKE, ks=256, v=FAKE, vs=256, kp=FAKE, vp=FAKE, bt=FAKE, sl=FAKE, cu=FAKE,
                 table=FAKE, rows=10, rot=64, inter=0, pos=None, q=FAKE, qs=512, qo=FAKE, qos=512, ko=None, kos=0, B=2,
                 T=6, Hq=8, Hkv=4, D=64, P=9, LH=6, h0=2, page=16, cols=3, out=None, st=None)
        a.update(kw)
        return L.sv_page_append(*a.values(), None)
    refuses(append, [dict(dt=binding.SV_F32)], binding.SV_ERR_DTYPE)
    refuses(append, [dict(B=-1), dict(B=65536), dict(T=-1), dict(Hq=-1), dict(Hkv=0), dict(D=12), dict(D=264), dict(P=0),
                     dict(LH=5), dict(h0=-1), dict(h0=3), dict(page=0), dict(cols=0), dict(ks=248), dict(vs=250),
                     dict(qs=8), dict(qos=8), dict(ko=FAKE, kos=16), dict(rot=65), dict(rot=0), dict(rows=0),
                     dict(table=None), dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(bt=None),
                     dict(sl=None), dict(cu=None), dict(q=None), dict(qo=None), dict(k=FAKE + 8), dict(v=FAKE + 8),
                     dict(kp=FAKE + 8), dict(vp=FAKE + 8), dict(q=FAKE + 8), dict(qo=FAKE + 8),
                     dict(ko=FAKE + 8, kos=256), dict(bt=FAKE + 1), dict(sl=FAKE + 2), dict(cu=FAKE + 2),
                     dict(pos=FAKE + 2), dict(out=FAKE), dict(out=FAKE + 4), dict(st=FAKE + 2), dict(ko=FAKE, kos=264)])
    assert append(B=0, k=None) == binding.SV_OK
    if HERE:
        assert append() == binding.SV_ERR_CUDA
        assert append(table=None, q=None, qo=None, Hq=0) == binding.SV_ERR_CUDA


def append8(L, **kw):
    a = dict(dt=binding.SV_BF16, k=FAKE, ks=256, v=FAKE, vs=256, kp=FAKE, vp=FAKE, ksc=FAKE, vsc=FAKE, bt=FAKE, sl=FAKE,
             cu=FAKE, table=None, rows=0, rot=0, inter=0, pos=None, B=2, T=6, Hkv=4, D=64, P=9, LH=6, h0=2, page=32,
             block=16, cols=3, out=None, st=None)
    a.update(kw)
    return L.sv_page_append8(*a.values(), None)


def commit8(L, **kw):
    a = dict(dt=binding.SV_F16, kp=FAKE, vp=FAKE, ksc=FAKE, vsc=FAKE, kn=FAKE, vn=FAKE, bt=FAKE, sl=FAKE, nodes=FAKE,
             acc=FAKE, B=2, LH=3, N=5, D=128, P=9, page=32, block=16, cols=4, out=FAKE, st=None)
    a.update(kw)
    return L.sv_page_commit8(*a.values(), None)


def attn8(L, **kw):
    a = dict(dt=binding.SV_BF16, q=FAKE, k=FAKE, v=FAKE, ksc=FAKE, vsc=FAKE, bt=FAKE, sl=FAKE, kn=FAKE, vn=FAKE, par=FAKE,
             scale=0.1, B=2, N=5, Hq=8, Hkv=4, D=64, P=10, LH=4, h0=0, page=32, block=16, cols=3, out=FAKE, ws=FAKE,
             wsb=1 << 40, st=None)
    a.update(kw)
    return L.sv_tree_attn8(*a.values(), None)


SHAPES8 = [dict(D=8), dict(D=72), dict(D=144), dict(D=0), dict(block=0), dict(block=4), dict(block=24), dict(block=256),
           dict(block=64), dict(page=24), dict(page=0), dict(cols=0), dict(P=0), dict(B=-1), dict(B=65536), dict(LH=0)]


@pytest.mark.parametrize("call", [append8, commit8, attn8])
def test_8_bit_refusals(L, call):
    refuses(lambda **kw: call(L, **kw), [dict(dt=binding.SV_F32), dict(dt=-1)], binding.SV_ERR_DTYPE)
    refuses(lambda **kw: call(L, **kw), SHAPES8)
    names = {append8: ("k", "v", "kp", "vp", "ksc", "vsc", "bt", "sl", "cu"),
             commit8: ("kp", "vp", "ksc", "vsc", "kn", "vn", "bt", "sl", "acc", "out"),
             attn8: ("q", "k", "v", "ksc", "vsc", "bt", "sl", "kn", "vn", "out")}[call]
    for p in names:
        assert call(L, **{p: None}) == BAD, p
        if p not in ("ksc", "vsc"):  # scales are bytes
            assert call(L, **{p: FAKE + 2}) == BAD, p
    assert call(L, st=FAKE + 2) == BAD
    assert call(L, B=0, bt=None) == binding.SV_OK


def test_other_8_bit_refusals(L):
    refuses(lambda **kw: append8(L, **kw), [dict(T=-1), dict(Hkv=0), dict(Hkv=65536), dict(h0=3), dict(h0=-1),
                                            dict(ks=248), dict(vs=260), dict(table=FAKE, rows=0, rot=64),
                                            dict(table=FAKE, rows=4, rot=66), dict(table=FAKE, rows=4, rot=3),
                                            dict(out=FAKE), dict(out=FAKE + 4), dict(pos=FAKE + 1), dict(cu=FAKE + 1)])
    refuses(lambda **kw: commit8(L, **kw), [dict(N=0), dict(N=(1 << 20) + 1), dict(out=FAKE + 4), dict(nodes=FAKE + 2)])
    refuses(lambda **kw: attn8(L, **kw), [dict(N=0), dict(N=257), dict(Hq=6), dict(Hkv=0), dict(h0=1), dict(h0=-1),
                                          dict(page=1 << 17, block=128), dict(scale=0.0), dict(scale=float("nan")),
                                          dict(scale=3e38), dict(B=65535, LH=1 << 16), dict(par=FAKE + 1)])
    for w in (dict(ws=None), dict(ws=FAKE + 16), dict(wsb=64)):
        assert attn8(L, **w) == binding.SV_ERR_WORKSPACE, w
    if HERE:
        assert append8(L) == commit8(L) == commit8(L, out=FAKE + 64, nodes=None) == binding.SV_ERR_CUDA
        assert attn8(L) == attn8(L, par=None) == binding.SV_ERR_CUDA


def test_binding_refuses_wrong_shapes():
    """The binding's own checks raise before the library is asked."""
    z, i32, bf = torch.zeros, torch.int32, torch.bfloat16
    q, k = z(6, 8, 64, dtype=bf), z(6, 4, 64, dtype=bf)
    kp, p8 = z(5, 4, 16, 64, dtype=bf), z(5, 4, 16, 64, dtype=ku.E4M3)
    sc = z(5, 4, 2, dtype=torch.uint8).view(ku.E8M0)
    bt, sl, cu, tab = z(2, 3, dtype=i32), z(2, dtype=i32), z(3, dtype=i32), z(9, 2, 32)
    pos, ws = z(6, dtype=i32), z(8, dtype=torch.uint8)
    calls = [
        lambda: binding.sv_rope(q, k, pos, tab, q, k),  # CPU tensors are refused last
        lambda: binding.sv_rope(q[0], k, pos, tab, q, k),
        lambda: binding.sv_rope(q, k[:3], pos, tab, q, k),
        lambda: binding.sv_rope(q, k, pos, tab, q),
        lambda: binding.sv_rope_table(tab),
        lambda: binding.sv_page_append(k, k, kp, kp, bt, sl, cu, tab),
        lambda: binding.sv_page_append(k, k[:5], kp, kp, bt, sl, cu, tab),
        lambda: binding.sv_page_append(k, k, kp, kp, bt, sl, cu, tab, q=q),
        lambda: binding.sv_page_append8(k, k, p8, p8, sc, sc, bt, sl, cu),
        lambda: binding.sv_page_append8(k[..., :32], k, p8, p8, sc, sc, bt, sl, cu),
        lambda: binding.sv_page_append8(k, k, p8, p8, sc[..., :0], sc, bt, sl, cu),
        lambda: binding.sv_page_commit8(p8, p8, sc, sc, k, k, bt, sl, None, sl, sl),
        lambda: binding.sv_tree_attn8(q[None], p8, p8, sc, sc, bt, sl, k[None], k[None], None, q[None], ws),
        lambda: binding.sv_tree_attn8(q, p8, p8, sc, sc, bt, sl, k[None], k[None], None, q, ws),
    ]
    for call in calls:
        with pytest.raises(binding.SpecVerifyError):
            call()
    text = open(binding.__file__).read()
    for name in (*binding.EXPORTED_ROPE, *binding.EXPORTED_KV8[:3]):
        body = text[text.index(f"def {name}("):]
        assert "_cuda_device(" in body[:body.index("_check(")], name


# ------------------------------------------------------------------ the definitions the GPU tests go by

def test_e4m3_of_the_definition_is_the_types():
    """to_e4m3 against torch's conversion: every value of the format, every midpoint between two, and values beside them."""
    bits = torch.arange(256, dtype=torch.uint8).view(ku.E4M3).float()
    fine = torch.sort(bits[bits.isfinite()].unique()).values.double()
    mid = (fine[1:] + fine[:-1]) / 2
    x = torch.cat([fine, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20), torch.tensor([1e-9, -1e-9, 0.0])])
    assert torch.equal(ku.to_e4m3(x), x.float().to(ku.E4M3).double())
    assert ku.to_e4m3(torch.tensor([1e4, -1e4, float("inf"), float("nan")]).double()).tolist()[:2] == [448.0, -448.0]


def test_exponents_of_the_definition():
    x = torch.tensor([[448.0], [448.0 * (1 + 2.0 ** -30)], [1.0], [1.75], [1.7500001], [0.0], [1e38], [float("inf")]],
                     dtype=torch.float64)
    e = ku.exponent(x.double(), torch.bfloat16).tolist()
    assert e == [0, 1, -8, -8, -7, -117, 118, -117]
    assert ku.exponent(x.double(), torch.float16).tolist() == [0, 1, -8, -8, -7, -15, 7, -15]


def test_a_planted_mistake_is_found():
    """The bounds notice a rotation by the wrong sign and a value one step off (planted in the definition, on the CPU)."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 2, 64, generator=g).to(torch.bfloat16)
    cs = ku.angles(5, 32).float()
    good = ku.rotate32(x, cs, False).to(torch.bfloat16)
    ku.check_rotated(good, x, cs, False)
    for wrong in (ku.rotate32(x, cs * torch.tensor([1.0, -1.0])[None, :, None], False).to(torch.bfloat16),
                  ku.rotate32(x, cs, True).to(torch.bfloat16), torch.where(good != 0, good * (1 + 2.0 ** -7), good)):
        with pytest.raises(AssertionError):
            ku.check_rotated(wrong, x, cs, False)


def test_attention_workspace_sizes():
    """0 for sizes that the calls refuse; it grows with the batch and covers every call that may follow."""
    ask = binding.sv_attn8_workspace_bytes
    for B, N, Hq, Hkv, D in [(1, 1, 1, 1, 16), (64, 22, 16, 16, 128), (65535, 1, 8, 2, 64), (3, 128, 4, 4, 32)]:
        n = ask(B, N, Hq, Hkv, D)
        assert n > 0 and n >= ask(max(1, B // 2), N, Hq, Hkv, D)
        assert ask(2 * B if B < 30000 else B, N, Hq, Hkv, D) >= n
    for bad in [(-1, 1, 1, 1, 16), (65536, 1, 1, 1, 16), (1, 0, 1, 1, 16), (1, 1, 3, 2, 16), (1, 1, 1, 1, 24), (1, 1, 1, 1, 0),
                (1, 1, 1, 1, 144), (1, 1, 0, 1, 16), (1, 1, 1, 0, 16), (1, 1 << 20, 1, 1, 16)]:
        assert ask(*bad) == 0, bad
    with pytest.raises(binding.SpecVerifyError):
        binding.make_attn_workspace(1, 0, 1, 1, 16, "cpu")
    make, both = binding.make_attn_workspace, (ask(400, 3, 2, 1, 32), binding.sv_attn_workspace_bytes(3, 2, 1, 32))
    assert make(400, 3, 2, 1, 32, "cpu").numel() == max(both)
    assert make(400, 3, 2, 1, 32, "cpu", 8).numel() == both[0] and make(400, 3, 2, 1, 32, "cpu", 16).numel() == both[1]
    assert make(2, 3, 2, 1, 24, "cpu").numel() == binding.sv_attn_workspace_bytes(3, 2, 1, 24)
    for bits, D in ((4, 32), (8, 24)):
        with pytest.raises(binding.SpecVerifyError):
            make(2, 3, 2, 1, D, "cpu", bits)
