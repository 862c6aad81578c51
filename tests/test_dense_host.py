"""The dense operators' refusals: every wrong argument returns its code (or
raises in the binding) before a device is touched."""
import ctypes

import pytest
import torch

from quantized_routed_expert_amd import moe

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
P = 0x10000  # never dereferenced: validation fails first (or T = 0 launches nothing)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return moe.lib()


def linear(L, **k):
    a = dict(x=P, xd=1, T=4, inner=64, w=P, out=64, bias=None, act=0, res=None, rd=1, z=None, y=P, yd=1, ws=P, n=BIG)
    a.update(k)
    return L.moe_linear(a["x"], a["xd"], a["T"], a["inner"], a["w"], a["out"], a["bias"], a["act"], a["res"], a["rd"],
                        a["z"], a["y"], a["yd"], a["ws"], a["n"], 0)


def linear_backward(L, **k):
    a = dict(dy=P, T=4, inner=64, out=64, x=P, w=P, z=None, act=0, dx=P, dw=P, db=P, wd=1, acc=0, ws=P, n=BIG)
    a.update(k)
    return L.moe_linear_backward(a["dy"], a["T"], a["inner"], a["out"], a["x"], a["w"], a["z"], a["act"], a["dx"], a["dw"],
                                 a["db"], a["wd"], a["acc"], a["ws"], a["n"], 0)


def ffn_of(**k):
    a = dict(gate=P, up=P, down=P, hidden=64, ffn=64, act=1)
    a.update(k)
    return ctypes.byref(moe.DenseFFN(a["gate"], a["up"], a["down"], a["hidden"], a["ffn"], a["act"]))


def gated(L, f=None, **k):
    a = dict(x=P, xd=1, T=4, res=None, rd=1, gu=None, y=P, yd=1, ws=P, n=BIG)
    a.update(k)
    return L.moe_gated_ffn(a["x"], a["xd"], a["T"], f or ffn_of(), a["res"], a["rd"], a["gu"], a["y"], a["yd"], a["ws"],
                           a["n"], 0)


def gated_backward(L, f=None, **k):
    a = dict(dy=P, x=P, T=4, gu=P, dx=P, dg=P, du=P, dd=P, wd=1, acc=0, ws=P, n=BIG)
    a.update(k)
    return L.moe_gated_ffn_backward(a["dy"], a["x"], a["T"], f or ffn_of(), a["gu"], a["dx"], a["dg"], a["du"], a["dd"],
                                    a["wd"], a["acc"], a["ws"], a["n"], 0)


@pytest.mark.parametrize("call", [linear, gated])
def test_forward_refusals(L, call):
    for k in ("x", "y", "ws"):
        assert call(L, **{k: None}) == INVALID, k
        assert call(L, **{k: P + 8}) == INVALID, k  # not 16-byte aligned
    assert call(L, xd=2) == INVALID and call(L, yd=-1) == INVALID
    assert call(L, res=P, rd=7) == INVALID
    assert call(L, res=P + 2) == INVALID
    assert call(L, T=-1) == INVALID
    assert call(L, T=(1 << 24) + 1) == UNSUPPORTED
    assert call(L, n=1000) == WORKSPACE
    assert call(L, T=0, x=None, y=None, ws=None, n=0) == OK  # nothing to do


def test_linear_refusals(L):
    assert linear(L, w=None) == INVALID and linear(L, w=P + 4) == INVALID
    assert linear(L, bias=P + 4) == INVALID and linear(L, z=P + 2) == INVALID
    assert linear(L, act=5) == INVALID and linear(L, act=-1) == INVALID
    for k in ("inner", "out"):
        assert linear(L, **{k: 0}) == INVALID
        assert linear(L, **{k: -8}) == INVALID
        assert linear(L, **{k: 60}) == UNSUPPORTED
        assert linear(L, **{k: (1 << 20) + 8}) == UNSUPPORTED


def test_linear_backward_refusals(L):
    assert linear_backward(L, dx=None, dw=None, db=None) == INVALID
    for k in ("dy", "x", "w", "ws"):
        assert linear_backward(L, **{k: None}) == INVALID, k
    for k in ("dy", "x", "w", "dx", "dw", "db", "ws"):
        assert linear_backward(L, **{k: P + 8}) == INVALID, k
    assert linear_backward(L, act=1) == INVALID  # needs z
    assert linear_backward(L, act=9, z=P) == INVALID
    assert linear_backward(L, wd=3) == INVALID
    assert linear_backward(L, T=-2) == INVALID
    assert linear_backward(L, inner=12) == UNSUPPORTED
    assert linear_backward(L, n=100) == WORKSPACE


def test_gated_refusals(L):
    assert L.moe_gated_ffn(P, 1, 4, None, None, 0, None, P, 1, P, BIG, 0) == INVALID
    for k in ("gate", "up", "down"):
        assert gated(L, ffn_of(**{k: None})) == INVALID, k
        assert gated(L, ffn_of(**{k: P + 8})) == INVALID, k
    assert gated(L, ffn_of(act=5)) == INVALID
    assert gated(L, gu=P + 8) == INVALID
    for k in ("hidden", "ffn"):
        assert gated(L, ffn_of(**{k: 0})) == INVALID
        assert gated(L, ffn_of(**{k: 100})) == UNSUPPORTED


def test_gated_backward_refusals(L):
    assert L.moe_gated_ffn_backward(P, P, 4, None, P, P, P, P, P, 1, 0, P, BIG, 0) == INVALID
    assert gated_backward(L, dx=None, dg=None, du=None, dd=None) == INVALID
    for k in ("dy", "x", "gu", "ws"):
        assert gated_backward(L, **{k: None}) == INVALID, k
    for k in ("dy", "x", "gu", "dx", "dg", "du", "dd", "ws"):
        assert gated_backward(L, **{k: P + 8}) == INVALID, k
    for k in ("gate", "up", "down"):
        assert gated_backward(L, ffn_of(**{k: None})) == INVALID, k
    assert gated_backward(L, wd=2) == INVALID
    assert gated_backward(L, ffn_of(act=-1)) == INVALID
    assert gated_backward(L, ffn_of(ffn=20)) == UNSUPPORTED
    assert gated_backward(L, T=-1) == INVALID
    assert gated_backward(L, n=4096) == WORKSPACE


def test_workspace_sizes(L):
    """Enough for fewer rows too: the size does not fall with T."""
    for f in (moe.linear_workspace_bytes, moe.gated_ffn_workspace_bytes):
        last = 0
        for T in (0, 1, 4, 5, 16, 17, 64, 65, 100, 128, 257, 1000, 2048, 8192, 100000):
            n = f(T, 2048, 768)
            assert n >= last
            last = n
        for bad, code in (((-1, 64, 64), INVALID), ((4, 0, 64), INVALID), ((4, 64, 12), UNSUPPORTED),
                          ((4, 1 << 21, 64), UNSUPPORTED)):
            with pytest.raises(moe.MoeError) as e:
                f(*bad)
            assert e.value.status == code


def test_binding_refuses_host_tensors():
    x, w, ws = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        moe.linear(x, w, ws)
    with pytest.raises(ValueError):
        moe.gated_ffn(x, moe.dense_ffn(w, w, w), ws)
    with pytest.raises(TypeError):
        moe.dense_ffn(w.float(), w, w)
    with pytest.raises(ValueError):
        moe.dense_ffn(w, w[:32], w)
    with pytest.raises(ValueError):
        moe.dense_ffn(w, w.T, w)
