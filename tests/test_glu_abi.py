"""Argument checks of the gated units, on the CPU: no call here launches a kernel."""
import ctypes

import pytest
import torch

import mlp_step_gb300 as M
from mlp_step_gb300 import build

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
F32, BF16, U8, F16 = M.MLP_DTYPE_F32, M.MLP_DTYPE_BF16, M.MLP_DTYPE_U8, M.MLP_DTYPE_F16
OK, BAD, ALIGN, SHAPE = 0, 1, 2, 3
CK = dict(gq=P, ldgq=96, gs=P, ldgs=3, uq=P, lduq=96, us=P, ldus=3)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return M.load()


def test_forward(lib):
    def fwd(x=P, ldx=64, wg=P, ldwg=96, wu=P, ldwu=96, T=16, k=64, n=96, dt=BF16, bg=P, bu=P,
            act=5, y=P, ldy=96, g=None, ldg=0, u=None, ldu=0, gq=None, ldgq=0, gs=None, ldgs=0,
            uq=None, lduq=0, us=None, ldus=0, ws=None, wsn=0):
        return lib.mlp_glu_fwd(x, ldx, wg, ldwg, wu, ldwu, T, k, n, dt, bg, bu, act,
                               ctypes.c_float(0.5), y, ldy, g, ldg, u, ldu, gq, ldgq, gs, ldgs, uq,
                               lduq, us, ldus, ws, wsn, None)
    assert fwd(T=0, x=None, wg=None, wu=None, y=None) == OK
    for bad in (dict(T=-1), dict(k=0), dict(n=0), dict(dt=U8), dict(act=6), dict(act=-1),
                dict(x=None), dict(wg=None), dict(wu=None), dict(y=None), dict(ldx=56),
                dict(ldwg=88), dict(ldwu=88), dict(ldy=95), dict(g=P, ldg=96),
                dict(u=P, ldu=96), dict(g=P, u=P, ldg=95, ldu=96), dict(g=P, u=P, ldg=96, ldu=95),
                dict(g=P, u=P, ldg=96, ldu=96, **CK), *({**CK, m: None} for m in CK if CK[m] is P),
                *({**CK, m: CK[m] - 1} for m in CK if CK[m] is not P)):
        assert fwd(**bad) == BAD, bad
    for m in ("x", "wg", "wu", "bg", "bu", "y", "ws"):
        assert fwd(**{m: ODD}) == ALIGN, m
    for m in ("gq", "gs", "uq", "us"):
        assert fwd(**{**CK, m: ODD}) == ALIGN, m
    assert fwd(g=ODD, u=P, ldg=96, ldu=96) == ALIGN
    # 16-bit rows start on 16 bytes
    assert fwd(ldx=66) == ALIGN and fwd(ldwg=100) == ALIGN and fwd(ldwu=100) == ALIGN
    assert fwd(k=(1 << 24) + 1) == SHAPE and fwd(n=(1 << 24) + 1) == SHAPE
    # split sums, and fp32 sums, need their workspace
    need = M.mlp_glu_workspace_bytes(64, 8192, 128, torch.bfloat16)
    assert need > 0 and M.mlp_glu_workspace_bytes(1, 8192, 128, torch.bfloat16) == 0
    long = dict(T=64, k=8192, n=128, ldx=8192, ldwg=128, ldwu=128, ldy=128)
    assert fwd(**long) == BAD and fwd(**long, ws=P, wsn=need - 1) == BAD
    assert M.mlp_glu_workspace_bytes(65536, 512, 1408, torch.bfloat16) == 0
    assert M.mlp_glu_workspace_bytes(100, 64, 96, torch.float32) == 2 * 100 * 96 * 4
    for wrong in ((0, 64, 96), (16, 0, 96), (16, 64, 1 << 25)):
        assert M.mlp_glu_workspace_bytes(*wrong, torch.bfloat16) == 0
        assert M.mlp_glu_bwd_workspace_bytes(*wrong, torch.bfloat16) == 0


def test_backward(lib):
    need = M.mlp_glu_bwd_workspace_bytes(16, 96, 64, torch.bfloat16)

    def bwd(dy=P, lddy=64, w=P, ldw=64, T=16, n=96, k=64, dt=BF16, act=5, g=P, ldg=96, u=P, ldu=96,
            gq=None, ldgq=0, gs=None, ldgs=0, uq=None, lduq=0, us=None, ldus=0, dg=P, lddg=96, du=P,
            lddu=96, dbg=None, dbu=None, a=None, lda=0, ws=P, wsn=need):
        return lib.mlp_glu_bwd(dy, lddy, w, ldw, T, n, k, dt, act, ctypes.c_float(0.5), g, ldg, u,
                               ldu, gq, ldgq, gs, ldgs, uq, lduq, us, ldus, dg, lddg, du, lddu, dbg,
                               dbu, a, lda, ws, wsn, None)
    none = dict(g=None, u=None)
    assert bwd(T=0, dy=None, w=None, dg=None, du=None, **none) == OK
    for bad in (dict(T=-1), dict(k=0), dict(n=0), dict(dt=U8), dict(act=6), dict(dy=None),
                dict(w=None), dict(dg=None), dict(du=None), dict(lddy=56), dict(ldw=56),
                dict(lddg=95), dict(lddu=95), dict(ldg=95), dict(ldu=95), dict(g=None),
                dict(u=None), none, CK, dict(a=P, lda=95), dict(dbg=P), dict(dbu=P),
                *({**none, **CK, m: None} for m in CK if CK[m] is P),
                *({**none, **CK, m: CK[m] - 1} for m in CK if CK[m] is not P),
                dict(dbg=P, dbu=P, ws=None), dict(dbg=P, dbu=P, wsn=need - 1)):
        assert bwd(**bad) == BAD, bad
    for m in ("dy", "w", "g", "u", "dg", "du", "ws"):
        assert bwd(**{m: ODD}) == ALIGN, m
    assert bwd(dbg=ODD, dbu=P) == ALIGN and bwd(dbg=P, dbu=ODD) == ALIGN
    assert bwd(T=0, dbg=ODD, dbu=P) == ALIGN and bwd(a=ODD, lda=96) == ALIGN
    for m in ("gq", "gs", "uq", "us"):
        assert bwd(**{**none, **CK, m: ODD}) == ALIGN, m
    assert bwd(lddy=68) == ALIGN and bwd(ldw=68) == ALIGN
    assert bwd(k=(1 << 24) + 1) == SHAPE


def test_binding_refuses_what_the_library_cannot_read():
    x, w = torch.zeros(4, 64), torch.zeros(64, 96)
    with pytest.raises(ValueError, match="CUDA device"):
        M.mlp_glu_fwd(x, w, w, torch.zeros(4, 96))
    with pytest.raises(ValueError, match="CUDA device"):
        M.mlp_glu_bwd(x, w.t(), torch.zeros(4, 96), torch.zeros(4, 96))
    with pytest.raises(TypeError):
        M.mlp_glu_workspace_bytes(4, 64, 64, torch.float64)
    with pytest.raises(ValueError, match="at most"):
        M.mlp_glu_workspace_bytes(4, 1 << 31, 64, torch.bfloat16)
