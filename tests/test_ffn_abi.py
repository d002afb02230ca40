"""Argument checks of the feed-forward operators (layer norm, linear layers,
8-bit checkpoints), on the CPU: no call here launches a kernel."""
import ctypes

import pytest
import torch

import mlp_step_gb300 as M
from mlp_step_gb300 import build

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
F32, BF16, U8, F16 = M.MLP_DTYPE_F32, M.MLP_DTYPE_BF16, M.MLP_DTYPE_U8, M.MLP_DTYPE_F16
OK, BAD, ALIGN, SHAPE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return M.load()


def test_ckpt8(lib):
    assert [M.mlp_ckpt8_scale_cols(c) for c in (-1, 0, 1, 32, 33, 512)] == [0, 0, 1, 1, 2, 16]
    enc = lambda x=P, dt=BF16, r=4, c=64, ldx=64, q=P, ldq=64, s=P, lds=2: \
        lib.mlp_ckpt8_encode(x, dt, r, c, ldx, q, ldq, s, lds, None)
    dec = lambda q=P, ldq=64, s=P, lds=2, r=4, c=64, o=P, dt=F16, ldo=64: \
        lib.mlp_ckpt8_decode(q, ldq, s, lds, r, c, o, dt, ldo, None)
    assert enc(r=0, x=None) == OK and enc(c=0) == OK and dec(r=0, o=None) == OK
    for bad in (dict(dt=U8), dict(dt=9), dict(r=-1), dict(c=-1), dict(q=None), dict(s=None),
                dict(ldq=63), dict(lds=1)):
        assert enc(**bad) == BAD and dec(**bad) == BAD, bad
    assert enc(x=None) == BAD and enc(ldx=63) == BAD and dec(o=None) == BAD and dec(ldo=63) == BAD
    assert enc(x=ODD) == ALIGN and enc(q=ODD) == ALIGN and dec(s=ODD) == ALIGN
    assert dec(o=ODD) == ALIGN
    big = (1 << 24) + 1
    assert enc(c=big, ldx=big, ldq=big, lds=big) == SHAPE


def test_layernorm(lib):
    f = ctypes.c_float
    fwd = lambda x=P, dt=BF16, ldx=64, g=P, s=P, T=4, d=64, eps=1e-5, y=P, ldy=64, m=P, r=P, q=None, \
        ldq=0, sc=None, lds=0: lib.mlp_layernorm_fwd(x, dt, ldx, g, s, T, d, f(eps), y, ldy, m, r,
                                                     q, ldq, sc, lds, None)
    assert fwd(T=0, x=None, y=None) == OK
    for bad in (dict(T=-1), dict(d=0), dict(dt=U8), dict(eps=-1.0), dict(eps=float("nan")),
                dict(x=None), dict(y=None), dict(ldx=63), dict(ldy=63), dict(q=P, ldq=64),
                dict(sc=P, lds=2), dict(q=P, sc=P, ldq=63, lds=2), dict(q=P, sc=P, ldq=64, lds=1)):
        assert fwd(**bad) == BAD, bad
    assert fwd(d=65537, ldx=65537, ldy=65537) == SHAPE
    for k in ("x", "y", "g", "s", "m", "r"):
        assert fwd(**{k: ODD}) == ALIGN, k

    need = M.mlp_layernorm_workspace_bytes(4, 64)
    assert need > 0 and M.mlp_layernorm_workspace_bytes(0, 64) == 0
    assert M.mlp_layernorm_workspace_bytes(1 << 20, 512) == 304 * 2 * 512 * 4

    def bwd(dy=P, dt=BF16, lddy=64, x=P, ldx=64, q=None, ldq=0, sc=None, lds=0, m=P, r=P, g=P,
            dr=None, ldr=0, T=4, d=64, dx=P, lddx=64, dg=P, ds=P, ws=P, n=need):
        return lib.mlp_layernorm_bwd(dy, dt, lddy, x, ldx, q, ldq, sc, lds, m, r, g, dr, ldr, T, d,
                                     dx, lddx, dg, ds, ws, n, None)
    for bad in (dict(T=-1), dict(d=0), dict(dt=U8), dict(dg=None), dict(ds=None), dict(dy=None),
                dict(dx=None), dict(m=None), dict(r=None), dict(lddy=63), dict(lddx=63),
                dict(ldx=63), dict(x=None), dict(q=P, sc=P, ldq=64, lds=2),  # both forms
                dict(x=None, q=P, ldq=64), dict(x=None, q=P, sc=P, ldq=64, lds=1),
                dict(sc=P, lds=2), dict(dr=P, ldr=63), dict(ws=None), dict(n=need - 1)):
        assert bwd(**bad) == BAD, bad
    assert bwd(d=65537) == SHAPE
    for k in ("dy", "x", "m", "r", "g", "dx", "dg", "ds", "ws"):
        assert bwd(**{k: ODD}) == ALIGN, k
    assert bwd(dr=ODD, ldr=64) == ALIGN


def test_linear(lib):
    f = ctypes.c_float

    def fwd(x=P, ldx=64, w=P, ldw=96, T=16, k=64, n=96, dt=BF16, b=P, act=3, r=None, ldr=0, y=P,
            ldy=96, ydt=BF16, u=None, ldu=0, q=None, ldq=0, sc=None, lds=0, ws=None, wsn=0):
        return lib.mlp_linear_fwd(x, ldx, w, ldw, T, k, n, dt, b, act, f(0.5), r, ldr, y, ldy, ydt,
                                  u, ldu, q, ldq, sc, lds, ws, wsn, None)
    assert fwd(T=0, x=None, w=None, y=None) == OK
    for bad in (dict(T=-1), dict(k=0), dict(n=0), dict(dt=U8), dict(act=6), dict(act=-1),
                dict(ydt=F16), dict(ydt=U8), dict(dt=F32, ydt=BF16), dict(x=None), dict(w=None),
                dict(y=None), dict(ldx=56), dict(ldw=88), dict(ldy=95), dict(r=P, ldr=95),
                dict(u=P, ldu=95), dict(q=P, ldq=96), dict(q=P, sc=P, ldq=96, lds=2)):
        assert fwd(**bad) == BAD, bad
    for k in ("x", "w", "b", "y", "ws"):
        assert fwd(**{k: ODD}) == ALIGN, k
    # 16-bit rows start on 16 bytes
    assert fwd(ldx=66) == ALIGN and fwd(ldw=100) == ALIGN
    assert fwd(k=(1 << 24) + 1) == SHAPE
    # split sums need their workspace
    need = M.mlp_linear_workspace_bytes(64, 8192, 128, torch.bfloat16)
    assert need > 0 and M.mlp_linear_workspace_bytes(1, 8192, 128, torch.bfloat16) == 0
    long = dict(T=64, k=8192, n=128, ldx=8192, ldw=128, ldy=128)
    assert fwd(**long) == BAD and fwd(**long, ws=P, wsn=need - 1) == BAD
    assert M.mlp_linear_workspace_bytes(65536, 512, 1536, torch.bfloat16) == 0
    assert M.mlp_linear_workspace_bytes(100, 64, 96, torch.float32) == 100 * 96 * 4 \
        + (-100 * 96 * 4) % 256

    def bwd(dy=P, lddy=96, w=P, ldw=96, T=16, di=64, do=96, dt=BF16, act=3, u=P, ldu=64, q=None,
            ldq=0, sc=None, lds=0, du=P, lddu=64, dudt=BF16, db=None, a=None, lda=0, ws=None,
            wsn=0):
        return lib.mlp_linear_bwd(dy, lddy, w, ldw, T, di, do, dt, act, f(0.5), u, ldu, q, ldq, sc,
                                  lds, du, lddu, dudt, db, a, lda, ws, wsn, None)
    assert bwd(T=0, dy=None, w=None, du=None, u=None) == OK
    for bad in (dict(T=-1), dict(di=0), dict(do=0), dict(dt=U8), dict(act=6), dict(dudt=F16),
                dict(dy=None), dict(w=None), dict(du=None), dict(lddy=88), dict(ldw=88),
                dict(lddu=63), dict(ldu=63), dict(u=None), dict(q=P, sc=P, ldq=64, lds=2),
                dict(u=None, q=P, ldq=64), dict(u=None, act=0, a=P, lda=64), dict(a=P, lda=63),
                dict(db=P)):
        assert bwd(**bad) == BAD, bad
    for k in ("dy", "w", "u", "du", "db", "ws"):
        assert bwd(**{k: ODD}) == ALIGN, k
    assert bwd(lddy=100) == ALIGN and bwd(ldw=100) == ALIGN
    assert bwd(db=P, ws=P, wsn=M.mlp_linear_bwd_workspace_bytes(16, 64, 96, torch.bfloat16) - 1) == BAD

    def act(dy=P, lddy=64, T=16, n=64, dt=F32, act=3, u=P, ldu=64, q=None, ldq=0, sc=None, lds=0,
            du=P, lddu=64, db=None, a=None, lda=0, ws=None, wsn=0):
        return lib.mlp_act_bwd(dy, lddy, T, n, dt, act, f(0.5), u, ldu, q, ldq, sc, lds, du, lddu,
                               db, a, lda, ws, wsn, None)
    assert act(T=0, dy=None, du=None, u=None) == OK
    for bad in (dict(T=-1), dict(n=0), dict(dt=U8), dict(act=6), dict(dy=None), dict(du=None),
                dict(lddy=63), dict(lddu=63), dict(ldu=63), dict(u=None), dict(a=P, lda=63),
                dict(q=P, sc=P, ldq=64, lds=2), dict(db=P),
                dict(db=P, ws=P, wsn=M.mlp_act_bwd_workspace_bytes(16, 64) - 1)):
        assert act(**bad) == BAD, bad
    for k in ("dy", "u", "du", "db", "ws"):
        assert act(**{k: ODD}) == ALIGN, k


def test_stack_with_8bit_checkpoints(lib):
    f = ctypes.c_float
    st = [P, P, P, P, P, P, f(0.02), f(0.95), P, P]
    need = M.mlp_stack_ckpt8_workspace_bytes(3, 8, 512, 1536)
    call = lambda n, T, h, ws, a=st: lib.mlp_stack_train_step_ckpt8(n, T, 512, h, f(1e-6), f(0.5),
                                                                    *a, ws, None)
    assert need > 0 and M.mlp_stack_ckpt8_workspace_bytes(3, 8, 512, 1000) == 0
    assert call(0, 8, 1536, need) == BAD and call(3, -1, 1536, need) == BAD
    assert call(3, 8, 1536, need - 1) == BAD and call(3, 8, 1000, need) == SHAPE
    assert call(3, 0, 1536, 0) == OK
    assert call(3, 8, 1536, need, [ODD] + st[1:]) == ALIGN
    # the kept activations halve (and their scales: 1/32)
    full = M.mlp_stack_workspace_bytes(11, 262144, 512, 1536)
    small = M.mlp_stack_ckpt8_workspace_bytes(11, 262144, 512, 1536)
    td = 262144 * 512
    assert full - small == 11 * td * 2 - 10 * (td + td // 32) - td * 2


def test_binding_refuses_what_the_library_cannot_read():
    """Host tensors, other shapes and types never reach a kernel."""
    x = torch.zeros(4, 64)
    v = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA device"):
        M.mlp_layernorm_fwd(x, x)
    with pytest.raises(ValueError, match="CUDA device"):
        M.mlp_ckpt8_encode(x, x.to(torch.int8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA device"):
        M.mlp_linear_fwd(x, torch.zeros(64, 64), x)
    with pytest.raises(ValueError, match="CUDA device"):
        M.mlp_act_bwd(x, x, u=x)
    with pytest.raises(ValueError, match=r"\[4, 64\]"):
        M._mat(x[:, :32], "y", 4, 64, 0)
    with pytest.raises(TypeError):
        M._mat(x, "y", 4, 64, 0, torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        M._mat(x, "y", 4, 64, 0)
    with pytest.raises(ValueError, match="adjacent"):
        M._mat(torch.zeros(64, 4).t(), "y", 4, 64, -1)
    with pytest.raises(ValueError):
        M._vec(v[:32], "gain", 64, 0)
    with pytest.raises(TypeError):
        M._vec(v.double(), "gain", 64, 0)
    with pytest.raises(ValueError, match="CUDA device"):
        M._ws(x, 0)
    with pytest.raises(TypeError):
        M.mlp_linear_workspace_bytes(4, 64, 64, torch.float64)
