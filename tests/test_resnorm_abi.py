"""Argument checks of dropout and the residual norm, on the CPU (no call here
launches a kernel), and the tests' own generator against its published vectors."""
import ctypes

import pytest
import torch

import mlp_step_gb300 as M
from mlp_step_gb300 import build
from philox import LOW, factor, keep_mask, philox

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
ODD4 = ctypes.c_void_p(0x10004)
F32, BF16, U8 = M.MLP_DTYPE_F32, M.MLP_DTYPE_BF16, M.MLP_DTYPE_U8
OK, BAD, ALIGN, SHAPE = 0, 1, 2, 3
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return M.load()


def test_generator_gives_the_published_numbers():
    for counter, key, words in (
            ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
            ([LOW] * 4, [LOW] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
             [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])):
        got = philox([torch.tensor(v) for v in counter], key)
        assert [int(w) for w in got] == words
    m = keep_mask(64, 100, 0.25, 5, 6, 7, device="cpu")
    assert m.shape == (64, 100) and abs(float(m.double().mean()) - 0.75) < 0.03
    assert torch.equal(m[:, :33], keep_mask(64, 33, 0.25, 5, 6, 7, device="cpu"))
    assert (factor(4, 8, 1.0, 1, 2, 3, device="cpu") == 0).all()
    assert (factor(4, 8, 2.0 ** -18, 1, 2, 3, device="cpu") == 1).all()


def test_dropout(lib):
    def drop(x=P, ldx=64, r=None, ldr=0, T=4, d=64, dt=BF16, p=0.5, rng=P, site=0, y=P, ldy=64):
        return lib.mlp_dropout(x, ldx, r, ldr, T, d, dt, ctypes.c_float(p), rng, site, y, ldy, None)
    assert drop(T=0, x=None, y=None) == OK
    for bad in (dict(T=-1), dict(d=0), dict(dt=U8), dict(p=-0.1), dict(p=1.5), dict(p=NAN),
                dict(rng=None), dict(x=None), dict(y=None), dict(ldx=63), dict(ldy=63),
                dict(r=P, ldr=63)):
        assert drop(**bad) == BAD, bad
    for m in ("x", "y"):
        assert drop(**{m: ODD}) == ALIGN, m
    assert drop(r=ODD, ldr=64) == ALIGN and drop(rng=ODD4) == ALIGN
    assert drop(d=(1 << 24) + 1) == SHAPE


def test_forward(lib):
    def fwd(x=P, ldx=64, b=P, ldb=64, dt=BF16, post=1, pg=P, z=P, ldz=64, act=1, scale=0.5, p=0.5,
            rng=P, site=0, T=4, d=64, eps=1e-6, ng=P, h=P, ldh=64, n=P, ldn=64, br=P, hr=P):
        return lib.mlp_resnorm_fwd(x, ldx, b, ldb, dt, post, pg, z, ldz, act, ctypes.c_float(scale),
                                   ctypes.c_float(p), rng, site, T, d, ctypes.c_float(eps), ng, h,
                                   ldh, n, ldn, br, hr, None)
    assert fwd(T=0, x=None, b=None, h=None, n=None) == OK
    alone = dict(b=None, post=0, pg=None, z=None, p=0.0, h=None, br=None)
    for bad in (dict(T=-1), dict(d=0), dict(dt=U8), dict(eps=-1.0), dict(eps=NAN), dict(p=1.1),
                dict(p=NAN), dict(rng=None), dict(act=2), dict(x=None), dict(h=None),
                dict(b=None), dict(n=None), dict(n=None, ng=None), dict(n=None, hr=None),
                dict(post=0), *({**alone, m: v} for m, v in
                                (("post", 1), ("pg", P), ("z", P), ("p", 0.5), ("h", P), ("n", None),
                                 ("br", P))),
                *({m: 63} for m in ("ldx", "ldb", "ldz", "ldh", "ldn"))):
        assert fwd(**bad) == BAD, bad
    for m in ("x", "b", "pg", "z", "ng", "h", "n", "br", "hr"):
        assert fwd(**{m: ODD}) == ALIGN, m
    assert fwd(rng=ODD4) == ALIGN
    assert fwd(d=65537, ldx=1 << 17) == SHAPE


def test_backward(lib):
    need = M.mlp_resnorm_workspace_bytes(4, 64)
    assert need > 0 and M.mlp_resnorm_workspace_bytes(0, 64) == 0
    assert M.mlp_resnorm_workspace_bytes(4, 65537) == 0

    def bwd(dh=P, lddh=64, dn=P, lddn=64, h=P, ldh=64, hr=P, ng=P, b=P, ldb=64, dt=BF16, post=1,
            pg=P, br=P, z=P, ldz=64, act=1, scale=0.5, p=0.5, rng=P, site=0, T=4, d=64, dx=P,
            lddx=64, db=P, lddb=64, dz=P, lddz=64, dpg=P, dng=P, ws=P, wsn=need):
        return lib.mlp_resnorm_bwd(dh, lddh, dn, lddn, h, ldh, hr, ng, b, ldb, dt, post, pg, br, z,
                                   ldz, act, ctypes.c_float(scale), ctypes.c_float(p), rng, site, T,
                                   d, dx, lddx, db, lddb, dz, lddz, dpg, dng, ws, wsn, None)
    assert bwd(T=0, dh=None, dn=None, dx=None, dpg=None, dng=None) == OK
    alone = dict(b=None, db=None, post=0, pg=None, br=None, z=None, dz=None, p=0.0, dpg=None)
    rest = dict(dn=None, h=None, hr=None, ng=None, dng=None)
    for bad in (dict(T=-1), dict(d=0), dict(dt=U8), dict(p=-1.0), dict(rng=None), dict(act=-1),
                dict(dx=None), dict(h=None), dict(hr=None), dict(dn=None),
                {**rest, "ng": P}, {**rest, "dng": P}, {**rest, "dh": None}, dict(b=None),
                dict(db=None), dict(br=None), dict(z=None), dict(dz=None), dict(ws=None),
                dict(wsn=need - 1),
                *({**alone, m: v} for m, v in (("post", 1), ("pg", P), ("z", P), ("dz", P),
                                               ("db", P), ("p", 0.5), ("dpg", P))),
                *({m: 63} for m in ("lddh", "lddn", "ldh", "ldb", "ldz", "lddx", "lddb", "lddz"))):
        assert bwd(**bad) == BAD, bad
    for m in ("dh", "dn", "h", "hr", "ng", "b", "pg", "br", "z", "dx", "db", "dz", "dpg", "dng",
              "ws"):
        assert bwd(**{m: ODD}) == ALIGN, m
    assert bwd(T=0, dpg=ODD) == ALIGN and bwd(rng=ODD4) == ALIGN
    assert bwd(d=65537, lddh=1 << 17) == SHAPE


def test_binding_refuses_what_the_library_cannot_read():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        M.mlp_dropout(x, x, 0.5)
    with pytest.raises(ValueError, match="CUDA device"):
        M.mlp_resnorm_fwd(x, n=x)
    with pytest.raises(ValueError, match="CUDA device"):
        M.mlp_resnorm_bwd(x, dh=x)
    with pytest.raises(ValueError, match="site"):
        M._site(-1)
    with pytest.raises(ValueError, match="site"):
        M._site(1 << 32)
    M._load_torch()
    for wrong in (torch.zeros(3, dtype=torch.int64), torch.zeros(2), torch.zeros(4, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError, match="int64"):
            M._rng(wrong, 0)
    with pytest.raises(ValueError, match="CUDA device"):
        M._rng(torch.zeros(2, dtype=torch.int64), 0)
    with pytest.raises(ValueError, match="at most"):
        M.mlp_resnorm_workspace_bytes(1 << 31, 64)
