"""Gated units (both projections, activation and product; the backward through
the down projection and the gate) against plain 64-bit implementations.

Tolerances are sums of the roundings an output goes through, as in
test_gpu_ffn.py: half a step of its type, and for the sums in fp32 before it the
number of additions times 2^-24 (2^-23 on the tensor cores, whose additions may
truncate) of the sum of magnitudes, carried through the formulas."""
import math

import pytest
import torch

import mlp_step_gb300 as M
from test_gpu_ffn import (ACT_ERR, ACTS, BF16, F16, F32, SLOPE, U24, Guarded, act_ref, ckpt_ref,
                          ckpt_values, near, new_ckpt, rnd, rounding, vec)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    M.load()
    yield
    assert M.get_device_status() == M.MLP_OK


def bytes_for(n):
    """A workspace of n bytes that holds NaN."""
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


def near_ckpt(q, s, ref, err, what):
    """The 8-bit form (Guarded q, s) of values within err of ref."""
    lo, hi = ckpt_ref((ref.abs() - err).clamp(min=0))[1], ckpt_ref(ref.abs() + err)[1]
    assert ((s.v >= lo) & (s.v <= hi)).all(), what
    step = (s.v.to(torch.int64) - 133 + 1023).bitwise_left_shift(52).view(torch.float64)
    step = step.repeat_interleave(32, 1)[:, :ref.shape[1]]
    near(ckpt_values(q.v, s.v), ref, step * torch.where(q.v.abs() == 127, 1.0, 0.5) + err, what)
    assert q.intact() and s.intact(), what


def product(x, w, bias=None):
    """x w + bias in 64 bits, and a bound of the kernels' error."""
    k = x.shape[1]
    r = x.double() @ w.double()
    e = (k + 8) * 2 * U24 * (x.double().abs() @ w.double().abs())
    if bias is not None:
        r = r + bias.double()
        e = e + U24 * r.abs() + U24 * bias.double().abs()
    return r, e


def forward_ref(x, wg, wu, bg, bu, act):
    """(g, error of g, u, error of u, y, error of y before its rounding)"""
    (g, eg), (u, eu) = product(x, wg, bg), product(x, wu, bu)
    f, df, curve = act_ref(g, act)
    ef = (1.0 if act == "relu" else df.abs()) * eg + curve * eg * eg
    if act not in ("none", "relu"):
        ef = ef + ACT_ERR * (1 + g.abs()) * (1 + f.abs())
    y = f * u
    return g, eg, u, eu, y, ef * (u.abs() + eu) + f.abs() * eu + 2 * U24 * y.abs() + 1e-30


def backward_ref(dy, w, g, u, act):
    """da f'(g) u, da f(g), f(g) u and bounds of their errors before the rounding"""
    da, eda = product(dy, w.t())
    f, df, _ = act_ref(g, act)
    ef = ACT_ERR * (1 + g.abs()) * (act not in ("none", "relu"))
    dg, du, a = da * df * u, da * f, f * u
    edg = u.abs() * (eda * df.abs() + (da.abs() + eda) * ef) + 3 * U24 * dg.abs() + 1e-30
    edu = eda * f.abs() + (da.abs() + eda) * ef * (1 + f.abs()) + 2 * U24 * du.abs() + 1e-30
    return dg, edg, du, edu, a, ef * (1 + f.abs()) * u.abs() + 2 * U24 * a.abs() + 1e-30


# few rows, split and unsplit tiles of one CTA, pairs with short and long K;
# ragged everywhere
SHAPES = [(1, 1, 1), (1, 512, 1408), (2, 784, 10), (3, 1000, 257), (5, 2056, 136), (8, 77, 72),
          (9, 512, 256), (33, 4096, 200), (100, 784, 256), (128, 1000, 1000), (257, 72, 2000),
          (1500, 520, 1001), (2000, 136, 1600), (4100, 200, 768), (3300, 1160, 1100)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,k,n", SHAPES)
def test_forward(T, k, n, dtype):
    for i, act in enumerate(ACTS):
        form = ("same", "ckpt", "none")[i % 3]
        x = rnd(40, T, k, dtype)
        wg, wu = rnd(41, k, n, dtype, std=k ** -0.5), rnd(42, k, n, dtype, std=k ** -0.5)
        bg, bu = vec(43, n) if i != 5 else None, vec(44, n) if i > 1 else None
        y, g, u = (Guarded(T, n, dtype) for _ in range(3))
        (gq, gs), (uq, us) = new_ckpt(T, n), new_ckpt(T, n)
        ws = bytes_for(M.mlp_glu_workspace_bytes(T, k, n, dtype))
        kw = {"same": dict(g=g.v, u=u.v), "none": {},
              "ckpt": dict(g_ckpt=(gq.v, gs.v), u_ckpt=(uq.v, us.v))}[form]
        M.mlp_glu_fwd(x, wg, wu, y.v, b_gate=bg, b_up=bu, act=ACTS[act], slope=SLOPE,
                      workspace=ws, **kw)
        rg, eg, ru, eu, ry, ey = forward_ref(x, wg, wu, bg, bu, act)
        near(y.v, ry, rounding(dtype, ry) + ey, "y %s" % act)
        assert y.intact()
        if form == "same":
            near(g.v, rg, rounding(dtype, rg) + eg + 1e-30, "g")
            near(u.v, ru, rounding(dtype, ru) + eu + 1e-30, "u")
            assert g.intact() and u.intact()
        elif form == "ckpt":
            near_ckpt(gq, gs, rg, eg, "8-bit g")
            near_ckpt(uq, us, ru, eu, "8-bit u")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,k,n", SHAPES)
def test_backward(T, k, n, dtype):
    for i, act in enumerate(ACTS):
        ck, again, sums = i % 2 == 1, i % 3 != 0, i != 2
        dy, w = rnd(50, T, k, dtype, std=0.1), rnd(51, n, k, dtype, std=n ** -0.5)
        g, u = rnd(52, T, n, dtype, std=1.5), rnd(53, T, n, dtype, std=1.5)
        kw, sg, su = dict(g=g, u=u), g.double(), u.double()
        if ck:
            cg, cu = ([m.v for m in new_ckpt(T, n)] for _ in range(2))
            M.mlp_ckpt8_encode(g, *cg)
            M.mlp_ckpt8_encode(u, *cu)
            kw, sg, su = dict(g_ckpt=cg, u_ckpt=cu), ckpt_values(*cg), ckpt_values(*cu)
        ws = bytes_for(M.mlp_glu_bwd_workspace_bytes(T, n, k, dtype))

        def call():
            out = [Guarded(T, n, dtype) for _ in range(3)]
            db = [torch.full((n,), math.nan, device="cuda") for _ in range(2)]
            M.mlp_glu_bwd(dy, w, out[0].v, out[1].v, act=ACTS[act], slope=SLOPE,
                          db_gate=db[0] if sums else None, db_up=db[1] if sums else None,
                          a=out[2].v if again else None, workspace=ws, **kw)
            return out, db
        (dg, du, a), db = call()
        rdg, edg, rdu, edu, ra, ea = backward_ref(dy, w, sg, su, act)
        near(dg.v, rdg, rounding(dtype, rdg) + edg, "dg %s" % act)
        near(du.v, rdu, rounding(dtype, rdu) + edu, "du %s" % act)
        assert dg.intact() and du.intact()
        if again:
            near(a.v, ra, rounding(dtype, ra) + ea, "a %s" % act)
            assert a.intact()
        else:
            assert (a.buf == -77).all()
        if sums:
            near(db[0], rdg.sum(0), edg.sum(0) + (T + 8) * U24 * rdg.abs().sum(0), "db_gate")
            near(db[1], rdu.sum(0), edu.sum(0) + (T + 8) * U24 * rdu.abs().sum(0), "db_up")
        (dg2, du2, a2), db2 = call()  # the same bits again
        assert torch.equal(dg.v, dg2.v) and torch.equal(du.v, du2.v)
        assert not sums or (torch.equal(db[0], db2[0]) and torch.equal(db[1], db2[1]))


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,k,n", [(3, 512, 200), (40, 4096, 200), (300, 520, 1001),
                                   (4100, 200, 776), (3300, 1160, 1100)])
def test_pitches_and_halves_of_one_matrix(T, k, n, dtype, odd):
    """W_gate and W_up as the halves of one matrix, and everything of the
    epilogue in matrices whose rows TMA can and cannot address."""
    n8 = (n + 7) // 8 * 8
    pitch = n + 3 if odd else None
    x = rnd(60, T, k, dtype)
    w = rnd(61, k, n8 + n, dtype, std=k ** -0.5)
    wg, wu = w[:, :n], w[:, n8:]
    y, g, u = (Guarded(T, n, dtype, pitch) for _ in range(3))
    (gq, gs), (uq, us) = new_ckpt(T, n, pitch), new_ckpt(T, n, pitch)
    ws = bytes_for(M.mlp_glu_workspace_bytes(T, k, n, dtype))
    rg, eg, ru, eu, ry, ey = forward_ref(x, wg, wu, None, None, "silu")
    for kw in (dict(g=g.v, u=u.v), dict(g_ckpt=(gq.v, gs.v), u_ckpt=(uq.v, us.v))):
        y.v.fill_(math.nan)
        M.mlp_glu_fwd(x, wg, wu, y.v, workspace=ws, **kw)
        near(y.v, ry, rounding(dtype, ry) + ey, "y")
        assert y.intact()
    near(g.v, rg, rounding(dtype, rg) + eg + 1e-30, "g")
    near(u.v, ru, rounding(dtype, ru) + eu + 1e-30, "u")
    assert g.intact() and u.intact()
    near_ckpt(gq, gs, rg, eg, "8-bit g")
    near_ckpt(uq, us, ru, eu, "8-bit u")
    # backward of dy = x through W_down = (x's width -> n)
    wd = rnd(62, n, k, dtype, std=k ** -0.5)
    bws = bytes_for(M.mlp_glu_bwd_workspace_bytes(T, n, k, dtype))
    for kw, sg, su in ((dict(g=g.v, u=u.v), g.v.double(), u.v.double()),
                       (dict(g_ckpt=(gq.v, gs.v), u_ckpt=(uq.v, us.v)),
                        ckpt_values(gq.v, gs.v), ckpt_values(uq.v, us.v))):
        dg, du, a = (Guarded(T, n, dtype, pitch) for _ in range(3))
        db = torch.empty(2, n8, device="cuda")[:, :n]
        M.mlp_glu_bwd(x, wd, dg.v, du.v, db_gate=db[0], db_up=db[1], a=a.v, workspace=bws, **kw)
        rdg, edg, rdu, edu, ra, ea = backward_ref(x, wd, sg, su, "silu")
        near(dg.v, rdg, rounding(dtype, rdg) + edg, "dg")
        near(du.v, rdu, rounding(dtype, rdu) + edu, "du")
        near(a.v, ra, rounding(dtype, ra) + ea, "a")
        near(db[0], rdg.sum(0), edg.sum(0) + (T + 8) * U24 * rdg.abs().sum(0), "db_gate")
        near(db[1], rdu.sum(0), edu.sum(0) + (T + 8) * U24 * rdu.abs().sum(0), "db_up")
        assert dg.intact() and du.intact() and a.intact()
        # the gradients in the saved values' place
        if "g" in kw:
            M.mlp_glu_bwd(x, wd, g.v, u.v, db_gate=db[0], db_up=db[1], workspace=bws, **kw)
            assert torch.equal(g.v, dg.v) and torch.equal(u.v, du.v)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward_is_the_derivative(dtype):
    """dg and du against differences of sum(dy * (f(g) u W_down)) in 64 bits."""
    T, k, n = 5, 24, 40
    dy, w = rnd(70, T, k, dtype), rnd(71, n, k, dtype)
    g, u = rnd(72, T, n, dtype), rnd(73, T, n, dtype)
    for act in ("gelu", "gelu_tanh", "silu", "leaky2"):
        def loss(g_, u_):
            return (dy.double() * ((act_ref(g_, act)[0] * u_) @ w.double())).sum()
        dg, du = torch.empty_like(g), torch.empty_like(u)
        ws = bytes_for(M.mlp_glu_bwd_workspace_bytes(T, n, k, dtype))
        M.mlp_glu_bwd(dy, w, dg, du, act=ACTS[act], slope=SLOPE, g=g, u=u, workspace=ws)
        h = 1e-5
        for m, d in ((0, dg), (1, du)):
            for r, c in ((0, 0), (2, 17), (4, 39)):
                z = [g.double(), u.double()]
                z[m] = z[m].clone()
                z[m][r, c] += h
                up = loss(*z)
                z[m][r, c] -= 2 * h
                diff = (up - loss(*z)) / (2 * h)
                # the difference's own error: h^2 f''' (of the order of 10) and
                # rounding 1e-16 / h; the kernel's: its rounding and fp32 sums
                tol = float(rounding(dtype, diff.abs())) + 1e-5 * (1 + abs(float(diff)))
                assert abs(float(d[r, c]) - float(diff)) <= tol, (act, m, r, c)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,k,n", [(1, 64, 96), (40, 64, 96), (300, 1024, 96)])
def test_values_that_are_not_finite(T, k, n, dtype):
    """Infinite pre-activations give the limits of f; NaN stays where it is."""
    x = torch.zeros(T, k, dtype=dtype, device="cuda")
    x[:, 0] = 1
    wg, wu = (torch.zeros(k, n, dtype=dtype, device="cuda") for _ in range(2))
    wg[0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 2.0])
    wg[1] = 1.0
    wu[0] = 3.0
    wu[0, 40] = math.inf
    # columns with an infinity meet zeros of x only where k > 0, whose products are 0 * finite
    y = torch.empty(T, n, dtype=dtype, device="cuda")
    (gq, gs), (uq, us) = new_ckpt(T, n), new_ckpt(T, n)
    ws = bytes_for(M.mlp_glu_workspace_bytes(T, k, n, dtype))
    M.mlp_glu_fwd(x, wg, wu, y, act=M.MLP_ACT_SILU, g_ckpt=(gq.v, gs.v), u_ckpt=(uq.v, us.v),
                  workspace=ws)
    assert (y[:, 0] == math.inf).all() and (y[:, 1] == 0).all() and y[:, 2].isnan().all()
    assert (y[:, 3].double() - 2 / (1 + math.exp(-2)) * 3).abs().max() < 0.05
    assert (y[:, 4:40] == 0).all() and y[:, 40].isnan().all() and (y[:, 41:] == 0).all()
    assert (gs.v[:, 0] == 255).all() and (gs.v[:, 1:] != 255).all()
    assert (us.v[:, 1] == 255).all() and (us.v[:, 0] != 255).all() and (us.v[:, 2:] != 255).all()


def test_no_rows():
    w = torch.zeros(64, 96, dtype=BF16, device="cuda")
    none = torch.empty(0, 64, dtype=BF16, device="cuda")
    out = [torch.empty(0, 96, dtype=BF16, device="cuda") for _ in range(3)]
    M.mlp_glu_fwd(none, w, w, out[0], g=out[1], u=out[2])
    db = torch.full((2, 96), math.nan, device="cuda")
    M.mlp_glu_bwd(none, w.t().contiguous(), *out[:2], g=out[1], u=out[2], db_gate=db[0],
                  db_up=db[1])
    assert (db == 0).all()
