"""The gated feed-forward sublayer's operators where a block, a cluster or a thread
takes several rows, chunks or pieces one after the other, and every form of a call
beside every other; against the 64-bit formulas and tolerances of their own
modules."""
import math

import pytest
import torch

import mlp_step_gb300 as M
import test_gpu_glu as glu
import test_gpu_resnorm as rn
import test_gpu_sublayer as sublayer
from philox import factor, keep_mask
from test_gpu_ffn import (ACTS, BF16, F16, F32, SLOPE, U24, Guarded, ckpt_values, near, new_ckpt,
                          rnd, rounding, vec)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    M.load()
    yield
    assert M.get_device_status() == M.MLP_OK


# ------------------------------------------------------------ rows one after the other

# More rows than a launch holds at once: 152 SMs with one to four blocks, or some
# twenty to seventy clusters of eight to two blocks.  Row sums exchanged many
# times, both turns of the rings, fp32 rows of more than 4,096 columns (no row
# ahead), partial sums over the rows of a block or cluster; rows that start
# anywhere beside whole pieces.
WALKS = [(10_007, 512, 513), (9000, 200, None), (2000, 1024, None), (2000, 2000, 2001),
         (2000, 4096, None), (700, 4100, 4101), (700, 8192, None), (2000, 8200, 8201),
         (2000, 16384, None), (400, 20000, None), (100, 65536, None)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", WALKS)
def test_resnorm_forward(T, d, pitch, dtype):
    rn.test_forward(T, d, pitch, dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", WALKS)
def test_resnorm_backward(T, d, pitch, dtype):
    rn.test_backward(T, d, pitch, dtype)


# Pieces of a thread's that wrap to later rows, several times over.
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", [(20_011, 1001, 1003), (300_007, 33, 35), (150, 65_537, None)])
def test_dropout(T, d, pitch, dtype):
    rn.test_dropout(T, d, pitch, dtype)


# ------------------------------------------------------------ forms of the residual norm

def unit(m):
    """The same inputs with gains of 1."""
    return {**m, "pg": torch.ones_like(m["pg"]), "ng": torch.ones_like(m["ng"])}


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", [(37, 512, None), (300, 333, 335), (40, 8200, 8201)])
def test_resnorm_without_gains(T, d, pitch, dtype):
    """Gains left out are ones, in the values and in the gradients that are wanted
    all the same; each of the two sums alone, and neither."""
    m = rn.inputs(T, d, dtype, pitch)
    ones = unit(m)
    rstd = rn.rstds(m)
    ws = glu.bytes_for(M.mlp_resnorm_workspace_bytes(T, d))
    rng = rn.state()
    for form in rn.FORMS:
        k = factor(T, d, form["p"], rn.SEED, rn.STEP, rn.SITE)
        out = {o: torch.full_like(m["x"], math.nan) for o in ("h", "n")}
        out.update({r: torch.full((T,), math.nan, device="cuda") for r in ("b_rstd", "h_rstd")})
        rn.run_forward({**m, "pg": None, "ng": None}, form, 0.5, out, rng=rng)
        for o, (v, e) in rn.forward_ref(ones, form, 0.5, k).items():
            near(out[o], v, rounding(F32 if v.dim() == 1 else dtype, v) + e + 1e-30,
                 "%s %s" % (o, form))
        ref = rn.backward_ref(ones, form, 0.5, k, True, rstd)
        for post, nxt in ((True, True), (True, False), (False, True), (False, False)):
            g = {o: torch.full_like(m["x"], math.nan) for o in ("dx", "db", "dz")}
            g["dpost"] = torch.full((d,), math.nan, device="cuda") if post else None
            g["dnext"] = torch.full((d,), math.nan, device="cuda") if nxt else None
            rn.run_backward({**m, "pg": None, "ng": None}, form, 0.5, True, rstd, g,
                            ws if post or nxt else None, rng=rng)
            for o, (v, e) in ref.items():
                if g[o] is not None:
                    near(g[o], v, rounding(F32 if v.dim() == 1 else dtype, v) + e + 1e-30,
                         "%s %s" % (o, form))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", [(5, 64, None), (300, 333, 335), (700, 8192, None),
                                       (60, 8200, 8201)])
def test_resnorm_in_the_blocks_place(T, d, pitch, dtype):
    """h in b's place, as it is and with x and b one matrix."""
    m = rn.inputs(T, d, dtype, pitch)
    for form in rn.FORMS[:6]:
        for same in (False, True):
            q = dict(m, x=m["b"]) if same else dict(m)
            new = lambda: {**{o: rnd(9, T, d, dtype, pitch=pitch) for o in ("h", "n")},  # noqa: E731
                           **{r: torch.zeros(T, device="cuda") for r in ("b_rstd", "h_rstd")}}
            want, got = new(), new()
            rn.run_forward(q, form, 0.5, want, rng=rn.state())
            b = rnd(11, T, d, dtype, pitch=pitch)
            b.copy_(m["b"])
            q["b"] = got["h"] = b
            if same:
                q["x"] = b
            rn.run_forward(q, form, 0.5, got, rng=rn.state())
            for o in want:
                assert torch.equal(got[o], want[o]), (o, form, same)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d", [(3, 40), (400, 1000), (50, 9000)])
def test_resnorm_with_everything_dropped(T, d, dtype):
    """p = 1: h is x, and nothing reaches the block."""
    m = rn.inputs(T, d, dtype, None)
    m["b"][0, 0] = math.inf
    form = dict(rn.FORMS[0], p=1.0, post=False)
    out = {o: torch.full_like(m["x"], math.nan) for o in ("h", "n")}
    out["h_rstd"] = torch.zeros(T, device="cuda")
    rn.run_forward(m, form, 0.5, out, rng=rn.state())
    n, r = torch.empty_like(m["x"]), torch.empty(T, device="cuda")
    M.mlp_resnorm_fwd(m["x"], n=n, next_gain=m["ng"], h_rstd=r, eps=rn.EPS)
    assert torch.equal(out["h"], m["x"]) and torch.equal(out["n"], n)
    assert torch.equal(out["h_rstd"], r)
    rstd = rn.rstds(m)
    g = {o: torch.full_like(m["x"], math.nan) for o in ("dx", "db", "dz")}
    g.update({o: torch.full((d,), math.nan, device="cuda") for o in ("dpost", "dnext")})
    ws = glu.bytes_for(M.mlp_resnorm_workspace_bytes(T, d))
    m["b"][0, 0] = 1
    rn.run_backward(m, form, 0.5, True, rstd, g, ws, rng=rn.state())
    assert all((g[o] == 0).all() for o in ("db", "dz", "dpost"))
    alone = {o: torch.full_like(t, math.nan) for o, t in g.items()}
    rn.run_backward(m, rn.FORMS[6], 0.5, True, rstd, alone, ws)
    assert torch.equal(g["dx"], alone["dx"])
    near(g["dnext"], alone["dnext"], 2 * (T + 10) * U24 *
         (m["dn"].double() * m["x"].double() * rstd["h"].double()[:, None]).abs().sum(0), "dnext")


def test_masks_of_the_two_operators_agree():
    """The residual norm drops the places that dropout alone drops."""
    T, d, p = 301, 777, 0.3
    one, zero = torch.ones(T, d, device="cuda"), torch.zeros(T, d, device="cuda")
    h = torch.empty_like(one)
    M.mlp_resnorm_fwd(zero, b=one, h=h, p=p, rng=rn.state(), site=rn.SITE)
    y = torch.empty_like(one)
    M.mlp_dropout(one, y, p, rn.state(), site=rn.SITE)
    assert torch.equal(h, y)
    assert torch.equal(h != 0, keep_mask(T, d, p, rn.SEED, rn.STEP, rn.SITE))


# ------------------------------------------------------------ gated units

# Few rows whose slice of K takes a CTA several chunks, with clusters that the
# number of resident CTAs limits, and with more CTAs than are resident.
@pytest.mark.parametrize("T,k,n,dtype", [(8, 1500, 9000, F32), (6, 600, 11_008, F32),
                                         (4, 4500, 6001, F32), (1, 40_000, 1001, F32),
                                         (1, 9000, 19_001, BF16), (2, 4500, 20_000, F16),
                                         (1, 200, 40_003, F16)])
def test_few_rows_in_several_chunks(T, k, n, dtype):
    x = rnd(40, T, k, dtype)
    wg, wu = rnd(41, k, n, dtype, std=k ** -0.5), rnd(42, k, n, dtype, std=k ** -0.5)
    bg, bu = vec(43, n), vec(44, n)
    y, g, u = (Guarded(T, n, dtype) for _ in range(3))
    (gq, gs), (uq, us) = new_ckpt(T, n), new_ckpt(T, n)
    ws = glu.bytes_for(M.mlp_glu_workspace_bytes(T, k, n, dtype))
    rg, eg, ru, eu, ry, ey = glu.forward_ref(x, wg, wu, bg, bu, "silu")
    for kw in (dict(g=g.v, u=u.v), dict(g_ckpt=(gq.v, gs.v), u_ckpt=(uq.v, us.v))):
        y.v.fill_(math.nan)
        M.mlp_glu_fwd(x, wg, wu, y.v, b_gate=bg, b_up=bu, workspace=ws, **kw)
        near(y.v, ry, rounding(dtype, ry) + ey, "y")
    near(g.v, rg, rounding(dtype, rg) + eg + 1e-30, "g")
    near(u.v, ru, rounding(dtype, ru) + eu + 1e-30, "u")
    glu.near_ckpt(gq, gs, rg, eg, "8-bit g")
    glu.near_ckpt(uq, us, ru, eu, "8-bit u")
    assert y.intact() and g.intact() and u.intact()


# A shape of each path: few rows, one CTA's tiles with and without a split of K,
# pairs with ragged and with whole pieces.
PATHS = [(2, 520, 136), (40, 2056, 200), (300, 136, 1001), (4100, 200, 776), (2600, 72, 1152)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T,k,n", PATHS)
def test_every_activation_in_every_form(T, k, n, act, dtype):
    x = rnd(40, T, k, dtype)
    wg, wu = rnd(41, k, n, dtype, std=k ** -0.5), rnd(42, k, n, dtype, std=k ** -0.5)
    bg, bu = vec(43, n), vec(44, n)
    ws = glu.bytes_for(max(M.mlp_glu_workspace_bytes(T, k, n, dtype),
                           M.mlp_glu_bwd_workspace_bytes(T, n, k, dtype)))
    rg, eg, ru, eu, ry, ey = glu.forward_ref(x, wg, wu, bg, bu, act)
    for form in ("none", "same", "ckpt"):
        y, g, u = (Guarded(T, n, dtype) for _ in range(3))
        (gq, gs), (uq, us) = new_ckpt(T, n), new_ckpt(T, n)
        kw = {"same": dict(g=g.v, u=u.v), "none": {},
              "ckpt": dict(g_ckpt=(gq.v, gs.v), u_ckpt=(uq.v, us.v))}[form]
        M.mlp_glu_fwd(x, wg, wu, y.v, b_gate=bg, b_up=bu, act=ACTS[act], slope=SLOPE,
                      workspace=ws, **kw)
        near(y.v, ry, rounding(dtype, ry) + ey, "y %s" % form)
        if form == "same":
            near(g.v, rg, rounding(dtype, rg) + eg + 1e-30, "g")
            near(u.v, ru, rounding(dtype, ru) + eu + 1e-30, "u")
        elif form == "ckpt":
            glu.near_ckpt(gq, gs, rg, eg, "8-bit g")
            glu.near_ckpt(uq, us, ru, eu, "8-bit u")
        assert y.intact() and g.intact() and u.intact()
    # backward
    dy, w = rnd(50, T, k, dtype, std=0.1), rnd(51, n, k, dtype, std=n ** -0.5)
    g, u = rnd(52, T, n, dtype, std=1.5), rnd(53, T, n, dtype, std=1.5)
    cg, cu = ([m.v for m in new_ckpt(T, n)] for _ in range(2))
    M.mlp_ckpt8_encode(g, *cg)
    M.mlp_ckpt8_encode(u, *cu)
    for kw, sg, su in ((dict(g=g, u=u), g.double(), u.double()),
                       (dict(g_ckpt=cg, u_ckpt=cu), ckpt_values(*cg), ckpt_values(*cu))):
        rdg, edg, rdu, edu, ra, ea = glu.backward_ref(dy, w, sg, su, act)
        for again in (False, True):
            for sums in (False, True):
                dg, du, a = (Guarded(T, n, dtype) for _ in range(3))
                db = [torch.full((n,), math.nan, device="cuda") for _ in range(2)]
                M.mlp_glu_bwd(dy, w, dg.v, du.v, act=ACTS[act], slope=SLOPE,
                              db_gate=db[0] if sums else None, db_up=db[1] if sums else None,
                              a=a.v if again else None, workspace=ws, **kw)
                near(dg.v, rdg, rounding(dtype, rdg) + edg, "dg")
                near(du.v, rdu, rounding(dtype, rdu) + edu, "du")
                if again:
                    near(a.v, ra, rounding(dtype, ra) + ea, "a")
                if sums:
                    for got, r, e in ((db[0], rdg, edg), (db[1], rdu, edu)):
                        near(got, r.sum(0), e.sum(0) + (T + 8) * U24 * r.abs().sum(0), "db")
                assert dg.intact() and du.intact() and a.intact()


# ------------------------------------------------------------ a training step

@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,hidden", [(1, 64, 96), (77, 128, 232), (3000, 512, 1376)])
def test_training_step_call_by_call(T, d, hidden, dtype, ckpt):
    """Every output of a step against the 64-bit formula of what the calls before
    it left, to the roundings of its own call."""
    s = sublayer.Sublayer(T, d, hidden, dtype, ckpt)
    s.forward()
    s.backward()
    o, gain = s.out, s.gains
    norm, both = rn.FORMS[6], dict(rn.FORMS[0], p=sublayer.P)
    seed, step = s.rng.tolist()
    k = factor(T, d, sublayer.P, seed, step, sublayer.SITE)

    def check(name, ref, err, got=None):
        got = o[name] if got is None else got
        near(got, ref, rounding(got.dtype, ref) + err + 1e-30, name)

    # forward
    ref = rn.forward_ref(dict(x=s.x, ng=gain[0]), norm, 1.0, None)
    check("n0", *ref["n"])
    check("r0", *ref["h_rstd"])
    rg, eg, ru, eu, ry, ey = glu.forward_ref(o["n0"], *s.halves(s.w), None, None, "silu")
    check("y", ry, ey)
    if not ckpt:
        check("g", rg, eg, s.kept[0])
        check("u", ru, eu, s.kept[1])
    check("b", *glu.product(o["y"], s.wd))
    m = dict(x=s.x, b=o["b"], z=s.z, pg=gain[1], ng=gain[2])
    ref = rn.forward_ref(m, both, sublayer.SCALE, k)
    for name, key in (("h", "h"), ("n1", "n"), ("rb", "b_rstd"), ("rh", "h_rstd")):
        check(name, *ref[key])
    # backward
    m.update(x=o["h"], dh=s.dh, dn=s.dn)
    ref = rn.backward_ref(m, both, sublayer.SCALE, k, True, dict(h=o["rh"], b=o["rb"]))
    for name, key in (("dx1", "dx"), ("db", "db"), ("dz", "dz"), ("dpost", "dpost"),
                      ("dnext", "dnext")):
        check(name, *ref[key])
    g, u = (ckpt_values(*v) if ckpt else v.double() for v in s.kept)
    rdg, edg, rdu, edu, ra, ea = glu.backward_ref(o["db"], s.wd, g, u, "silu")
    dg, du = s.halves(o["dgu"])
    check("dg", rdg, edg, dg)
    check("du", rdu, edu, du)
    check("a", ra, ea)
    check("dwd", *glu.product(o["a"].t(), o["db"]))
    check("dn0", *glu.product(o["dgu"], s.w.t()))
    check("dw", *glu.product(o["n0"].t(), o["dgu"]))
    ref = rn.backward_ref(dict(x=s.x, dh=o["dx1"], dn=o["dn0"], ng=gain[0]), norm, 1.0, None, True,
                          dict(h=o["r0"]))
    check("dx", *ref["dx"])
    check("dgain0", *ref["dnext"])
