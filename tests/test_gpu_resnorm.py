"""Dropout and the residual norm (norm of a block's output, gate, dropout, scaled
residual, norm before the next block; and the backward) against plain 64-bit
implementations.

Tolerances count roundings as in test_gpu_ffn.py: U24 = 2^-24 per fp32 operation
relative to its result, S of them for a row's sum (16 values per thread, then a
tree over up to 512 threads and 8 blocks), carried through the formulas, and half
a step of the output's type."""
import math

import pytest
import torch

import mlp_step_gb300 as M
from philox import factor, keep_mask
from test_gpu_ffn import BF16, F16, F32, U24, Guarded, near, rnd, rounding, vec

pytestmark = pytest.mark.gpu

EPS = 1e-6
S = 16 + 10 + 8 + 8
SEED, STEP, SITE = 0x1234_5678_9ABC_DEF0, 7, 3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    M.load()
    yield
    assert M.get_device_status() == M.MLP_OK


def state(seed=SEED, step=STEP):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


# ------------------------------------------------------------ dropout

SHAPES = [(1, 1, None), (1, 512, None), (2, 7, 9), (9, 33, 40), (300, 256, None),
          (1001, 512, 520), (77, 520, 523), (515, 1000, 1000), (130, 2000, None),
          (65, 4099, 4100), (33, 8192, None), (7, 8200, 8201), (5, 20000, None),
          (3, 65536, None)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", SHAPES)
def test_dropout(T, d, pitch, dtype):
    x, r = rnd(1, T, d, dtype, std=2.0, pitch=pitch), rnd(2, T, d, dtype, pitch=pitch)
    for p in (0.0, 0.1, 0.5, 1.0):
        k = factor(T, d, p, SEED, STEP, SITE)
        for res in (None, r):
            y = Guarded(T, d, dtype, pitch)
            M.mlp_dropout(x, y.v, p, state(), site=SITE, residual=res)
            ref = x.double() * k
            tol = 2 * U24 * ref.abs()
            if res is not None:
                ref = ref + res.double()
                tol = tol + U24 * ref.abs()
            near(y.v, ref, rounding(dtype, ref) + tol, "y p %g" % p)
            assert y.intact()
            if res is None:
                assert torch.equal(y.v == 0, (k == 0) | (x == 0))
    y = x.clone()  # in place, as it is and as the residual
    M.mlp_dropout(y, y, 0.5, state(), site=SITE)
    z = r.clone()
    M.mlp_dropout(x, z, 0.5, state(), site=SITE, residual=z)
    once = torch.empty_like(x)
    M.mlp_dropout(x, once, 0.5, state(), site=SITE)
    assert torch.equal(y, once)
    M.mlp_dropout(x, once, 0.5, state(), site=SITE, residual=r)
    assert torch.equal(z, once)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dropout_masks(dtype):
    """The same place gives the same bit in every type and direction; other seeds,
    steps and sites give other masks, of the wanted share."""
    T, d, p = 1000, 777, 0.3
    one = torch.ones(T, d, dtype=dtype, device="cuda")
    y = torch.empty_like(one)
    seen = []
    for seed, step, site in ((SEED, STEP, SITE), (SEED + 1, STEP, SITE), (SEED, STEP + 1, SITE),
                             (SEED, STEP, SITE + 1), (-1, (1 << 32) - 1, (1 << 32) - 1),
                             (SEED + (1 << 32), STEP, SITE), (0, 0, 0)):
        M.mlp_dropout(one, y, p, state(seed, step), site=site)
        assert torch.equal(y != 0, keep_mask(T, d, p, seed, step, site)), (seed, step, site)
        seen.append((y != 0).clone())
        # 777,000 draws: five standard deviations of the share are 0.0026
        assert abs(float((y == 0).double().mean()) - p) < 0.0026
    for i, a in enumerate(seen):
        for b in seen[:i]:
            # two independent masks agree at p^2 + (1 - p)^2 = 0.58 of the places
            assert abs(float((a == b).double().mean()) - 0.58) < 0.003
    # the step counts by its low 32 bits
    M.mlp_dropout(one, y, p, state(SEED, STEP + (5 << 32)), site=SITE)
    assert torch.equal(y != 0, seen[0])
    # rows of a slice are rows of their own
    M.mlp_dropout(one[:500], y[:500], p, state(), site=SITE)
    assert torch.equal(y[:500] != 0, seen[0][:500])


def test_dropped_values_give_zero():
    x = torch.full((64, 96), math.nan, device="cuda")
    x[:, ::2] = math.inf
    y = torch.empty_like(x)
    M.mlp_dropout(x, y, 0.5, state(), site=SITE)
    keep = keep_mask(64, 96, 0.5, SEED, STEP, SITE)
    assert (y[~keep] == 0).all() and torch.equal(y.isnan(), x.isnan() & keep)
    M.mlp_dropout(x, y, 1.0, state())
    assert (y == 0).all()
    M.mlp_dropout(x, y, 2.0 ** -18, state())  # rounds to no dropout
    assert torch.equal(y.isnan(), x.isnan())
    M.mlp_dropout(x[:0], y[:0], 0.5, state())


def test_dropout_rows_past_32_bits_of_elements():
    """The last rows of a matrix of more than 2^31 values."""
    T, d = 33_000, 65_536
    x = torch.zeros(T, d, dtype=BF16, device="cuda")
    x[-2:] = 1
    M.mlp_dropout(x, x, 0.25, state(), site=SITE)
    k = factor(T, 8, 0.25, SEED, STEP, SITE)[-2:]
    assert torch.equal(x[-2:, :8].double() != 0, k != 0)
    assert (x[:-2].view(torch.int16).count_nonzero(dim=1) == 0).all()


# ------------------------------------------------------------ residual norm

# block, norm of its output, gate, dropout, norm before the next block
FORMS = [dict(block=True, post=True, gate="sigmoid", p=0.25, next=True),
         dict(block=True, post=True, gate=None, p=0.0, next=True),
         dict(block=True, post=False, gate="plain", p=0.1, next=True),
         dict(block=True, post=True, gate="plain", p=0.0, next=False),
         dict(block=True, post=False, gate="sigmoid", p=0.0, next=False),
         dict(block=True, post=False, gate=None, p=0.5, next=True),
         dict(block=False, post=False, gate=None, p=0.0, next=True)]


def inputs(T, d, dtype, pitch, gains=True, gate=True):
    m = {k: rnd(10 + i, T, d, dtype, std=s, shift=c, pitch=pitch)
         for i, (k, s, c) in enumerate((("x", 2.0, 0.3), ("b", 1.5, -0.2), ("z", 2.0, 0.0),
                                        ("dh", 0.1, 0.0), ("dn", 0.1, 0.0)))}
    m["pg"], m["ng"] = vec(20, d, 1.0), vec(21, d, 1.0)
    return m


def gate_of(form, z):
    """(G, G', relative error of either in U24)"""
    if form["gate"] is None:
        return 1.0, None, 0.0
    z = z.double()
    if form["gate"] == "plain":
        return z, torch.ones_like(z), 0.0
    s = torch.sigmoid(z)
    # e^(-z): its argument's rounding |z| 2^-24 (twice in the hardware's base-2
    # form), two ulp; sum, reciprocal or quotient, two ulp; the product
    # (beyond 100 either is exact: 0 or 1)
    return s, s * torch.sigmoid(-z), 8 * z.abs().clamp(max=100) + 40


def forward_ref(m, form, scale, k):
    """{output: (value, error before its rounding)}"""
    x = m["x"].double()
    T, d = x.shape
    out = {}
    h, eh = x, torch.zeros_like(x)
    if form["block"]:
        c, rel = m["b"].double(), 0.0
        if form["post"]:
            rb = 1 / ((c * c).mean(1, keepdim=True) + EPS).sqrt()
            out["b_rstd"] = rb[:, 0], (S / 2 + 4) * U24 * rb[:, 0]
            c, rel = c * rb, S / 2 + 5
        c = c * m["pg"].double()
        G, _, eg = gate_of(form, m["z"])
        e = scale * c * k * G
        h = x + e
        eh = (rel + eg + 6) * U24 * e.abs() + U24 * (x.abs() + h.abs())
        out["h"] = h, eh
    if form["next"]:
        q = (h * h).mean(1, keepdim=True) + EPS
        rh = 1 / q.sqrt()
        er = (h.abs() * eh).mean(1, keepdim=True) / q + (S / 2 + 4) * U24  # relative
        out["h_rstd"] = rh[:, 0], (rh * er)[:, 0]
        n = h * rh * m["ng"].double()
        out["n"] = n, n.abs() * (er + 3 * U24) + eh * (rh * m["ng"].double()).abs()
    return out


def run_forward(m, form, scale, out, site=SITE, rng=None, x=None):
    kw = {}
    if form["block"]:
        kw.update(b=m["b"], h=out["h"], post_norm=form["post"], post_gain=m["pg"], scale=scale,
                  p=form["p"], rng=rng, site=site)
        if form["post"]:
            kw["b_rstd"] = out["b_rstd"]
        if form["gate"]:
            kw.update(gate=m["z"], gate_act=M.MLP_GATE_SIGMOID if form["gate"] == "sigmoid"
                      else M.MLP_GATE_PLAIN)
    if form["next"]:
        kw.update(n=out["n"], next_gain=m["ng"], h_rstd=out["h_rstd"])
    M.mlp_resnorm_fwd(m["x"] if x is None else x, eps=EPS, **kw)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", SHAPES)
def test_forward(T, d, pitch, dtype):
    m = inputs(T, d, dtype, pitch)
    for form in FORMS:
        k = factor(T, d, form["p"], SEED, STEP, SITE)
        ref = forward_ref(m, form, 0.5, k)
        g = {o: Guarded(T, d, dtype, pitch) for o in ("h", "n")}
        out = {"h": g["h"].v, "n": g["n"].v,
               **{r: torch.full((T,), math.nan, device="cuda") for r in ("b_rstd", "h_rstd")}}
        run_forward(m, form, 0.5, out, rng=state())
        for o, (v, e) in ref.items():
            near(out[o], v, rounding(dtype if o in g else F32, v) + e + 1e-30, "%s %s" % (o, form))
        assert g["h"].intact() and g["n"].intact()
        for o in g:
            assert o in ref or (g[o].buf == -77).all()
        if form["block"]:  # h in x's place
            x = m["x"].clone() if pitch is None else rnd(10, T, d, dtype, 2.0, 0.3, pitch)
            x.copy_(m["x"])
            again = dict(out, h=x, n=torch.empty_like(x))
            run_forward(m, form, 0.5, again, rng=state(), x=x)
            assert torch.equal(x, out["h"])
            assert not form["next"] or torch.equal(again["n"], out["n"])


def backward_ref(m, form, scale, k, with_dh, rstd):
    dh = m["dh"].double() if with_dh else torch.zeros_like(m["x"].double())
    T, d = dh.shape
    out = {}
    dx, ex = dh, torch.zeros_like(dh)
    if form["next"]:
        r = rstd["h"].double()[:, None]
        hh, dn, g = m["x"].double() * r, m["dn"].double(), m["ng"].double()
        t = dn * g
        mean, mabs = (t * hh).mean(1, keepdim=True), (t * hh).abs().mean(1, keepdim=True)
        dx = dh + r * (t - hh * mean)
        ex = (r * (4 * U24 * (t.abs() + (hh * mean).abs()) + hh.abs() * (S + 4) * U24 * mabs)
              + 2 * U24 * (dh.abs() + dx.abs()))
        w = (dn * hh).abs().sum(0)
        out["dnext"] = (dn * hh).sum(0), (T + 10) * U24 * w
    out["dx"] = dx, ex
    if form["block"]:
        rb = rstd["b"].double()[:, None] if form["post"] else 1.0
        bb, pg = m["b"].double() * rb, m["pg"].double()
        G, dG, eg = gate_of(form, m["z"])
        v = scale * dx * k * G
        ev = (scale * k * G).abs() * ex if form["gate"] else scale * k * ex
        ev = ev + v.abs() * (eg + 6) * U24
        if form["gate"]:
            dz = scale * dx * bb * pg * k * dG
            out["dz"] = dz, ((scale * bb * pg * k * dG).abs() * ex
                             + dz.abs() * (2 * eg + 10) * U24)
        out["dpost"] = (v * bb).sum(0), ((ev + 2 * U24 * v.abs()) * bb.abs()).sum(0) \
            + (T + 10) * U24 * (v * bb).abs().sum(0)
        vg, evg = v * pg, ev * pg.abs() + U24 * (v * pg).abs()
        db, edb = vg, evg
        if form["post"]:
            mean, mabs = (vg * bb).mean(1, keepdim=True), (vg * bb).abs().mean(1, keepdim=True)
            em = (evg * bb.abs()).mean(1, keepdim=True) + (S + 4) * U24 * mabs
            db = rb * (vg - bb * mean)
            edb = rb * (evg + 4 * U24 * (vg.abs() + (bb * mean).abs()) + bb.abs() * em) \
                + 2 * U24 * db.abs()
        out["db"] = db, edb
    return out


def run_backward(m, form, scale, with_dh, rstd, out, ws, rng=None, site=SITE):
    kw = {}
    if with_dh:
        kw["dh"] = m["dh"]
    if form["next"]:
        kw.update(dn=m["dn"], h=m["x"], h_rstd=rstd["h"], next_gain=m["ng"],
                  dnext_gain=out["dnext"])
    if form["block"]:
        kw.update(b=m["b"], db=out["db"], post_norm=form["post"], post_gain=m["pg"], scale=scale,
                  p=form["p"], rng=rng, site=site, dpost_gain=out["dpost"])
        if form["post"]:
            kw["b_rstd"] = rstd["b"]
        if form["gate"]:
            kw.update(gate=m["z"], dgate=out["dz"],
                      gate_act=M.MLP_GATE_SIGMOID if form["gate"] == "sigmoid"
                      else M.MLP_GATE_PLAIN)
    M.mlp_resnorm_bwd(out["dx"], workspace=ws, **kw)


def rstds(m):
    return {k: torch.rsqrt(m[v].float().square().mean(1) + EPS) for k, v in (("h", "x"), ("b", "b"))}


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", SHAPES)
def test_backward(T, d, pitch, dtype):
    m = inputs(T, d, dtype, pitch)  # x stands for the saved h
    rstd = rstds(m)
    ws = torch.full((M.mlp_resnorm_workspace_bytes(T, d),), 255, dtype=torch.uint8, device="cuda")
    for i, form in enumerate(FORMS):
        with_dh = i != 1 or not form["next"]
        k = factor(T, d, form["p"], SEED, STEP, SITE)
        ref = backward_ref(m, form, 0.5, k, with_dh, rstd)

        def call():
            g = {o: Guarded(T, d, dtype, pitch) for o in ("dx", "db", "dz")}
            out = {**{o: g[o].v for o in g},
                   **{o: torch.full((d,), math.nan, device="cuda") for o in ("dpost", "dnext")}}
            run_backward(m, form, 0.5, with_dh, rstd, out, ws, rng=state())
            assert all(o.intact() for o in g.values())
            return out
        out, again = call(), call()
        for o, (v, e) in ref.items():
            near(out[o], v, rounding(F32 if o in ("dpost", "dnext") else dtype, v) + e + 1e-30,
                 "%s %s" % (o, form))
            assert torch.equal(out[o], again[o]), o
        # the gradients in their inputs' place
        own = {**m, **{o: m[o].clone() for o in ("b", "z", "dh", "dn")}}
        place = {"dx": own["dh"] if with_dh else own["dn"], "db": own["b"], "dz": own["z"],
                 "dpost": torch.empty(d, device="cuda"), "dnext": torch.empty(d, device="cuda")}
        run_backward(own, form, 0.5, with_dh, rstd, place, ws, rng=state())
        for o in ref:
            assert torch.equal(place[o], out[o]), o


def test_backward_is_the_derivative():
    """All gradients against differences of a 64-bit loss."""
    T, d, scale = 3, 40, 0.7
    m = inputs(T, d, F32, None)
    k = factor(T, d, 0.25, SEED, STEP, SITE)
    for form in FORMS[:1] + FORMS[2:5]:
        form = dict(form, p=0.25)

        def loss(**change):
            q = {n: change.get(n, m[n].double()) for n in ("x", "b", "z", "pg", "ng")}
            out = forward_ref(q, form, scale, k)
            s = (m["dh"].double() * out["h"][0]).sum()
            return s + ((m["dn"].double() * out["n"][0]).sum() if form["next"] else 0)
        new = lambda: torch.empty(T, d, device="cuda")  # noqa: E731
        out = {"h": new(), "n": new(), "b_rstd": torch.empty(T, device="cuda"),
               "h_rstd": torch.empty(T, device="cuda")}
        run_forward(m, form, scale, out, rng=state())
        grads = {"dx": new(), "db": new(), "dz": new(), "dpost": torch.empty(d, device="cuda"),
                 "dnext": torch.empty(d, device="cuda")}
        ws = torch.empty(M.mlp_resnorm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
        run_backward({**m, "x": out["h"]}, form, scale, True,
                     {"h": out["h_rstd"], "b": out["b_rstd"]}, grads, ws, rng=state())
        step = 1e-5
        for name, grad in (("x", "dx"), ("b", "db"), ("z", "dz"), ("pg", "dpost"), ("ng", "dnext")):
            if (name == "z" and not form["gate"]) or (name == "ng" and not form["next"]):
                continue
            for at in ((0, 0), (1, 17), (2, 39)):
                at = at if m[name].dim() == 2 else at[1:]
                v = m[name].double().clone()
                v[at] += step
                up = loss(**{name: v})
                v[at] -= 2 * step
                diff = float(up - loss(**{name: v})) / (2 * step)
                # the difference: step^2 times a third derivative of the order of 10,
                # 1e-16 / step; the kernel: some tens of fp32 roundings of terms
                # of the order of 1
                assert abs(float(grads[grad][at]) - diff) <= 1e-5 * (1 + abs(diff)), (name, at)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_gates_at_their_limits_and_rows_of_zeros(dtype):
    T, d = 4, 48
    m = inputs(T, d, dtype, None)
    m["z"][:, 0], m["z"][:, 1] = math.inf, -math.inf
    m["b"][1] = 0  # a block output of zeros: eps alone under the root
    m["b"][2, 5] = math.nan
    form = FORMS[0]
    k = factor(T, d, form["p"], SEED, STEP, SITE)
    out = {"h": torch.empty_like(m["x"]), "n": torch.empty_like(m["x"]),
           "b_rstd": torch.empty(T, device="cuda"), "h_rstd": torch.empty(T, device="cuda")}
    run_forward(m, form, 0.5, out, rng=state())
    rows = torch.tensor([0, 1, 3], device="cuda")
    ref = {o: (v[rows], e[rows]) for o, (v, e) in forward_ref(m, form, 0.5, k).items()}
    for o, (v, e) in ref.items():
        assert v.isfinite().all()
        near(out[o][rows], v, rounding(F32 if v.dim() == 1 else dtype, v) + e + 1e-30, o)
    assert out["n"][2].isnan().all()
    assert torch.equal(out["h"][2].isnan(), k[2] != 0)
    grads = {**{o: torch.empty_like(m["x"]) for o in ("dx", "db", "dz")},
             "dpost": torch.empty(d, device="cuda"), "dnext": torch.empty(d, device="cuda")}
    ws = torch.empty(M.mlp_resnorm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    run_backward(m, form, 0.5, True, rstds(m), grads, ws, rng=state())
    for o in ("dx", "db", "dz"):
        assert grads[o][rows].isfinite().all(), o
    assert (grads["dz"][rows][:, :2] == 0).all()


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    g = torch.full((2, 64), math.nan, device="cuda")
    M.mlp_resnorm_fwd(x, b=x, h=x, n=x)
    M.mlp_resnorm_bwd(x, dh=x, dn=x, h=x, h_rstd=torch.empty(0, device="cuda"), b=x, db=x,
                      dpost_gain=g[0], dnext_gain=g[1])
    assert (g == 0).all()
