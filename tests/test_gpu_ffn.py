"""The feed-forward operators (layer norm, linear layers with a fused epilogue,
8-bit activation checkpoints) against plain 64-bit implementations.

Tolerances are sums of the roundings an output goes through: half a step of
its type relative to its value (`torch.finfo(t).eps / 2`), and for what is
summed in fp32 before it the number of additions times 2^-24 (2^-23 for tensor-core sums,
whose additions may truncate) of the sum of magnitudes."""
import math

import pytest
import torch

import mlp_step_gb300 as M

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = {"none": M.MLP_ACT_NONE, "relu": M.MLP_ACT_RELU, "leaky2": M.MLP_ACT_LEAKY_RELU_SQ,
        "gelu": M.MLP_ACT_GELU, "gelu_tanh": M.MLP_ACT_GELU_TANH, "silu": M.MLP_ACT_SILU}
SLOPE = 0.5
U24 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    M.load()
    yield
    assert M.get_device_status() == M.MLP_OK


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(dtype, ref):
    """One rounding of ref to dtype: half a step.  Steps are eps 2^e for values
    in [2^e, 2^(e+1)), at most eps |ref|, down to the smallest normal; below it
    they are all the smallest subnormal (2^-24 in fp16: a rounding there is off
    by up to 2^-25 however small the value)."""
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    return (half(dtype) * ref.abs()).clamp(min=tiny / 2)


class Guarded:
    """A [rows, cols] view inside a larger buffer of a sentinel: `intact()`
    says that nothing outside the view was written."""

    def __init__(self, rows, cols, dtype, pitch=None, fill=-77):
        pitch = pitch or (cols + 15) // 16 * 16
        self.buf = torch.full((rows + 3, pitch), fill, dtype=dtype, device="cuda")
        self.v = self.buf[:rows, :cols]
        self.fill, self.rows, self.cols = fill, rows, cols

    def intact(self):
        return bool((self.buf[self.rows:] == self.fill).all()
                    and (self.buf[:self.rows, self.cols:] == self.fill).all())


def rnd(seed, rows, cols, dtype, std=1.0, shift=0.0, pitch=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = Guarded(rows, cols, dtype, pitch).v
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda") * std + shift)
    return t


def vec(seed, n, mean=0.0, std=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return mean + std * torch.randn(n, generator=g, device="cuda")


def near(got, ref, tol, what):
    got, ref = got.double(), ref.double()
    bad = ~((got - ref).abs() <= tol) & ~((got == ref) | (got.isnan() & ref.isnan()))
    assert not bad.any(), "%s: %d of %d off, worst %g over the tolerance (of %g)" % (
        what, int(bad.sum()), bad.numel(), float(((got - ref).abs() / tol).nan_to_num(1e9)[bad].max()),
        float(torch.as_tensor(tol).max()))


# ------------------------------------------------------------ 8-bit checkpoints

def ckpt_ref(x):
    """(q, b) of the format's definition, in 64 bits."""
    T, d = x.shape
    G = -(-d // 32)
    v = torch.zeros(T, G * 32, dtype=torch.float64, device=x.device)
    v[:, :d] = x.double()
    v = v.view(T, G, 32)
    amax = v.abs().amax(2)
    e = torch.frexp(amax)[1] - 1
    bad = ~torch.isfinite(amax)
    b = torch.where(amax == 0, torch.full_like(e, 7), (e + 127).clamp(min=7))
    step = (b.to(torch.int64) - 133 + 1023).bitwise_left_shift(52).view(torch.float64)
    q = torch.round(v / step[:, :, None]).clamp(-127, 127)
    q = torch.where(bad[:, :, None], torch.zeros_like(q), q)
    b = torch.where(bad, torch.full_like(b, 255), b)
    return q.view(T, G * 32)[:, :d].to(torch.int8), b.to(torch.uint8)


def ckpt_values(q, b):
    T, d = q.shape
    step = (b.to(torch.int64) - 133 + 1023).bitwise_left_shift(52).view(torch.float64)
    step = torch.where(b == 255, torch.full_like(step, math.nan), step)
    return q.double() * step.repeat_interleave(32, 1)[:, :d]


def new_ckpt(T, d, pitch=None):
    return Guarded(T, d, torch.int8, pitch), Guarded(T, -(-d // 32), torch.uint8, fill=211)


SHAPES = [(1, 1, None), (1, 512, None), (3, 31, 33), (5, 32, 32), (7, 33, 41), (130, 1000, 1000),
          (129, 1001, 1003), (64, 4100, 4104)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", SHAPES)
def test_ckpt8_round_trip(T, d, pitch, dtype):
    x = rnd(1, T, d, dtype, std=3.0, pitch=pitch)
    x[::2] *= 2.0 ** -9
    q, s = new_ckpt(T, d, pitch)
    M.mlp_ckpt8_encode(x, q.v, s.v)
    qr, br = ckpt_ref(x)
    assert torch.equal(q.v, qr) and torch.equal(s.v, br)
    assert q.intact() and s.intact()
    for odt in (BF16, F16, F32):
        out = Guarded(T, d, odt, pitch)
        M.mlp_ckpt8_decode(q.v, s.v, out.v)
        # the values have 7 bits: exact in bf16 and fp32, one rounding in fp16's subnormals
        assert torch.equal(out.v, ckpt_values(qr, br).to(odt))
        assert out.intact()


def test_ckpt8_special_values():
    x = torch.zeros(9, 64, device="cuda")
    x[1, 3] = math.inf
    x[2, 40] = -math.inf
    x[3, 0] = math.nan
    x[4] = torch.finfo(F32).max
    x[5] = torch.finfo(F32).tiny
    x[6] = 2.0 ** -149
    x[7, ::2] = 127.5     # rounds to 128: held to 127
    x[7, 1::2] = -127.75
    x[8, :32] = torch.arange(32, device="cuda") + 0.5  # steps of 1/4: exact
    x[8, 32:] = torch.arange(32, device="cuda") * 4 + 2.0 * 0.5  # steps of 1
    q, s = new_ckpt(9, 64)
    M.mlp_ckpt8_encode(x, q.v, s.v)
    qr, br = ckpt_ref(x)
    assert torch.equal(s.v, br) and torch.equal(q.v, qr)
    out = torch.empty_like(x)
    M.mlp_ckpt8_decode(q.v, s.v, out)
    ref = ckpt_values(qr, br).float()
    assert torch.equal(out.isnan(), ref.isnan())
    assert torch.equal(out.nan_to_num(), ref.nan_to_num())
    assert out[1, :32].isnan().all() and not out[1, 32:].isnan().any()
    assert (out[7, ::2] == 127).all() and (out[7, 1::2] == -127).all()


def test_ckpt8_empty():
    q, s = new_ckpt(4, 32)
    M.mlp_ckpt8_encode(torch.empty(0, 32, device="cuda"), q.v[:0], s.v[:0])
    M.mlp_ckpt8_decode(q.v[:0], s.v[:0], torch.empty(0, 32, device="cuda"))
    assert (q.buf == -77).all()


# ------------------------------------------------------------ layer norm

def ln_ref(x, gain, shift, eps):
    x = x.double()
    mu = x.mean(1, keepdim=True)
    rho = 1 / ((x - mu).square().mean(1, keepdim=True) + eps).sqrt()
    y = (x - mu) * rho
    if gain is not None:
        y = y * gain.double()
    if shift is not None:
        y = y + shift.double()
    return y, mu[:, 0], rho[:, 0]


def ln_slack(x, rho, d):
    """Error of xh from the fp32 mean and scale: a thread adds 16 values (a
    wide row's thread d/512), then a tree of at most 10 levels."""
    adds = max(16, d // 512) + 10
    big = x.double().abs().amax(1, keepdim=True)
    return (2 * adds + 8) * U24 * big * rho[:, None]


LN_SHAPES = [(1, 1, None), (1, 512, None), (2, 7, 9), (9, 33, 40), (300, 256, None),
             (1001, 512, 520), (77, 520, 523), (515, 1000, 1000), (130, 2000, None),
             (65, 4099, 4100), (33, 8192, None), (7, 8200, 8201), (5, 20000, None)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", LN_SHAPES)
def test_layernorm_forward(T, d, pitch, dtype):
    x = rnd(2, T, d, dtype, std=2.0, shift=1.5, pitch=pitch)
    gain, shift = vec(3, d, 1.0), vec(4, d)
    y, q, s = Guarded(T, d, dtype, pitch), *new_ckpt(T, d, pitch)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    M.mlp_layernorm_fwd(x, y.v, gain=gain, shift=shift, mean=mean, rstd=rstd, ckpt=(q.v, s.v))
    ref, mu, rho = ln_ref(x, gain, shift, 1e-5)
    slack = ln_slack(x, rho, d)
    near(y.v, ref, rounding(dtype, ref) + slack * gain.abs() + 8 * U24 * (ref.abs() + 1), "y")
    near(mean, mu, (slack / rho[:, None])[:, 0], "mean")
    # relative error of rho: half that of the variance, whose terms are off by 2 |c| err
    near(rstd, rho, rho * (4 * slack[:, 0] + 40 * U24), "rstd")
    qr, br = ckpt_ref(x)
    assert torch.equal(q.v, qr) and torch.equal(s.v, br)
    assert y.intact() and q.intact() and s.intact()
    y2 = Guarded(T, d, dtype, pitch)
    M.mlp_layernorm_fwd(x, y2.v)  # gain 1, shift 0, nothing saved
    ref, _, rho = ln_ref(x, None, None, 1e-5)
    near(y2.v, ref, rounding(dtype, ref) + slack + 8 * U24 * (ref.abs() + 1), "plain y")


def test_layernorm_large_mean():
    """The variance is taken about the mean: a row of mean 4096 and spread 1
    in fp32 keeps its spread."""
    x = rnd(5, 64, 512, F32, shift=4096.0)
    y = torch.empty(64, 512, device="cuda")
    M.mlp_layernorm_fwd(x, y)
    ref, _, rho = ln_ref(x, None, None, 1e-5)
    near(y, ref, ln_slack(x, rho, 512) + 8 * U24 * (ref.abs() + 1), "y")


def test_layernorm_rows_are_separate():
    """A row that is not finite, or constant, leaves the others alone."""
    for d in (512, 1000, 4096, 20000):
        x = rnd(6, 12, d, F32)
        x[3, 5], x[5, d - 1], x[7] = math.inf, math.nan, 0.25
        y = torch.empty(12, d, device="cuda")
        M.mlp_layernorm_fwd(x, y)
        ref, _, rho = ln_ref(x, None, None, 1e-5)
        assert y[3].isnan().all() and y[5].isnan().all() and (y[7] == 0).all()
        rest = [0, 1, 2, 4, 6, 8, 9, 10, 11]
        near(y[rest], ref[rest], ln_slack(x, rho, d)[rest] + 8 * U24 * (ref[rest].abs() + 1), "y")


def ln_bwd_ref(dy, x, mu, rho, gain, dres):
    dy, x = dy.double(), x.double()
    xh = (x - mu.double()[:, None]) * rho.double()[:, None]
    g = dy if gain is None else dy * gain.double()
    dx = rho.double()[:, None] * (g - g.mean(1, keepdim=True)
                                  - xh * (g * xh).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * xh).sum(0), dy.sum(0), xh, g


@pytest.mark.parametrize("ck", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d,pitch", LN_SHAPES)
def test_layernorm_backward(T, d, pitch, dtype, ck):
    x = rnd(7, T, d, dtype, std=2.0, shift=0.5, pitch=pitch)
    dy = rnd(8, T, d, dtype, std=0.1, pitch=pitch)
    dres = rnd(9, T, d, dtype, std=0.1, pitch=pitch) if T % 2 else None
    gain = vec(10, d, 1.0) if d != 512 else None
    _, mu, rho = ln_ref(x, None, None, 1e-5)
    mean, rstd = mu.float(), rho.float()
    kw = {"x": x}
    seen = x
    if ck:
        q, s = new_ckpt(T, d, pitch)
        M.mlp_ckpt8_encode(x, q.v, s.v)
        kw = {"ckpt": (q.v, s.v)}
        seen = ckpt_values(q.v, s.v)
    dx = Guarded(T, d, dtype, pitch)
    dg, ds = (torch.full((d,), math.nan, device="cuda") for _ in range(2))
    ws = torch.empty(M.mlp_layernorm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    M.mlp_layernorm_bwd(dy, mean, rstd, dx.v, dg, ds, ws, gain=gain, dres=dres, **kw)
    rdx, rdg, rds, xh, g = ln_bwd_ref(dy, seen, mean, rstd, gain, dres)
    adds = max(16, d // 512) + 10
    r = rstd.double()[:, None]
    # xh is off by 3 roundings of (|x| + |mu|) rho; the row means by `adds` more
    exh = 3 * U24 * (seen.double().abs() + mean.double().abs()[:, None]) * r
    mean_g = g.abs().mean(1, keepdim=True)
    mean_gx = (g * xh).abs().mean(1, keepdim=True)
    e2 = (g.abs() * exh).mean(1, keepdim=True) + (adds + 3) * U24 * mean_gx
    slack = r * (8 * U24 * (g.abs() + mean_g + xh.abs() * mean_gx) + adds * U24 * mean_g
                 + xh.abs() * e2 + exh * mean_gx) + 4 * U24 * rdx.abs()
    near(dx.v, rdx, rounding(dtype, rdx) + slack + 1e-30, "dx")
    assert dx.intact()
    # parameter gradients: at most T / 304 + 8 rows in a chain per block, then 304 blocks
    n = T + 16
    near(dg, rdg, n * U24 * (dy.double() * xh).abs().sum(0) + (dy.double().abs() * exh).sum(0)
         + 1e-30, "dgain")
    near(ds, rds, n * U24 * dy.double().abs().sum(0) + 1e-30, "dshift")
    # the same bits again
    dg2, ds2, dx2 = torch.empty_like(dg), torch.empty_like(ds), Guarded(T, d, dtype, pitch)
    M.mlp_layernorm_bwd(dy, mean, rstd, dx2.v, dg2, ds2, ws, gain=gain, dres=dres, **kw)
    assert torch.equal(dg, dg2) and torch.equal(ds, ds2) and torch.equal(dx.v, dx2.v)
    if dres is not None:  # dx over dres
        M.mlp_layernorm_bwd(dy, mean, rstd, dres, dg2, ds2, ws, gain=gain, dres=dres, **kw)
        assert torch.equal(dres, dx.v)


def test_layernorm_backward_against_differences():
    """d/dh of sum(dy . y) along random directions of x, gain and shift."""
    T, d = 6, 70
    x, dy = rnd(11, T, d, F32), rnd(12, T, d, F32)
    gain, shift = vec(13, d, 1.0), vec(14, d)
    _, mu, rho = ln_ref(x, gain, shift, 1e-5)
    dx = torch.empty(T, d, device="cuda")
    dg, ds = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(M.mlp_layernorm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    M.mlp_layernorm_bwd(dy, mu.float(), rho.float(), dx, dg, ds, ws, x=x, gain=gain)
    h = 1e-5
    for grad, arg in ((dx, 0), (dg, 1), (ds, 2)):
        base = [x.double(), gain.double(), shift.double()]
        v = torch.randn(base[arg].shape, dtype=torch.float64, device="cuda")
        f = []
        for sgn in (1, -1):
            a = list(base)
            a[arg] = a[arg] + sgn * h * v
            f.append((ln_ref(a[0], a[1], a[2], 1e-5)[0] * dy.double()).sum())
        slope = float((f[0] - f[1]) / (2 * h))
        # central differences: h^2 of a third derivative of order 10, and fp32 gradients
        scale = float((grad.double() * v).abs().sum())
        assert abs(float((grad.double() * v).sum()) - slope) <= 1e-5 * scale


def test_layernorm_empty():
    e = torch.empty(0, 64, device="cuda")
    f = torch.empty(0, device="cuda")
    dg, ds = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    M.mlp_layernorm_fwd(e, e)
    M.mlp_layernorm_bwd(e, f, f, e, dg, ds, None, x=e)
    assert (dg == 0).all() and (ds == 0).all()


# ------------------------------------------------------------ linear layers

def act_ref(u, act):
    """(f(u), f'(u), a bound of |f''| times 2) in 64 bits."""
    one = torch.ones_like(u)
    if act == "none":
        return u, one, 0.0
    if act == "relu":
        return u.clamp(min=0), (u > 0).double(), 0.0
    if act == "leaky2":
        t = torch.where(u > 0, one, SLOPE * one)
        return (t * u) ** 2, 2 * t * t * u, 4.0
    if act == "gelu":
        p = torch.special.erfc(-u / math.sqrt(2)) / 2
        return u * p, p + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi), 2.0
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (u + 0.044715 * u ** 3))
        return (u * (1 + t) / 2,
                (1 + t) / 2 + u * (1 - t * t) / 2 * c * (1 + 3 * 0.044715 * u * u), 2.0)
    s = torch.sigmoid(u)
    return u * s, s * (1 + u * (1 - s)), 2.0


# error of the evaluated activations themselves, of (1 + |u|): the rational
# approximation's 1.5e-7 and a few roundings of fp32 exponentials
ACT_ERR = 1e-6

# few rows, narrow and split tiles, 128-wide tiles, pairs; ragged everywhere
LIN_SHAPES = [(1, 1, 1), (1, 512, 1536), (2, 784, 10), (3, 1000, 257), (5, 2056, 136), (8, 77, 72),
              (9, 512, 256), (33, 4096, 200), (100, 784, 256), (128, 1000, 1000), (257, 72, 2000),
              (1500, 520, 1001), (2000, 136, 1600), (4100, 200, 768)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,k,n", LIN_SHAPES)
def test_linear_forward(T, k, n, dtype):
    for i, act in enumerate(ACTS):
        res, save, f32 = i % 2 == 0, ("u", "ckpt", "both", "none")[i % 4], i == 3
        odt = F32 if f32 else dtype
        x = rnd(20, T, k, dtype)
        w = rnd(21, k, n, dtype, std=k ** -0.5)
        bias = vec(22, n) if i != 5 else None
        r = rnd(23, T, n, odt) if res else None
        y, u = Guarded(T, n, odt), Guarded(T, n, dtype)
        q, s = new_ckpt(T, n)
        ws = torch.empty(M.mlp_linear_workspace_bytes(T, k, n, dtype), dtype=torch.uint8,
                         device="cuda")
        M.mlp_linear_fwd(x, w, y.v, bias=bias, act=ACTS[act], slope=SLOPE, residual=r,
                         u=u.v if save in ("u", "both") else None,
                         ckpt=(q.v, s.v) if save in ("ckpt", "both") else None, workspace=ws)
        ru = x.double() @ w.double()
        eu = (k + 8) * 2 * U24 * (x.double().abs() @ w.double().abs())
        if bias is not None:
            ru = ru + bias.double()
            eu = eu + U24 * ru.abs() + U24 * bias.double().abs()
        f, df, curve = act_ref(ru, act)
        # |f(u + e) - f(u)| <= |f'| e + |f''| e^2 / 2
        ef = (1.0 if act == "relu" else df.abs()) * eu + curve * eu * eu
        if act != "none":
            ef = ef + ACT_ERR * (1 + ru.abs()) * (1 + f.abs())
        ref = f + r.double() if res else f
        near(y.v, ref, rounding(odt, ref) + ef + 2 * U24 * (ref.abs() + f.abs()),
             "y %s" % act)
        assert y.intact()
        if save in ("u", "both"):
            near(u.v, ru, rounding(dtype, ru) + eu + 1e-30, "u")
            assert u.intact()
        else:
            assert (u.buf == -77).all()
        if save in ("ckpt", "both"):
            _, b_lo = ckpt_ref((ru.abs() - eu).clamp(min=0))
            _, b_hi = ckpt_ref(ru.abs() + eu)
            assert ((s.v >= b_lo) & (s.v <= b_hi)).all()
            step = (s.v.to(torch.int64) - 133 + 1023).bitwise_left_shift(52).view(torch.float64)
            step = step.repeat_interleave(32, 1)[:, :n]
            held = q.v.abs() == 127
            near(ckpt_values(q.v, s.v), ru, step * torch.where(held, 1.0, 0.5) + eu, "8-bit u")
            assert q.intact() and s.intact()
        else:
            assert (q.buf == -77).all() and (s.buf == 211).all()


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,n", [(3, 512, 200), (40, 4096, 200), (300, 520, 1001),
                                   (1500, 328, 1200), (4100, 200, 776), (3300, 1160, 1100)])
def test_linear_mixed_outputs(T, k, n, dtype, odd):
    """fp32 outputs beside 16-bit and 8-bit ones, all at once, in matrices whose
    rows TMA can address and in ones that it cannot."""
    pitch = n + 3 if odd else None
    x, w = rnd(100, T, k, dtype), rnd(101, k, n, dtype, std=k ** -0.5)
    wt = w.t().contiguous()
    if n % 8:
        wt = rnd(102, n, k, dtype)
        wt.copy_(w.t())
    bias, r = vec(103, n), rnd(104, T, n, F32, pitch=pitch)
    ru = x.double() @ w.double() + bias.double()
    eu = (k + 8) * 2 * U24 * (x.double().abs() @ w.double().abs()) + 2 * U24 * ru.abs()
    f, df, _ = act_ref(ru, "silu")
    for odt in (F32, dtype):
        y, u, (q, s) = Guarded(T, n, odt, pitch), Guarded(T, n, dtype, pitch), new_ckpt(T, n, pitch)
        res = r if odt == F32 else rnd(104, T, n, dtype, pitch=pitch)
        ws = torch.empty(M.mlp_linear_workspace_bytes(T, k, n, dtype), dtype=torch.uint8,
                         device="cuda")
        M.mlp_linear_fwd(x, w, y.v, bias=bias, act=M.MLP_ACT_SILU, residual=res, u=u.v,
                         ckpt=(q.v, s.v), workspace=ws)
        ref = f + res.double()
        near(y.v, ref, rounding(odt, ref) + (df.abs() + 0.1) * eu + ACT_ERR * (1 + ru.abs()),
             "y")
        near(u.v, ru, rounding(dtype, ru) + eu, "u")
        step = (s.v.to(torch.int64) - 133 + 1023).bitwise_left_shift(52).view(torch.float64)
        near(ckpt_values(q.v, s.v), ru,
             step.repeat_interleave(32, 1)[:, :n] * torch.where(q.v.abs() == 127, 1.0, 0.5) + eu,
             "8-bit u")
        assert y.intact() and u.intact() and q.intact() and s.intact()
        # backward: dy = x, so that da = x w
        da = x.double() @ w.double()
        uin = rnd(105, T, n, dtype, std=1.5, pitch=pitch)
        M.mlp_ckpt8_encode(uin, q.v, s.v)
        bws = torch.empty(M.mlp_linear_bwd_workspace_bytes(T, n, k, dtype), dtype=torch.uint8,
                          device="cuda")
        for kw, seen in (({"u": uin}, uin.double()),
                         ({"ckpt": (q.v, s.v)}, ckpt_values(q.v, s.v))):
            du, a = Guarded(T, n, odt, pitch), Guarded(T, n, dtype, pitch)
            db = torch.empty(n, device="cuda")
            M.mlp_linear_bwd(x, wt, du.v, act=M.MLP_ACT_GELU, dbias=db, a=a.v, workspace=bws, **kw)
            fg, dfg, _ = act_ref(seen, "gelu")
            rdu = da * dfg
            e = eu * dfg.abs() + (da.abs() + eu) * ACT_ERR * (1 + seen.abs()) + 2 * U24 * rdu.abs()
            near(du.v, rdu, rounding(odt, rdu) + e, "du")
            near(a.v, fg, rounding(dtype, fg) + ACT_ERR * (1 + seen.abs()) * (1 + fg.abs()), "a")
            near(db, rdu.sum(0), e.sum(0) + (T + 8) * U24 * rdu.abs().sum(0), "dbias")
            assert du.intact() and a.intact()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,k,n", [(4, 512, 200), (64, 2048, 96), (300, 520, 1001),
                                   (4100, 200, 768)])
def test_linear_forward_in_place_residual(T, k, n, dtype):
    x, w = rnd(24, T, k, dtype), rnd(25, k, n, dtype, std=k ** -0.5)
    r, y = rnd(26, T, n, dtype), torch.empty(T, (n + 7) // 8 * 8, dtype=dtype, device="cuda")[:, :n]
    ws = torch.empty(M.mlp_linear_workspace_bytes(T, k, n, dtype), dtype=torch.uint8, device="cuda")
    M.mlp_linear_fwd(x, w, y, act=M.MLP_ACT_SILU, residual=r, workspace=ws)
    M.mlp_linear_fwd(x, w, r, act=M.MLP_ACT_SILU, residual=r, workspace=ws)
    assert torch.equal(y, r)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,k,n", LIN_SHAPES)
def test_linear_backward(T, k, n, dtype):
    for i, act in enumerate(ACTS):
        ck, again, f32 = i % 2 == 1, i % 3 != 0, i == 4
        odt = F32 if f32 else dtype
        dy = rnd(30, T, k, dtype, std=0.1)
        w = rnd(31, n, k, dtype, std=n ** -0.5)
        u = rnd(32, T, n, dtype, std=1.5)
        kw = {"u": u}
        seen = u.double()
        if ck:
            q, s = new_ckpt(T, n)
            M.mlp_ckpt8_encode(u, q.v, s.v)
            kw, seen = {"ckpt": (q.v, s.v)}, ckpt_values(q.v, s.v)
        if act == "none" and not again:
            kw = {}
        du, a = Guarded(T, n, odt), Guarded(T, n, dtype)
        db = torch.full((n,), math.nan, device="cuda")
        ws = torch.empty(M.mlp_linear_bwd_workspace_bytes(T, n, k, dtype), dtype=torch.uint8,
                         device="cuda")
        M.mlp_linear_bwd(dy, w, du.v, act=ACTS[act], slope=SLOPE, dbias=db,
                         a=a.v if again else None, workspace=ws, **kw)
        f, df, _ = act_ref(seen, act)
        da = dy.double() @ w.double().t()
        eda = (k + 8) * 2 * U24 * (dy.double().abs() @ w.double().abs().t())
        ref = da * df
        e = eda * df.abs() + 2 * U24 * ref.abs()
        if act not in ("none", "relu"):
            e = e + (da.abs() + eda) * ACT_ERR * (1 + seen.abs())
        near(du.v, ref, rounding(odt, ref) + e + 1e-30, "du %s" % act)
        near(db, ref.sum(0), e.sum(0) + (T + 8) * U24 * ref.abs().sum(0) + 1e-30, "dbias %s" % act)
        assert du.intact()
        if again:
            near(a.v, f, rounding(dtype, f) + ACT_ERR * (1 + seen.abs()) * (1 + f.abs())
                 * (act not in ("none", "relu")) + 1e-30, "a %s" % act)
            assert a.intact()
        else:
            assert (a.buf == -77).all()
        db2, du2 = torch.empty_like(db), Guarded(T, n, odt)
        M.mlp_linear_bwd(dy, w, du2.v, act=ACTS[act], slope=SLOPE, dbias=db2, workspace=ws, **kw)
        assert torch.equal(db, db2) and torch.equal(du.v, du2.v)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,n,pitch", [(1, 1, None), (1, 512, None), (31, 33, 35), (32, 32, 32),
                                       (33, 1001, 1001), (1000, 1536, None), (300, 4099, 4101)])
def test_act_backward(T, n, pitch, dtype):
    for i, act in enumerate(ACTS):
        ck, again = i % 2 == 0, i % 3 == 0
        dy, u = rnd(40, T, n, dtype, pitch=pitch), rnd(41, T, n, dtype, std=2.0, pitch=pitch)
        kw, seen = {"u": u}, u.double()
        if ck:
            q, s = new_ckpt(T, n, pitch)
            M.mlp_ckpt8_encode(u, q.v, s.v)
            kw, seen = {"ckpt": (q.v, s.v)}, ckpt_values(q.v, s.v)
        du, a = Guarded(T, n, dtype, pitch), Guarded(T, n, dtype, pitch)
        db = torch.full((n,), math.nan, device="cuda")
        ws = torch.empty(M.mlp_act_bwd_workspace_bytes(T, n), dtype=torch.uint8, device="cuda")
        M.mlp_act_bwd(dy, du.v, act=ACTS[act], slope=SLOPE, dbias=db, a=a.v if again else None,
                      workspace=ws, **kw)
        f, df, _ = act_ref(seen, act)
        ref = dy.double() * df
        e = 2 * U24 * ref.abs() + dy.double().abs() * ACT_ERR * (1 + seen.abs())
        near(du.v, ref, rounding(dtype, ref) + e, "du %s" % act)
        near(db, ref.sum(0), e.sum(0) + (T + 8) * U24 * ref.abs().sum(0), "dbias %s" % act)
        assert du.intact()
        if again:
            near(a.v, f, rounding(dtype, f) + ACT_ERR * (1 + seen.abs()) * (1 + f.abs()),
                 "a %s" % act)
            assert a.intact()


def test_activation_derivatives_against_differences():
    """f' of every activation against central differences of its f, in 64 bits."""
    u = torch.linspace(-9, 9, 1441, device="cuda").view(1, -1)
    u = u[:, (u[0] != 0)]
    dy, du, a = torch.ones_like(u), torch.empty_like(u), torch.empty_like(u)
    h = 1e-5
    for act in ACTS:
        M.mlp_act_bwd(dy, du, act=ACTS[act], slope=SLOPE, u=u, a=a)
        slope = (act_ref(u.double() + h, act)[0] - act_ref(u.double() - h, act)[0]) / (2 * h)
        # h^2 times a third derivative below 4, and 64-bit noise of 1e-16 |f| / h
        tol = ACT_ERR * (1 + u.double().abs()) + 1e-9
        if act == "relu":
            # f' jumps by 1 at 0: a quotient over an interval with 0 inside
            # (|u| < h) lies anywhere between the two sides
            tol = tol + (u.double().abs() < h)
        elif act == "leaky2":
            # f'' jumps at 0, so there the quotient is only good to h max|f''| = 2 h
            tol = tol + 2 * h * (u.double().abs() < h)
        near(du, slope, tol, act)


@pytest.mark.parametrize("act", list(ACTS))
def test_activation_limits(act):
    """Large and infinite pre-activations: the limits, not 0 times infinity."""
    u = torch.tensor([[1e4, -1e4, 3e38, -3e38, math.inf, -math.inf, 0.0, math.nan]], device="cuda")
    dy, du = torch.ones_like(u), torch.empty_like(u)
    for dtype in (F32, BF16):
        d = torch.empty(1, 8, dtype=dtype, device="cuda")
        M.mlp_act_bwd(dy.to(dtype), d, act=ACTS[act], slope=SLOPE, u=u.to(dtype))
        d = d.float()[0]
        if act in ("gelu", "gelu_tanh", "silu", "relu"):
            assert d[[0, 2, 4]].tolist() == [1, 1, 1]
            assert d[[1, 3, 5]].abs().max() < 1e-30
        if act != "relu":
            assert act == "none" or d[7].isnan()


def test_linear_empty():
    e, w = torch.empty(0, 64, dtype=BF16, device="cuda"), rnd(50, 64, 64, BF16)
    db = torch.ones(64, device="cuda")
    M.mlp_linear_fwd(e, w, e)
    M.mlp_linear_bwd(e, w, e, dbias=db)
    assert (db == 0).all()
    db.fill_(1)
    M.mlp_act_bwd(e, e, dbias=db)
    assert (db == 0).all()


# ------------------------------------------------------------ together

def feed_forward(x, P, ck, ws, out):
    """y = x + W2 gelu(W1 LN(x) + b1) + b2, and from dy its gradients, through
    the library; ck: x and the pre-activations kept in 8 bits."""
    T, d = x.shape
    h = P["w1"].shape[1]
    o = out
    M.mlp_layernorm_fwd(x, o["n"], gain=P["g"], shift=P["s"], mean=o["mean"], rstd=o["rstd"],
                        ckpt=o["xq"] if ck else None)
    M.mlp_linear_fwd(o["n"], P["w1"], o["a"], bias=P["b1"], act=M.MLP_ACT_GELU,
                     u=None if ck else o["u"], ckpt=o["uq"] if ck else None, workspace=ws)
    M.mlp_linear_fwd(o["a"], P["w2"], o["y"], bias=P["b2"], residual=x, workspace=ws)
    kw = {"ckpt": o["uq"]} if ck else {"u": o["u"]}
    M.mlp_colsum(P["dy"], o["db2"], workspace=ws)
    M.mlp_linear_bwd(P["dy"], P["w2"], o["du"], act=M.MLP_ACT_GELU, dbias=o["db1"], a=o["a2"],
                     workspace=ws, **kw)
    M.mlp_gemm(o["a2"], P["dy"], o["dw2"], h, d, T, a_trans=True)
    M.mlp_gemm(o["n"], o["du"], o["dw1"], d, h, T, a_trans=True)
    M.mlp_gemm(o["du"], P["w1"], o["dn"], T, d, h, b_trans=True)
    M.mlp_layernorm_bwd(o["dn"], o["mean"], o["rstd"], o["dx"], o["dg"], o["ds"], ws,
                        x=None if ck else x, ckpt=o["xq"] if ck else None, gain=P["g"],
                        dres=P["dy"])


def ff_problem(T, d, h, dtype, seed=60):
    P = {"w1": rnd(seed, d, h, dtype, d ** -0.5), "w2": rnd(seed + 1, h, d, dtype, h ** -0.5),
         "b1": vec(seed + 2, h), "b2": vec(seed + 3, d), "g": vec(seed + 4, d, 1.0),
         "s": vec(seed + 5, d), "dy": rnd(seed + 6, T, d, dtype, 0.1)}
    e = lambda r, c, t=dtype: torch.empty(r, c, dtype=t, device="cuda")  # noqa: E731
    f = lambda n: torch.empty(n, device="cuda")  # noqa: E731
    out = {"n": e(T, d), "a": e(T, h), "a2": e(T, h), "u": e(T, h), "y": e(T, d), "du": e(T, h),
           "dn": e(T, d), "dx": e(T, d), "mean": f(T), "rstd": f(T), "db1": f(h), "db2": f(d),
           "dg": f(d), "ds": f(d), "dw1": e(d, h, F32), "dw2": e(h, d, F32),
           "xq": (e(T, d, torch.int8), e(T, -(-d // 32), torch.uint8)),
           "uq": (e(T, h, torch.int8), e(T, -(-h // 32), torch.uint8))}
    need = max(M.mlp_layernorm_workspace_bytes(T, d), M.mlp_linear_workspace_bytes(T, d, h, dtype),
               M.mlp_linear_workspace_bytes(T, h, d, dtype),
               M.mlp_linear_bwd_workspace_bytes(T, h, d, dtype),
               M.mlp_colsum_workspace_bytes(T, d))
    return P, out, torch.empty(need, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("ck", [False, True])
@pytest.mark.parametrize("T,d,h,dtype", [(1, 512, 1536, BF16), (200, 256, 784, BF16),
                                         (3000, 512, 1536, BF16), (1000, 512, 1024, F16)])
def test_feed_forward_block(T, d, h, dtype, ck):
    """The operators as a pre-norm feed-forward block uses them, against
    autograd in 64 bits with the kept activations as the library kept them."""
    x = rnd(70, T, d, dtype, shift=0.3)
    P, o, ws = ff_problem(T, d, h, dtype)
    feed_forward(x, P, ck, ws, o)
    D = {k: v.double().requires_grad_(k != "dy") for k, v in P.items()}
    xd = x.double().requires_grad_()
    mu = xd.mean(1, keepdim=True)
    rho = 1 / ((xd - mu).square().mean(1, keepdim=True) + 1e-5).sqrt()
    n = (xd - mu) * rho * D["g"] + D["s"]
    u = n @ D["w1"] + D["b1"]
    a = torch.nn.functional.gelu(u)
    y = xd + a @ D["w2"] + D["b2"]
    (y * D["dy"]).sum().backward()
    ref = {"y": y, "dx": xd.grad, "dw1": D["w1"].grad, "dw2": D["w2"].grad, "db1": D["b1"].grad,
           "db2": D["b2"].grad, "dg": D["g"].grad, "ds": D["s"].grad}
    # 2-norms: every intermediate is rounded to 16 bits once (n, a, u, du, dn:
    # five half steps at most in a chain).  In 8 bits a value is off by at most
    # half a step, 1/128 of its group's largest magnitude, itself at most
    # sqrt(32) of the group's root mean square: 0.045 of the norm for x (in xh)
    # and, with |gelu''| <= 0.8 against a derivative whose root mean square is
    # at least half, 0.08 for the chain through u.
    tol = 5 * half(dtype) + (0.13 if ck else 0)
    for k, r in ref.items():
        r = r.detach()
        t = 3 * half(dtype) if k == "y" else tol
        err = float((o[k].double() - r).norm() / r.norm())
        assert err <= t, (k, err, t)


def test_feed_forward_block_captured():
    """A captured run of the block replays to the same bits on new inputs, and
    runs on a side stream."""
    T, d, h = 500, 256, 512
    x = rnd(71, T, d, BF16)
    P, o, ws = ff_problem(T, d, h, BF16)
    feed_forward(x, P, True, ws, o)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        feed_forward(x, P, True, ws, o)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        feed_forward(x, P, True, ws, o)
    x.copy_(rnd(72, T, d, BF16))
    P["dy"].copy_(rnd(73, T, d, BF16))
    g.replay()
    keep = {k: o[k].clone() for k in ("y", "dx", "dw1", "dw2", "db1", "dg", "ds")}
    for k in keep:
        o[k].fill_(float("nan"))
    feed_forward(x, P, True, ws, o)
    for k, v in keep.items():
        assert torch.equal(v, o[k]), k


@pytest.mark.parametrize("T", [1, 5, 8, 9, 100])
@pytest.mark.parametrize("k,n", [(1, 1), (63, 65), (300, 129), (1030, 1500)])
def test_linear_f32_odd_pitches(T, k, n):
    """fp32 operands at any pitch, few and many rows."""
    x, w = rnd(120, T, k, F32, pitch=k + 1), rnd(121, k, n, F32, std=k ** -0.5, pitch=n + 3)
    wt = rnd(122, n, k, F32, pitch=k + 5)
    wt.copy_(w.t())
    y, du = Guarded(T, n, F32, n + 1), Guarded(T, n, F32, n + 2)
    ws = torch.empty(max(M.mlp_linear_workspace_bytes(T, k, n, F32),
                         M.mlp_linear_bwd_workspace_bytes(T, n, k, F32)), dtype=torch.uint8,
                     device="cuda")
    u = rnd(123, T, n, F32, std=1.5, pitch=n + 1)
    db = torch.empty(n, device="cuda")
    M.mlp_linear_fwd(x, w, y.v, act=M.MLP_ACT_GELU, workspace=ws)
    M.mlp_linear_bwd(x, wt, du.v, act=M.MLP_ACT_GELU, u=u, dbias=db, workspace=ws)
    ru = x.double() @ w.double()
    e = (k + 8) * 2 * U24 * (x.double().abs() @ w.double().abs())
    f, df, _ = act_ref(ru, "gelu")
    near(y.v, f, (df.abs() + 0.1) * e + ACT_ERR * (1 + ru.abs()), "y")
    rdu = ru * act_ref(u.double(), "gelu")[1]
    e = 1.2 * e + (ru.abs() + e) * ACT_ERR * (1 + u.double().abs()) + 2 * U24 * rdu.abs()
    near(du.v, rdu, e, "du")
    near(db, rdu.sum(0), e.sum(0) + (T + 8) * U24 * rdu.abs().sum(0), "dbias")
    assert y.intact() and du.intact()


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with a workspace of its own."""
    T, k, n = 64, 4096, 256
    jobs = []
    for i in range(2):
        x, w, dy = rnd(110 + i, T, k, BF16), rnd(112 + i, k, n, BF16, k ** -0.5), rnd(114 + i, T, n,
                                                                                      BF16)
        ws = torch.empty(max(M.mlp_linear_workspace_bytes(T, k, n, BF16),
                             M.mlp_layernorm_workspace_bytes(T, n)), dtype=torch.uint8,
                         device="cuda")
        o = [torch.empty(T, n, dtype=BF16, device="cuda") for _ in range(3)]
        f = [torch.empty(z, device="cuda") for z in (T, T, n, n)]
        jobs.append((x, w, dy, ws, o, f, torch.cuda.Stream()))

    def one(x, w, dy, ws, o, f, stream):
        M.mlp_linear_fwd(x, w, o[0], act=M.MLP_ACT_GELU, workspace=ws, stream=stream)
        M.mlp_layernorm_fwd(o[0], o[1], mean=f[0], rstd=f[1], stream=stream)
        M.mlp_layernorm_bwd(dy, f[0], f[1], o[2], f[2], f[3], ws, x=o[0], stream=stream)

    ref = []
    for j in jobs:
        one(*j)
        torch.cuda.synchronize()
        ref.append([t.clone() for t in j[4] + j[5]])
    for _ in range(20):
        for j in jobs:
            one(*j)
    torch.cuda.synchronize()
    for j, r in zip(jobs, ref):
        for a, b in zip(j[4] + j[5], r):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n_blocks,T", [(1, 200), (2, 300), (3, 1000), (4, 257)])
def test_stack_with_8bit_checkpoints(n_blocks, T):
    """The step equals, bit for bit, the public block calls with every kept
    block output passed through an 8-bit checkpoint; its loss equals the step's
    without checkpoints."""
    d, h, lr, mom = 512, 512, 0.02, 0.9
    per = 2 * d * h
    x0, tgt = rnd(90, T, d, BF16).contiguous(), rnd(91, T, d, BF16).contiguous()
    p0 = (0.02 * vec(92, n_blocks * per, std=1.0)).to(BF16)

    def buffers():
        p = p0.float()
        return p, torch.zeros_like(p), torch.zeros_like(p), p0.clone(), torch.zeros(4, device="cuda")

    P, V, G, W, L = buffers()
    ws = torch.empty(M.mlp_stack_ckpt8_workspace_bytes(n_blocks, T, d, h), dtype=torch.uint8,
                     device="cuda")
    M.mlp_stack_train_step_ckpt8(n_blocks, T, d, h, x0, tgt, P, V, G, W, lr, mom, L, ws)
    P1, V1, G1, W1, L1 = buffers()
    ws1 = torch.empty(M.mlp_stack_workspace_bytes(n_blocks, T, d, h), dtype=torch.uint8,
                      device="cuda")
    M.mlp_stack_train_step(n_blocks, T, d, h, x0, tgt, P1, V1, G1, W1, lr, mom, L1, ws1)
    assert torch.equal(L[0], L1[0])

    wg = lambda l: p0[l * per:l * per + d * h].view(d, h)  # noqa: E731
    wd = lambda l: p0[l * per + d * h:(l + 1) * per].view(h, d)  # noqa: E731
    xs, rs = [x0], []
    for l in range(n_blocks):
        y, r = torch.empty_like(x0), torch.empty(T, device="cuda")
        M.mlp_block_fwd(xs[-1], wg(l), wd(l), y, r)
        xs.append(y)
        rs.append(r)
    dy, loss = torch.empty_like(x0), torch.zeros(4, device="cuda")
    M.mse_loss_fwd_bwd(xs[-1], tgt, loss, dy,
                       torch.empty(M.mse_workspace_bytes(T * d), dtype=torch.uint8, device="cuda"))
    bws = torch.empty(M.mlp_block_workspace_bytes(T, d, h), dtype=torch.uint8, device="cuda")
    for l in reversed(range(n_blocks)):
        x = xs[l]
        if l:
            x = ckpt_values(*ckpt_ref(x)).to(BF16)
        dx, dg, dd = torch.empty_like(x0), torch.empty(d, h, device="cuda"), torch.empty(
            h, d, device="cuda")
        M.mlp_block_bwd(x, rs[l], wg(l), wd(l), dy, dx, dg, dd, bws)
        assert torch.equal(G[l * per:l * per + d * h].view(d, h), dg), l
        assert torch.equal(G[l * per + d * h:(l + 1) * per].view(h, d), dd), l
        dy = dx
    # and the gradients are those of the exact inputs up to the inputs' 8-bit
    # error: at most 1/128 of a group's largest magnitude, sqrt(32)/128 = 0.045
    # of its norm, in each of the two factors that depend on the input
    if n_blocks > 1:
        assert float((G - G1).norm() / G1.norm()) < 0.09
    else:
        assert torch.equal(G, G1)


def test_offsets_past_32_bits():
    """Rows so far apart that element offsets pass 2^31."""
    T, d, ld = 70_000, 64, 40_000
    base = torch.empty(T, ld, dtype=BF16, device="cuda")
    x = base[:, 128:192]
    x.copy_(rnd(80, T, d, BF16))
    last = slice(T - 300, T)
    y, out = base[:, 512:576], base[:, 1024:1088]
    M.mlp_layernorm_fwd(x, y)
    z = torch.empty(300, d, dtype=BF16, device="cuda")
    M.mlp_layernorm_fwd(x[last].contiguous(), z)
    assert torch.equal(y[last], z)
    qb = torch.empty(T, ld, dtype=torch.int8, device="cuda")
    q, s = qb[:, 32:96], torch.empty(T, 2, dtype=torch.uint8, device="cuda")
    M.mlp_ckpt8_encode(x, q, s)
    M.mlp_ckpt8_decode(q, s, out)
    assert torch.equal(out[last], ckpt_values(*ckpt_ref(x[last])).to(BF16))
    w = rnd(81, d, d, BF16, 0.125)
    M.mlp_linear_fwd(x, w, y, act=M.MLP_ACT_RELU, residual=out)
    M.mlp_linear_fwd(x[last].contiguous(), w, z, act=M.MLP_ACT_RELU,
                     residual=out[last].contiguous())
    near(y[last], z, 2 * half(BF16) * z.double().abs() + 1e-6, "y")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,n", [(2001, 72, 1600), (3300, 1160, 1088), (4097, 512, 832)])
def test_linear_whole_pieces(T, k, n, dtype):
    """Outputs and saved values that rows of 16-byte pieces let TMA move, against
    the same call at odd pitches (the general form: the same arithmetic, so the
    same bits) and, for y and du, the formula; every combination of them."""
    x, w, bias = rnd(130, T, k, dtype), rnd(131, k, n, dtype, std=k ** -0.5), vec(132, n)
    wt = w.t().contiguous()
    if k % 8:
        wt = rnd(133, n, k, dtype)
        wt.copy_(w.t())
    r = rnd(134, T, n, dtype)
    r_odd = rnd(135, T, n, dtype, pitch=n + 1)
    r_odd.copy_(r)
    raw = x.double() @ w.double()
    eraw = (k + 8) * 2 * U24 * (x.double().abs() @ w.double().abs())
    ru = raw + bias.double()
    eu = eraw + U24 * (ru.abs() + bias.double().abs())
    f, df, curve = act_ref(ru, "gelu_tanh")
    ef = df.abs() * eu + curve * eu * eu + ACT_ERR * (1 + ru.abs()) * (1 + f.abs())
    for res in (False, True):
        for save in ("none", "u", "ckpt", "both"):
            got = []
            for pitch in (None, n + 1):
                y, u = Guarded(T, n, dtype, pitch), Guarded(T, n, dtype, pitch)
                q, s = new_ckpt(T, n, pitch)
                M.mlp_linear_fwd(x, w, y.v, bias=bias, act=M.MLP_ACT_GELU_TANH,
                                 residual=(r_odd if pitch else r) if res else None,
                                 u=u.v if save in ("u", "both") else None,
                                 ckpt=(q.v, s.v) if save in ("ckpt", "both") else None)
                assert y.intact() and u.intact() and q.intact() and s.intact()
                got.append((y.v, u.v, q.v, s.v))
            assert all(torch.equal(a, b) for a, b in zip(*got)), (res, save)
            ref = f + r.double() if res else f
            near(got[0][0], ref, rounding(dtype, ref) + ef + 2 * U24 * (ref.abs() + f.abs()), "y")
    u = rnd(136, T, n, dtype, std=1.5)
    u_odd = rnd(137, T, n, dtype, pitch=n + 1)
    u_odd.copy_(u)
    ws = torch.empty(M.mlp_linear_bwd_workspace_bytes(T, n, k, dtype), dtype=torch.uint8,
                     device="cuda")
    for saved in ("none", "u", "ckpt"):
        seen = u.double()
        for again in (False, True):
            if saved == "none" and again:
                continue
            got = []
            for pitch in (None, n + 1):
                kw = {"u": u_odd if pitch else u}
                if saved == "ckpt":
                    q, s = new_ckpt(T, n, pitch)
                    M.mlp_ckpt8_encode(u, q.v, s.v)
                    kw, seen = {"ckpt": (q.v, s.v)}, ckpt_values(q.v, s.v)
                du, a = Guarded(T, n, dtype, pitch), Guarded(T, n, dtype, pitch)
                db = torch.full((n,), math.nan, device="cuda")
                M.mlp_linear_bwd(x, wt, du.v, dbias=db, a=a.v if again else None, workspace=ws,
                                 **({"act": M.MLP_ACT_SILU, **kw} if saved != "none" else {}))
                assert du.intact() and a.intact()
                got.append((du.v, a.v, db))
            assert all(torch.equal(a, b) for a, b in zip(*got)), (saved, again)
            d = act_ref(seen, "silu")[1] if saved != "none" else torch.ones_like(raw)
            ref = raw * d
            e = eraw * d.abs() + 2 * U24 * ref.abs() + (raw.abs() + eraw) * ACT_ERR * (
                1 + seen.abs()) * (saved != "none")
            near(got[0][0], ref, rounding(dtype, ref) + e + 1e-30, "du")
            near(got[0][2], ref.sum(0), e.sum(0) + (T + 8) * U24 * ref.abs().sum(0) + 1e-30,
                 "dbias")


@pytest.mark.parametrize("T,d", [(1, 8200), (9, 10477), (380, 8209), (2500, 8200)])
def test_layernorm_backward_wide_rows(T, d):
    """Rows wider than a block's registers: eight of them to a partial row."""
    x, dy = rnd(140, T, d, F32, shift=0.3), rnd(141, T, d, F32, std=0.1)
    _, mu, rho = ln_ref(x, None, None, 1e-5)
    dx, dg, ds = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(M.mlp_layernorm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    M.mlp_layernorm_bwd(dy, mu.float(), rho.float(), dx, dg, ds, ws, x=x)
    mu, rho = mu.float().double(), rho.float().double()
    xh = (x.double() - mu[:, None]) * rho[:, None]
    t = dy.double() * xh
    # a term: the difference (half a step of |x - mu|, which is |xh| / rho), two
    # products and the sum of T of them in any order
    near(dg, t.sum(0), (T + 8) * U24 * t.abs().sum(0) + 1e-30, "dgain")
    near(ds, dy.double().sum(0), (T + 8) * U24 * dy.double().abs().sum(0), "dshift")


@pytest.mark.parametrize("T,n", [(1, 10242), (8, 130), (9, 1001), (448, 10242)])
def test_act_backward_few_rows(T, n):
    """Fewer rows to a warp where there are few: their column sums."""
    dy, u = rnd(150, T, n, BF16), rnd(151, T, n, BF16, std=2.0)
    du, a = Guarded(T, n, BF16), Guarded(T, n, BF16)
    db = torch.full((n,), math.nan, device="cuda")
    ws = torch.empty(M.mlp_act_bwd_workspace_bytes(T, n), dtype=torch.uint8, device="cuda")
    M.mlp_act_bwd(dy, du.v, act=M.MLP_ACT_RELU, u=u, dbias=db, a=a.v, workspace=ws)
    ref = dy.double() * (u > 0)
    assert torch.equal(du.v.double(), ref) and torch.equal(a.v, u.clamp(min=0))
    near(db, ref.sum(0), (T + 8) * U24 * ref.abs().sum(0) + 1e-30, "dbias")
    assert du.intact() and a.intact()


def test_linear_f32_many_rows():
    """More row tiles than a grid's second dimension holds."""
    T, k, n = 65535 * 128 + 5, 4, 3
    x, w, bias = rnd(160, T, k, F32), rnd(161, k, n, F32), vec(162, n)
    y = Guarded(T, n, F32, 3)
    ws = torch.empty(M.mlp_linear_workspace_bytes(T, k, n, F32), dtype=torch.uint8, device="cuda")
    M.mlp_linear_fwd(x, w, y.v, bias=bias, act=M.MLP_ACT_RELU, workspace=ws)
    u = x.double() @ w.double() + bias.double()
    # four products and four sums, each off by at most half a step of the sum
    # of the terms' magnitudes
    e = 8 * U24 * (x.double().abs() @ w.double().abs() + bias.double().abs())
    near(y.v, u.clamp(min=0), e, "y")
    assert y.intact()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ckpt8_again_is_the_same(dtype):
    """Encoding what was decoded gives the same bytes (q has at most 8 bits)."""
    x = rnd(163, 300, 1001, dtype, std=3.0) * torch.logspace(-30, 30, 300, device="cuda")[:, None]
    x = x.to(dtype)
    q, s, q2, s2 = *new_ckpt(300, 1001), *new_ckpt(300, 1001)
    out = torch.empty(300, 1001, dtype=dtype, device="cuda")
    M.mlp_ckpt8_encode(x, q.v, s.v)
    M.mlp_ckpt8_decode(q.v, s.v, out)
    M.mlp_ckpt8_encode(out, q2.v, s2.v)
    assert torch.equal(q.v, q2.v) and torch.equal(s.v, s2.v)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_ckpt8_special_values_at_odd_pitches(dtype):
    """Infinities, NaNs, zeros, tiny values and largest magnitudes that round to
    128, in rows that start anywhere: the bytes of the same rows aligned."""
    d = 1001
    x = rnd(164, 40, d, dtype, std=2.0)
    tiny = torch.finfo(dtype).smallest_normal
    for i, v in enumerate((math.inf, -math.inf, math.nan, 0.0, tiny, -tiny / 4, 1.9999, -255 / 128,
                           torch.finfo(dtype).max)):
        x[4 * i, 31 * i::97] = v
        x[4 * i + 1] = v
        x[4 * i + 2, d - 1] = v
    odd = rnd(165, 40, d, dtype, pitch=d)
    odd.copy_(x)
    q, s, q2, s2 = *new_ckpt(40, d), *new_ckpt(40, d, d)
    M.mlp_ckpt8_encode(x, q.v, s.v)
    M.mlp_ckpt8_encode(odd, q2.v, s2.v)
    assert torch.equal(q.v, q2.v) and torch.equal(s.v, s2.v) and s2.intact()
    a, b = Guarded(40, d, dtype), Guarded(40, d, dtype, d)
    M.mlp_ckpt8_decode(q.v, s.v, a.v)
    M.mlp_ckpt8_decode(q.v, s.v, b.v)
    ra, rb = (t.v.contiguous().view(torch.int32 if dtype == F32 else torch.int16) for t in (a, b))
    assert torch.equal(a.v.isnan(), b.v.isnan())
    assert torch.equal(ra[~a.v.isnan()], rb[~b.v.isnan()]) and a.intact() and b.intact()


def test_act_backward_workspace_of_fewer_rows():
    """Fewer rows may need a larger workspace: one too small for them is refused,
    the largest of the sizes serves all."""
    n, counts = 128, (58_400, 58_300, 700)
    sizes = [M.mlp_act_bwd_workspace_bytes(T, n) for T in counts]
    assert sizes[1] > sizes[0]
    dy, u = rnd(170, counts[0], n, BF16), rnd(171, counts[0], n, BF16)
    du, db = torch.empty_like(dy), torch.empty(n, device="cuda")
    small = torch.empty(sizes[0], dtype=torch.uint8, device="cuda")
    with pytest.raises(M.MlpError):
        M.mlp_act_bwd(dy[:counts[1]], du[:counts[1]], u=u[:counts[1]], act=M.MLP_ACT_RELU,
                      dbias=db, workspace=small)
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    for T in counts:
        M.mlp_act_bwd(dy[:T], du[:T], u=u[:T], act=M.MLP_ACT_RELU, dbias=db, workspace=ws)
        ref = dy[:T].double() * (u[:T] > 0)
        assert torch.equal(du[:T].double(), ref)
        near(db, ref.sum(0), (T + 8) * U24 * ref.abs().sum(0), "dbias")
