"""The feed-forward operators where values, pitches and callers are unusual."""
import math
import threading

import pytest
import torch

import mlp_step_gb300 as M
from test_gpu_ffn import ACTS, BF16, F16, F32, SLOPE, Guarded, near, rnd, rounding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    M.load()
    yield
    assert M.get_device_status() == M.MLP_OK


def bytes_for(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------ activations

LIMIT_INPUTS = [math.inf, -math.inf, 3e38, -3e38, 1e4, -1e4, 0.0, math.nan]


def check_limits(got, u, act, what):
    """f of LIMIT_INPUTS in turn along the rows of u: infinities and the largest
    values go to their limits."""
    most = torch.finfo(got.dtype).max
    got, u = got.double(), u.double()
    assert torch.equal(got.isnan(), u.isnan()), what
    if act == "leaky2":
        f = torch.where(u > 0, u, SLOPE * u) ** 2
        assert torch.equal(got.isinf(), f > most), what
        return
    if act == "none":
        assert torch.equal(got.nan_to_num(7.0), u.nan_to_num(7.0)), what
        return
    up, down = u > 0, u < 0
    assert torch.equal(got[up], u[up]), what
    assert (got[down].abs() < 1e-30).all() and (got[u == 0] == 0).all(), what


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_activation_values_at_their_limits(act, dtype):
    """f(u) of infinite and very large u, forward and backward, in every kernel:
    the limits 0 and u, not 0 times infinity (and not -infinity in fp32, where
    Phi(-14) is not yet 0)."""
    col = torch.tensor(LIMIT_INPUTS, device="cuda")
    if dtype == F16:
        col = col.clamp(-6e4, 6e4).where(col.isfinite(), col)
    if act == "leaky2":
        col = col.where(col.abs() != 1e4, col / 1e3)  # squares of 16-bit values stay finite
    col = col.to(dtype)
    # the activation's backward alone, four columns a lane and one
    for pitch in (None, 13):
        u = rnd(1, 12, 8, dtype, pitch=pitch)
        u.copy_(col.expand(12, 8))
        du, a = Guarded(12, 8, dtype, pitch), Guarded(12, 8, dtype, pitch)
        dy = rnd(2, 12, 8, dtype, pitch=pitch)
        M.mlp_act_bwd(dy, du.v, act=ACTS[act], slope=SLOPE, u=u, a=a.v)
        check_limits(a.v, u, act, "a")
        assert a.intact()
    # a product of one term: few rows, single tiles, split sums, pairs
    for T, k, n in ((1, 1, 64), (8, 1, 96), (16, 4096, 64), (300, 1, 200), (4100, 1, 776)):
        rows = col[torch.arange(T, device="cuda") % 8]
        x = torch.zeros(T, (k + 7) // 8 * 8, dtype=dtype, device="cuda")[:, :k]
        x[:, 0] = rows
        w = torch.zeros(k, n, dtype=dtype, device="cuda")
        w[0] = 1
        u = rows[:, None].expand(T, n)
        ws = bytes_for(M.mlp_linear_workspace_bytes(T, k, n, dtype))
        for odt in {F32, dtype}:
            y = Guarded(T, n, odt)
            M.mlp_linear_fwd(x, w, y.v, act=ACTS[act], slope=SLOPE, workspace=ws)
            check_limits(y.v, u, act, ("y", T, odt))
        # and the activations again, beside a gradient of zero
        dy, wt = (torch.zeros(r, (k + 7) // 8 * 8, dtype=dtype, device="cuda") for r in (T, n))
        us = rnd(3, T, n, dtype)
        us.copy_(u)
        du, a = Guarded(T, n, dtype), Guarded(T, n, dtype)
        ws = bytes_for(M.mlp_linear_bwd_workspace_bytes(T, n, k, dtype))
        M.mlp_linear_bwd(dy[:, :k], wt[:, :k], du.v, act=ACTS[act], slope=SLOPE, u=us, a=a.v, workspace=ws)
        check_limits(a.v, u, act, ("a", T))


def act_terms(u, act):
    """f(u), its derivative, the sum of magnitudes of the derivative's two terms,
    and the argument of the exponential in it, in 64 bits."""
    if act == "gelu":
        p = torch.special.erfc(-u / math.sqrt(2)) / 2
        b = u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
        return u * p, p + b, p + b.abs(), u * u / 2
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        z, dz = c * (u + 0.044715 * u ** 3), c * (1 + 3 * 0.044715 * u * u)
    else:
        z, dz = u, torch.ones_like(u)
    s = 1 / (1 + torch.exp(-z))
    b = u * s / (1 + torch.exp(z)) * dz
    return u * s, s + b, s + b.abs(), z


def act_error(u, act, fp32):
    """Relative error of f(u), and of f'(u) against its two terms."""
    z = act_terms(u, act)[3].abs()
    if fp32:
        # the argument is off by two roundings (four for the cubic), which the
        # exponential turns into |z| times as much (erfc of u / sqrt 2 into
        # u^2 = 2 z); the functions are good to 4 ulp, the division to 2, and
        # some roundings of products and sums
        return (8 * z + 20) * 2.0 ** -24
    if act == "gelu":
        # the polynomial's 2.7e-6 with the functions' few 2^-23, and the
        # exponent u^2 / 2 after two roundings
        return 4e-6 + u * u * 2.0 ** -24
    # the exponent's four roundings, the hardware functions' few 2^-23
    return (4 * z + 16) * 2.0 ** -23


# what reads as 0: the fast division's quotients by more than 2^126 (times |u|),
# subnormal results of the hardware exponential
LOST = 2.0 ** -118


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_activation_tails(act, dtype):
    """f and f' of negative pre-activations are as exact relative to their own
    (small) values as they are near 0: in outputs of the operand type, and in fp32 ones
    of a 16-bit layer."""
    n = 2048
    u = torch.linspace(-1, 0, n, device="cuda") * (40 if act == "silu" else 12)
    u = torch.stack([u, u.flip(0) * 0.37]).to(dtype)
    ud = u.double()
    f, df, terms, _ = act_terms(ud, act)
    e = act_error(ud, act, dtype == F32)
    du, a = torch.empty_like(u), torch.empty_like(u)
    M.mlp_act_bwd(torch.ones_like(u), du, act=ACTS[act], u=u, a=a)
    # (the error comes before the rounding: both, and the error's own rounding)
    r = lambda ref, err, t: rounding(t, ref) * (1 + 1e-3) + err + LOST  # noqa: E731
    near(a, f, r(f, e * f.abs(), dtype), "f")
    near(du, df, r(df, e * terms, dtype), "f'")
    # a product that gives u (forward) or 1 (backward) exactly, fp32 outputs:
    # few rows, single tiles, pairs
    for T in (2, 200, 4100):
        x = torch.zeros(T, 8, dtype=dtype, device="cuda")
        x[::2, 0], x[1::2, 1] = 1, 1
        w = torch.zeros(8, n, dtype=dtype, device="cuda")
        w[:2] = u
        rows = torch.arange(T, device="cuda") % 2
        ws = bytes_for(M.mlp_linear_workspace_bytes(T, 8, n, dtype))
        for odt in {F32, dtype}:
            y = torch.empty(T, n, dtype=odt, device="cuda")
            M.mlp_linear_fwd(x, w, y, act=ACTS[act], workspace=ws)
            near(y, f[rows], r(f, e * f.abs(), odt)[rows], ("y", T, odt))
        one = torch.ones(n, 8, dtype=dtype, device="cuda")
        us = u[rows].contiguous()
        ws = bytes_for(M.mlp_linear_bwd_workspace_bytes(T, n, 8, dtype))
        for odt in {F32, dtype}:
            g = torch.empty(T, n, dtype=odt, device="cuda")
            a = torch.empty(T, n, dtype=dtype, device="cuda")
            M.mlp_linear_bwd(x, one, g, act=ACTS[act], u=us, a=a, workspace=ws)
            near(g, df[rows], r(df, e * terms, odt)[rows], ("du", T, odt))
            near(a, f[rows], r(f, e * f.abs(), dtype)[rows], ("a", T, odt))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_activations_above_zero(act, dtype):
    """Beside 0 and above it errors are absolute: 3e-7 of 1 + |u|.  (The tanh
    form's f' = s + u s (1 - s) z' has u z' of up to 38 beside 1 - s, which is
    off by the 2 ulp of s, 2^-23, until s is 1 for z above 24 ln 2 = 16.7.)"""
    u = torch.linspace(-1, 30, 4096, device="cuda").view(1, -1).to(dtype)
    f, df, _, _ = act_terms(u.double(), act)
    du, a = torch.empty_like(u), torch.empty_like(u)
    M.mlp_act_bwd(torch.ones_like(u), du, act=ACTS[act], u=u, a=a)
    e = 3e-7 * (1 + u.double().abs())
    near(a, f, rounding(dtype, f) * (1 + 1e-3) + e, "f")
    if act == "gelu_tanh":
        ud = u.double()
        dz = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * ud * ud)
        z = act_terms(ud, act)[3]
        e = e + ud.abs() * dz * torch.where(z < 18, 2.0 ** -23, torch.exp(-z))
    near(du, df, rounding(dtype, df) * (1 + 1e-3) + e, "f'")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_activation_derivatives_at_their_limits(dtype):
    """f' of infinite and largest u where it has no limit in [0, 1], and of NaN."""
    big = 6e4 if dtype == F16 else 3e38
    u = torch.tensor([[math.inf, -math.inf, big, -big, 4.0, -4.0, 0.0, math.nan]],
                     device="cuda").to(dtype)
    dy, du = torch.full_like(u, 0.5), torch.empty_like(u)
    inf = math.inf
    for act, want in (("none", [0.5] * 8), ("relu", [0.5, 0, 0.5, 0, 0.5, 0, 0, None]),
                      # 0.5 * 2 slope^2 u
                      ("leaky2", [inf, -inf, None, None, 4, -1, 0, math.nan])):
        M.mlp_act_bwd(dy, du, act=ACTS[act], slope=SLOPE, u=u)
        for got, ref in zip(du[0].tolist(), want):
            assert ref is None or got == ref or (math.isnan(ref) and math.isnan(got)), (act, got, ref)
    for act in ("gelu", "gelu_tanh", "silu"):
        M.mlp_act_bwd(dy, du, act=ACTS[act], u=u)
        assert du[0, [0, 2]].tolist() == [0.5, 0.5] and du[0, 7].isnan(), act
        assert (du[0, [1, 3]].double().abs() < 1e-30).all() and abs(du[0, 6].item() - 0.25) < 1e-6, act


# ------------------------------------------------------------ mixed pitches

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,n", [(200, 520, 200), (1500, 520, 1001), (2000, 72, 2000),
                                   (4100, 200, 776), (3300, 1160, 1088)])
def test_linear_input_by_tma_output_by_copies(T, k, n, dtype):
    """A residual (u) that TMA brings into the box of a unit whose output leaves
    by the warp's own copies, its rows at an odd pitch or its last columns ragged:
    the same bits as where all of them are moved value by value."""
    x, w, bias = rnd(4, T, k, dtype), rnd(5, k, n, dtype, std=k ** -0.5), torch.randn(n, device="cuda")
    wt = rnd(6, n, k, dtype)
    wt.copy_(w.t())
    r, u = rnd(7, T, n, dtype), rnd(8, T, n, dtype, std=1.5)
    odd = [rnd(9, T, n, dtype, pitch=n + 1) for _ in range(2)]
    odd[0].copy_(r)
    odd[1].copy_(u)
    ws = bytes_for(max(M.mlp_linear_workspace_bytes(T, k, n, dtype),
                       M.mlp_linear_bwd_workspace_bytes(T, n, k, dtype)))
    got = []
    for res, saved, pitch in ((odd[0], odd[1], n + 1), (r, u, n + 1), (r, u, None)):
        y, du = Guarded(T, n, dtype, pitch), Guarded(T, n, dtype, pitch)
        db = torch.empty(n, device="cuda")
        for _ in range(3):  # the same again, over itself
            M.mlp_linear_fwd(x, w, y.v, bias=bias, act=M.MLP_ACT_RELU, residual=res, workspace=ws)
            M.mlp_linear_bwd(x, wt, du.v, act=M.MLP_ACT_RELU, u=saved, dbias=db, workspace=ws)
        assert y.intact() and du.intact()
        got.append((y.v, du.v, db))
    for a in got[1:]:
        assert all(torch.equal(p, q) for p, q in zip(got[0], a))
    # and of the formula: a term's rounding in fp32 each, then one to 16 bits
    ru = x.double() @ w.double()
    e = (k + 8) * 2.0 ** -23 * (x.double().abs() @ w.double().abs())
    ref = (ru + bias.double()).clamp(min=0) + r.double()
    near(got[0][0], ref, rounding(dtype, ref) + e + 2.0 ** -22 * (ref.abs() + bias.double().abs()), "y")
    ref = ru * (u.double() > 0)
    near(got[0][1], ref, rounding(dtype, ref) + e + 1e-30, "du")


# ------------------------------------------------------------ callers

def test_host_threads_at_once():
    """Calls from several host threads, each on a stream and a workspace of its
    own: the bits of the same calls one after another."""
    T, k, n = 96, 1040, 784
    jobs = []
    for i, dtype in enumerate((BF16, F16, F32, BF16, F16, F32)):
        x, w = rnd(20 + i, T, k, dtype), rnd(30 + i, k, n, dtype, std=k ** -0.5)
        o = [torch.empty(T, n, dtype=dtype, device="cuda") for _ in range(4)]
        f = [torch.empty(z, device="cuda") for z in (T, T, n, n, n)]
        ws = bytes_for(max(M.mlp_linear_workspace_bytes(T, k, n, dtype),
                           M.mlp_layernorm_workspace_bytes(T, n),
                           M.mlp_act_bwd_workspace_bytes(T, n)))
        jobs.append((x, w, o, f, ws, torch.cuda.Stream()))

    def one(x, w, o, f, ws, stream):
        M.mlp_linear_fwd(x, w, o[0], act=M.MLP_ACT_GELU, workspace=ws, stream=stream)
        M.mlp_layernorm_fwd(o[0], o[1], mean=f[0], rstd=f[1], stream=stream)
        M.mlp_layernorm_bwd(o[1], f[0], f[1], o[2], f[2], f[3], ws, x=o[0], stream=stream)
        M.mlp_act_bwd(o[2], o[3], act=M.MLP_ACT_SILU, u=o[0], dbias=f[4], workspace=ws,
                      stream=stream)

    def run(job):
        with torch.cuda.device(0):
            for _ in range(25):
                one(*job)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    got = [[t.clone() for t in j[2] + j[3]] for j in jobs]
    for j, g in zip(jobs, got):
        for t in j[2] + j[3]:
            t.fill_(math.nan)
        torch.cuda.synchronize()
        one(*j)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(j[2] + j[3], g))


def test_host_thread_without_a_context():
    """The first CUDA call of a host thread may be one of ours: products whose
    tensor maps a driver call encodes work in it."""
    T, k, n = 96, 1040, 784
    x, w, c = rnd(40, T, k, BF16), rnd(41, k, n, BF16, std=k ** -0.5), torch.empty(T, n, device="cuda")
    y = torch.empty(T, n, dtype=BF16, device="cuda")
    ws = bytes_for(M.mlp_linear_workspace_bytes(T, k, n, BF16))
    calls = [lambda: M.mlp_linear_fwd(x, w, y, workspace=ws), lambda: M.mlp_gemm(x, w, c, T, n, k)]
    for call, out in zip(calls, (y, c)):
        call()  # here first, so that nothing is left to set up
        torch.cuda.synchronize()
        want, raised = out.clone(), []
        out.fill_(math.nan)
        torch.cuda.synchronize()

        def run():
            try:
                call()
            except M.MlpError as e:
                raised.append(e)
        t = threading.Thread(target=run)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not raised and torch.equal(out, want)


# ------------------------------------------------------------ products with ragged rows

@pytest.mark.parametrize("out", [F32, None])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,n,k", [(2048, 1001, 136), (1040, 1015, 64), (20000, 1004, 72)])
def test_gemm_leaves_what_lies_behind_its_columns(T, n, k, dtype, out):
    """mlp_gemm (the weight gradients of these layers) into wider rows: nothing
    past the last column is written, and the values are the product's."""
    x, w = rnd(50, T, k, dtype), rnd(51, k, n, dtype, std=k ** -0.5)
    for pitch in (n, n + 3, 1024, 1032):
        c = Guarded(T, n, out or dtype, pitch)
        M.mlp_gemm(x, w, c.v, T, n, k)
        ref = x.double() @ w.double()
        e = (k + 8) * 2.0 ** -23 * (x.double().abs() @ w.double().abs())
        near(c.v, ref, rounding(out or dtype, ref) + e, "c")
        assert c.intact(), pitch


@pytest.mark.parametrize("prec,dtype", [(M.MLP_PREC_BF16, BF16), (M.MLP_PREC_FP16, F16)])
def test_bias_gradients_behind_odd_hidden_widths(prec, dtype):
    """A hidden width that is no whole number of 16-byte pieces at a large batch:
    the column of ones behind the layer's values, which gives the next layer's
    bias gradient, stays."""
    dims, batch = [64, 1001, 16], 2048
    n = M.mlp_param_count(dims)
    p0 = 0.05 * torch.randn(n, generator=torch.Generator().manual_seed(3))
    net = M.MLP(dims, prec=prec, max_batch=batch, params=p0)
    x = torch.rand(batch, 64, device="cuda")
    dl = (0.01 * torch.randn(batch, 16, device="cuda")).to(dtype)
    for _ in range(2):
        net.forward(x, torch.empty(batch, 16, device="cuda"))
        net.backward(dl, batch)
    torch.cuda.synchronize()
    db = net.grads[-16:].double()
    ref = dl.double()  # summed in fp32
    near(db, ref.sum(0), (batch + 8) * 2.0 ** -23 * ref.abs().sum(0), "db")


# ------------------------------------------------------------ in place

@pytest.mark.parametrize("ck", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d", [(1, 512), (300, 512), (77, 523), (130, 2000), (65, 4099),
                                 (40, 8192), (380, 8209), (50, 20000)])
def test_layernorm_backward_over_its_gradients(T, d, dtype, ck):
    """dx over dy, and over a dres that is dy: the bits of the call with a dx of
    its own, whatever the width."""
    x, dy = rnd(60, T, d, dtype, shift=0.3), rnd(61, T, d, dtype, std=0.1)
    gain = 1 + 0.2 * torch.randn(d, device="cuda")
    mean = x.float().mean(1)
    rstd = 1 / (x.float().var(1, unbiased=False) + 1e-5).sqrt()
    kw = {"x": x}
    if ck:
        q = torch.empty(T, d, dtype=torch.int8, device="cuda")
        s = torch.empty(T, M.mlp_ckpt8_scale_cols(d), dtype=torch.uint8, device="cuda")
        M.mlp_ckpt8_encode(x, q, s)
        kw = {"ckpt": (q, s)}
    ws = bytes_for(M.mlp_layernorm_workspace_bytes(T, d))
    for through in (False, True):
        want, got = Guarded(T, d, dtype), rnd(62, T, d, dtype)
        got.copy_(dy)
        sums = [torch.empty(d, device="cuda") for _ in range(4)]
        M.mlp_layernorm_bwd(dy, mean, rstd, want.v, sums[0], sums[1], ws, gain=gain,
                            dres=dy if through else None, **kw)
        M.mlp_layernorm_bwd(got, mean, rstd, got, sums[2], sums[3], ws, gain=gain,
                            dres=got if through else None, **kw)
        assert torch.equal(want.v, got)
        assert torch.equal(sums[0], sums[2]) and torch.equal(sums[1], sums[3])


# ------------------------------------------------------------ captured calls

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T", [1, 5, 300])
def test_operators_captured(T, dtype):
    """Every operator in one captured graph, replayed on new inputs: the bits of
    the calls one by one."""
    k, n = 520, 1001
    x, w = rnd(70, T, k, dtype), rnd(71, k, n, dtype, std=k ** -0.5)
    wt = rnd(72, n, k, dtype)
    wt.copy_(w.t())
    f = lambda z: torch.empty(z, device="cuda")  # noqa: E731
    e = lambda c, t=dtype: Guarded(T, c, t)  # noqa: E731
    o = {"n": e(k), "y": e(n), "u": e(n), "du": e(n), "a": e(n), "d2": e(n), "dx": e(k), "dec": e(k)}
    v = {"mean": f(T), "rstd": f(T), "dg": f(k), "ds": f(k), "db": f(n), "db2": f(n)}
    xq = (e(k, torch.int8).v, e(-(-k // 32), torch.uint8).v)
    uq = (e(n, torch.int8).v, e(-(-n // 32), torch.uint8).v)
    ws = [bytes_for(z) for z in (M.mlp_linear_workspace_bytes(T, k, n, dtype),
                                 M.mlp_linear_bwd_workspace_bytes(T, n, k, dtype),
                                 M.mlp_act_bwd_workspace_bytes(T, n),
                                 M.mlp_layernorm_workspace_bytes(T, k))]

    def calls():
        M.mlp_layernorm_fwd(x, o["n"].v, mean=v["mean"], rstd=v["rstd"], ckpt=xq)
        M.mlp_linear_fwd(o["n"].v, w, o["y"].v, act=M.MLP_ACT_SILU, u=o["u"].v, ckpt=uq,
                         workspace=ws[0])
        M.mlp_linear_bwd(o["n"].v, wt, o["du"].v, act=M.MLP_ACT_GELU, ckpt=uq, dbias=v["db"],
                         a=o["a"].v, workspace=ws[1])
        M.mlp_act_bwd(o["y"].v, o["d2"].v, act=M.MLP_ACT_GELU_TANH, u=o["u"].v, dbias=v["db2"],
                      workspace=ws[2])
        M.mlp_layernorm_bwd(o["n"].v, v["mean"], v["rstd"], o["dx"].v, v["dg"], v["ds"], ws[3],
                            ckpt=xq)
        M.mlp_ckpt8_decode(*xq, o["dec"].v)

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    x.copy_(rnd(73, T, k, dtype))
    outs = [t.v for t in o.values()] + list(v.values())
    calls()
    want = [t.clone() for t in outs]
    for _ in range(2):
        for t in outs:
            t.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert all(t.intact() for t in o.values())


@pytest.mark.parametrize("n_blocks,T", [(1, 1), (3, 1), (3, 257)])
def test_stack_with_8bit_checkpoints_captured(n_blocks, T):
    """The stack's step with 8-bit checkpoints from a single token on, eager and
    as a replayed graph."""
    d, h, per = 512, 512, 2 * 512 * 512
    x0, tgt = rnd(80, T, d, BF16).contiguous(), rnd(81, T, d, BF16).contiguous()
    g0 = torch.Generator(device="cuda").manual_seed(82)
    p0 = (0.02 * torch.randn(n_blocks * per, generator=g0, device="cuda")).to(BF16)
    P, W = p0.float(), p0.clone()
    V, G, L = torch.zeros_like(P), torch.zeros_like(P), torch.zeros(4, device="cuda")
    ws = bytes_for(M.mlp_stack_ckpt8_workspace_bytes(n_blocks, T, d, h))

    def reset():
        P.copy_(p0.float())
        W.copy_(p0)
        V.zero_()
        G.fill_(math.nan)
        ws.fill_(255)

    def step():
        M.mlp_stack_train_step_ckpt8(n_blocks, T, d, h, x0, tgt, P, V, G, W, 0.02, 0.9, L, ws)

    reset()
    step()
    want = [t.clone() for t in (P, V, G, W, L)]
    assert want[2].isfinite().all() and want[4][0] > 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    reset()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((P, V, G, W, L), want))


# ------------------------------------------------------------ far offsets

def test_backward_offsets_past_32_bits():
    """Gradients and saved values in rows so far apart that element offsets pass
    2^31: the last rows' values are those of a call on these rows alone."""
    T, d, ld = 70_000, 64, 40_000
    base = torch.empty(T, ld, dtype=BF16, device="cuda")
    qb = torch.empty(T, ld, dtype=torch.int8, device="cuda")
    col = lambda i: base[:, 128 * i:128 * i + d]  # noqa: E731
    dy, u, du, a, dx = (col(i) for i in range(5))
    dy.copy_(rnd(90, T, d, BF16))
    u.copy_(rnd(91, T, d, BF16, std=1.5))
    q, s = qb[:, 32:32 + d], torch.empty(T, 2, dtype=torch.uint8, device="cuda")
    M.mlp_ckpt8_encode(u, q, s)
    w = rnd(92, d, d, BF16, 0.125)
    mean, rstd = u.float().mean(1), 1 / u.float().std(1)
    db, dg, ds = (torch.empty(d, device="cuda") for _ in range(3))
    last = slice(T - 300, T)
    e = lambda: torch.empty(300, d, dtype=BF16, device="cuda")  # noqa: E731
    ws = bytes_for(max(f(t) for t in (T, 300) for f in (
        lambda t: M.mlp_act_bwd_workspace_bytes(t, d), lambda t: M.mlp_layernorm_workspace_bytes(t, d),
        lambda t: M.mlp_linear_bwd_workspace_bytes(t, d, d, BF16))))
    end = lambda t: t[last].clone(memory_format=torch.contiguous_format)  # noqa: E731
    for kw, kw_end in (({"u": u}, {"u": end(u)}), ({"ckpt": (q, s)}, {"ckpt": (end(q), end(s))})):
        M.mlp_act_bwd(dy, du, act=M.MLP_ACT_SILU, dbias=db, a=a, workspace=ws, **kw)
        g, h = e(), e()
        M.mlp_act_bwd(end(dy), g, act=M.MLP_ACT_SILU, a=h, **kw_end)
        assert torch.equal(du[last], g) and torch.equal(a[last], h)
        M.mlp_linear_bwd(dy, w, du, act=M.MLP_ACT_RELU, dbias=db, a=a, workspace=ws, **kw)
        M.mlp_linear_bwd(end(dy), w, g, act=M.MLP_ACT_RELU, a=h, workspace=ws, **kw_end)
        # 64 terms in another kernel's order, then one rounding each
        near(du[last], g, 2 * rounding(BF16, g.double()) + 64 * 2.0 ** -22, "du")
        assert torch.equal(a[last], h)
        x_kw = {("x" if k == "u" else k): v for k, v in kw.items()}
        x_end = {("x" if k == "u" else k): v for k, v in kw_end.items()}
        M.mlp_layernorm_bwd(dy, mean, rstd, dx, dg, ds, ws, dres=dy, **x_kw)
        M.mlp_layernorm_bwd(end(dy), end(mean), end(rstd), g, dg, ds, ws, dres=end(dy), **x_end)
        assert torch.equal(dx[last], g)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 8, 64])
def test_linear_weights_past_32_bits(T, dtype):
    """Weights of more than 2^31 elements: their last rows and columns are read
    where they are."""
    k, n, few = 60_000, 40_000, 40
    w = torch.zeros(k, n, dtype=dtype, device="cuda")
    w[-1] = rnd(93, 1, n, dtype)[0]
    x = torch.zeros(T, k, dtype=dtype, device="cuda")
    x[:, -1] = torch.arange(1, T + 1, device="cuda").to(dtype)
    y = torch.empty(T, n, dtype=dtype, device="cuda")
    ws = bytes_for(max(M.mlp_linear_workspace_bytes(T, k, n, dtype),
                       M.mlp_linear_bwd_workspace_bytes(T, k, n, dtype)))
    M.mlp_linear_fwd(x, w, y, workspace=ws)
    ref = x[:, -1:].double() * w[-1].double()
    near(y, ref, rounding(dtype, ref), "y")
    # backward: du[:, -1] is dy . w[-1], the others 0
    dy = torch.zeros(T, n, dtype=dtype, device="cuda")
    dy[:, -few:] = rnd(94, T, few, dtype)
    du = torch.empty(T, k, dtype=dtype, device="cuda")
    M.mlp_linear_bwd(dy, w, du, workspace=ws)
    p = dy[:, -few:].double() * w[-1, -few:].double()
    ref = p.sum(1)
    near(du[:, -1], ref, rounding(dtype, ref) + few * 2.0 ** -22 * p.abs().sum(1), "du")
    assert (du[:, :-1] == 0).all()
