"""The gated feed-forward sublayer's operators together, as a training step and a
serving step use them, and their calls captured, on several streams and threads,
and in rows past 2^31 elements."""
import math
import threading

import pytest
import torch

import mlp_step_gb300 as M
from philox import factor
from test_gpu_ffn import BF16, F16, F32, near, rnd, rounding, vec

pytestmark = pytest.mark.gpu

EPS, SCALE, P, SITE = 1e-6, 0.5, 0.25, 11


@pytest.fixture(scope="module", autouse=True)
def _lib():
    M.load()
    yield
    assert M.get_device_status() == M.MLP_OK


def bytes_for(n):
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


class Sublayer:
    """norm -> gated unit -> down projection -> norm, gate, dropout, residual and
    the next norm, with every gradient; weights of gate and up side by side."""

    def __init__(self, T, d, hidden, dtype, ckpt, seed=0):
        r = lambda i, rows, cols, std=1.0: rnd(100 * seed + i, rows, cols, dtype, std)  # noqa: E731
        self.T, self.d, self.n, self.dtype, self.ckpt = T, d, hidden, dtype, ckpt
        n = hidden
        self.x, self.z = r(1, T, d, 2.0), r(2, T, d)
        self.w, self.wd = r(3, d, 2 * n, d ** -0.5), r(4, n, d, n ** -0.5)
        self.dh, self.dn = r(5, T, d, 0.1), r(6, T, d, 0.1)
        self.gains = [vec(7 + i, d, 1.0) for i in range(3)]  # first, post, next
        self.rng = torch.tensor([1234567 + seed, 5], dtype=torch.int64, device="cuda")
        m = lambda rows, cols: torch.full((rows, cols), math.nan, dtype=dtype,  # noqa: E731
                                          device="cuda")
        v = lambda k: torch.full((k,), math.nan, device="cuda")  # noqa: E731
        self.out = dict(n0=m(T, d), r0=v(T), y=m(T, n), b=m(T, d), h=m(T, d), n1=m(T, d), rb=v(T),
                        rh=v(T), dx1=m(T, d), db=m(T, d), dz=m(T, d), dgu=m(T, 2 * n), a=m(T, n),
                        dn0=m(T, d), dx=m(T, d), dw=torch.empty(d, 2 * n, device="cuda"),
                        dwd=torch.empty(n, d, device="cuda"), dgain0=v(d), dpost=v(d), dnext=v(d))
        if ckpt:
            g = -(-n // 32)
            self.kept = [(torch.empty(T, n, dtype=torch.int8, device="cuda"),
                          torch.empty(T, g, dtype=torch.uint8, device="cuda")) for _ in range(2)]
        else:
            self.kept = [m(T, n), m(T, n)]
        sizes = [M.mlp_glu_workspace_bytes(T, d, n, dtype),
                 M.mlp_linear_workspace_bytes(T, n, d, dtype),
                 M.mlp_resnorm_workspace_bytes(T, d),
                 M.mlp_glu_bwd_workspace_bytes(T, n, d, dtype),
                 M.mlp_linear_bwd_workspace_bytes(T, d, 2 * n, dtype)]
        self.ws = bytes_for(max(sizes))

    def halves(self, m):
        return m[:, :self.n], m[:, self.n:]

    def forward(self, stream=None):
        o, s = self.out, dict(stream=stream)
        M.mlp_resnorm_fwd(self.x, n=o["n0"], next_gain=self.gains[0], h_rstd=o["r0"], eps=EPS, **s)
        kept = dict(zip(("g_ckpt", "u_ckpt") if self.ckpt else ("g", "u"), self.kept))
        M.mlp_glu_fwd(o["n0"], *self.halves(self.w), o["y"], workspace=self.ws, **kept, **s)
        M.mlp_linear_fwd(o["y"], self.wd, o["b"], workspace=self.ws, **s)
        M.mlp_resnorm_fwd(self.x, b=o["b"], h=o["h"], n=o["n1"], post_norm=True,
                          post_gain=self.gains[1], b_rstd=o["rb"], gate=self.z,
                          gate_act=M.MLP_GATE_SIGMOID, scale=SCALE, p=P, rng=self.rng, site=SITE,
                          next_gain=self.gains[2], h_rstd=o["rh"], eps=EPS, **s)

    def backward(self, stream=None):
        o, s = self.out, dict(stream=stream)
        M.mlp_resnorm_bwd(o["dx1"], dh=self.dh, dn=self.dn, h=o["h"], h_rstd=o["rh"],
                          next_gain=self.gains[2], b=o["b"], db=o["db"], post_norm=True,
                          post_gain=self.gains[1], b_rstd=o["rb"], gate=self.z, dgate=o["dz"],
                          gate_act=M.MLP_GATE_SIGMOID, scale=SCALE, p=P, rng=self.rng, site=SITE,
                          dpost_gain=o["dpost"], dnext_gain=o["dnext"], workspace=self.ws, **s)
        kept = dict(zip(("g_ckpt", "u_ckpt") if self.ckpt else ("g", "u"), self.kept))
        M.mlp_glu_bwd(o["db"], self.wd, *self.halves(o["dgu"]), a=o["a"], workspace=self.ws, **kept,
                      **s)
        M.mlp_gemm(o["a"], o["db"], o["dwd"], self.n, self.d, self.T, a_trans=True, **s)
        M.mlp_linear_bwd(o["dgu"], self.w, o["dn0"], workspace=self.ws, **s)
        M.mlp_gemm(o["n0"], o["dgu"], o["dw"], self.d, 2 * self.n, self.T, a_trans=True, **s)
        M.mlp_resnorm_bwd(o["dx"], dh=o["dx1"], dn=o["dn0"], h=self.x, h_rstd=o["r0"],
                          next_gain=self.gains[0], dnext_gain=o["dgain0"], workspace=self.ws, **s)

    def reference(self):
        """The same in 64 bits, the gradients by automatic differentiation."""
        leaf = lambda t: t.double().clone().requires_grad_()  # noqa: E731
        x, z, w, wd = (leaf(t) for t in (self.x, self.z, self.w, self.wd))
        gain = [leaf(g) for g in self.gains]
        norm = lambda t: t / ((t * t).mean(1, keepdim=True) + EPS).sqrt()  # noqa: E731
        n0 = norm(x) * gain[0]
        g, u = self.halves(n0 @ w)
        y = g * torch.sigmoid(g) * u
        b = y @ wd
        seed, step = self.rng.tolist()
        c = norm(b) * gain[1] * factor(self.T, self.d, P, seed, step, SITE)
        h = x + SCALE * torch.sigmoid(z) * c
        n1 = norm(h) * gain[2]
        ((h * self.dh.double()).sum() + (n1 * self.dn.double()).sum()).backward()
        return dict(n0=n0, y=y, b=b, h=h, n1=n1, dx=x.grad, dz=z.grad, dw=w.grad, dwd=wd.grad,
                    dgain0=gain[0].grad, dpost=gain[1].grad, dnext=gain[2].grad)


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,d,hidden", [(1, 64, 96), (77, 128, 232), (3000, 512, 1376)])
def test_training_step(T, d, hidden, dtype, ckpt):
    s = Sublayer(T, d, hidden, dtype, ckpt)
    s.forward()
    s.backward()
    # In the norm of each tensor: up to ten roundings of half a step lie on the
    # path of an output (stored activations and gradients, operands), each of
    # which norms, products and the activation pass on at most about doubled;
    # 8-bit g and u are off by up to half a step of 2^-6 of their group's largest
    # magnitude, three to four times the usual value: 2^-7 3.5 / sqrt(3), for both,
    # also doubled.  fp32: the sums of up to 2 hidden terms, as roundings each.
    tol = 20 * torch.finfo(dtype).eps / 2
    if dtype == F32:
        tol = 2 * (2 * hidden + T) * 2.0 ** -24
    for k, v in s.reference().items():
        got = s.out[k].double()
        assert got.isfinite().all(), k
        if ckpt and k.startswith("d") and k not in ("dnext", "dpost", "dz"):
            limit = tol + 2 * 2 * 2.0 ** -7 * 3.5 / 3 ** 0.5
        else:
            limit = tol
        off = float((got - v.detach()).norm() / v.detach().norm())
        assert off <= limit, (k, off, limit)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_serving_step_row_by_row(dtype):
    """A token's forward alone is its row of a batch's, but for the order of sums."""
    T, d, hidden = 40, 128, 232
    s = Sublayer(T, d, hidden, dtype, False)
    s.forward()
    batch = {k: s.out[k].double().clone() for k in ("n0", "y", "b")}
    one = Sublayer(1, d, hidden, dtype, False)
    one.w, one.wd, one.gains = s.w, s.wd, s.gains
    # Two orders of a sum of k terms differ by at most 2 (k + 8) 2^-23 of the sum of
    # magnitudes (the tensor cores truncate).  So g and u by e below, y = f(g) u by
    # e (1.1 |u| + |f|) (|f'| <= 1.1) and its rounding, up to two half steps; b by
    # that of its own sum, by the sum of y's differences, and its rounding.
    eps = torch.finfo(dtype).eps
    w, wd = s.w.double().abs(), s.wd.double().abs()
    for t in (0, 17, 39):
        one.x = s.x[t:t + 1]
        one.forward()
        n0, y, b = (batch[k][t] for k in ("n0", "y", "b"))
        assert torch.equal(one.out["n0"][0].double(), n0)
        e = 2 * (d + 8) * 2.0 ** -23 * (n0.abs() @ w)
        g, u = (n0 @ s.w.double()).split(hidden)
        ey = e[:hidden] * (1.1 * u.abs()) + e[hidden:] * g.abs() + eps * y.abs() + 1e-6 * eps
        near(one.out["y"][0], y, ey, "y")
        eb = 2 * (hidden + 8) * 2.0 ** -23 * (y.abs() @ wd) + ey @ wd + eps * b.abs()
        near(one.out["b"][0], b, eb, "b")


@pytest.mark.parametrize("dtype,ckpt", [(BF16, True), (F16, False), (F32, True)])
@pytest.mark.parametrize("T", [1, 300])
def test_captured_step_draws_new_masks(T, dtype, ckpt):
    """A captured step, replayed: the bits of the same calls made one by one, at
    every step of the generator, which the graph itself counts."""
    s = Sublayer(T, 128, 328, dtype, ckpt)
    one = torch.tensor([0, 1], dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.forward()
        s.backward()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.rng.add_(one)
        s.forward()
        s.backward()
    seen = []
    for step in range(6, 9):
        s.rng[1] = step - 1
        for t in s.out.values():
            t.fill_(math.nan)
        s.ws.fill_(255)
        graph.replay()
        got = {k: t.clone() for k, t in s.out.items()}
        assert s.rng.tolist()[1] == step
        s.forward()
        s.backward()
        torch.cuda.synchronize()
        for k, t in s.out.items():
            assert torch.equal(got[k], t), (k, step)
        seen.append(got["h"])
    assert T == 1 or not torch.equal(seen[0], seen[1])


def test_two_streams_and_host_threads_at_once():
    """Steps that overlap on streams of their own, from host threads of their own."""
    make = lambda i: Sublayer(500 + i, 256, 488, (BF16, F16, F32, BF16)[i], i % 2 == 0,  # noqa: E731
                              seed=i)
    alone = [make(i) for i in range(4)]
    for s in alone:
        s.forward()
        s.backward()
    both = [make(i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    wrong = []

    def work(s, stream):
        try:
            for _ in range(5):
                s.forward(stream=stream)
                s.backward(stream=stream)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(both, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong
    for a, b in zip(alone, both):
        for k in a.out:
            assert torch.equal(a.out[k], b.out[k]), k


def test_rows_far_apart():
    """Rows whose element offsets pass 2^31: the last rows' values are those of a
    call on these rows alone."""
    T, d, ld = 70_000, 64, 40_000
    base = torch.empty(T, ld, dtype=BF16, device="cuda")
    qb = torch.empty(T, ld, dtype=torch.int8, device="cuda")
    col = lambda i: base[:, 128 * i:128 * i + d]  # noqa: E731
    for i in range(5):
        col(i).copy_(rnd(200 + i, T, d, BF16))
    x, b, z, dn, dh = (col(i) for i in range(5))
    o = [col(i) for i in range(5, 10)]
    last = slice(T - 300, T)
    end = lambda t: t[last].clone(memory_format=torch.contiguous_format)  # noqa: E731
    new = lambda: torch.empty(300, d, dtype=BF16, device="cuda")  # noqa: E731
    g = vec(210, d, 1.0)
    kw = dict(post_norm=True, post_gain=g, gate_act=M.MLP_GATE_SIGMOID, scale=0.5)
    M.mlp_resnorm_fwd(x, n=o[1], next_gain=g, b=b, h=o[0], gate=z, **kw)
    h, n = new(), new()
    M.mlp_resnorm_fwd(end(x), n=n, next_gain=g, b=end(b), h=h, gate=end(z), **kw)
    assert torch.equal(o[0][last], h) and torch.equal(o[1][last], n)
    rs = torch.ones(T, device="cuda")
    M.mlp_resnorm_bwd(o[2], dh=dh, dn=dn, h=x, h_rstd=rs, next_gain=g, b=b, db=o[3], b_rstd=rs,
                      gate=z, dgate=o[4], **kw)
    e = [new() for _ in range(3)]
    M.mlp_resnorm_bwd(e[0], dh=end(dh), dn=end(dn), h=end(x), h_rstd=rs[:300], next_gain=g,
                      b=end(b), db=e[1], b_rstd=rs[:300], gate=end(z), dgate=e[2], **kw)
    assert all(torch.equal(a[last], c) for a, c in zip(o[2:], e))
    # the gated unit, its 8-bit values and its gradients
    w = rnd(211, d, 2 * d, BF16, 0.125)
    cg, cu = ((qb[:, 128 * i:128 * i + d], torch.empty(T, 2, dtype=torch.uint8, device="cuda"))
              for i in range(2))
    M.mlp_glu_fwd(x, w[:, :d], w[:, d:], o[0], g=o[1], u=o[2])
    M.mlp_glu_fwd(x, w[:, :d], w[:, d:], o[0], g_ckpt=cg, u_ckpt=cu)
    e = [new() for _ in range(3)]
    ws = bytes_for(max(M.mlp_glu_workspace_bytes(300, d, d, BF16),
                       M.mlp_glu_bwd_workspace_bytes(300, d, d, BF16)))
    M.mlp_glu_fwd(end(x), w[:, :d], w[:, d:], e[0], g=e[1], u=e[2], workspace=ws)
    for a, c in zip(o, e):
        # 64 terms in another kernel's order, then one rounding each
        near(a[last], c, 2 * rounding(BF16, c.double()) + 64 * 2.0 ** -22, "glu")
    dgu = [col(i) for i in range(10, 13)]
    for saved, saved_end in ((dict(g=o[1], u=o[2]), dict(g=end(o[1]), u=end(o[2]))),
                             (dict(g_ckpt=cg, u_ckpt=cu),
                              dict(g_ckpt=tuple(map(end, cg)), u_ckpt=tuple(map(end, cu))))):
        M.mlp_glu_bwd(dn, w[:, d:], *dgu[:2], a=dgu[2], **saved)
        M.mlp_glu_bwd(end(dn), w[:, d:], *e[:2], a=e[2], workspace=ws, **saved_end)
        for a, c in zip(dgu, e):
            near(a[last], c, 2 * rounding(BF16, c.double()) + 64 * 2.0 ** -22, "glu backward")
    del base, qb


def test_more_than_2_31_values():
    T, k, n = 1_600_000, 16, 1_376
    x, w = rnd(220, T, k, BF16), rnd(221, k, 2 * n, BF16, 0.25)
    y = torch.empty(T, n, dtype=BF16, device="cuda")
    M.mlp_glu_fwd(x, w[:, :n], w[:, n:], y)
    g, u = (x[-500:].double() @ w.double()).split(n, 1)
    ref = g * torch.sigmoid(g) * u
    near(y[-500:], ref, rounding(BF16, ref) + 1e-5 * (1 + ref.abs()), "y")
    dy, wd = x, w[:, :n].t().contiguous()
    dg, du = torch.empty_like(y), torch.empty_like(y)
    M.mlp_glu_bwd(dy, wd, dg, du, act=M.MLP_ACT_NONE, g=y, u=y)
    da = dy[-500:].double() @ wd.double().t()
    ref = da * y[-500:].double()
    for got in (dg, du):
        near(got[-500:], ref, rounding(BF16, ref) + 1e-5 * (1 + ref.abs()), "dg")
