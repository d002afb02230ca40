"""Workloads of the gated feed-forward sublayer's operators: the gated linear
unit (both projections, activation and product, and the backward through all
of them), the residual norm (norms before and after a block with its gate,
residual scale and dropout, and its backward) and dropout from a counter-based
generator.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``run()`` makes one pass: with ``own`` false in elementary torch operations in
32 bits, with ``own`` true through ``mlp_step_gb300``.  ``exact()`` computes
the same outputs from the definitions in 64 bits.

Matrices of 16-bit values have their row pitch rounded up to 8 elements (whole
16-byte rows, as the library's tensor-core path asks), so a width may be odd.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ESZ = {"bf16": 2, "f16": 2, "f32": 4}
_SLOPE = 0.5
_EPS = 1e-6
_ACTS = ("none", "relu", "leaky_relu_sq", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # serving one token of the 512-wide model: latency
        {"name": "glu_token", "op": "glu_fwd", "T": 1, "k": 512, "n": 1408, "dtype": "bf16",
         "act": "silu", "bias": False, "save": "none"},
        # one token of an 8,192-wide model: both weights are read once
        {"name": "glu_token_wide", "op": "glu_fwd", "T": 1, "k": 8192, "n": 8192,
         "dtype": "bf16", "act": "silu", "bias": False, "save": "none"},
        # training the 512-wide block over 65,536 tokens, pre-activations kept in 8 bits
        {"name": "glu_train_ckpt8", "op": "glu_fwd", "T": 65536, "k": 512, "n": 1408,
         "dtype": "bf16", "act": "silu", "bias": False, "save": "ckpt"},
        # a wide gated layer, fp16, biases, pre-activations kept as they are
        {"name": "glu_wide", "op": "glu_fwd", "T": 4096, "k": 8192, "n": 8192, "dtype": "f16",
         "act": "gelu_tanh", "bias": True, "save": "same"},
        # the gradient through the down projection and the gated unit, from 8-bit
        # pre-activations, with both bias gradients and the activations again
        {"name": "glu_bwd_ckpt8", "op": "glu_bwd", "T": 65536, "k": 512, "n": 1408,
         "dtype": "bf16", "act": "silu", "bias": True, "saved": "ckpt", "again": True},
        # a ragged fp32 batch of the small network's widths
        {"name": "glu_bwd_f32", "op": "glu_bwd", "T": 1003, "k": 784, "n": 1001,
         "dtype": "f32", "act": "gelu", "bias": True, "saved": "same", "again": False},
        # serving one token: norm of the block's output, residual, norm of the next block
        {"name": "resnorm_token", "op": "rn_fwd", "T": 1, "d": 512, "dtype": "bf16",
         "block": True, "post": True, "gate": "none", "next": True, "p": 0.0},
        # between two blocks in training: norm, gate from a projection, dropout,
        # scaled residual, norm of the next block
        {"name": "resnorm_train", "op": "rn_fwd", "T": 65536, "d": 512, "dtype": "bf16",
         "block": True, "post": True, "gate": "sigmoid", "next": True, "p": 0.1},
        # its gradients
        {"name": "resnorm_train_bwd", "op": "rn_bwd", "T": 65536, "d": 512, "dtype": "bf16",
         "block": True, "post": True, "gate": "sigmoid", "next": True, "p": 0.1},
        # gradients in the 8,192-wide network, no gate and no dropout
        {"name": "resnorm_wide_bwd", "op": "rn_bwd", "T": 16384, "d": 8192, "dtype": "f16",
         "block": True, "post": True, "gate": "none", "next": True, "p": 0.0},
        # dropout of a sublayer's output and the residual sum over 262,144 tokens
        {"name": "dropout_stack", "op": "drop", "T": 262144, "d": 512, "dtype": "bf16",
         "p": 0.1, "residual": True},
        # a ragged fp32 matrix
        {"name": "dropout_f32", "op": "drop", "T": 10007, "d": 1001, "dtype": "f32", "p": 0.25,
         "residual": False},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glu_fwd", "glu_fwd", "glu_fwd", "glu_bwd", "glu_bwd", "rn_fwd", "rn_fwd",
                     "rn_bwd", "rn_bwd", "drop"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    c = {"op": op, "dtype": dtype}
    if op in ("rn_fwd", "rn_bwd", "drop"):
        d = _spread(rng, 8, 16384)
        c.update({"T": min(_spread(rng, 1, 262144), (1 << 25) // d + 1), "d": d,
                  "p": rng.choice([0.0, 0.1, 0.5])})
        if op == "drop":
            c.update({"p": rng.choice([0.1, 0.25, 0.5]), "residual": rng.random() < 0.5})
            return c
        c.update({"block": rng.random() < 0.8, "post": False, "gate": "none", "next": True})
        if c["block"]:
            c.update({"post": rng.random() < 0.6, "next": rng.random() < 0.8,
                      "gate": rng.choice(["none", "plain", "sigmoid"])})
        else:
            c["p"] = 0.0
        return c
    k, n = _spread(rng, 8, 8192), _spread(rng, 8, 8192)
    most = 2 ** (35 if dtype == "f32" else 37)  # multiply-adds: fp32 has no tensor cores
    T = min(_spread(rng, 1, 65536), (1 << 25) // max(k, n) + 1, most // (k * n) + 1)
    c.update({"T": T, "k": k, "n": n, "act": rng.choice(_ACTS), "bias": rng.random() < 0.5})
    if op == "glu_fwd":
        c["save"] = rng.choice(["none", "same", "ckpt"])
    else:
        c.update({"saved": rng.choice(["same", "ckpt"]), "again": rng.random() < 0.5})
    return c


# ------------------------------------------------------------------ inputs

def _rows(rows, cols, dtype):
    """An uninitialised matrix whose 16-bit rows start on 16 bytes."""
    pitch = cols if dtype == torch.float32 else (cols + 7) // 8 * 8
    return torch.empty(rows, pitch, dtype=dtype, device="cuda")[:, :cols]


def _randn(g, rows, cols, dtype, std=1.0, shift=None, scale=None):
    out = _rows(rows, cols, dtype)
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        v = torch.randn(min(step, rows - r), cols, generator=g, device="cuda")
        v *= std
        if scale is not None:
            v *= scale
        if shift is not None:
            v += shift
        out[r:r + step] = v
    return out


def _stream_rows(g, rows, cols, dtype):
    """Rows of a residual stream: a shift and a scale per channel, and a few
    channels an order of magnitude larger than the rest."""
    scale = 0.5 + torch.rand(cols, generator=g, device="cuda")
    scale[torch.randint(0, cols, (max(1, cols // 128),), generator=g, device="cuda")] *= 12.0
    shift = 0.2 * torch.randn(cols, generator=g, device="cuda")
    return _randn(g, rows, cols, dtype, shift=shift, scale=scale)


def _vec(g, n, mean=0.0, std=0.1):
    return mean + std * torch.randn(n, generator=g, device="cuda")


def _ckpt_buffers(T, d):
    return (torch.empty(T, d, dtype=torch.int8, device="cuda"),
            torch.empty(T, (d + 31) // 32, dtype=torch.uint8, device="cuda"))


def _rng(seed, p):
    """The generator's state, on the device: seed and step."""
    return torch.tensor([(seed + 1) * 0x9E3779B97F4A7C15 % (1 << 63), seed % 1000],
                        dtype=torch.int64, device="cuda") if p > 0 else None


def _rstd_of(x):
    return torch.rsqrt(x.float().square().mean(1) + _EPS)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _DT[case["dtype"]]
    op, T = case["op"], case["T"]
    s = {"case": case, "dt": dt}
    f32 = dict(dtype=torch.float32, device="cuda")
    if op == "glu_fwd":
        k, n = case["k"], case["n"]
        s.update(x=_randn(g, T, k, dt), wg=_randn(g, k, n, dt, k ** -0.5),
                 wu=_randn(g, k, n, dt, k ** -0.5),
                 bg=_vec(g, n) if case["bias"] else None, bu=_vec(g, n) if case["bias"] else None,
                 y=_rows(T, n, dt))
        same, ck = case["save"] == "same", case["save"] == "ckpt"
        s.update({m: _rows(T, n, dt) if same else None for m in ("g", "u")})
        s.update({m: _ckpt_buffers(T, n) if ck else None for m in ("gq", "uq")})
    elif op == "glu_bwd":
        k, n = case["k"], case["n"]
        s.update(dy=_randn(g, T, k, dt, 0.1), w=_randn(g, n, k, dt, n ** -0.5), g=None, u=None,
                 gq=None, uq=None, dg=_rows(T, n, dt), du=_rows(T, n, dt),
                 dbg=torch.empty(n, **f32) if case["bias"] else None,
                 dbu=torch.empty(n, **f32) if case["bias"] else None,
                 a=_rows(T, n, dt) if case["again"] else None)
        for m in ("g", "u"):
            v = _randn(g, T, n, dt, 1.5)
            if case["saved"] == "ckpt":
                s[m + "q"] = _quantise(v)
            else:
                s[m] = v
    elif op in ("rn_fwd", "rn_bwd"):
        d, gate = case["d"], case["gate"] != "none"
        s.update(b=_stream_rows(g, T, d, dt) if case["block"] else None,
                 z=_randn(g, T, d, dt) if gate else None, scale=0.5,
                 post_gain=_vec(g, d, 1.0) if case["post"] else None,
                 next_gain=_vec(g, d, 1.0) if case["next"] else None,
                 rng=_rng(seed, case["p"]))
        if op == "rn_fwd":
            s.update(x=_stream_rows(g, T, d, dt), h=_rows(T, d, dt) if case["block"] else None,
                     n=_rows(T, d, dt) if case["next"] else None,
                     b_rstd=torch.empty(T, **f32) if case["post"] else None,
                     h_rstd=torch.empty(T, **f32) if case["next"] else None)
        else:
            h = _stream_rows(g, T, d, dt)
            s.update(h=h if case["next"] else None,
                     dn=_randn(g, T, d, dt, 0.1) if case["next"] else None,
                     dh=_randn(g, T, d, dt, 0.1), dx=_rows(T, d, dt),
                     h_rstd=_rstd_of(h) if case["next"] else None,
                     b_rstd=_rstd_of(s["b"]) if case["post"] else None,
                     db=_rows(T, d, dt) if case["block"] else None,
                     dz=_rows(T, d, dt) if gate else None,
                     dpost=torch.empty(d, **f32) if case["post"] else None,
                     dnext=torch.empty(d, **f32) if case["next"] else None)
    else:
        d = case["d"]
        s.update(x=_stream_rows(g, T, d, dt), y=_rows(T, d, dt), rng=_rng(seed, 1),
                 res=_stream_rows(g, T, d, dt) if case["residual"] else None)
    if own:
        import mlp_step_gb300 as M
        need = {"glu_fwd": lambda: M.mlp_glu_workspace_bytes(T, case["k"], case["n"], dt),
                "glu_bwd": lambda: M.mlp_glu_bwd_workspace_bytes(T, case["n"], case["k"], dt),
                "rn_bwd": lambda: M.mlp_resnorm_workspace_bytes(T, case["d"])}
        s["ws"] = torch.empty(need[op]() if op in need else 0, dtype=torch.uint8, device="cuda")
        s["act"] = {"none": M.MLP_ACT_NONE, "relu": M.MLP_ACT_RELU,
                    "leaky_relu_sq": M.MLP_ACT_LEAKY_RELU_SQ, "gelu": M.MLP_ACT_GELU,
                    "gelu_tanh": M.MLP_ACT_GELU_TANH,
                    "silu": M.MLP_ACT_SILU}[case.get("act", "none")]
        s["gate_act"] = M.MLP_GATE_SIGMOID if case.get("gate") == "sigmoid" else M.MLP_GATE_PLAIN
    return s


# ------------------------------------------------------------------ plain forms

def _power(e):
    """2^e as float32 for whole e in [-126, 127], by its bits."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(x):
    """(int8 values, scale bytes) of x, 32 values of a row to a scale: the
    exponent of the group's largest magnitude, 255 where a value is not finite."""
    T, d = x.shape
    g = (d + 31) // 32
    v = torch.zeros(T, g * 32, dtype=torch.float32, device=x.device)
    v[:, :d] = x
    v = v.view(T, g, 32)
    top = (v.abs().amax(2).view(torch.int32) >> 23).clamp(min=7)  # NaN passes through amax
    q = torch.round(v * _power(133 - top.clamp(max=254))[:, :, None]).clamp(-127, 127)
    q = torch.where((top == 255)[:, :, None], torch.zeros_like(q), q)
    return q.to(torch.int8).view(T, g * 32)[:, :d].contiguous(), top.to(torch.uint8)


def _values(ckpt):
    """The float32 values that an 8-bit checkpoint stands for."""
    q, b = ckpt
    T, d = q.shape
    e = b.to(torch.int32)
    step = torch.where(e == 255, torch.full_like(_power(e * 0), float("nan")),
                       _power(e.clamp(7, 254) - 133))
    return q.to(torch.float32) * step.repeat_interleave(32, dim=1)[:, :d]


def _act(u, act):
    if act == "none":
        return u
    if act == "relu":
        return torch.where(u > 0, u, torch.zeros_like(u))
    if act == "leaky_relu_sq":
        return torch.where(u > 0, u, _SLOPE * u) ** 2
    if act == "gelu":
        return 0.5 * u * torch.special.erfc(-u * math.sqrt(0.5))
    if act == "gelu_tanh":
        return u / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
    return u / (1 + torch.exp(-u))


def _act_grad(u, act):
    if act == "none":
        return torch.ones_like(u)
    if act == "relu":
        return (u > 0).to(u.dtype)
    if act == "leaky_relu_sq":
        return 2 * torch.where(u > 0, u, _SLOPE * _SLOPE * u)
    if act == "gelu":
        return (0.5 * torch.special.erfc(-u * math.sqrt(0.5)) +
                u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-c * (u + 0.044715 * u ** 3)))
        return s + u * s * (1 - s) * c * (1 + 3 * 0.044715 * u * u)
    s = 1 / (1 + torch.exp(-u))
    return s + u * s * (1 - s)


_LOW = 0xFFFFFFFF


def _random16(rng, site, T, d):
    """[T, d] random whole numbers in [0, 2^16): Philox4x32-10 (Salmon, Moraes,
    Dror and Shaw 2011) of the counter (column / 8, row, site, step) under the
    key `seed`; its four words are eight numbers, low halves first."""
    dev = rng.device
    c0 = torch.arange((d + 7) // 8, device=dev).expand(T, -1)
    c1 = torch.arange(T, device=dev)[:, None].expand_as(c0)
    c2, c3 = torch.full_like(c0, site), (rng[1] & _LOW).expand_as(c0)
    k0, k1 = rng[0] & _LOW, (rng[0] >> 32) & _LOW
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64 bits, wrapping
        c0, c1, c2, c3 = (((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW,
                          ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW)
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    w = torch.stack((c0, c1, c2, c3), dim=2)
    return torch.stack((w & 0xFFFF, w >> 16), dim=3).reshape(T, -1)[:, :d]


def _threshold(p):
    """p in steps of 2^-16: a value whose random number is below it is dropped."""
    return math.floor(p * 65536 + 0.5)


def _dropped(x, case, rng):
    if case["p"] == 0:
        return x
    t = _threshold(case["p"])
    keep = _random16(rng, _SITE, *x.shape) >= t
    return torch.where(keep, x * (65536 / (65536 - t)), torch.zeros_like(x))


_SITE = 3  # which of a model's dropout places this one is


def _run_plain(s):
    case, dt = s["case"], s["dt"]
    op = case["op"]
    if op == "glu_fwd":
        x = s["x"].float()
        g, u = x @ s["wg"].float(), x @ s["wu"].float()
        if case["bias"]:
            g, u = g + s["bg"], u + s["bu"]
        out = {"y": (_act(g, case["act"]) * u).to(dt)}
        if case["save"] == "same":
            out.update(g=g.to(dt), u=u.to(dt))
        elif case["save"] == "ckpt":
            out.update(g=_values(_quantise(g)).to(torch.bfloat16),
                       u=_values(_quantise(u)).to(torch.bfloat16))
        return out
    if op == "glu_bwd":
        da = s["dy"].float() @ s["w"].float().t()
        ck = case["saved"] == "ckpt"
        g, u = [_values(s[m + "q"]) if ck else s[m].float() for m in ("g", "u")]
        f = _act(g, case["act"])
        dg, du = da * u * _act_grad(g, case["act"]), da * f
        out = {"dg": dg.to(dt), "du": du.to(dt)}
        if case["bias"]:
            out.update(dbg=dg.sum(0), dbu=du.sum(0))
        if case["again"]:
            out["a"] = (f * u).to(dt)
        return out
    if op == "rn_fwd":
        h = s["x"].float()
        out = {}
        if case["block"]:
            c = s["b"].float()
            if case["post"]:
                out["b_rstd"] = torch.rsqrt((c * c).mean(1) + _EPS)
                c = c * out["b_rstd"][:, None] * s["post_gain"]
            c = _dropped(c, case, s["rng"])
            if case["gate"] != "none":
                z = s["z"].float()
                c = c * (1 / (1 + torch.exp(-z)) if case["gate"] == "sigmoid" else z)
            h = h + s["scale"] * c
            out["h"] = h.to(dt)
        if case["next"]:
            out["h_rstd"] = torch.rsqrt((h * h).mean(1) + _EPS)
            out["n"] = (h * out["h_rstd"][:, None] * s["next_gain"]).to(dt)
        return out
    if op == "rn_bwd":
        dh = s["dh"].float()
        out = {}
        if case["next"]:
            nh, dn = s["h"].float() * s["h_rstd"][:, None], s["dn"].float()
            t = dn * s["next_gain"]
            dh = dh + s["h_rstd"][:, None] * (t - nh * (t * nh).mean(1)[:, None])
            out["dnext"] = (dn * nh).sum(0)
        out["dx"] = dh.to(dt)
        if case["block"]:
            v = s["b"].float()
            if case["post"]:
                v = v * s["b_rstd"][:, None]
            c = v * s["post_gain"] if case["post"] else v
            dc = s["scale"] * dh
            if case["gate"] != "none":
                z = s["z"].float()
                sg = 1 / (1 + torch.exp(-z)) if case["gate"] == "sigmoid" else z
                dz = dc * _dropped(c, case, s["rng"])
                out["dz"] = (dz * sg * (1 - sg) if case["gate"] == "sigmoid" else dz).to(dt)
                dc = dc * sg
            dc = _dropped(dc, case, s["rng"])
            if case["post"]:
                out["dpost"] = (dc * v).sum(0)
                dc = dc * s["post_gain"]
                dc = s["b_rstd"][:, None] * (dc - v * (dc * v).mean(1)[:, None])
            out["db"] = dc.to(dt)
        return out
    y = _dropped(s["x"].float(), case, s["rng"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(dt)}


# ------------------------------------------------------------------ the library

def _run_own(s):
    import mlp_step_gb300 as M
    case = s["case"]
    op = case["op"]
    if op == "glu_fwd":
        M.mlp_glu_fwd(s["x"], s["wg"], s["wu"], s["y"], b_gate=s["bg"], b_up=s["bu"],
                      act=s["act"], slope=_SLOPE, g=s["g"], u=s["u"], g_ckpt=s["gq"],
                      u_ckpt=s["uq"], workspace=s["ws"])
        out = {"y": s["y"]}
        if case["save"] == "same":
            out.update(g=s["g"], u=s["u"])
        elif case["save"] == "ckpt":
            for m in ("g", "u"):
                out[m] = torch.empty(case["T"], case["n"], dtype=torch.bfloat16, device="cuda")
                M.mlp_ckpt8_decode(*s[m + "q"], out[m])
        return out
    if op == "glu_bwd":
        M.mlp_glu_bwd(s["dy"], s["w"], s["dg"], s["du"], act=s["act"], slope=_SLOPE, g=s["g"],
                      u=s["u"], g_ckpt=s["gq"], u_ckpt=s["uq"], db_gate=s["dbg"],
                      db_up=s["dbu"], a=s["a"], workspace=s["ws"])
        return {m: s[m] for m in ("dg", "du", "dbg", "dbu", "a") if s[m] is not None}
    if op == "rn_fwd":
        M.mlp_resnorm_fwd(s["x"], b=s["b"], h=s["h"], n=s["n"], post_norm=case["post"],
                          post_gain=s["post_gain"], b_rstd=s["b_rstd"], gate=s["z"],
                          gate_act=s["gate_act"], scale=s["scale"], p=case["p"], rng=s["rng"],
                          site=_SITE, next_gain=s["next_gain"], h_rstd=s["h_rstd"], eps=_EPS)
        return {m: s[m] for m in ("b_rstd", "h", "h_rstd", "n") if s[m] is not None}
    if op == "rn_bwd":
        M.mlp_resnorm_bwd(s["dx"], dh=s["dh"], dn=s["dn"], h=s["h"], h_rstd=s["h_rstd"],
                          next_gain=s["next_gain"], b=s["b"], db=s["db"],
                          post_norm=case["post"], post_gain=s["post_gain"], b_rstd=s["b_rstd"],
                          gate=s["z"], dgate=s["dz"], gate_act=s["gate_act"], scale=s["scale"],
                          p=case["p"], rng=s["rng"], site=_SITE, dpost_gain=s["dpost"],
                          dnext_gain=s["dnext"], workspace=s["ws"])
        return {m: s[m] for m in ("dnext", "dx", "dz", "dpost", "db") if s[m] is not None}
    M.mlp_dropout(s["x"], s["y"], case["p"], s["rng"], site=_SITE, residual=s["res"])
    return {"y": s["y"]}


def run(state):
    out = _run_own(state) if own else _run_plain(state)
    return {k: out[k] for k in sorted(out)}


def work(case):
    op, T, e = case["op"], case["T"], _ESZ[case["dtype"]]
    if op in ("glu_fwd", "glu_bwd"):
        k, n = case["k"], case["n"]
        m = T * n
        if op == "glu_fwd":
            b = e * (T * k + 2 * k * n + m) + (8 * n if case["bias"] else 0)
            b += 2 * e * m if case["save"] == "same" else 0
            # written once, then read back and expanded
            b += 2 * (2 * (1 + 1 / 32) + 2) * m if case["save"] == "ckpt" else 0
            return {"bytes": b, "flops": 4 * T * k * n}
        b = e * (T * k + k * n + 2 * m) + (8 * n if case["bias"] else 0)
        b += 2 * ((1 + 1 / 32) if case["saved"] == "ckpt" else e) * m
        b += e * m if case["again"] else 0
        return {"bytes": b, "flops": 2 * T * k * n}
    m = T * case["d"]
    if op == "drop":
        return {"bytes": e * m * (3 if case["residual"] else 2), "flops": 2 * m}
    mats = (3 if case["block"] else 1) + (case["gate"] != "none") + case["next"]
    rows = case["post"] + case["next"]
    if op == "rn_bwd":
        # dh, dx; b, db; z, dz; dn, h
        mats = 2 + 2 * (case["block"] + (case["gate"] != "none") + case["next"])
    return {"bytes": e * m * mats + 4 * rows * (T + case["d"] * (2 if op == "rn_bwd" else 1)),
            "flops": 10 * m}


# ------------------------------------------------------------------ 64 bits

def _two_to(e):
    """2^e in float64, from the bits of the number (a library power may be an ulp off,
    which would move values halfway between two steps)."""
    return (e.to(torch.int64) + 1023).bitwise_left_shift(52).view(torch.float64)


def _exact_ckpt(x):
    """What the 8-bit form of x stands for, group by group: a step of
    2^(floor(log2 largest) - 6), halves to even, at most 127 steps."""
    T, d = x.shape
    g = -(-d // 32)
    v = torch.nn.functional.pad(x.double(), (0, g * 32 - d)).reshape(T, g, 32)
    big = v.abs().max(dim=2, keepdim=True).values
    _, e = torch.frexp(big)  # big = m 2^e, m in [1/2, 1)
    e = torch.where(big == 0, torch.full_like(e, -120), e - 1).clamp(min=-120)
    step = _two_to(e - 6)
    q = torch.round(v / step)
    return (torch.clamp(q, -127, 127) * step).reshape(T, g * 32)[:, :d]


def _exact_act(u, act):
    """(f(u), f'(u))"""
    one = torch.ones_like(u)
    if act == "none":
        return u, one
    if act == "relu":
        return u.clamp(min=0), (u > 0).double()
    if act == "leaky_relu_sq":
        t = torch.where(u > 0, one, _SLOPE * one)
        return (t * u) ** 2, 2 * t * t * u
    if act == "gelu":
        cdf = (1 + torch.erf(u / 2 ** 0.5)) / 2
        return u * cdf, cdf + u * torch.exp(-u * u / 2) / (2 * math.pi) ** 0.5
    if act == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (u + 0.044715 * u * u * u))
        return u * (1 + t) / 2, (1 + t) / 2 + u * (1 - t * t) / 2 * c * (1 + 0.134145 * u * u)
    s = torch.sigmoid(u)
    return u * s, s * (1 + u * (1 - s))


def _exact_factor(case, rng):
    """[T, d] factors 0 or 1 / (1 - p) of dropout, the generator in numpy's
    unsigned 64-bit arithmetic, a stretch of rows at a time."""
    T, d = case["T"], case["d"]
    t = int(np.floor(np.float64(case["p"]) * 65536 + 0.5))
    seed, step = [int(v) for v in rng.cpu().tolist()]
    seed &= (1 << 64) - 1
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    groups = (d + 7) // 8
    out = torch.empty(T, d, dtype=torch.bool, device="cuda")
    rows = max(1, (1 << 20) // groups)
    for r in range(0, T, rows):
        m = min(rows, T - r)
        x = [np.tile(np.arange(groups, dtype=np.uint64), m),
             np.repeat(np.arange(r, r + m, dtype=np.uint64), groups),
             np.full(m * groups, _SITE, np.uint64),
             np.full(m * groups, step & 0xFFFFFFFF, np.uint64)]
        for i in range(10):
            key = [np.uint64(((seed & 0xFFFFFFFF) + i * 0x9E3779B9) & 0xFFFFFFFF),
                   np.uint64(((seed >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)]
            p0, p1 = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
            x = [(p1 >> half) ^ x[1] ^ key[0], p1 & low, (p0 >> half) ^ x[3] ^ key[1], p0 & low]
        n = np.stack([x[i // 2] >> np.uint64(16 * (i % 2)) & np.uint64(0xFFFF)
                      for i in range(8)], axis=1).reshape(m, groups * 8)[:, :d]
        out[r:r + m] = torch.from_numpy(n >= t).to("cuda")
    return out.double() / (1 - t / 65536)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    out = {}
    if op == "glu_fwd":
        x = s["x"].double()
        g, u = torch.matmul(x, s["wg"].double()), torch.matmul(x, s["wu"].double())
        if case["bias"]:
            g += s["bg"].double()
            u += s["bu"].double()
        out["y"] = _exact_act(g, case["act"])[0].mul_(u)
        if case["save"] != "none":
            out["g"], out["u"] = (g, u) if case["save"] == "same" else map(_exact_ckpt, (g, u))
    elif op == "glu_bwd":
        da = torch.matmul(s["dy"].double(), s["w"].double().t())
        gu = []
        for m in ("g", "u"):
            if case["saved"] == "ckpt":
                q, b = s[m + "q"]
                step = _two_to(b.to(torch.int32) - 133).repeat_interleave(32, dim=1)
                gu.append(q.double() * step[:, :case["n"]])
            else:
                gu.append(s[m].double())
        f, df = _exact_act(gu[0], case["act"])
        out["dg"], out["du"] = da * df * gu[1], da * f
        if case["bias"]:
            out["dbg"], out["dbu"] = out["dg"].sum(0), out["du"].sum(0)
        if case["again"]:
            out["a"] = f * gu[1]
    elif op == "drop":
        out["y"] = s["x"].double() * _exact_factor(case, s["rng"])
        if case["residual"]:
            out["y"] += s["res"].double()
    else:
        d = case["d"]
        rms = lambda v: 1 / torch.sqrt((v ** 2).sum(1, keepdim=True) / d + _EPS)  # noqa: E731
        factor = s["scale"] * (_exact_factor(case, s["rng"]) if case["p"] else 1.0)
        gate, dgate = 1.0, None
        if case["gate"] != "none":
            gate = s["z"].double()
            dgate = torch.ones_like(gate)
            if case["gate"] == "sigmoid":
                gate = torch.sigmoid(gate)
                dgate = gate * (1 - gate)
        if op == "rn_fwd":
            h = s["x"].double()
            if case["block"]:
                c = s["b"].double()
                if case["post"]:
                    r = rms(c)
                    out["b_rstd"] = r[:, 0]
                    c = c * r * s["post_gain"].double()
                h = h + c * factor * gate
                out["h"] = h
            if case["next"]:
                r = rms(h)
                out["h_rstd"] = r[:, 0]
                out["n"] = h * r * s["next_gain"].double()
        else:
            dh = s["dh"].double()
            if case["next"]:
                r = s["h_rstd"].double()[:, None]
                unit = s["h"].double() * r
                pull = s["dn"].double() * s["next_gain"].double()
                dh = dh + r * (pull - unit * (pull * unit).sum(1, keepdim=True) / d)
                out["dnext"] = (s["dn"].double() * unit).sum(0)
            out["dx"] = dh
            if case["block"]:
                c = s["b"].double()
                if case["post"]:
                    r, w = s["b_rstd"].double()[:, None], s["post_gain"].double()
                    c = c * r
                    pull = dh * factor * gate
                    out["dpost"] = (pull * c).sum(0)
                    pull = pull * w
                    out["db"] = r * (pull - c * (pull * c).sum(1, keepdim=True) / d)
                    c = c * w
                else:
                    out["db"] = dh * factor * gate
                if dgate is not None:
                    out["dz"] = dh * factor * c * dgate
    return {k: out[k] for k in sorted(out)}
