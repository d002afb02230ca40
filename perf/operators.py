"""Workloads of the feed-forward operators: layer norm (forward, backward with
the parameter gradients), the linear layer with bias, activation and residual
in its epilogue (and the backward through the activation), and 8-bit
activation checkpoints.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``run()`` makes one pass: with ``own`` false in elementary torch operations in
32 bits, with ``own`` true through ``mlp_step_gb300``.  ``exact()`` computes
the same outputs from the definitions in 64 bits.

Matrices of 16-bit values have their row pitch rounded up to 8 elements (whole
16-byte rows, as the library's tensor-core path asks), so a width may be odd.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ESZ = {"bf16": 2, "f16": 2, "f32": 4}
_SLOPE = 0.5
_EPS = 1e-5
_ACTS = ("none", "relu", "leaky_relu_sq", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # serving one token of the 512-wide model: the norm is pure latency
        {"name": "ln_token", "op": "ln_fwd", "T": 1, "d": 512, "dtype": "bf16"},
        # training the 512-wide block over 65,536 tokens, its input kept in 8 bits
        {"name": "ln_train_ckpt8", "op": "ln_train", "T": 65536, "d": 512, "dtype": "bf16",
         "ckpt": True, "dres": True},
        # the 8,192-wide network's rows, fp16, input kept as it is
        {"name": "ln_train_wide", "op": "ln_train", "T": 16384, "d": 8192, "dtype": "f16",
         "ckpt": False, "dres": False},
        # a ragged fp32 batch of the 1,000-wide head
        {"name": "ln_train_f32", "op": "ln_train", "T": 4099, "d": 1000, "dtype": "f32",
         "ckpt": False, "dres": True},
        # one token through an 8,192 x 8,192 layer: the weights are read once
        {"name": "linear_token", "op": "lin_fwd", "T": 1, "k": 8192, "n": 8192, "dtype": "bf16",
         "act": "gelu", "residual": False, "save": "none"},
        # the block's up projection in training: GELU, pre-activation kept in 8 bits
        {"name": "linear_up_ckpt8", "op": "lin_fwd", "T": 65536, "k": 512, "n": 1536,
         "dtype": "bf16", "act": "gelu", "residual": False, "save": "ckpt"},
        # the block's down projection: bias and residual
        {"name": "linear_down", "op": "lin_fwd", "T": 65536, "k": 1536, "n": 512,
         "dtype": "bf16", "act": "none", "residual": True, "save": "none"},
        # the wide network's hidden layer at its full batch, fp16, SiLU and a skip connection
        {"name": "linear_wide", "op": "lin_fwd", "T": 16384, "k": 8192, "n": 8192,
         "dtype": "f16", "act": "silu", "residual": True, "save": "none"},
        # the gradient through the down projection and the activation, from 8-bit
        # pre-activations, with the bias gradient and the activations again
        {"name": "linear_bwd_ckpt8", "op": "lin_bwd", "T": 65536, "k": 512, "n": 1536,
         "dtype": "bf16", "act": "gelu", "saved": "ckpt", "again": True},
        # the gradient through an activation alone, ragged fp32
        {"name": "act_bwd_f32", "op": "act_bwd", "T": 10007, "n": 1001, "dtype": "f32",
         "act": "gelu_tanh", "saved": "same", "again": False},
        # a block input of the 262,144-token stack into 8 bits and back
        {"name": "ckpt8_stack", "op": "ckpt8", "T": 262144, "d": 512, "dtype": "bf16"},
        # a ragged fp32 matrix into 8 bits and back
        {"name": "ckpt8_f32", "op": "ckpt8", "T": 10007, "d": 1001, "dtype": "f32"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_train", "ln_train", "lin_fwd", "lin_fwd", "lin_fwd", "lin_bwd",
                     "lin_bwd", "act_bwd", "ckpt8"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    c = {"op": op, "dtype": dtype}
    if op in ("ln_fwd", "ln_train", "act_bwd", "ckpt8"):
        d = _spread(rng, 8, 16384)
        T = min(_spread(rng, 1, 262144), (1 << 26) // d + 1)
        c["T"] = T
        c["n" if op == "act_bwd" else "d"] = d
        if op == "ln_train":
            c["ckpt"] = rng.random() < 0.5
            c["dres"] = rng.random() < 0.5
        if op == "act_bwd":
            c["act"] = rng.choice(_ACTS[1:])
            c["saved"] = rng.choice(["same", "ckpt"])
            c["again"] = rng.random() < 0.5
        return c
    k, n = _spread(rng, 8, 8192), _spread(rng, 8, 8192)
    most = 2 ** (36 if dtype == "f32" else 38)  # multiply-adds: fp32 has no tensor cores
    T = min(_spread(rng, 1, 65536), (1 << 26) // max(k, n) + 1, most // (k * n) + 1)
    c.update({"T": T, "k": k, "n": n, "act": rng.choice(_ACTS)})
    if op == "lin_fwd":
        c["residual"] = rng.random() < 0.5
        c["save"] = rng.choice(["none", "same", "ckpt"])
    else:
        c["saved"] = rng.choice(["same", "ckpt"])
        c["again"] = rng.random() < 0.5
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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _DT[case["dtype"]]
    op, T = case["op"], case["T"]
    s = {"case": case, "dt": dt}
    f32 = dict(dtype=torch.float32, device="cuda")
    if op in ("ln_fwd", "ln_train"):
        d = case["d"]
        s.update(x=_stream_rows(g, T, d, dt), gain=_vec(g, d, 1.0), shift=_vec(g, d),
                 y=_rows(T, d, dt), mean=torch.empty(T, **f32), rstd=torch.empty(T, **f32))
        if op == "ln_train":
            s.update(dy=_randn(g, T, d, dt, 0.1), dx=_rows(T, d, dt),
                     dgain=torch.empty(d, **f32), dshift=torch.empty(d, **f32),
                     dres=_randn(g, T, d, dt, 0.1) if case["dres"] else None,
                     ckpt=_ckpt_buffers(T, d) if case["ckpt"] else None)
    elif op == "lin_fwd":
        k, n = case["k"], case["n"]
        s.update(x=_randn(g, T, k, dt), w=_randn(g, k, n, dt, k ** -0.5), bias=_vec(g, n),
                 residual=_stream_rows(g, T, n, dt) if case["residual"] else None,
                 y=_rows(T, n, dt), u=_rows(T, n, dt) if case["save"] != "none" else None,
                 ckpt=_ckpt_buffers(T, n) if case["save"] == "ckpt" else None)
    elif op in ("lin_bwd", "act_bwd"):
        n = case["n"]
        if op == "lin_bwd":
            k = case["k"]
            s.update(dy=_randn(g, T, k, dt, 0.1), w=_randn(g, n, k, dt, n ** -0.5))
        else:
            s.update(dy=_randn(g, T, n, dt, 0.1))
        u = _randn(g, T, n, dt, 1.5)
        s.update(u=None, ckpt=None, du=_rows(T, n, dt), dbias=torch.empty(n, **f32),
                 a=_rows(T, n, dt) if case["again"] else None)
        if case["saved"] == "ckpt":
            s["ckpt"] = _quantise(u)
        else:
            s["u"] = u
    else:
        d = case["d"]
        s.update(x=_stream_rows(g, T, d, dt), out=_rows(T, d, dt), ckpt=_ckpt_buffers(T, d))
    if own:
        import mlp_step_gb300 as M
        need = {"ln_train": lambda: M.mlp_layernorm_workspace_bytes(T, case["d"]),
                "lin_fwd": lambda: M.mlp_linear_workspace_bytes(T, case["k"], case["n"], dt),
                "lin_bwd": lambda: M.mlp_linear_bwd_workspace_bytes(T, case["n"], case["k"], dt),
                "act_bwd": lambda: M.mlp_act_bwd_workspace_bytes(T, case["n"])}
        s["ws"] = torch.empty(need[op]() if op in need else 0, dtype=torch.uint8, device="cuda")
        s["act"] = {"none": M.MLP_ACT_NONE, "relu": M.MLP_ACT_RELU,
                    "leaky_relu_sq": M.MLP_ACT_LEAKY_RELU_SQ, "gelu": M.MLP_ACT_GELU,
                    "gelu_tanh": M.MLP_ACT_GELU_TANH,
                    "silu": M.MLP_ACT_SILU}[case.get("act", "none")]
    return s


# ------------------------------------------------------------------ plain forms

def _ckpt_buffers(T, d):
    return (torch.empty(T, d, dtype=torch.int8, device="cuda"),
            torch.empty(T, (d + 31) // 32, dtype=torch.uint8, device="cuda"))


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


def _norm(x):
    mean = x.mean(1)
    c = x - mean[:, None]
    return mean, torch.rsqrt((c * c).mean(1) + _EPS)


def _run_plain(s):
    case, dt = s["case"], s["dt"]
    op = case["op"]
    if op in ("ln_fwd", "ln_train"):
        x = s["x"].float()
        mean, rstd = _norm(x)
        out = {"y": ((x - mean[:, None]) * rstd[:, None] * s["gain"] + s["shift"]).to(dt),
               "mean": mean, "rstd": rstd}
        if op == "ln_train":
            if case["ckpt"]:
                x = _values(_quantise(s["x"]))
            xh = (x - mean[:, None]) * rstd[:, None]
            dy = s["dy"].float()
            t = dy * s["gain"]
            dx = rstd[:, None] * (t - t.mean(1)[:, None] - xh * (t * xh).mean(1)[:, None])
            if s["dres"] is not None:
                dx = dx + s["dres"].float()
            out.update(dx=dx.to(dt), dgain=(dy * xh).sum(0), dshift=dy.sum(0))
        return out
    if op == "lin_fwd":
        u = s["x"].float() @ s["w"].float() + s["bias"]
        y = _act(u, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = {"y": y.to(dt)}
        if case["save"] == "same":
            out["u"] = u.to(dt)
        elif case["save"] == "ckpt":
            out["u"] = _values(_quantise(u)).to(torch.bfloat16)
        return out
    if op in ("lin_bwd", "act_bwd"):
        da = s["dy"].float()
        if op == "lin_bwd":
            da = da @ s["w"].float().t()
        u = _values(s["ckpt"]) if case["saved"] == "ckpt" else s["u"].float()
        du = da * _act_grad(u, case["act"])
        out = {"du": du.to(dt), "dbias": du.sum(0)}
        if case["again"]:
            out["a"] = _act(u, case["act"]).to(dt)
        return out
    return {"out": _values(_quantise(s["x"])).to(dt)}


# ------------------------------------------------------------------ the library

def _run_own(s):
    import mlp_step_gb300 as M
    case = s["case"]
    op = case["op"]
    if op == "ln_fwd":
        M.mlp_layernorm_fwd(s["x"], s["y"], gain=s["gain"], shift=s["shift"], mean=s["mean"],
                            rstd=s["rstd"], eps=_EPS)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "ln_train":
        ck = s["ckpt"]
        M.mlp_layernorm_fwd(s["x"], s["y"], gain=s["gain"], shift=s["shift"], mean=s["mean"],
                            rstd=s["rstd"], ckpt=ck, eps=_EPS)
        M.mlp_layernorm_bwd(s["dy"], s["mean"], s["rstd"], s["dx"], s["dgain"], s["dshift"],
                            s["ws"], x=None if ck is not None else s["x"], ckpt=ck,
                            gain=s["gain"], dres=s["dres"])
        return {k: s[k] for k in ("y", "mean", "rstd", "dx", "dgain", "dshift")}
    if op == "lin_fwd":
        save = case["save"]
        M.mlp_linear_fwd(s["x"], s["w"], s["y"], bias=s["bias"], act=s["act"], slope=_SLOPE,
                         residual=s["residual"], u=s["u"] if save == "same" else None,
                         ckpt=s["ckpt"], workspace=s["ws"])
        if save == "none":
            return {"y": s["y"]}
        u = s["u"]
        if save == "ckpt":
            u = torch.empty(case["T"], case["n"], dtype=torch.bfloat16, device="cuda")
            M.mlp_ckpt8_decode(s["ckpt"][0], s["ckpt"][1], u)
        return {"y": s["y"], "u": u}
    if op in ("lin_bwd", "act_bwd"):
        kw = dict(act=s["act"], slope=_SLOPE, u=s["u"], ckpt=s["ckpt"], dbias=s["dbias"],
                  a=s["a"], workspace=s["ws"])
        if op == "lin_bwd":
            M.mlp_linear_bwd(s["dy"], s["w"], s["du"], **kw)
        else:
            M.mlp_act_bwd(s["dy"], s["du"], **kw)
        out = {"du": s["du"], "dbias": s["dbias"]}
        if case["again"]:
            out["a"] = s["a"]
        return out
    M.mlp_ckpt8_encode(s["x"], s["ckpt"][0], s["ckpt"][1])
    M.mlp_ckpt8_decode(s["ckpt"][0], s["ckpt"][1], s["out"])
    return {"out": s["out"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, T, e = case["op"], case["T"], _ESZ[case["dtype"]]
    flops = 0
    if op in ("ln_fwd", "ln_train"):
        m = T * case["d"]
        b = 2 * e * m + 8 * case["d"] + 8 * T
        flops = 8 * m
        if op == "ln_train":
            # the backward runs later in a step: it reads x (or its 8-bit form) again
            kept = (1 + 1 / 32) * m if case["ckpt"] else 0
            b += kept + (kept or e * m) + 2 * e * m + 8 * T + 12 * case["d"]
            b += e * m if case["dres"] else 0
            flops += 12 * m
    elif op == "lin_fwd":
        k, n = case["k"], case["n"]
        m = T * n
        b = e * (T * k + k * n + m) + 4 * n + (e * m if case["residual"] else 0)
        b += e * m if case["save"] == "same" else 0
        # written once, then read back and expanded
        b += (2 * (1 + 1 / 32) + 2) * m if case["save"] == "ckpt" else 0
        flops = 2 * T * k * n
    elif op in ("lin_bwd", "act_bwd"):
        n = case["n"]
        m = T * n
        b = ((1 + 1 / 32) if case["saved"] == "ckpt" else e) * m + e * m + 4 * n
        b += e * m if case["again"] else 0
        if op == "lin_bwd":
            b += e * (T * case["k"] + case["k"] * n)
            flops = 2 * T * case["k"] * n
        else:
            b += e * m
            flops = 10 * m
    else:
        m = T * case["d"]
        b = 2 * e * m + 2 * (1 + 1 / 32) * m
    return {"bytes": b, "flops": flops}


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


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("ln_fwd", "ln_train"):
        out = {k: [] for k in ("y", "mean", "rstd", "dx")}
        dgain = dshift = 0
        gain, shift = s["gain"].double(), s["shift"].double()
        step = max(1, (1 << 26) // case["d"])
        for r in range(0, case["T"], step):
            x = s["x"][r:r + step].double()
            mu = x.mean(1, keepdim=True)
            rho = 1 / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + _EPS)
            out["y"].append((x - mu) * rho * gain + shift)
            out["mean"].append(mu[:, 0])
            out["rstd"].append(rho[:, 0])
            if op == "ln_train":
                if case["ckpt"]:
                    x = _exact_ckpt(s["x"][r:r + step])
                xh = (x - mu) * rho
                dy = s["dy"][r:r + step].double()
                t = dy * gain
                dx = rho * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
                if s["dres"] is not None:
                    dx += s["dres"][r:r + step].double()
                out["dx"].append(dx)
                dgain = dgain + (dy * xh).sum(0)
                dshift = dshift + dy.sum(0)
        if op == "ln_fwd":
            del out["dx"]
        out = {k: torch.cat(v) for k, v in out.items()}
        if op == "ln_train":
            out.update(dgain=dgain, dshift=dshift)
        return out
    if op == "lin_fwd":
        u = s["x"].double() @ s["w"].double() + s["bias"].double()
        y = _exact_act(u, case["act"])[0]
        if s["residual"] is not None:
            y += s["residual"].double()
        out = {"y": y}
        if case["save"] != "none":
            out["u"] = u if case["save"] == "same" else _exact_ckpt(u)
        return out
    if op in ("lin_bwd", "act_bwd"):
        da = s["dy"].double()
        if op == "lin_bwd":
            da = da @ s["w"].double().t()
        if case["saved"] == "ckpt":
            q, b = s["ckpt"]
            step = _two_to(b.to(torch.int32) - 133)
            u = q.double() * step.repeat_interleave(32, dim=1)[:, :case["n"]]
        else:
            u = s["u"].double()
        f, df = _exact_act(u, case["act"])
        out = {"du": da * df, "dbias": (da * df).sum(0)}
        if case["again"]:
            out["a"] = f
        return out
    return {"out": _exact_ckpt(s["x"])}
