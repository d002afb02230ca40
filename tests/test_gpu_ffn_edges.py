"""The feed-forward operators where values, pitches and callers are unusual."""
import math

import pytest
import torch

import mlp_step_gb300 as M
from test_gpu_ffn import ACTS, BF16, F16, F32, SLOPE, Guarded, rnd

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
