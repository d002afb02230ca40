"""The gated feed-forward sublayer's operators where values, sizes and forms of the
call are unusual."""
import math

import pytest
import torch

import mlp_step_gb300 as M
from test_gpu_ffn import BF16, F16, F32, U24, near, rounding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    M.load()
    yield
    assert M.get_device_status() == M.MLP_OK


# ------------------------------------------------------------ logistic gates

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_logistic_gate_in_its_far_tail(dtype):
    """The gate s and its derivative s (1 - s), relative to their own values, as
    far as they are normal numbers; below they may be 0."""
    T, d = 3, 488
    z = torch.linspace(-100, -70, T * d, device="cuda").view(T, d).to(dtype)
    g = torch.Generator(device="cuda").manual_seed(31)
    r = lambda: (1 + torch.rand(T, d, generator=g, device="cuda")).to(dtype)  # noqa: E731
    b, dh = r(), r()
    big = 2.0 ** 112  # brings e^-87 to 5e-5
    kw = dict(gate=z, gate_act=M.MLP_GATE_SIGMOID, scale=big)
    h, dx, db, dz = (torch.full_like(b, math.nan) for _ in range(4))
    M.mlp_resnorm_fwd(torch.zeros_like(b), b=b, h=h, **kw)
    M.mlp_resnorm_bwd(dx, dh=dh, b=b, db=db, dgate=dz, **kw)
    assert torch.equal(dx, dh)
    zd, bd, hd = z.double(), b.double(), dh.double()
    s, rest = torch.sigmoid(zd), torch.sigmoid(-zd)
    # In U24: e^(-z) 2 |z| from its argument (the product with log2 e and that
    # constant are off by half a step each) and 4 (two ulp); 1 + e^(-z) 1; its
    # reciprocal 4.  So s has 2 |z| + 9, s e^(-z) twice that at most and its own
    # product, s (1 - s) three times and both products; then three
    # products each, two of them with powers of two.
    rel = 2 * zd.abs() + 9
    # 1 / (1 + e^(-z)) reads as 0 where it is below 2^-126 (or off by rel of it)
    gone = s <= 2.0 ** -126 * (1 + rel * U24)
    for got, ref, e in ((h, s * bd * big, rel + 3), (db, s * hd * big, rel + 3),
                        (dz, s * rest * bd * hd * big, 3 * rel + 5)):
        near(got, ref, torch.where(gone, ref, e * U24 * ref + rounding(dtype, ref)), "z")
        assert (got >= 0).all()
