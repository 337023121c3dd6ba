"""silu behind products of microscaled operands, on every tile form, whole and in pieces: it
keeps its relative accuracy as far as the output's type reaches, and is the same on all of them."""
import pytest
import torch

from layer_wise_obs_amd import _lib as L
from tests.test_gpu_mx import BF, DEV, F32, _randn
from tests.test_mx_plan import JOINED, WHOLE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,b,c", [(*WHOLE[t][:1], 96, WHOLE[t][1]) for t in WHOLE] + JOINED[:1])
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_silu_keeps_its_relative_accuracy(n, b, c, form):
    """Arguments from -110 to 110 by the bias alone (X is 0). An argument's rounding in the
    exponential is |z| 2^-23 of the result, everything else five roundings of 2^-23 (units of
    the hardware's exponential and reciprocal among them); the output is rounded once, below its
    type's normal numbers to the next multiple of its lowest step, of which the steps in fp32 before
    it are as coarse as 2^-149 each."""
    print(f"[case] mx silu n={n} b={b} c={c} {form}", flush=True)
    X = L.mx_quantize(torch.zeros(n, b, dtype=BF, device=DEV), form)
    W = L.mx_quantize(_randn((c, b), 1).to(DEV), "e2m1")
    bias = torch.linspace(-110, 110, c).to(BF) if c > 100 else _randn((c,), 2, scale=60.0)
    bias[:8] = torch.tensor([-86.0, -87.5, -88.5, -89.0, -90.0, -91.5, -103.0, -0.0])
    z = bias.double()
    want = z / (1 + torch.exp(-z))
    for ydt in (BF, F32):
        Y = L.mx_linear(X, W, bias=bias.to(DEV), act="silu", out_dtype=ydt).double().cpu()
        tol = want.abs() * ((z.abs() + 5) * 2.0 ** -23)
        tol = tol + torch.finfo(ydt).eps / 2 * (want.abs() + tol) + 2 * 2.0 ** -149
        if ydt == BF:
            tol = tol + 2.0 ** -134
        bad = ~((Y - want).abs() <= tol)
        assert not bad.any(), (z[bad.any(0)], Y[:, bad.any(0)][0], want[bad.any(0)])
