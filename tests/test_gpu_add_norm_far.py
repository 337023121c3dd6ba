"""The norm behind an addition where an element is so far below its row's root mean square that
the two's quotient is no normal fp32 number, and the weight brings it back: outputs are still
those of the 64-bit definition, rounded once."""
import pytest
import torch

from layer_wise_obs_amd import _lib as L
from tests.test_gpu_add_norm import BF, DEV, F32, _check, _randn, _stream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,b", [(5, 96), (3, 4128)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [True, False])
def test_elements_far_below_their_rows_root_mean_square(n, b, dtype, residual):
    print(f"[case] add_rms_norm far elements n={n} b={b} {dtype} residual={residual}", flush=True)
    x, w = _randn((n, b), 1, F32), _randn((b,), 2, F32)
    x[:, 64:] *= 2.0 ** -40
    x[:, 5] = 2.0 ** 95  # of a block of its own
    x[:, 32:64] *= torch.exp2(-torch.arange(32.0) - 20)  # quotients 2^-115 to 2^-150
    w[32:64] *= 2.0 ** 80
    w[64:] *= 2.0 ** 100
    x, w = x.to(dtype), w.to(dtype)
    r = torch.zeros_like(x) if residual else None
    h = _stream(x, r)
    for out in ("e4m3", "e2m1", BF, F32):
        _, Y = L.add_rms_norm(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV), out=out)
        _check(Y, h, w, 1e-5)
