"""What the Python entry points of the forward steps refuse and how they make their outputs."""

import pytest
import torch

from layer_wise_obs_amd import _lib as thanos

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _t(*shape, dtype=BF):
    return torch.ones(shape, dtype=dtype, device="cuda")


def _gap(*shape, dtype=BF):  # last dimension not contiguous
    return torch.ones(shape + (2,), dtype=dtype, device="cuda")[..., 0]


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("bad,error", [
    (lambda n: thanos.rms_norm(_gap(n, 16), _t(16)), ValueError),
    (lambda n: thanos.rms_norm(_t(n, 16), _t(8)), ValueError),
    (lambda n: thanos.rms_norm(_t(n, 16), _t(16, dtype=torch.float32)), TypeError),
    (lambda n: thanos.rms_norm(_t(n, 16), _t(16).cpu()), ValueError),
    (lambda n: thanos.rms_norm(_t(n, 16), _t(16), Y=_gap(n, 16)), ValueError),
    (lambda n: thanos.rms_norm(_t(n, 16), _t(16), Y=_t(n + 1, 16)), ValueError),
    (lambda n: thanos.linear(_gap(n, 16), _t(8, 16)), ValueError),
    (lambda n: thanos.linear(_t(n, 16), _t(8, 24)), ValueError),
    (lambda n: thanos.linear(_t(n, 16), _t(8, 32)[:, :16]), ValueError),
    (lambda n: thanos.linear(_t(n, 16), _t(8, 16, dtype=torch.float32)), TypeError),
    (lambda n: thanos.linear(_t(n, 16), _t(8, 16), residual=_gap(n, 8)), ValueError),
    (lambda n: thanos.linear(_t(n, 16), _t(8, 16), residual=_t(n, 8), out_dtype=torch.float32),
     TypeError),
    (lambda n: thanos.linear(_t(n, 16), _t(8, 16), Y=_gap(n, 8)), ValueError),
    (lambda n: thanos.linear(_t(n, 16), _t(8, 16), bias=_t(9)), ValueError),
    (lambda n: thanos.rotary(_gap(n, 2, 16), None, _t(8, dtype=torch.float64)), ValueError),
    (lambda n: thanos.rotary(_t(n, 2, 16), _t(n, 1, 8), _t(8, dtype=torch.float64)), ValueError),
    (lambda n: thanos.rotary(_t(n, 2, 16), _t(n + 1, 1, 16), _t(8, dtype=torch.float64)),
     ValueError),
    (lambda n: thanos.rotary(_t(n, 2, 16), None, _t(8)), TypeError),
    (lambda n: thanos.rotary(_t(n, 2, 16), None, _t(8, dtype=torch.float64),
                             positions=_t(n, dtype=torch.int64)), TypeError),
    (lambda n: thanos.rotary(_t(n, 2, 16), None, _t(8, dtype=torch.float64), q_norm=_t(8)),
     ValueError),
    (lambda n: thanos.rotary(_t(n, 2, 16), None, _t(8, dtype=torch.float64),
                             k_out=_t(n, 2, 16)), ValueError),
    (lambda n: thanos.rotary(_t(n, 2, 16), None, _t(8, dtype=torch.float64),
                             q_out=_gap(n, 2, 16)), ValueError),
    (lambda n: thanos.attention(_gap(n, 2, 16), _t(n, 1, 16), _t(n, 1, 16)), ValueError),
    (lambda n: thanos.attention(_t(n, 2, 16), _t(n, 1, 16), _t(n, 2, 16)), ValueError),
    (lambda n: thanos.attention(_t(n, 2, 16), _t(n, 1, 16), _t(n, 1, 16),
                                q_start=_t(2, dtype=torch.int64)), TypeError),
    (lambda n: thanos.attention(_t(n, 2, 16), _t(n, 1, 16), _t(n, 1, 16),
                                k_start=_t(2, dtype=torch.int32)), ValueError),
    (lambda n: thanos.attention(_t(n, 2, 16), _t(n, 1, 16), _t(n, 1, 16), O=_gap(n, 2, 16)),
     ValueError),
])
def test_refuses(bad, error, n):
    with pytest.raises(error):
        bad(n)


def test_outputs_are_dense_whatever_the_inputs_strides():
    x = torch.randn(4, 6, 16, device="cuda").to(BF).permute(1, 0, 2)  # [6, 4, 16], heads outside
    freqs = thanos.rotary_freqs(16, device="cuda")
    q, k = thanos.rotary(x, x, freqs)
    assert q.is_contiguous() and k.is_contiguous()
    dense = thanos.rotary(x.contiguous(), None, freqs)[0]
    assert torch.equal(q, dense) and torch.equal(k, dense)
    o = thanos.attention(x, x, x)
    assert o.is_contiguous()
    assert torch.equal(o, thanos.attention(*(x.contiguous(),) * 3))


def test_single_rows_of_any_stride():
    x = torch.randn(1, 16, device="cuda").to(BF)
    odd = x.as_strided((1, 16), (3, 1))  # the stride of a single row means nothing
    w = torch.randn(8, 16, device="cuda").to(BF)
    assert torch.equal(thanos.linear(odd, w), thanos.linear(x, w))
    assert torch.equal(thanos.rms_norm(odd, w[0]), thanos.rms_norm(x, w[0]))
    h = odd.as_strided((1, 1, 16), (3, 5, 1))
    f = thanos.rotary_freqs(16, device="cuda")
    assert torch.equal(thanos.rotary(h, None, f)[0], thanos.rotary(x[:, None], None, f)[0])
    assert torch.equal(thanos.attention(h, h, h), x[:, None])


def test_no_rows():
    f = thanos.rotary_freqs(16, device="cuda")
    assert thanos.linear(_t(0, 16), _t(8, 16), bias=_t(8), act="gelu").shape == (0, 8)
    assert thanos.linear(_t(0, 16), _t(8, 16), residual=_t(0, 8)).shape == (0, 8)
    assert thanos.rms_norm(_t(0, 16), _t(16), out_dtype=torch.float32).dtype == torch.float32
    q, k = thanos.rotary(_t(0, 2, 16), _t(0, 1, 16), f, q_norm=_t(16))
    assert q.shape == (0, 2, 16) and k.shape == (0, 1, 16)
    starts = torch.zeros(4, dtype=torch.int32, device="cuda")  # three sequences, all empty
    assert thanos.attention(_t(0, 2, 16), _t(0, 1, 16), _t(0, 1, 16), starts).shape == (0, 2, 16)
    torch.cuda.synchronize()
