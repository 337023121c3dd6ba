"""The norm behind an addition to the residual stream against its fp64 definition.

Sums, root and products are in 64 bits: an output is off by half a step of its type, and by
at most b / 2 + 70 roundings of 2^-53 before it. Microscaled outputs are compared bit by bit
with the quantisation of the fp64 values; they could differ only where one of those lies
within 2^-43 of itself next to a border.
"""
import numpy as np
import pytest
import torch

import oracle as O
from layer_wise_obs_amd import _lib as L
from tests.test_gpu_mx import _codes

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _randn(shape, seed, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def _stream(x, r):
    return x if r is None else (x.double() + r.double()).to(x.dtype)


def _check(Y, h, w, eps):
    ref = O.rms_norm(h, w, eps)
    if isinstance(Y, L.MxMatrix):
        codes, scales = O.mx_quantize(ref, Y.type)
        got = _codes(Y)
        assert np.array_equal(got[1], scales) and np.array_equal(got[0], codes)
        return
    tol = np.abs(ref) * (torch.finfo(Y.dtype).eps / 2 * 1.0001) + 1e-44
    got = Y.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


@pytest.mark.parametrize("n,b", [(1, 32), (7, 4096), (3, 64), (33, 2048), (9, 2080), (5, 8192), (4, 8224),
                                 (2, 28672), (130, 544), (1, 17), (6, 1001), (5, 4095), (3, 9001)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [True, False])
def test_add_norm_matches_definition(n, b, dtype, residual):
    print(f"[case] add_rms_norm n={n} b={b} {dtype} residual={residual}", flush=True)
    x, w = _randn((n, b), 1, dtype, 2.0), 1 + _randn((b,), 2, dtype, 0.1)
    r = _randn((n, b), 3, dtype, 3.0) if residual else None
    h = _stream(x, r)
    for out in ["e4m3", "e2m1"] * (b % 32 == 0) + [BF, F32]:
        s, Y = L.add_rms_norm(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV),
                              eps=1e-5, out=out)
        assert torch.equal(s.cpu(), h)
        _check(Y, h, w, 1e-5)


@pytest.mark.parametrize("n,b", [(3, 544), (2, 9216)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_add_norm_in_place_and_memory_left_alone(n, b, dtype):
    print(f"[case] add_rms_norm in place n={n} b={b} {dtype}", flush=True)
    x, w, r = _randn((n, b), 1, dtype), _randn((b,), 2, dtype), _randn((n, b), 3, dtype)
    h = _stream(x, r)
    for where in ("x", "r", "own"):
        for pad in (8, 3):
            bufs = [torch.full((n + 2, b + 2 * pad), 5.0, dtype=dtype, device=DEV) for _ in range(3)]
            views = [t[1:n + 1, pad:pad + b] for t in bufs]
            views[0].copy_(x)
            views[1].copy_(r)
            to = views[{"x": 0, "r": 1, "own": 2}[where]]
            s, Y = L.add_rms_norm(views[0], w.to(DEV), residual=views[1], sum_out=to, out="e4m3")
            assert s is to and torch.equal(to.cpu(), h)
            _check(Y, h, w, 1e-5)
            for v in views:
                v.fill_(5.0)
            assert all(torch.all(t == 5.0) for t in bufs)
    y = torch.full((n + 2, b + 7), 5.0, device=DEV)
    _, Y = L.add_rms_norm(x.to(DEV), w.to(DEV), residual=r.to(DEV), out=y[1:n + 1, 3:3 + b])
    _check(Y, h, w, 1e-5)
    Y.fill_(5.0)
    assert torch.all(y == 5.0)
    # the sum is not wanted
    xd, rd, wd, out = x.to(DEV), r.to(DEV), w.to(DEV), torch.empty(n, b, device=DEV)
    assert L.lib().th_add_rms_norm(L._ptr(xd), b, L._ptr(rd), b, L._dtype_code(xd), n, b, L._ptr(wd),
                                   1e-5, None, 0, L._ptr(out), L.TH_F32, b, None,
                                   L._stream()) == L.TH_OK
    _check(out, h, w, 1e-5)
    assert torch.equal(xd.cpu(), x) and torch.equal(rd.cpu(), r)


def test_add_norm_far_values_zeros_and_numbers_that_are_none():
    """Squares past fp32's range are held; a row of zeros gives zeros; rows with a NaN or an
    infinity are no numbers, the others stay."""
    print("[case] add_rms_norm far values", flush=True)
    n, b = 6, 96
    x = _randn((n, b), 1, F32)
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = 0
    x[3, 50] = float("inf")
    x[4, 7] = float("nan")
    w = _randn((b,), 2, F32)
    for out in ("e4m3", "e2m1", F32, BF):
        _, Y = L.add_rms_norm(x.to(DEV), w.to(DEV), eps=1e-5, out=out)
        y = L.mx_dequantize(Y, out_dtype=F32) if isinstance(Y, L.MxMatrix) else Y
        y = y.float().cpu()
        # x / infinity is 0; infinity / infinity no number, nor its block
        assert torch.all(y[4].isnan()) and y[3, 50].isnan()
        assert torch.all(y[2] == 0) and torch.all(y[[0, 1, 2, 5]].isfinite())
        keep = [0, 1, 2, 5]
        if isinstance(Y, L.MxMatrix):
            codes, scales = O.mx_quantize(O.rms_norm(x[keep], w, 1e-5), Y.type)
            got = _codes(Y)
            assert np.array_equal(got[0][keep], codes) and np.array_equal(got[1][keep], scales)
        else:
            _check(Y[keep], x[keep], w, 1e-5)


def test_add_norm_many_rows_of_a_block_repeated_and_captured():
    print("[case] add_rms_norm captured", flush=True)
    n, b = 3000, 1056
    x, r, w = _randn((n, b), 1), _randn((n, b), 2), _randn((b,), 3)
    xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
    h, Y = L.add_rms_norm(xd, wd, residual=rd, out="e4m3")
    for _ in range(2):
        h2, Y2 = L.add_rms_norm(xd, wd, residual=rd, out="e4m3")
        assert torch.equal(h, h2) and torch.equal(Y.elements, Y2.elements)
        assert torch.equal(Y.scales, Y2.scales)
    pick = [0, 1, 1499, 2998, 2999]
    _check(L.MxMatrix("e4m3", Y.elements[pick], Y.scales[pick]), _stream(x, r)[pick], w, 1e-5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hg, Yg = L.add_rms_norm(xd, wd, residual=rd, out="e2m1")
    for i in range(3):
        xd.copy_(_randn((n, b), 10 + i))
        g.replay()
        he, Ye = L.add_rms_norm(xd, wd, residual=rd, out="e2m1")
        torch.cuda.synchronize()
        assert torch.equal(hg, he) and torch.equal(Yg.elements, Ye.elements)
        assert torch.equal(Yg.scales, Ye.scales)
