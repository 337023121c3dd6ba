"""Linear layer with its epilogue against its fp64 definition.

Tolerances: an output is off by at most half a step of its type plus the fp32 sums'
error. A sum of b products of bf16 values (exact in fp32) in any order is off by at
most (b + 4) roundings of the sum of magnitudes; the matrix cores add several
products at once and may cut rather than round, which the factor 2 covers. Bias and
residual add one rounding each; the activations' slopes are at most 1.13 and their
own error is below 8 roundings of the argument's size.
"""
import numpy as np
import pytest
import torch

import oracle as O
from layer_wise_obs_amd import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _randn(shape, seed, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def _check(Y, X, W, bias, act, residual):
    ref = O.forward_linear(X, W, bias, act, residual)
    size = np.abs(X.double().cpu().numpy()) @ np.abs(W.double().cpu().numpy()).T
    if bias is not None:
        size = size + np.abs(bias.double().cpu().numpy())
    tol = size * ((X.shape[1] + 4) * 2 * U * (1.13 if act != "none" else 1.0) + 9 * U)
    if residual is not None:
        tol = tol + 2 * U * (np.abs(residual.double().cpu().numpy()) + np.abs(ref))
    tol = tol + torch.finfo(Y.dtype).eps / 2 * (np.abs(ref) + tol) + 1e-38
    got = Y.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.max(np.abs(got - ref) / tol))


def _dev(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("n,b,c", [
    (1, 8, 1), (1, 4096, 4096), (2, 40, 7), (3, 1032, 515), (16, 2056, 129), (17, 264, 64),
    (33, 72, 1000), (64, 11008, 256), (65, 512, 2048), (100, 4096, 16), (127, 96, 127),
    (128, 128, 128), (129, 1000, 257), (300, 264, 200), (777, 2056, 1023), (1030, 40, 520),
    (2048, 512, 8200), (4100, 1032, 4352)])
@pytest.mark.parametrize("ydt", [BF, F32])
def test_linear_matches_definition(n, b, c, ydt):
    """Ragged in every dimension, contraction tails (b % 32 != 0), split contractions,
    both tile sizes."""
    print(f"[case] linear n={n} b={b} c={c} {ydt}", flush=True)
    X, W = _randn((n, b), n + b), _randn((c, b), c, scale=b ** -0.5)
    _check(L.linear(_dev(X), _dev(W), out_dtype=ydt), X, W, None, "none", None)


@pytest.mark.parametrize("n,c", [(5, 72), (5, 71), (300, 264), (300, 263), (40, 4097)])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_linear_epilogues(n, c, act):
    print(f"[case] linear epilogue n={n} c={c} {act}", flush=True)
    b = 392
    X, W, bias = _randn((n, b), 1), _randn((c, b), 2, scale=2 * b ** -0.5), _randn((c,), 3)
    for ydt in (BF, F32):
        R = _randn((n, c), 4, ydt, 2.0)
        for has_bias, has_res in ((True, False), (False, True), (True, True)):
            bi, r = bias if has_bias else None, R if has_res else None
            Y = L.linear(_dev(X), _dev(W), bias=_dev(bi), act=act, residual=_dev(r), out_dtype=ydt)
            _check(Y, X, W, bi, act, r)


@pytest.mark.parametrize("n,b,c", [(5, 264, 72), (300, 1032, 264), (70, 4096, 520)])
def test_linear_with_and_without_workspace_and_repeated(n, b, c):
    """A split contraction repeats bit for bit; without a workspace the call runs unsplit."""
    print(f"[case] linear workspace n={n} b={b} c={c}", flush=True)
    X, W = _randn((n, b), 5), _randn((c, b), 6, scale=b ** -0.5)
    Xd, Wd = _dev(X), _dev(W)
    first = L.linear(Xd, Wd, out_dtype=F32)
    for _ in range(3):
        assert torch.equal(L.linear(Xd, Wd, out_dtype=F32), first)
    Y = torch.empty(n, c, dtype=F32, device=DEV)
    st = L.lib().th_linear(L._ptr(Xd), b, L._ptr(Wd), L.TH_BF16, n, b, c, None, 0, None, 0,
                           L._ptr(Y), L.TH_F32, c, None, 0, L._stream())
    assert st == L.TH_OK
    _check(Y, X, W, None, "none", None)


@pytest.mark.parametrize("n", [3, 150])
def test_linear_strides_in_place_residual_and_memory_left_alone(n):
    print(f"[case] linear strides n={n}", flush=True)
    b, c = 136, 88
    X = _randn((n, 2 * b + 8), 7)[:, 8:8 + b]
    W = _randn((c, b), 8, scale=b ** -0.5)
    for ydt, pad in ((BF, 8), (BF, 3), (F32, 4), (F32, 1)):
        buf = torch.full((n + 2, c + 2 * pad), 5.0, dtype=ydt, device=DEV)
        R = _randn((n, c), 9, ydt)
        Y = buf[1:n + 1, pad:pad + c]
        Y.copy_(R.to(DEV))
        big = torch.zeros(n, 2 * b + 8, dtype=BF, device=DEV)
        big[:, 8:8 + b] = X.to(DEV)
        out = L.linear(big[:, 8:8 + b], W.to(DEV), residual=Y, Y=Y)
        assert out is Y
        _check(Y, X, W, None, "none", R)
        Y.fill_(5.0)
        assert torch.all(buf == 5.0)


def test_linear_nonfinite_values_stay_in_their_rows_and_channels():
    """Rows past the end and the contraction's tail are read again as fill; none of it
    may reach another row's or channel's output, infinities included."""
    print("[case] linear non-finite", flush=True)
    for n, b, c in ((5, 40, 9), (200, 72, 150), (600, 1032, 520)):
        X, W = _randn((n, b), 10), _randn((c, b), 11)
        X[n - 1, 0] = float("inf")
        X[1, b - 1] = float("nan")
        W[c - 1, 8] = float("-inf")
        Y = L.linear(X.to(DEV), W.to(DEV), act="relu").cpu()
        fin = torch.ones(n, c, dtype=torch.bool)
        fin[n - 1], fin[1], fin[:, c - 1] = False, False, False
        assert torch.all(Y[fin].isfinite()) and torch.all(Y[1].isnan())
        assert not torch.any(Y[n - 1].isfinite() & (Y[n - 1] != 0))


def test_linear_captured_and_replayed():
    """A split product and its join in a graph, replayed with eager work between."""
    print("[case] linear in a graph", flush=True)
    n, b, c = 9, 2056, 264
    X, W = _randn((n, b), 12).to(DEV), _randn((c, b), 13, scale=b ** -0.5).to(DEV)
    R = _randn((n, c), 14).to(DEV)
    L.linear(X, W, residual=R)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y = L.linear(X, W, act="silu", residual=R)
    for seed in (20, 21, 22):
        X.copy_(_randn((n, b), seed).to(DEV))
        g.replay()
        eager = L.linear(X, W, act="silu", residual=R)
        torch.cuda.synchronize()
        assert torch.equal(Y, eager)


def test_linear_full_size_sampled():
    """The block's o_proj over 131072 tokens: sampled rows against fp64."""
    print("[case] linear 131072 x 4096 -> 4096", flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    X = torch.randn(131072, 4096, generator=g, device=DEV).to(BF)
    W = (torch.randn(4096, 4096, generator=g, device=DEV) / 64).to(BF)
    R = torch.randn(131072, 4096, generator=g, device=DEV).to(BF)
    Y = L.linear(X, W, residual=R)
    rows = torch.tensor([0, 1, 255, 256, 65535, 65536, 100001, 131070, 131071])
    _check(Y[rows].cpu(), X[rows].cpu(), W.cpu(), None, "none", R[rows].cpu())


@pytest.mark.parametrize("n,b,c", [(3, 64, 19), (70, 4096, 75), (150, 72, 331), (700, 136, 523)])
@pytest.mark.parametrize("ydt", [BF, F32])
@pytest.mark.parametrize("at", [0, 1, 3])
def test_linear_rows_of_any_alignment(n, b, c, ydt, at):
    print(f"[case] linear n={n} b={b} c={c} {ydt} at={at}", flush=True)
    X, W, bias = _randn((n, b), n), _randn((c, b), c, scale=b ** -0.5), _randn((c,), 5)
    wide = _randn((n, c + 4), 6, ydt)
    R = wide[:, 4 - at:c + 4 - at]
    buf = torch.full((n, c + 5), 7.0, dtype=ydt, device=DEV)  # odd pitches for odd and even c
    Y = buf[:, at:at + c]
    L.linear(X.to(DEV), W.to(DEV), bias=bias.to(DEV), act="silu", residual=_dev(wide)[:, 4 - at:c + 4 - at],
             Y=Y)
    _check(Y, X, W, bias, "silu", R)
    assert bool((buf[:, :at] == 7).all()) and bool((buf[:, at + c:] == 7).all())


@pytest.mark.parametrize("n", [1, 12])
def test_linear_most_channels_of_few_tokens(n):
    """The widest accepted layer: a workgroup per 16 channels is 2^32 threads in all, more than
    one launch takes. Small whole numbers, so every output is exact."""
    print(f"[case] linear {n} x 8 -> 2^27 - 1", flush=True)
    b, c = 8, (1 << 27) - 1
    W = torch.empty(c, b, dtype=BF, device=DEV)
    q = torch.arange(c, dtype=torch.int32, device=DEV)
    for j in range(b):
        W[:, j] = (q + j) % 5
    X = torch.zeros(n, b, dtype=BF, device=DEV)
    X[:, 0], X[:, 1], X[:, 7] = 1, 2, torch.arange(n, device=DEV) % 3
    Y = torch.full((n, c), 99.0, dtype=BF, device=DEV)
    L.linear(X, W, Y=Y)
    for t in range(n):
        assert torch.equal(Y[t], (q % 5 + 2 * ((q + 1) % 5) + (t % 3) * ((q + 7) % 5)).to(BF))


@pytest.mark.parametrize("n", [1, 70])
def test_linear_gelu_keeps_its_bits_in_the_tails(n):
    """Arguments that are exact in fp32 (one weight of 8 bits, another of 8 bits 2^-9 below it):
    the result is off by at most (16 + 1.5 z^2) roundings of itself. Counted: the exponent's
    product of three rounded factors, 3 U z^2 / 2; the hardware's exponential and reciprocal,
    2 U each, the latter met up to 1.6 times with the 2 U of its argument and of itself; 4 U of
    the polynomial and its fit; 4 U of the last products."""
    print(f"[case] linear gelu tails n={n}", flush=True)
    z = torch.linspace(-12.5, 12.5, 9001)
    hi = z.to(BF)
    W = torch.zeros(z.numel(), 8, dtype=BF)
    W[:, 0], W[:, 3] = hi, ((z - hi.float())).to(BF)
    X = torch.zeros(n, 8, dtype=BF)
    X[:, 0] = X[:, 3] = 1.0
    zz = W[:, 0].double().numpy() + W[:, 3].double().numpy()
    assert np.array_equal(zz, zz.astype(np.float32))
    ref = O.forward_linear(X[:1], W, None, "gelu")[0]
    Y = L.linear(X.to(DEV), W.to(DEV), act="gelu", out_dtype=F32).cpu().double().numpy()
    tol = (16 + 1.5 * zz * zz) * U * np.abs(ref)
    assert np.all(np.abs(Y - ref) <= tol), np.max(np.abs(Y - ref) / tol)


def test_linear_gelu_of_infinities_and_zero():
    print("[case] linear gelu infinities", flush=True)
    W = torch.zeros(4, 8, dtype=BF)
    W[:, 0] = torch.tensor([float("inf"), 1e30, -1e30, 0.0])
    X = torch.zeros(1, 8, dtype=BF)
    X[0, 0] = 1.0
    Y = L.linear(X.to(DEV), W.to(DEV), act="gelu", out_dtype=F32).cpu()[0]
    assert Y[0] == float("inf") and Y[1] == W[1, 0].float() and Y[2] == 0 and Y[3] == 0


@pytest.mark.parametrize("n,b,c", [(1, 8192, 1024), (12, 8192, 100), (13, 11008, 64), (1, 28672, 17),
                                   (5, 11008, 512), (200, 28672, 40)])
def test_linear_few_channels_of_a_long_contraction(n, b, c):
    print(f"[case] linear n={n} b={b} c={c}", flush=True)
    X, W = _randn((n, b), n), _randn((c, b), c, scale=b ** -0.5)
    for ydt in (BF, F32):
        _check(L.linear(X.to(DEV), W.to(DEV), out_dtype=ydt), X, W, None, "none", None)
