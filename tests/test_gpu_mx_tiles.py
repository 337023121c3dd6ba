"""Products of microscaled operands on every tile form, whole and in pieces: ragged rows and
channels, contraction tails, blocks of no numbers, epilogues, sums that fp32 holds over the
widest spans of the elements, and how much an e4m3 X with a bf16 Y loses. Tolerances are those of
test_gpu_mx.py (its docstring derives them); test_mx_plan.py holds the shapes to their tiles."""
import numpy as np
import pytest
import torch

from layer_wise_obs_amd import _lib as L
from tests.test_gpu_mx import BF, DEV, F32, _check_product, _random_mx, _randn, _values
from tests.test_mx_plan import JOINED, PAST_CACHE, WHOLE, WHOLE_K

pytestmark = pytest.mark.gpu
LARGE = [(128, 128), (128, 256), (256, 256)]


def _operands(n, b, c, form, std=1.0):
    X = L.mx_quantize(_randn((n, b), n + b).to(DEV), form)
    W = L.mx_quantize(_randn((c, b), c, scale=std * b ** -0.5).to(DEV), "e2m1")
    return X, W


@pytest.mark.parametrize("tile", LARGE)
@pytest.mark.parametrize("b", WHOLE_K)
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_tiles_match_definition(tile, b, form):
    n, c = WHOLE[tile]
    print(f"[case] mx tile {tile} n={n} b={b} c={c} {form}", flush=True)
    X, W = _operands(n, b, c, form)
    v = _values(X), _values(W)
    for ydt in (BF, F32):
        _check_product(L.mx_linear(X, W, out_dtype=ydt), X, W, None, "none", None, v)


@pytest.mark.parametrize("tile", LARGE)
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_tiles_keep_blocks_of_no_numbers_in_their_rows_and_channels(tile, form):
    n, c = WHOLE[tile]
    b = 288
    print(f"[case] mx tile {tile} NaN blocks {form}", flush=True)
    x, w = _randn((n, b), 11), _randn((c, b), 12)
    x[2, 70], x[n - 1, b - 1], w[77, 5], w[c - 1, 280] = (float("nan"),) * 4
    X, W = L.mx_quantize(x.to(DEV), form), L.mx_quantize(w.to(DEV), "e2m1")
    want = torch.zeros(n, c, dtype=torch.bool)
    want[[2, n - 1]], want[:, [77, c - 1]] = True, True
    for ydt in (BF, F32):
        assert torch.equal(L.mx_linear(X, W, out_dtype=ydt).isnan().cpu(), want)


@pytest.mark.parametrize("tile", list(WHOLE))
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_scales_of_the_whole_range(tile, form):
    """Blocks of X with scales from 2^-127 to 2^127, those of W the other way round up to 2^3: either
    side's values may be past fp32's range, their products are not."""
    n, c = WHOLE[tile]
    b = 1056
    print(f"[case] mx tile {tile} scales {form}", flush=True)
    X, W = _random_mx(n, b, form, n), _random_mx(c, b, "e2m1", c)
    g = np.random.default_rng(1)
    scales = g.integers(0, 255, b // 32)
    scales[:8] = 0, 1, 2, 3, 251, 252, 253, 254
    other = np.clip(254 - scales + g.integers(-3, 4, b // 32), 0, 254)
    X.scales.copy_(torch.from_numpy(np.tile(scales.astype(np.uint8), (n, 1))))
    W.scales.copy_(torch.from_numpy(np.tile(other.astype(np.uint8), (c, 1))))
    v = _values(X), _values(W)
    for ydt in (BF, F32):
        _check_product(L.mx_linear(X, W, out_dtype=ydt), X, W, None, "none", None, v)


def _epilogues(n, b, c, form, act, pad):
    """Bias, residual in place at odd pitches, memory around Y left alone."""
    X, W = _operands(n, b, c, form, 2.0)
    v = _values(X), _values(W)
    bias = _randn((c,), 3)
    for ydt in (BF, F32):
        R = _randn((n, c), 4, ydt, 2.0)
        for has_bias, has_res in ((True, False), (False, True), (True, True)):
            buf = torch.full((n + 2, c + 2 * pad), 5.0, dtype=ydt, device=DEV)
            Y = buf[1:n + 1, pad:pad + c]
            if has_res:
                Y.copy_(R.to(DEV))
            L.mx_linear(X, W, bias=bias.to(DEV) if has_bias else None, act=act,
                        residual=Y if has_res else None, Y=Y)
            _check_product(Y, X, W, bias if has_bias else None, act, R if has_res else None, v)
            Y.fill_(5.0)
            assert torch.all(buf == 5.0)


@pytest.mark.parametrize("tile", LARGE)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_tiles_epilogues(tile, act, form):
    n, c = WHOLE[tile]
    print(f"[case] mx tile {tile} epilogue {act} {form}", flush=True)
    _epilogues(n, 96, c, form, act, 3)


@pytest.mark.parametrize("n,b,c", JOINED)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_epilogues_of_joined_pieces(n, b, c, act, form):
    print(f"[case] mx joined n={n} b={b} c={c} {act} {form}", flush=True)
    _epilogues(n, b, c, form, act, 1)


@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_outputs_past_the_caches_at_odd_places(form):
    """2^27 outputs and more, whose stores go past the caches: rows 2-byte aligned, sampled ones
    against the definition, the memory around them left alone."""
    n, b, c = PAST_CACHE
    print(f"[case] mx past the caches n={n} b={b} c={c} {form}", flush=True)
    X, W = _operands(n, b, c, form)
    buf = torch.full((n + 2, c + 2), 5.0, dtype=BF, device=DEV)
    Y = buf[1:n + 1, 1:c + 1]
    L.mx_linear(X, W, Y=Y)
    rows = sorted({0, 1, 255, 256, n - 1, n - 2, *(int(x) for x in np.linspace(0, n - 1, 300))})
    part = L.MxMatrix(form, X.elements[rows].contiguous(), X.scales[rows].contiguous())
    _check_product(Y[rows], part, W, None, "none", None)
    Y.fill_(5.0)
    assert torch.all(buf == 5.0)


@pytest.mark.parametrize("tile", list(WHOLE))
@pytest.mark.parametrize("form", ["e4m3", "e2m1"])
def test_sums_are_exact_over_the_widest_spans(tile, form):
    """All of one power, all codes of either side. e4m3 X: 448 times 6 beside elements from 2 on
    times 0.5 (2^11.4 beside multiples of 2^-3), 1.875 times 6 beside 2^-9 times 0.5 (2^3.5 beside
    2^-10), and both among the smallest. Every partial sum is a multiple of 2^-10 below 2^14: fp32
    holds each, and so an fp32 Y is exact, whatever the order, and a bf16 one of few tokens (or of an
    e2m1 X, whose products are multiples of 2^-2) is the sum rounded once."""
    n, c = WHOLE[tile]
    b = 640
    print(f"[case] mx exact tile {tile} {form}", flush=True)
    g = np.random.default_rng(n + c)
    w = g.integers(0, 16, (c, b))
    if form == "e4m3":
        x = np.zeros((n, b // 8, 8), dtype=np.int64)
        small = g.integers(1, 8, x.shape)  # multiples of 2^-9
        x[:] = small
        lead = np.arange(b // 8) % 4
        x[:, lead == 0, 3] = 63  # 1.875, the largest of the smaller part
        x[:, lead == 1] = np.where(g.random((n, b // 32, 8)) < 0.9, small[:, lead == 1], g.integers(8, 64, (n, b // 32, 8)))
        x[:, 6] = g.integers(64, 72, (n, 8))  # 2 .. 3.75, the smallest of the larger part
        x[:, 6, 5] = 126  # 448 beside them
        x[:, 46, 1::2] = g.integers(64, 70, (n, 4))
        x[:, 46, 2] = 126
        x[:, 46, 0] = 1  # and beside the very smallest
        x = (x + 128 * g.integers(0, 2, x.shape)).reshape(n, b).astype(np.uint8)
        w = np.where(g.random((c, b)) < 0.5, 1 + 8 * g.integers(0, 2, (c, b)), w)  # half of them 0.5
        w[:, 3::8] = 7 + 8 * g.integers(0, 2, (c, b // 8))  # 6 beside 1.875
        w[:, [6 * 8 + 5, 46 * 8 + 2]] = 7 + 8 * g.integers(0, 2, (c, 2))  # and beside 448
        w[: c // 2, [6 * 8 + 5, 46 * 8 + 2]] = 7
    else:
        x = g.integers(0, 256, (n, b // 2), dtype=np.uint8)
    X, W = L.MxMatrix.empty(n, b, form, DEV), L.MxMatrix.empty(c, b, "e2m1", DEV)
    X.elements.copy_(torch.from_numpy(x))
    W.elements.copy_(torch.from_numpy((w[:, 0::2] | (w[:, 1::2] << 4)).astype(np.uint8)))
    X.scales.fill_(127)
    W.scales.fill_(127)
    xv, wv = _values(X), _values(W)
    ref = xv @ wv.T  # exact in 64 bits
    assert (np.abs(xv) @ np.abs(wv).T).max() < 2.0 ** 14
    got = L.mx_linear(X, W, out_dtype=F32).double().cpu().numpy()
    assert np.array_equal(got, ref), (int((got != ref).sum()), np.abs(got - ref).max())
    if n <= 16 or form == "e2m1":
        assert torch.equal(L.mx_linear(X, W).cpu(), torch.from_numpy(ref).to(BF))


@pytest.mark.parametrize("tile", LARGE + [(64, 64)])
@pytest.mark.parametrize("b", [640, 4096])
def test_what_an_e4m3_input_with_a_bf16_output_loses(tile, b):
    """Over normal data the sums are off by 5e-6 of Y in root mean square. Rounded to bf16, such a
    Y differs from the exact one where a border lies within the error: for normal Y, spacings of 2^-8
    |Y| at least and a mean error of 0.8 x 5e-6, in E min(1, a / |y|) = 0.8 a (0.9 + ln 1/a) = 0.7% of
    the places, a = 0.8 x 5e-6 x 2^8. (fp32's own sums, 2e-7 of Y: 0.04%.)"""
    n, c = WHOLE[tile] if b == 640 else (2500, 1024)
    print(f"[case] mx loss tile {tile} n={n} b={b} c={c}", flush=True)
    X, W = _operands(n, b, c, "e4m3")
    ref = _values(X) @ _values(W).T
    Y = L.mx_linear(X, W).cpu()
    differ = float((Y != torch.from_numpy(ref).to(BF)).double().mean())
    assert differ < 0.008, differ
    off = float(np.sqrt(np.mean((Y.double().numpy() - ref) ** 2)))
    least = float(np.sqrt(np.mean((torch.from_numpy(ref).to(BF).double().numpy() - ref) ** 2)))
    assert off < 1.001 * least, (off, least)
