"""Row norm and rotary positions against their fp64 definitions.

Tolerances count roundings: an output is off by at most half a step of its type,
the fp32 arithmetic before it by the roundings listed at each check.
"""
import numpy as np
import pytest
import torch

import oracle as O
from layer_wise_obs_amd import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24  # one fp32 rounding, relative


def _randn(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def _close(got, ref, rel, extra=0.0):
    """|got - ref| <= half a step of got's type + rel |ref| + extra."""
    half = torch.finfo(got.dtype).eps / 2
    g = got.double().cpu().numpy()
    tol = (half * (1 + rel) + rel) * np.abs(ref) + extra + 1e-38
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.max(np.abs(g - ref) / np.maximum(tol, 1e-300)))


def _norm_rel(b):
    """Sum of squares: a thread adds at most 8 ceil(b / 512) + 8 products (64 threads for
    up to 1024 columns, 256 above: never more), then 6 lane and 4 wave steps; the mean,
    eps and the root halve; root, reciprocal and two products round once each."""
    return (0.5 * (8 * -(-b // 512) + 8 + 10 + 2) + 4) * U


@pytest.mark.parametrize("xdt,ydt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("n,b", [(1, 1), (3, 7), (5, 8), (2, 520), (4, 1024), (3, 1032), (7, 4096),
                                 (300, 257), (2, 8192), (2, 8200), (3, 20001), (1, 28672)])
def test_rms_norm_matches_definition(n, b, xdt, ydt):
    print(f"[case] rms norm n={n} b={b} {xdt}->{ydt}", flush=True)
    X, w = _randn((n, b), b, xdt, 3.0), _randn((b,), b + 1, xdt)
    Y = L.rms_norm(X.to(DEV), w.to(DEV), eps=1e-5, out_dtype=ydt)
    assert Y.dtype == ydt
    _close(Y, O.rms_norm(X, w, 1e-5), _norm_rel(b))


def test_rms_norm_strides_alignment_and_rows_left_alone():
    print("[case] rms norm strided", flush=True)
    for off, b, pitch in ((0, 64, 72), (1, 64, 72), (0, 65, 67), (8, 128, 168)):
        buf = _randn((6, pitch + off), 3, BF).to(DEV)
        X = buf[:, off:off + b]
        out = torch.full((8, pitch + 16), 7.0, dtype=BF, device=DEV)
        L.rms_norm(X, torch.ones(b, dtype=BF, device=DEV), eps=0.0, Y=out[1:7, 8:8 + b])
        _close(out[1:7, 8:8 + b], O.rms_norm(X, np.ones(b), 0.0), _norm_rel(b))
        out[1:7, 8:8 + b] = 7.0
        assert torch.all(out == 7.0)


@pytest.mark.parametrize("b", [96, 9000, 77])
def test_rms_norm_in_place_equals_out_of_place(b):
    print(f"[case] rms norm in place b={b}", flush=True)
    X, w = _randn((9, b), 5, F32).to(DEV), _randn((b,), 6, F32).to(DEV)
    Y = L.rms_norm(X, w)
    assert L.rms_norm(X, w, Y=X) is X and torch.equal(X, Y)


def test_rms_norm_zero_rows_and_infinities():
    print("[case] rms norm zeros, inf, nan", flush=True)
    X = torch.ones(5, 1032, dtype=F32)
    X[1] = 0.0
    X[2, 7] = float("inf")
    X[3, 1031] = float("nan")
    Y = L.rms_norm(X.to(DEV), torch.ones(1032, dtype=F32, device=DEV), eps=1e-5).cpu()
    assert torch.all(Y[1] == 0) and torch.all(Y[3].isnan())
    assert Y[2, 7].isnan() and torch.all(Y[2, :7] == 0)
    _close(Y[[0, 4]], np.full((2, 1032), 1 / np.sqrt(1 + 1e-5)), _norm_rel(1032))


def _rot_check(got, x, pos, freqs, layout, amp, norm, eps):
    """(cos, sin): the angle in half turns is rounded to fp32 (pi U), sine and cosine are
    good to 2 units (4 U), amplitude and the two products and the sum round once each:
    10 U of the pair's size. A norm adds 8 + 5 sums and 2 more, halved, and 4 U. Positions
    of p turns lose 3 fp64 roundings of p f."""
    y = O.rotary(x, pos, freqs, layout, amp, norm, eps)
    z = O.rotary(x, np.zeros(len(pos)), freqs, layout, 1.0, norm, eps)
    half, d = len(freqs), z.shape[2]
    e = np.arange(d)
    mate = e.copy()
    if layout == "half":
        mate[:half], mate[half:2 * half] = e[half:2 * half], e[:half]
    else:
        mate[:2 * half] = e[:2 * half] ^ 1
    size = np.abs(z) + np.where(mate != e, np.abs(z[:, :, mate]), 0.0)
    size[:, :, :2 * half] *= max(1.0, abs(amp))
    rel = (10 + (0 if norm is None else 0.5 * 15 + 4)) * U
    far = np.zeros(len(pos))
    if half:
        far = np.abs(np.asarray(pos, dtype=np.float64)) * np.max(freqs) * 3 * 2.0 ** -53
    _close(got, y, U, size * (rel + far[:, None, None]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,hq,hk,d,rot,normed", [
    (1, 1, 0, 2, 2, False), (3, 2, 1, 6, 4, True), (5, 32, 8, 128, 128, False),
    (5, 32, 8, 128, 128, True), (300, 4, 4, 64, 32, True), (33, 7, 1, 80, 48, False),
    (2, 3, 2, 256, 256, True), (9, 5, 5, 72, 72, True), (70, 1, 1, 96, 0, True),
    (40, 24, 4, 96, 48, True), (17, 2, 2, 130, 130, False), (1000, 1, 0, 8, 8, True)])
def test_rotary_matches_definition(n, hq, hk, d, rot, normed, layout, dtype):
    print(f"[case] rotary n={n} hq={hq} hk={hk} d={d} rot={rot} {layout} {dtype}", flush=True)
    qkv = _randn((n, hq + 2 * hk, d), n + d, dtype)
    dev = qkv.to(DEV)
    q, k = dev[:, :hq], (dev[:, hq:hq + hk] if hk else None)
    pos = torch.randint(0, 100000, (n,), generator=torch.Generator().manual_seed(n),
                        dtype=torch.int32)
    freqs = L.rotary_freqs(rot, base=500000.0, divide=8.0, bands=(8192, 1.0, 4.0))
    wq = _randn((d,), 8, dtype) if normed else None
    wk = _randn((d,), 9, dtype) if normed and hk else None
    qo, ko = L.rotary(q, k, freqs.to(DEV), positions=pos.to(DEV), layout=layout, amplitude=1.25,
                      q_norm=None if wq is None else wq.to(DEV),
                      k_norm=None if wk is None else wk.to(DEV), eps=1e-6)
    assert torch.equal(dev.cpu(), qkv)
    _rot_check(qo, qkv[:, :hq], pos.numpy(), freqs.numpy(), layout, 1.25, wq, 1e-6)
    if hk:
        _rot_check(ko, qkv[:, hq:hq + hk], pos.numpy(), freqs.numpy(), layout, 1.25, wk, 1e-6)
    else:
        assert ko is None


@pytest.mark.parametrize("d", [128, 20])
def test_rotary_default_positions_in_place_and_cache_layout(d):
    """Positions default to the row index; in place equals out of place; k written head by
    head into a cache [heads, room, d] leaves the cache's other rows alone."""
    print(f"[case] rotary in place, cache layout d={d}", flush=True)
    n, hq, hk = 21, 6, 3
    qkv = _randn((n, hq + 2 * hk, d), 4, BF).to(DEV)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    freqs = L.rotary_freqs(d, device=DEV)
    cache = torch.full((hk, 64, d), 3.0, dtype=BF, device=DEV)
    qo, ko = L.rotary(q, k, freqs, k_out=cache[:, 10:10 + n].transpose(0, 1))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    q2, k2 = L.rotary(q, k, freqs, positions=pos)
    assert torch.equal(qo, q2) and torch.equal(cache[:, 10:10 + n].transpose(0, 1), k2)
    assert torch.all(cache[:, :10] == 3.0) and torch.all(cache[:, 10 + n:] == 3.0)
    v = qkv[:, hq + hk:].clone()
    L.rotary(q, k, freqs, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, k2) and torch.equal(qkv[:, hq + hk:], v)


def test_rotary_far_and_negative_positions():
    print("[case] rotary far positions", flush=True)
    pos = torch.tensor([0, -1, 1, -100000, 1000000, 2 ** 31 - 1, -2 ** 31, 12345678],
                       dtype=torch.int32)
    x = _randn((8, 2, 64), 5, F32)
    freqs = L.rotary_freqs(64)
    for layout in ("half", "interleaved"):
        y, _ = L.rotary(x.to(DEV), None, freqs.to(DEV), positions=pos.to(DEV), layout=layout)
        _rot_check(y, x, pos.numpy(), freqs.numpy(), layout, 1.0, None, 1e-6)
        assert torch.equal(y[0].cpu(), x[0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary_keeps_infinities_of_the_unturned_part_and_of_other_heads(dtype):
    print("[case] rotary infinities", flush=True)
    x = _randn((4, 3, 64), 6, dtype)
    x[1, 1, 50] = float("inf")
    x[2, 0, 3] = float("nan")
    freqs = L.rotary_freqs(32)
    y, _ = L.rotary(x.to(DEV), None, freqs.to(DEV))
    y = y.cpu()
    assert torch.equal(y[:, :, 32:], x[:, :, 32:])
    bad = ~y.isfinite()
    want = torch.zeros_like(bad)
    want[1, 1, 50] = want[2, 0, 3] = want[2, 0, 19] = True
    assert torch.equal(bad, want)


def test_strides_past_32_bits_and_another_stream():
    """A row pitch that takes the last row past 2^32 elements, on a stream of its own."""
    print("[case] rows past 2^32 elements", flush=True)
    n, pitch, d = 5, (1 << 30) + 8, 64
    buf = torch.empty(n * pitch, dtype=BF, device=DEV)
    x = buf.as_strided((n, 1, d), (pitch, d, 1))
    src = _randn((n, 1, d), 7, BF)
    x.copy_(src.to(DEV))
    freqs = L.rotary_freqs(d, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, _ = L.rotary(x, None, freqs)
        z = L.rms_norm(x[:, 0], torch.ones(d, dtype=BF, device=DEV), eps=1e-5)
    side.synchronize()
    _rot_check(y, src, np.arange(n), freqs.cpu().numpy(), "half", 1.0, None, 1e-6)
    _close(z, O.rms_norm(src[:, 0], np.ones(d), 1e-5), _norm_rel(d))


def test_rms_norm_more_rows_than_a_launch_takes():
    n, b = (1 << 24) + 3, 8
    X = torch.empty(n, b, dtype=BF, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    w = torch.arange(1, b + 1, dtype=BF, device=DEV)
    Y = L.rms_norm(X, w)
    for a in (0, (1 << 23) - 2, 1 << 23, (1 << 24) - 2, n - 4):  # ends of the launches' ranges
        _close(Y[a:a + 4], O.rms_norm(X[a:a + 4].cpu(), w.cpu(), 1e-5), _norm_rel(b))
    # every other row against the same call on a part
    half = L.rms_norm(X[n // 2:], w)
    assert torch.equal(Y[n // 2:], half)


@pytest.mark.parametrize("d,n", [(6, (1 << 24) + 5), (8, (1 << 28) + 21)])
def test_rotary_more_tokens_than_a_launch_takes(d, n):
    x = torch.empty(n, 1, d, dtype=BF, device=DEV)
    x[:] = torch.arange(1, d + 1, device=DEV).to(BF)
    freqs = L.rotary_freqs(2, device=DEV)  # one pair, one radian a position
    y, _ = L.rotary(x, None, freqs, q_out=x)
    step = 1 << (23 if d == 6 else 27)
    for a in (0, step - 2, step, 2 * step - 2, n - 4):
        p = torch.arange(a, a + 4, dtype=torch.float64)
        want = torch.stack([p.cos() - 2 * p.sin(), 2 * p.cos() + p.sin()], 1)
        got = y[a:a + 4, 0].double().cpu()
        # the angle in turns is off by 2^-53 of itself, the sine and cosine by 2^-21 with it,
        # the two products by three roundings, the output by half a step
        assert ((got[:, :2] - want).abs() <= 2.0 ** -8 * want.abs() + 3 * 2.0 ** -20).all()
        assert torch.equal(got[:, 2:], torch.arange(3, d + 1, dtype=torch.float64).expand(4, -1))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,hq,hk,d,rot,normed", [
    (7, 9, 2, 88, 88, True), (5, 3, 1, 32, 28, True), (33, 2, 2, 64, 62, False),
    (4, 2, 1, 40, 40, False), (12, 3, 1, 256, 250, True), (300, 1, 1, 8, 6, True),
    (9, 5, 5, 104, 2, False), (3, 65, 3, 128, 126, True), (40, 4, 2, 136, 136, False)])
def test_rotary_pairs_and_rows_of_any_alignment(n, hq, hk, d, rot, normed, layout, dtype):
    print(f"[case] rotary n={n} hq={hq} hk={hk} d={d} rot={rot} {layout} {dtype}", flush=True)
    h = hq + hk
    x = _randn((n, h * d + 3), n + d, dtype)  # odd token pitch, first element at 1
    heads = lambda t: t[:, 1:1 + h * d].unflatten(1, (h, d))
    dev = x.to(DEV)
    q, k = heads(dev)[:, :hq], heads(dev)[:, hq:]
    out = torch.full((n, h * d + 5), 7.0, dtype=dtype, device=DEV)
    at = out[:, 3:3 + h * d].unflatten(1, (h, d))
    pos = torch.randint(0, 100000, (n,), generator=torch.Generator().manual_seed(n),
                        dtype=torch.int32)
    freqs = L.rotary_freqs(rot, base=500000.0)
    w = _randn((d,), 8, dtype) if normed else None
    dw = None if w is None else w.to(DEV)
    L.rotary(q, k, freqs.to(DEV), positions=pos.to(DEV), layout=layout, amplitude=0.75, q_norm=dw,
             k_norm=dw, eps=1e-6, q_out=at[:, :hq], k_out=at[:, hq:])
    _rot_check(at[:, :hq], heads(x)[:, :hq], pos.numpy(), freqs.numpy(), layout, 0.75, w, 1e-6)
    _rot_check(at[:, hq:], heads(x)[:, hq:], pos.numpy(), freqs.numpy(), layout, 0.75, w, 1e-6)
    assert bool((out[:, :3] == 7).all()) and bool((out[:, 3 + h * d:] == 7).all())
    same = dev.clone()  # in place
    L.rotary(heads(same)[:, :hq], heads(same)[:, hq:], freqs.to(DEV), positions=pos.to(DEV),
             layout=layout, amplitude=0.75, q_norm=dw, k_norm=dw, eps=1e-6,
             q_out=heads(same)[:, :hq], k_out=heads(same)[:, hq:])
    assert torch.equal(heads(same), at)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norms_of_zeros_at_the_smallest_eps(dtype):
    print(f"[case] norms of zeros, smallest eps {dtype}", flush=True)
    x, w = torch.zeros(3, 2, 64, dtype=dtype, device=DEV), torch.ones(64, dtype=dtype, device=DEV)
    assert torch.all(L.rms_norm(x[:, 0], w, eps=1.2e-38) == 0)
    y, _ = L.rotary(x, None, L.rotary_freqs(64, device=DEV), q_norm=w, eps=1.2e-38)
    assert torch.all(y == 0)


@pytest.mark.parametrize("d", [16, 10])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_small_sines_and_cosines_keep_their_bits(d, layout):
    """Pairs of (1, 0) become (cos, sin) themselves: each is formed in fp64 (good to a few units
    there) from an angle that is off by 3 roundings of itself, and rounded once."""
    print(f"[case] rotary sines and cosines d={d} {layout}", flush=True)
    n, pairs = 5000, d // 2
    x = torch.zeros(n, 1, d, dtype=F32)
    first = slice(0, pairs) if layout == "half" else slice(0, d, 2)
    second = slice(pairs, d) if layout == "half" else slice(1, d, 2)
    x[:, :, first] = 1.0
    pos = torch.randint(-100000, 100000, (n,), generator=torch.Generator().manual_seed(3),
                        dtype=torch.int32)
    freqs = torch.tensor(([1.0, 0.37, np.pi / 64, 1e-4, 2.0, 1e-6, 0.05, 1.5])[:pairs],
                         dtype=torch.float64)
    y, _ = L.rotary(x.to(DEV), None, freqs.to(DEV), positions=pos.to(DEV), layout=layout)
    angle = pos.numpy().astype(np.longdouble)[:, None] * freqs.numpy().astype(np.longdouble)
    got = y[:, 0].double().cpu().numpy()
    far = 3 * 2.0 ** -53 * np.abs(angle).astype(np.float64) + 2.0 ** -50
    for part, ref in ((first, np.cos(angle)), (second, np.sin(angle))):
        ref = ref.astype(np.float64)
        tol = U * np.abs(ref) + 1.01 * far
        err = np.abs(got[:, part] - ref)
        assert np.all(err <= tol), np.max(err / tol)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rms_norm_scale_is_rounded_once(dtype):
    """Rows (1, k, 0 ..): their sum of squares and its mean (of 2^m columns) are exact in fp32, so
    the output of the 1 is the scale itself, within half a step of fp32 (and what the last
    correction leaves, 2^-45)."""
    print(f"[case] rms norm scale {dtype}", flush=True)
    for b in (2, 64, 2048):
        k = torch.arange(1, 257 if dtype == BF else 4096, dtype=torch.float32)
        X = torch.zeros(k.numel(), b, dtype=dtype)
        X[:, 0], X[:, 1] = 1.0, k.to(dtype)
        Y = L.rms_norm(X.to(DEV), torch.ones(b, dtype=dtype, device=DEV), eps=0.0, out_dtype=F32)
        ref = 1.0 / np.sqrt((1.0 + k.double().numpy() ** 2) / b)
        err = np.abs(Y[:, 0].double().cpu().numpy() - ref)
        assert np.all(err <= (U + 2.0 ** -44) * ref), np.max(err / ref) / U
