"""What attention over pages adds to its output's own rounding. The weights enter the second
product as a bf16 value and its rest, also a bf16 value, whatever the number of rows that its
sequence or the others of the call have. bf16 has 8 significant bits, so half a step is 2^-8 of
the value at most (numbers between 1 and 2 are 2^-7 apart): a weight's rest is 2^-8 of it, and what
the rest's own rounding loses 2^-16. Scores and sums are fp32. So an output is off by at most
A (2^-16 + 2 e) before its rounding, A and e as in test_gpu_attention.py, where 2^-8 stands in the place
of 2^-16, and by 2^-8 of itself in it; and over normal data the root mean square of the error is
that of the rounding, to which what is lost adds its square, (2^-8)^2 of it."""
import numpy as np
import pytest
import torch

import oracle as O
from layer_wise_obs_amd import _lib as L
from tests.test_gpu_attention import U, _i32, _randn, _starts
from tests.test_gpu_paged import BF, DEV, Cache

pytestmark = pytest.mark.gpu


def _closer(got, Q, K, V, qs, ks, causal=True):
    d = Q.shape[2]
    ref = O.attention(Q, K, V, qs, ks, causal)
    A = O.attention(Q, K, V.float().abs(), qs, ks, causal)
    size = Q.double().abs().amax((1, 2)).numpy() * K.double().abs().sum(2).max().item() * d ** -0.5
    longest = max(b - a for a, b in zip(ks[:-1], ks[1:]))
    e = size * (2 * (d + 4) + 5) * U + (2 + longest / 2 + 70) * U
    tol = A * (2.0 ** -16 + 2 * e[:, None, None]) * 1.01 + 2.0 ** -8 * np.abs(ref) + 1e-38
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.max(np.abs(g - ref) / tol))
    own = np.sqrt(np.mean((torch.from_numpy(ref).to(BF).double().numpy() - ref) ** 2))
    off = np.sqrt(np.mean((g - ref) ** 2))
    assert off <= 1.01 * own, (off, own)


CASES = [
    ([(300, 300), (65, 65), (1, 1), (130, 700)], 8, 2, 128, 16),
    ([(200, 3000)], 4, 4, 64, 64),  # keys cut into pieces
    ([(70, 150), (40, 400), (0, 5)], 6, 2, 80, 32), ([(129, 129), (40, 555)], 4, 1, 40, 16),
    ([(150, 200)] * 3, 4, 2, 96, 16), ([(150, 200), (64, 1000)], 2, 2, 112, 128), ([(100, 120)] * 2, 2, 1, 24, 16),
    ([(260, 900)], 2, 1, 120, 16), ([(90, 90)], 2, 2, 48, 16),
    ([(400, 700)] + [(1, 600)] * 9, 4, 2, 128, 16),  # a prompt among single tokens
    ([(1, 900)] * 40 + [(50, 800)], 8, 2, 128, 16),  # few rows on average
    ([(40, 90)] * 70, 2, 1, 64, 16)]


@pytest.mark.parametrize("lens,hq,hk,d,page", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_weights_enter_with_their_rest(lens, hq, hk, d, page, causal):
    print(f"[case] paged precision {lens[:4]} hq={hq} hk={hk} d={d} causal={causal}", flush=True)
    qs = _starts([a for a, _ in lens])
    c = Cache([b for _, b in lens], hk, d, page)
    Q = _randn((qs[-1], hq, d), 1, 2.0)
    got = L.paged_attention(Q.to(DEV), *c.dev(), _i32(qs), causal=causal)
    _closer(got, Q, c.K, c.V, qs, c.starts, causal)


@pytest.mark.parametrize("lens", [[(300, 300), (65, 90)], [(200, 2000)], [(3, 700)]])
@pytest.mark.parametrize("d", [64, 128, 72])
def test_infinite_values_that_rows_see(lens, d):
    """An infinity that a row sees stays one, though the rest of its weight may be 0 or of the
    other sign; both signs, or a NaN, give none; other rows and channels keep their precision."""
    print(f"[case] paged infinities seen {lens} d={d}", flush=True)
    hq, hk = 4, 2
    qs = _starts([a for a, _ in lens])
    c = Cache([b for _, b in lens], hk, d, 16)
    n0 = c.k_len[0]
    inf, nan = float("inf"), float("nan")
    for key, h, e, x in ((n0 - 2, 0, 3, inf), (n0 - 2, 0, 9, -inf), (n0 // 2, 0, 4, inf), (n0 // 2, 1, 4, -inf),
                         (0, 0, 6, -inf), (n0 - 3, 1, 7, inf), (n0 - 1, 1, 7, -inf), (n0 - 2, 1, 2, nan)):
        c.v[c.pages[0, key // 16].long(), key % 16, h, e] = x
        c.V[key, h, e] = x
    Q = _randn((qs[-1], hq, d), 12)
    got = L.paged_attention(Q.to(DEV), *c.dev(), _i32(qs)).double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref = O.attention(Q, c.K, c.V, qs, c.starts)
    special = ~np.isfinite(ref)
    assert special.any() and np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    zeros = c.V.float().nan_to_num(0, 0, 0)
    A = O.attention(Q, c.K, zeros.abs(), qs, c.starts)
    tol = A * (2.0 ** -16 + 2.0 ** -13) + 2.0 ** -8 * np.abs(ref) + 1e-38
    with np.errstate(invalid="ignore"):
        assert np.all((np.abs(got - ref) <= tol) | special)
