"""Attention over packed sequences against its fp64 definition.

Tolerance: with A = sum p |v| / sum p, an output is off by at most
  A (2^-8 + 2 e) + 2^-8 |o|:
2^-8 for the weights' rounding to bf16 and for the output's own; e for the relative
error of a weight, met in numerator and denominator: the score's sum of d products
(2 (d + 4) roundings of the sum of magnitudes, scaled), the rounding of its product
with scale log2(e) and of the maximum (3 roundings of its size), the exponential
(2 units) and the sums over nk keys in fp32 (each weight enters at most nk / 2 + 70
additions of one lane and the joins).
"""
import numpy as np
import pytest
import torch

import oracle as O
from layer_wise_obs_amd import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
U = 2.0 ** -24


def _randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF)


def _starts(lens):
    return [0] + list(np.cumsum(lens))


def _i32(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device=DEV)


def _check(got, Q, K, V, qs, ks, causal=True, scale=None, rows=None):
    """Rows `rows` (default: every row of a sequence) of got."""
    d = Q.shape[2]
    sc = d ** -0.5 if scale is None else scale
    ref = O.attention(Q, K, V, qs, ks, causal, scale)
    with np.errstate(invalid="ignore"):
        A = O.attention(Q, K, V.float().abs(), qs, ks, causal, scale)
    kf = K.float().abs().nan_to_num(0, 0, 0).numpy()
    qf = Q.float().abs().nan_to_num(0, 0, 0).numpy()
    size = np.max(qf, axis=(1, 2)) * np.max(kf.sum(2), initial=0.0) * sc  # bounds |q||k| scale
    longest = max([b - a for a, b in zip(ks[:-1], ks[1:])] + [1])
    e = size * (2 * (d + 4) + 5) * U + (2 + longest / 2 + 70) * U
    tol = A * (2.0 ** -8 + 2 * e[:, None, None]) * 1.01 + 2.0 ** -8 * np.abs(ref) + 1e-38
    g = got.double().cpu().numpy()
    sel = np.arange(qs[0], qs[-1]) if rows is None else np.asarray(rows)
    g, ref, tol = g[sel], ref[sel], tol[sel]
    special = ~np.isfinite(ref)
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    assert np.array_equal(g[special & ~np.isnan(ref)], ref[special & ~np.isnan(ref)])
    with np.errstate(invalid="ignore"):
        bad = ~special & ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.max((np.abs(g - ref) / tol)[~special]))


CASES = [
    ([(1, 1)], 1, 1, 8), ([(1, 1)], 4, 2, 128), ([(1, 300)], 8, 8, 128), ([(3, 3)], 2, 1, 16),
    ([(64, 64), (65, 65), (0, 0), (1, 1), (130, 130)], 8, 2, 64),
    ([(5, 3), (4, 0), (0, 7), (1, 1), (0, 0)], 4, 4, 64),  # rows that see no key
    ([(1, 1000), (2, 63), (1, 64), (3, 65), (1, 129)], 16, 2, 128),
    ([(1, 5000), (1, 100), (1, 4097), (2, 1)], 8, 2, 128),  # keys split over workgroups
    ([(7, 3000)], 4, 1, 72), ([(300, 300)], 3, 3, 80), ([(200, 1000)], 7, 1, 128),
    ([(33, 33)] * 5, 6, 3, 40), ([(1025, 1025)], 2, 1, 96), ([(17, 9), (9, 17)], 9, 3, 24),
    ([(1, 2)] * 70 + [(2, 5)] * 70, 4, 2, 32),
    ([(40, 20000)], 2, 2, 120),
]


@pytest.mark.parametrize("lens,hq,hk,d", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_definition(lens, hq, hk, d, causal):
    print(f"[case] attention {lens[:5]} hq={hq} hk={hk} d={d} causal={causal}", flush=True)
    qs, ks = _starts([a for a, _ in lens]), _starts([b for _, b in lens])
    Q, K, V = _randn((qs[-1], hq, d), 1, 2.0), _randn((ks[-1], hk, d), 2), _randn((ks[-1], hk, d), 3)
    got = L.attention(Q.to(DEV), K.to(DEV), V.to(DEV), _i32(qs), k_start=_i32(ks), causal=causal)
    _check(got, Q, K, V, qs, ks, causal)


@pytest.mark.parametrize("d", list(range(8, 129, 8)))
@pytest.mark.parametrize("lens", [[(70, 70), (0, 5), (40, 150)], [(1, 75), (2, 2)]])
def test_attention_every_head_size(lens, d):
    print(f"[case] attention lens={lens} d={d}", flush=True)
    qs, ks = _starts([a for a, _ in lens]), _starts([b for _, b in lens])
    Q, K, V = (_randn((n, h, d), d + i) for i, (n, h) in enumerate(
        [(qs[-1], 6), (ks[-1], 2), (ks[-1], 2)]))
    got = L.attention(Q.to(DEV), K.to(DEV), V.to(DEV), _i32(qs), k_start=_i32(ks))
    _check(got, Q, K, V, qs, ks)


def test_attention_default_starts_and_scale():
    """k_start defaults to q_start; without either all rows are one sequence."""
    print("[case] attention defaults", flush=True)
    Q, K, V = _randn((150, 4, 64), 4), _randn((150, 2, 64), 5), _randn((150, 2, 64), 6)
    d = [t.to(DEV) for t in (Q, K, V)]
    _check(L.attention(*d), Q, K, V, [0, 150], [0, 150])
    _check(L.attention(*d, q_start=_i32([0, 70, 150]), scale=0.5), Q, K, V, [0, 70, 150],
           [0, 70, 150], scale=0.5)
    K2, V2 = _randn((9, 2, 64), 7), _randn((9, 2, 64), 8)
    got = L.attention(d[0], K2.to(DEV), V2.to(DEV), causal=False)
    _check(got, Q, K2, V2, [0, 150], [0, 9], causal=False)


def test_attention_no_keys_at_all():
    print("[case] attention without keys", flush=True)
    Q = _randn((5, 2, 64), 9).to(DEV)
    E = torch.empty(0, 1, 64, dtype=BF, device=DEV)
    assert torch.all(L.attention(Q, E, E) == 0)
    assert L.attention(Q[:0], E, E).shape == (0, 2, 64)


@pytest.mark.parametrize("lens", [[(40, 40), (25, 25)], [(1, 9000), (1, 8500)]])
def test_attention_strides_and_rows_of_no_sequence(lens):
    """q, k, v as views of one tensor or a head-major cache; O inside a larger tensor; rows
    before the first and behind the last sequence are left as they were."""
    print(f"[case] attention strides {lens}", flush=True)
    hq, hk, d, front, back = 8, 4, 80, 3, 5
    qs = [front + v for v in _starts([a for a, _ in lens])]
    ks = [7 + v for v in _starts([b for _, b in lens])]
    nq, nk = qs[-1] + back, ks[-1] + 9
    qall = _randn((nq, hq + 6, d + 16), 10)
    cache = _randn((2, hk, nk, d), 11)
    Q, K, V = qall[:, 2:2 + hq, 8:8 + d], cache[0].transpose(0, 1), cache[1].transpose(0, 1)
    cd, qd = cache.to(DEV), qall.to(DEV)
    buf = torch.full((nq, hq + 1, d + 8), 9.0, dtype=BF, device=DEV)
    out = buf[:, :hq, 8:]
    got = L.attention(qd[:, 2:2 + hq, 8:8 + d], cd[0].transpose(0, 1), cd[1].transpose(0, 1),
                      _i32(qs), k_start=_i32(ks), O=out)
    assert got is out
    _check(got, Q, K, V, qs, ks)
    out[front:nq - back] = 9.0
    assert torch.all(buf == 9.0)


@pytest.mark.parametrize("lens", [[(70, 70), (90, 90)], [(3, 5000), (2, 4000)]])
def test_attention_hidden_keys_never_enter(lens):
    """NaN and infinities in keys and values that a query does not see (later ones, other
    sequences', rows of no sequence) leave it as it is; queries that see them get them."""
    print(f"[case] attention hidden non-finite {lens}", flush=True)
    hq, hk, d = 4, 2, 64
    qs, ks = _starts([a for a, _ in lens]), _starts([b for _, b in lens])
    nk = ks[-1] + 30
    Q, K, V = _randn((qs[-1], hq, d), 12), _randn((nk, hk, d), 13), _randn((nk, hk, d), 14)
    K[ks[-1]:], V[ks[-1]:] = float("nan"), float("inf")
    # the first sequence's last two keys: seen by its last (two) queries only
    V[ks[1] - 1, 0, 5] = float("inf")
    V[ks[1] - 1, 1, 7] = float("nan")
    K[ks[1] - 2, 1] = float("nan")
    got = L.attention(Q.to(DEV), K.to(DEV), V.to(DEV), _i32(qs), k_start=_i32(ks))
    _check(got, Q, K, V, qs, ks)
    g = got.float().cpu()
    assert torch.all(g[:qs[1] - 2].isfinite()) and torch.all(g[qs[1]:].isfinite())
    assert torch.all(g[qs[1] - 1, :2, 5] == float("inf")) and torch.all(g[qs[1] - 1, 2:].isnan())


def test_attention_infinite_scores():
    """Scores of -inf weigh nothing; a row that has no others, or one of +inf, has no softmax."""
    print("[case] attention infinite scores", flush=True)
    hq, hk, d, nk = 2, 1, 64, 6000
    for nq in (1, 3):
        Q = _randn((nq, hq, d), 15).abs()
        K, V = _randn((nk, hk, d), 16), _randn((nk, hk, d), 17)
        K[:2500] = float("-inf")  # whole split pieces among them
        qs, ks = [0, nq], [0, nk]
        _check(L.attention(Q.to(DEV), K.to(DEV), V.to(DEV), causal=False), Q, K, V, qs, ks, False)
        K[:] = float("-inf")
        assert torch.all(L.attention(Q.to(DEV), K.to(DEV), V.to(DEV)).isnan())
        K = _randn((nk, hk, d), 16)
        K[100] = float("inf")
        assert torch.all(L.attention(Q.to(DEV), K.to(DEV), V.to(DEV)).isnan())


def test_attention_large_scores_move_the_reference():
    """Scores that grow along the keys, by far more than fp32's exponent range in all."""
    print("[case] attention growing scores", flush=True)
    n, d = 700, 64
    Q = torch.ones(n, 1, d, dtype=BF)
    K = (torch.arange(n).float()[:, None, None] / 8).to(BF).expand(n, 1, d).contiguous()
    V = _randn((n, 1, d), 18)
    for k in (K, K.flip(0).contiguous(), -K):
        _check(L.attention(Q.to(DEV), k.to(DEV), V.to(DEV), scale=1.0), Q, k, V, [0, n], [0, n],
               scale=1.0)


def test_attention_start_values_outside_the_tensors():
    """They are moved to the ends; starts that do not ascend stay inside the tensors too."""
    print("[case] attention bad starts", flush=True)
    Q, K, V = _randn((40, 2, 64), 19), _randn((40, 2, 64), 20), _randn((40, 2, 64), 21)
    d = [t.to(DEV) for t in (Q, K, V)]
    got = L.attention(*d, q_start=_i32([-7, 25, 1000]))
    _check(got, Q, K, V, [0, 25, 40], [0, 25, 40])
    buf = torch.full((60, 2, 64), 9.0, dtype=BF, device=DEV)
    L.attention(*d, q_start=_i32([30, 2 ** 31 - 1, 5, -2 ** 31, 38]), k_start=_i32([9, 3, 50, 1, 0]),
                O=buf[10:50])
    torch.cuda.synchronize()
    assert torch.all(buf[:10] == 9.0) and torch.all(buf[50:] == 9.0)


@pytest.mark.parametrize("lens", [[(130, 130), (1, 70)], [(1, 7000), (1, 100)]])
def test_attention_repeats_with_and_without_workspace_and_on_a_stream(lens):
    print(f"[case] attention repeats {lens}", flush=True)
    qs, ks = _starts([a for a, _ in lens]), _starts([b for _, b in lens])
    Q, K, V = _randn((qs[-1], 8, 128), 22), _randn((ks[-1], 2, 128), 23), _randn((ks[-1], 2, 128), 24)
    d = [t.to(DEV) for t in (Q, K, V)]
    first = L.attention(*d, _i32(qs), k_start=_i32(ks))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = L.attention(*d, _i32(qs), k_start=_i32(ks))
    side.synchronize()
    assert torch.equal(first, again)
    out = torch.empty_like(first)
    p = L.AttentionParams(qs[-1], ks[-1], 8, 2, 128, 1024, 128, 256, 128, 256, 128, 1024, 128,
                          len(lens), 1, 128 ** -0.5)
    qd, kd = _i32(qs), _i32(ks)
    assert L.lib().th_attention(*[L._ptr(t) for t in d], L.TH_BF16, L._ptr(qd), L._ptr(kd), p,
                                L._ptr(out), None, 0, L._stream()) == L.TH_OK
    _check(out, Q, K, V, qs, ks)


def test_attention_captured_and_replayed_with_new_lengths():
    """Single tokens over a cache in a graph: keys, queries and lengths change between
    replays, eager work runs between them."""
    print("[case] attention in a graph", flush=True)
    nseq, room, hq, hk, d = 3, 4000, 8, 2, 128
    Q, K, V = (_randn((nseq, hq, d), 25).to(DEV), _randn((nseq * room, hk, d), 26).to(DEV),
               _randn((nseq * room, hk, d), 27).to(DEV))
    qs, ks = _i32([0, 1, 2, 3]), _i32([0, 10, 20, 30])
    L.attention(Q, K, V, qs, k_start=ks)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = L.attention(Q, K, V, qs, k_start=ks)
    for i, lens in enumerate(([1, 2, 3], [4000, 1, 3999], [64, 65, 4000])):
        ks.copy_(_i32(_starts(lens)))
        Q.copy_(_randn((nseq, hq, d), 30 + i))
        g.replay()
        eager = L.attention(Q, K, V, qs, k_start=ks)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        _check(out, Q.cpu(), K.cpu(), V.cpu(), [0, 1, 2, 3], _starts(lens))


def test_attention_offsets_past_32_bits():
    print("[case] attention keys past 2^32 elements", flush=True)
    n, pitch, d = 600, (1 << 23) + 8, 64
    buf = torch.empty(n * pitch + 2 * d, dtype=BF, device=DEV)
    K = buf.as_strided((n, 1, d), (pitch, d, 1))
    V = buf.as_strided((n, 1, d), (pitch, d, 1), d)
    k, v, q = _randn((n, 1, d), 31), _randn((n, 1, d), 32), _randn((5, 3, d), 33)
    K.copy_(k.to(DEV))
    V.copy_(v.to(DEV))
    _check(L.attention(q.to(DEV), K, V), q, k, v, [0, 5], [0, n])


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("n", [168, 300, 450])
def test_attention_second_pass_with_waves_that_end_early(n, d, causal, value):
    """The last value row is not finite, so the row blocks that meet it (hidden, or behind the
    sequence's end) take a second pass. In the last block some waves have no rows, or none that
    see the last tile (of an odd number, so that it lies in the first buffer): they write their
    rows while the others may still be at it, and none of those may notice."""
    print(f"[case] attention second pass n={n} d={d} causal={causal} {value}", flush=True)
    Q, K, V = _randn((n, 2, d), 40), _randn((n, 2, d), 41), _randn((n, 2, d), 42)
    V[n - 1] = value
    V[n - 1, :, 8:] = 1.0  # the other channels stay finite in every row
    dev = [t.to(DEV) for t in (Q, K, V)]
    first = L.attention(*dev, causal=causal)
    _check(first, Q, K, V, [0, n], [0, n], causal)
    assert torch.all(first[:, :, 8:].isfinite())
    for _ in range(4):
        assert torch.equal(L.attention(*dev, causal=causal).nan_to_num(9.0), first.nan_to_num(9.0))


@pytest.mark.parametrize("nq,h,nk", [(1, 1, 1000), (1, 3, 1100), (3, 5, 3000), (101, 1, 2000)])
def test_attention_odd_numbers_of_partial_rows(nq, h, nk):
    print(f"[case] attention odd partial rows nq={nq} h={h} nk={nk}", flush=True)
    Q, K, V = _randn((nq, h, 128), 50), _randn((nk, h, 128), 51), _randn((nk, h, 128), 52)
    _check(L.attention(*(t.to(DEV) for t in (Q, K, V)), causal=False), Q, K, V, [0, nq], [0, nk], False)


@pytest.mark.parametrize("lens", [[(70, 70), (3, 1)], [(1, 900), (2, 1)]])
def test_attention_smallest_scale_weighs_all_visible_keys_alike(lens):
    print(f"[case] attention smallest scale {lens}", flush=True)
    qs, ks = _starts([a for a, _ in lens]), _starts([b for _, b in lens])
    Q, K, V = _randn((qs[-1], 2, 64), 60), _randn((ks[-1], 1, 64), 61), _randn((ks[-1], 1, 64), 62)
    got = L.attention(Q.to(DEV), K.to(DEV), V.to(DEV), _i32(qs), k_start=_i32(ks), scale=8.2e-39)
    _check(got, Q, K, V, qs, ks, scale=8.2e-39)


@pytest.mark.parametrize("nk", [5, 40, 700])
@pytest.mark.parametrize("d", [64, 72, 128])
def test_attention_single_tokens_weigh_in_more_than_16_bits(nk, d):
    """Single tokens' weights enter the second product as a bf16 value and its rest, 2^-16 of
    themselves at most being left (half a step of half a step). Values of +-1 that mostly
    cancel, so that the output's own rounding hides nothing of it. Small scores: the same
    bound of a weight's fp32 error as everywhere is then about 2^-13."""
    print(f"[case] attention weights nk={nk} d={d}", flush=True)
    nseq, h = 60, 4
    qs, ks = list(range(nseq + 1)), [nk * i for i in range(nseq + 1)]
    Q, K = _randn((nseq, h, d), 70, 0.5), _randn((nk * nseq, h, d), 71, 0.25)
    V = torch.ones(nk * nseq, h, d, dtype=BF)
    V[1::2] = -1.0
    V[:, :, 1::2] *= -1.0
    got = L.attention(Q.to(DEV), K.to(DEV), V.to(DEV), _i32(qs), k_start=_i32(ks)).double().cpu().numpy()
    ref = O.attention(Q, K, V, qs, ks)
    size = float(Q.float().norm(dim=2).max() * K.float().norm(dim=2).max()) * d ** -0.5
    e = size * (2 * (d + 4) + 5) * U + (2 + nk / 2 + 70) * U
    tol = 2.0 ** -16 + 2 * e + 2.0 ** -8 * np.abs(ref)  # sum p |v| / sum p is 1
    assert e < 2.0 ** -13
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("lens", [[(1, 100), (2, 31)], [(1, 6000), (3, 5000)]])
def test_attention_single_tokens_over_values_that_are_not_finite(lens, d, value):
    """A visible infinity stays one (times a weight, whose rest may be 0 or negative), in its
    channel alone; hidden ones enter nowhere."""
    print(f"[case] attention visible non-finite {lens} d={d} {value}", flush=True)
    qs, ks = _starts([a for a, _ in lens]), _starts([b for _, b in lens])
    Q, K, V = _randn((qs[-1], 4, d), 73), _randn((ks[-1], 2, d), 74), _randn((ks[-1], 2, d), 75)
    V[10, 0, 3] = value           # seen by the first sequence
    V[ks[-1] - 1, 1, 9] = value   # by the second one's last token only
    got = L.attention(Q.to(DEV), K.to(DEV), V.to(DEV), _i32(qs), k_start=_i32(ks))
    _check(got, Q, K, V, qs, ks)
    fin = got.isfinite().cpu()
    want = torch.ones_like(fin)
    want[0, :2, 3] = want[-1, 2:, 9] = False
    assert torch.equal(fin, want)


@pytest.mark.parametrize("lens,hq,hk,d", [
    ([(1, 700)] * 20 + [(400, 400)] + [(1, 90)] * 43, 2, 2, 64),  # averages below 32 rows
    ([(1, 33)] * 9 + [(3, 9000)] + [(0, 50)] * 3, 8, 2, 128),     # pieces by a short average
    ([(1, 100)] * 31 + [(1, 20000)] + [(1, 1)] * 32, 16, 2, 128),
    ([(600, 700), (1, 1), (1, 5000)], 4, 1, 80)])                 # averages above
def test_attention_sequences_far_from_their_average(lens, hq, hk, d):
    """A prompt among single tokens, and lengths a factor of 200 apart: the kernel and the number
    of pieces follow the average lengths, the results must not."""
    print(f"[case] attention uneven {len(lens)} sequences hq={hq} hk={hk} d={d}", flush=True)
    qs, ks = _starts([a for a, _ in lens]), _starts([b for _, b in lens])
    Q, K, V = _randn((qs[-1], hq, d), 80, 2.0), _randn((ks[-1], hk, d), 81), _randn((ks[-1], hk, d), 82)
    _check(L.attention(Q.to(DEV), K.to(DEV), V.to(DEV), _i32(qs), k_start=_i32(ks)), Q, K, V, qs, ks)


def test_attention_calibration_size():
    """16 sequences of 2048 tokens, 32 heads of 128: several rounds of workgroups. Sampled rows
    against fp64, each alone: its query over the keys that it sees."""
    print("[case] attention 16 x 2048, 32 heads of 128", flush=True)
    n, seqs, h, d = 2048, 16, 32, 128
    g = torch.Generator(device=DEV).manual_seed(90)
    Q, K, V = (torch.randn(seqs * n, h, d, generator=g, device=DEV).to(BF) for _ in range(3))
    got = L.attention(Q, K, V, _i32([n * i for i in range(seqs + 1)]))
    for s, i in ((0, 0), (0, 63), (3, 1000), (7, 127), (7, 128), (11, 2047), (15, 1), (15, 2047)):
        a = s * n
        k, v = K[a:a + i + 1].cpu(), V[a:a + i + 1].cpu()
        _check(got[a + i:a + i + 1], Q[a + i:a + i + 1].cpu(), k, v, [0, 1], [0, i + 1])
    assert torch.all(got.isfinite())
    again = L.attention(Q, K, V, _i32([n * i for i in range(seqs + 1)]))
    assert torch.equal(got, again)
