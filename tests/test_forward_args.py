"""Argument checks of the block's forward steps (linear, row norm, rotary positions, attention),
answered
before anything touches the GPU, and the host-side frequencies of the rotation."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O
from layer_wise_obs_amd import _lib as L

FAKE = 0x100000  # never dereferenced: every call below fails its checks first
NAN, INF = float("nan"), float("inf")


def _norm_args(**kw):
    a = dict(X=FAKE, xdt=L.TH_BF16, n=4, b=64, ldx=64, w=FAKE, eps=1e-5, Y=2 * FAKE,
             ydt=L.TH_BF16, ldy=64)
    a.update(kw)
    return list(a.values()) + [None]


@pytest.mark.parametrize("bad", [
    dict(X=None), dict(Y=None), dict(w=None), dict(xdt=2), dict(ydt=-1), dict(n=-1),
    dict(n=1 << 31), dict(b=0), dict(ldx=63), dict(ldy=63), dict(eps=-1.0), dict(eps=NAN),
    dict(eps=INF), dict(Y=FAKE, ydt=L.TH_F32), dict(Y=FAKE, ldy=128)])
def test_rms_norm_refuses(bad):
    assert L.lib().th_rms_norm(*_norm_args(**bad)) == L.TH_ERR_INVALID_ARG


def _linear_args(**kw):
    a = dict(X=FAKE, ldx=64, W=2 * FAKE, dt=L.TH_BF16, n=4, b=64, c=32, bias=None, act=0,
             residual=None, ldr=0, Y=3 * FAKE, ydt=L.TH_BF16, ldy=32, ws=None, ws_bytes=0)
    a.update(kw)
    return list(a.values()) + [None]


@pytest.mark.parametrize("bad", [
    dict(X=None), dict(W=None), dict(Y=None), dict(dt=L.TH_F32), dict(dt=9), dict(ydt=3),
    dict(n=-1), dict(b=0), dict(b=4, ldx=8), dict(b=60), dict(b=1 << 22, ldx=1 << 22), dict(c=0),
    dict(ldx=56), dict(ldx=68), dict(ldx=1 << 22), dict(ldy=31), dict(act=4), dict(act=-1),
    dict(X=FAKE + 8), dict(W=FAKE + 2), dict(residual=FAKE, ldr=31), dict(n=1 << 37),
    dict(n=1 << 38, c=1, ldy=1), dict(c=1 << 31, ldy=1 << 31),
    dict(residual=3 * FAKE, ldr=64), dict(ws=FAKE + 4, ws_bytes=1 << 20)])
def test_linear_refuses(bad):
    assert L.lib().th_linear(*_linear_args(**bad)) == L.TH_ERR_INVALID_ARG


@pytest.mark.parametrize("n,b,c", [  # a launch has less than 2^32 threads
    (1, 8, 1 << 27), (1 << 31, 8, 8), ((1 << 30) - 960, 8, 8), (1 << 18, 64, 1 << 18),
    (((1 << 24) - 16) * 64 + 1, 8, 64)])
def test_linear_refuses_more_than_a_launch_takes(n, b, c):
    assert L.lib().th_linear(*_linear_args(n=n, b=b, ldx=b, c=c, ldy=c)) == L.TH_ERR_INVALID_ARG
    out = ctypes.c_size_t(0)
    assert (L.lib().th_linear_workspace_size(n, b, c, ctypes.byref(out)) == L.TH_ERR_INVALID_ARG)


@pytest.mark.parametrize("n,b,c", [
    (1, 8, (1 << 27) - 1), (((1 << 24) - 16) * 64, 8, 64), (64, 64, (1 << 27) - 1)])
def test_linear_accepts_what_a_launch_takes(n, b, c):
    assert L.linear_workspace_size(n, b, c) == 0


@pytest.mark.parametrize("call", [
    lambda: L.lib().th_linear(*_linear_args(Y=FAKE, ldy=64)),
    lambda: L.lib().th_linear(*_linear_args(Y=2 * FAKE)),
    lambda: L.lib().th_linear(*_linear_args(bias=3 * FAKE)),
    lambda: L.lib().th_rms_norm(*_norm_args(X=3 * FAKE, Y=FAKE)),
    lambda: _attention(Q=2 * FAKE), lambda: _attention(K=2 * FAKE), lambda: _attention(V=2 * FAKE)])
def test_outputs_that_are_inputs_are_refused(call):
    assert call() == L.TH_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,ok", [
    (dict(nq=8, nseq=(1 << 24) - 1, hq=1, hk=1, o_token=64), True),
    (dict(nq=8, nseq=1 << 23, hq=2, hk=2, o_token=128), False),
    # row blocks of a key head: floor(nq / 128) + 1, times 4: 2^24 - 4, then 2^24
    (dict(nq=(1 << 29) - 129, nk=0, nseq=1, hq=4, hk=4, d=8, o_token=32, o_head=8), True),
    (dict(nq=(1 << 29) - 64, nk=0, nseq=1, hq=4, hk=4, d=8, o_token=32, o_head=8), False),
    (dict(nq=1 << 29, nk=0, nseq=1, hq=4, hk=4, d=8, o_token=32, o_head=8), False),
    (dict(nq=1 << 23, nk=0, nseq=1 << 23, hq=1, hk=1, d=8, o_token=8), True),
    (dict(nq=1 << 28, nk=0, nseq=1 << 23, hq=1, hk=1, d=8, o_token=8), False)])
def test_attention_workgroups_of_a_launch(kw, ok):
    p, out = _attention_params(**kw), ctypes.c_size_t(0)
    got = L.lib().th_attention_workspace_size(ctypes.byref(p), ctypes.byref(out))
    assert got == (L.TH_OK if ok else L.TH_ERR_INVALID_ARG)


def test_linear_workspace_query():
    lib, out = L.lib(), ctypes.c_size_t(0)
    for n, b, c in ((-1, 64, 8), (4, 60, 8), (4, 64, 0), (4, 0, 8)):
        assert lib.th_linear_workspace_size(n, b, c, ctypes.byref(out)) == L.TH_ERR_INVALID_ARG
    assert lib.th_linear_workspace_size(4, 64, 8, None) == L.TH_ERR_INVALID_ARG
    assert L.linear_workspace_size(0, 4096, 4096) == 0
    assert L.linear_workspace_size(131072, 4096, 4096) == 0  # enough tiles: nothing is split
    need = L.linear_workspace_size(70, 4096, 519)
    assert need > 0 and need % (70 * 520 * 4) == 0
    a = dict(n=70, b=4096, ldx=4096, c=519, ldy=519, ws=FAKE)
    assert lib.th_linear(*_linear_args(ws_bytes=need - 1, **a)) == L.TH_ERR_WORKSPACE


def _attention_params(**kw):
    a = dict(nq=6, nk=9, hq=8, hk=2, d=64, q_token=512, q_head=64, k_token=128, k_head=64,
             v_token=128, v_head=64, o_token=512, o_head=64, nseq=2, causal=1, scale=0.125)
    a.update(kw)
    return L.AttentionParams(*a.values())


def _attention(Q=FAKE, K=FAKE, V=FAKE, dt=L.TH_BF16, qs=FAKE, ks=None, O=2 * FAKE, ws=None,
               ws_bytes=0, **kw):
    return L.lib().th_attention(Q, K, V, dt, qs, ks, ctypes.byref(_attention_params(**kw)), O, ws,
                                ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(Q=None), dict(K=None), dict(V=None), dict(O=None), dict(dt=L.TH_F32), dict(Q=FAKE + 8),
    dict(K=FAKE + 2), dict(V=FAKE + 8), dict(O=FAKE + 8), dict(ws=FAKE + 8, ws_bytes=1 << 30),
    dict(qs=None), dict(qs=None, nseq=1, ks=FAKE), dict(nq=-1), dict(nk=-1), dict(nk=1 << 31),
    dict(nq=1 << 62), dict(hq=0), dict(hk=0), dict(hk=3), dict(hq=-8), dict(d=4), dict(d=60),
    dict(d=136, q_head=136, o_head=136, o_token=1088), dict(hq=1 << 17, o_token=1 << 24),
    dict(nseq=0), dict(nseq=1 << 24), dict(q_token=-512), dict(k_head=60), dict(v_token=132),
    dict(k_token=1 << 24), dict(v_token=1 << 30), dict(o_head=56), dict(o_token=504), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN),
    dict(scale=INF), dict(nq=1 << 30, hq=64, hk=8, o_token=4096)])
def test_attention_refuses(bad):
    assert _attention(**bad) == L.TH_ERR_INVALID_ARG


def test_attention_workspace_query():
    lib, out = L.lib(), ctypes.c_size_t(0)
    p = _attention_params(scale=0.0)
    assert lib.th_attention_workspace_size(ctypes.byref(p), ctypes.byref(out)) == L.TH_ERR_INVALID_ARG
    assert lib.th_attention_workspace_size(None, ctypes.byref(out)) == L.TH_ERR_INVALID_ARG
    assert L.attention_workspace_size(_attention_params()) == 0  # short: nothing is split
    long = dict(nq=2, nk=100000)
    need = L.attention_workspace_size(_attention_params(**long))
    assert need > 0 and need % (2 * 8 * (64 + 2) * 4) == 0
    assert _attention(ws=FAKE, ws_bytes=need - 1, **long) == L.TH_ERR_WORKSPACE


def test_no_rows_is_no_work():
    assert _attention(nq=0, Q=None, O=None) == L.TH_OK
    assert L.lib().th_linear(*_linear_args(n=0, X=None, Y=None)) == L.TH_OK
    assert L.lib().th_rms_norm(*_norm_args(n=0, X=None, Y=None)) == L.TH_OK
    h = _heads(x=None, y=None)
    assert L.lib().th_rotary(*_rotary_args(q=h, k=None, n=0)) == L.TH_OK
    h = _heads(x=None, y=None, heads=0)
    assert L.lib().th_rotary(*_rotary_args(q=h, k=h)) == L.TH_OK


def _heads(**kw):
    a = dict(x=FAKE, y=2 * FAKE, norm=None, heads=4, x_token=512, x_head=128, y_token=512,
             y_head=128)
    a.update(kw)
    return L.Heads(*a.values())


def _rotary_args(**kw):
    a = dict(q=_heads(), k=_heads(heads=2), dt=L.TH_BF16, n=3, d=128, rot=128, layout=0,
             pos=None, freqs=FAKE, amp=1.0, eps=1e-6)
    a.update(kw)
    a["q"] = None if a["q"] is None else ctypes.byref(a["q"])
    a["k"] = None if a["k"] is None else ctypes.byref(a["k"])
    return list(a.values()) + [None]


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(dt=5), dict(n=-1), dict(n=(1 << 31) // 6 + 1), dict(d=0), dict(d=257),
    dict(rot=127), dict(rot=130), dict(rot=-2), dict(layout=2), dict(freqs=None), dict(amp=NAN),
    dict(eps=-1e-6), dict(eps=INF), dict(q=_heads(x=None)), dict(k=_heads(y=None)),
    dict(q=_heads(heads=-1)), dict(q=_heads(x_head=-128)),
    dict(q=_heads(y_head=127)), dict(q=_heads(y_token=511)), dict(k=_heads(y_token=0)),
    dict(q=_heads(y=FAKE, y_token=1024))])
def test_rotary_refuses(bad):
    assert L.lib().th_rotary(*_rotary_args(**bad)) == L.TH_ERR_INVALID_ARG


def test_head_major_outputs_are_not_refused_as_overlapping():
    """y as [heads, n, d] (a cache's layout): the checks pass up to the dtype one."""
    h = _heads(y_token=128, y_head=3 * 128)
    assert L.lib().th_rotary(*_rotary_args(q=h, k=None, d=128, n=0)) == L.TH_OK
    h = _heads(y_token=128, y_head=3 * 128 - 1)
    assert L.lib().th_rotary(*_rotary_args(q=h, k=None)) == L.TH_ERR_INVALID_ARG


@pytest.mark.parametrize("rot,kw", [
    (128, {}), (2, {}), (0, {}), (64, dict(base=500000.0)), (96, dict(divide=4.0)),
    (128, dict(base=500000.0, divide=8.0, bands=(8192, 1.0, 4.0))),
    (250, dict(divide=32.0, bands=(2048, 0.0, 2.5)))])
def test_rotary_freqs_match_the_definition(rot, kw):
    """Three roundings of fp64 and the power's own (below 4 units) at most."""
    got = L.rotary_freqs(rot, **kw).numpy()
    ref = O.rotary_freqs(rot, **kw)
    assert got.shape == ref.shape == (rot // 2,)
    assert np.all(np.abs(got - ref) <= 16 * np.finfo(np.float64).eps * ref)


def test_rotary_freqs_bands_keep_fast_pairs_and_divide_slow_ones():
    f = L.rotary_freqs(128, base=500000.0).numpy()
    g = L.rotary_freqs(128, base=500000.0, divide=8.0, bands=(8192, 1.0, 4.0)).numpy()
    turns = 8192 * f / (2 * math.pi)
    assert (turns >= 4).any() and (turns <= 1).any() and ((turns > 1) & (turns < 4)).any()
    assert np.array_equal(g[turns >= 4], f[turns >= 4])
    assert np.array_equal(g[turns <= 1], f[turns <= 1] / 8.0)
    mid = (turns > 1) & (turns < 4)
    assert np.all((g[mid] < f[mid]) & (g[mid] > f[mid] / 8.0))


@pytest.mark.parametrize("rot,kw", [
    (3, {}), (258, {}), (-2, {}), (8, dict(base=0.0)), (8, dict(base=INF)), (8, dict(divide=0.0)),
    (8, dict(divide=NAN)), (8, dict(bands=(0.0, 1.0, 4.0))), (8, dict(bands=(2048, 4.0, 4.0))),
    (8, dict(bands=(2048, -1.0, 4.0))), (8, dict(bands=(NAN, 1.0, 4.0)))])
def test_rotary_freqs_refuses(rot, kw):
    with pytest.raises(L.ThanosError) as e:
        L.rotary_freqs(rot, **kw)
    assert e.value.status == L.TH_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(ValueError):
        L.rms_norm(x, w)
    with pytest.raises(ValueError):
        L.rotary(torch.zeros(2, 1, 8), None, torch.zeros(4, dtype=torch.float64))


@pytest.mark.parametrize("nq,hq,hk,nk", [(1, 1, 1, 1000), (1, 3, 3, 1000), (5, 1, 1, 3000), (2, 8, 2, 9000)])
def test_attention_partial_rows_are_16_byte_aligned(nq, hq, hk, nk):
    """The pieces' (maximum, sum) pairs are followed by their rows of d floats, moved 16 bytes at
    a time: where the pairs are odd in number, their block is rounded up."""
    d = 64
    need = L.attention_workspace_size(_attention_params(nq=nq, nk=nk, hq=hq, hk=hk, nseq=1, o_token=hq * d))
    pieces = need // (nq * hq * (d * 4 + 8))
    assert pieces > 1 and need % 16 == 0
    assert need == -(-pieces * nq * hq * 8 // 16) * 16 + pieces * nq * hq * d * 4


@pytest.mark.parametrize("scale", [1e-300, 1e-46, 8e-39, 2.4e38, 1e300])
def test_attention_refuses_scales_that_fp32_does_not_hold(scale):
    """Times log2(e) they are 0, short of bits or infinite in fp32, where a hidden key's score
    of -inf or a score of 0 would become NaN."""
    assert _attention(scale=scale) == L.TH_ERR_INVALID_ARG
    p, out = _attention_params(scale=scale), ctypes.c_size_t(0)
    assert L.lib().th_attention_workspace_size(ctypes.byref(p), ctypes.byref(out)) == L.TH_ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [8.2e-39, 1e-30, 1e30, 2.35e38])
def test_attention_takes_scales_that_fp32_holds(scale):
    assert L.attention_workspace_size(_attention_params(scale=scale)) == 0


@pytest.mark.parametrize("eps", [1e-300, 1e-46, 1.1e-38, 3.5e38, 1e300])
def test_norms_refuse_eps_that_fp32_does_not_hold(eps):
    """Added in fp32 it would be 0 (a row of zeros: 0 / 0), short of bits or infinite."""
    assert L.lib().th_rms_norm(*_norm_args(eps=eps)) == L.TH_ERR_INVALID_ARG
    assert L.lib().th_rotary(*_rotary_args(eps=eps)) == L.TH_ERR_INVALID_ARG


@pytest.mark.parametrize("eps", [0.0, 1.2e-38, 3.4e38])
def test_norms_take_eps_that_fp32_holds(eps):
    assert L.lib().th_rms_norm(*_norm_args(eps=eps, n=0)) == L.TH_OK
    assert L.lib().th_rotary(*_rotary_args(eps=eps, n=0)) == L.TH_OK


@pytest.mark.parametrize("amp,ok", [(1e39, False), (-1e300, False), (1e-39, False), (INF, False),
                                    (0.0, True), (-3.4e38, True), (1.2e-38, True)])
def test_rotary_amplitude_is_one_that_fp32_holds(amp, ok):
    """Infinite in fp32, it would make NaN of an element of 0."""
    got = L.lib().th_rotary(*_rotary_args(amp=amp, n=0))
    assert got == (L.TH_OK if ok else L.TH_ERR_INVALID_ARG)


@pytest.mark.parametrize("q,k", [
    (dict(x=FAKE, y=FAKE), dict(x=FAKE, y=2 * FAKE)), (dict(x=FAKE, y=2 * FAKE), dict(x=FAKE, y=FAKE)),
    (dict(x=FAKE, y=2 * FAKE), dict(x=3 * FAKE, y=2 * FAKE)),
    (dict(x=FAKE, y=FAKE), dict(x=FAKE, y=FAKE))])
def test_rotary_refuses_outputs_that_the_other_side_uses(q, k):
    """One side would be written while the other is still read, in no fixed order."""
    q, k = _heads(**q), _heads(**k, heads=2)
    assert L.lib().th_rotary(*_rotary_args(q=q, k=k)) == L.TH_ERR_INVALID_ARG
