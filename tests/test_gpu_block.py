"""The block's forward steps run together, as sequential.prune_block_whole uses them."""
import numpy as np
import pytest
import torch

import oracle as O
from layer_wise_obs_amd import _lib as L
from layer_wise_obs_amd import sequential, synth
from tests import test_gpu_attention as A
from tests import test_gpu_linear as T
from tests import test_gpu_norm_rotary as N

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def _weights(b, kv, f, seed):
    shapes = {"q": (b, b), "k": (kv, b), "v": (kv, b), "o": (b, b), "gate": (f, b), "up": (f, b),
              "down": (b, f)}
    return {nm: T._randn(s, seed + i, scale=s[1] ** -0.5) for i, (nm, s) in enumerate(shapes.items())}


def _forward(x, w, ones, freqs, pos, starts, head):
    """One pass of a block, every intermediate kept."""
    r = {}
    n = x.shape[0]
    r["x1"] = L.rms_norm(x, ones)
    for nm in "qkv":
        r[nm] = L.linear(r["x1"], w[nm]).view(n, -1, head)
    r["qr"], r["kr"] = L.rotary(r["q"], r["k"], freqs, positions=pos)
    r["a"] = L.attention(r["qr"], r["kr"], r["v"], starts).view(n, -1)
    r["h"] = L.linear(r["a"], w["o"], residual=x)
    r["x2"] = L.rms_norm(r["h"], ones)
    r["f"] = L.gated_ffn_input(r["x2"], w["gate"], w["up"])
    r["y"] = L.linear(r["f"], w["down"], residual=r["h"])
    return r


def _setup(lens, head, hk, b, f, seed):
    n = sum(lens)
    w = _weights(b, hk * head, f, seed)
    x = T._randn((n, b), seed + 20, scale=2.0)
    pos = np.concatenate([np.arange(v) for v in lens])
    qs = A._starts(lens)
    dev = dict(w={k: v.to(DEV) for k, v in w.items()}, ones=torch.ones(b, dtype=BF, device=DEV),
               freqs=L.rotary_freqs(head, device=DEV),
               pos=torch.tensor(pos, dtype=torch.int32, device=DEV), starts=A._i32(qs), head=head)
    return w, x, pos, qs, dev


def test_block_step_by_step_matches_the_definitions():
    """Every step against the fp64 definition on the inputs it got (the previous step's
    rounded outputs), each within its own tolerance."""
    print("[case] block step by step", flush=True)
    lens, head, hk, b, f = [65, 1, 130, 17], 64, 2, 256, 392
    w, x, pos, qs, dev = _setup(lens, head, hk, b, f, 40)
    r = {k: v.cpu() for k, v in _forward(x.to(DEV), **dev).items()}
    freqs = dev["freqs"].cpu().numpy()
    N._close(r["x1"], O.rms_norm(x, np.ones(b), 1e-5), N._norm_rel(b))
    for nm in "qkv":
        T._check(r[nm].view(sum(lens), -1), r["x1"], w[nm], None, "none", None)
    N._rot_check(r["qr"], r["q"], pos, freqs, "half", 1.0, None, 0)
    N._rot_check(r["kr"], r["k"], pos, freqs, "half", 1.0, None, 0)
    A._check(r["a"].view(sum(lens), -1, head), r["qr"], r["kr"], r["v"], qs, qs)
    T._check(r["h"], r["a"], w["o"], None, "none", x)
    N._close(r["x2"], O.rms_norm(r["h"], np.ones(b), 1e-5), N._norm_rel(b))
    T._check(r["y"], r["f"], w["down"], None, "none", r["h"])


def test_block_decodes_to_the_same_values_as_the_whole_prompt():
    """The last token of each sequence alone, over the others' keys and values, agrees with
    the whole prompt's row: both are within the attention's tolerance of the definition."""
    print("[case] block single tokens", flush=True)
    lens, head, hk, b, f = [200, 3, 129], 64, 2, 256, 392
    _, x, _, qs, dev = _setup(lens, head, hk, b, f, 60)
    r = _forward(x.to(DEV), **dev)
    last = torch.tensor([v - 1 for v in qs[1:]], device=DEV)
    q = r["qr"][last]
    one = L.attention(q, r["kr"], r["v"], A._i32([0, 1, 2, 3]), k_start=dev["starts"])
    A._check(one, q.cpu(), r["kr"].cpu(), r["v"].cpu(), [0, 1, 2, 3], qs)
    step = (2.0 ** -7 + 2.0 ** -7) * r["v"].float().abs().max()
    assert torch.all((one.view(3, -1).float() - r["a"][last].float()).abs() <= step)


def test_block_captured_and_replayed():
    print("[case] block in a graph", flush=True)
    lens, head, hk, b, f = [65, 40], 64, 2, 256, 392
    _, x, _, _, dev = _setup(lens, head, hk, b, f, 80)
    xd = x.to(DEV)
    _forward(xd, **dev)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = _forward(xd, **dev)["y"]
    for seed in (90, 91, 92):
        xd.copy_(T._randn(x.shape, seed, scale=2.0))
        g.replay()
        eager = _forward(xd, **dev)["y"]
        torch.cuda.synchronize()
        assert torch.equal(held, eager)


def _small_config(n=1100, b=256, f=512):
    cfg = synth.Config(9, 12345, BF, BF, 0.06, block=64)
    cfg.streams["attn_in"] = synth.Stream("attn_in", b, n, 3, 20.0, False, 1)
    cfg.layers = [synth.Layer("q_proj", b, b, "attn_in"), synth.Layer("k_proj", 128, b, "attn_in"),
                  synth.Layer("v_proj", 128, b, "attn_in"), synth.Layer("o_proj", b, b, "attn_in"),
                  synth.Layer("gate_proj", f, b, "attn_in"), synth.Layer("up_proj", f, b, "attn_in"),
                  synth.Layer("down_proj", b, f, "attn_in")]
    return cfg


def test_prune_block_whole_composes_the_steps():
    """Each layer's weights are what th_prune_layer gives on the input formed by the steps
    called one by one with the pruned predecessors, bit for bit; so is the block's output."""
    print("[case] prune_block_whole", flush=True)
    cfg = _small_config()
    params = L.make_params(pattern=(2, 4), block=64)
    lines = []
    out, hidden, times = sequential.prune_block_whole(cfg, params, head=64, tokens=256,
                                                      report=lines.append)
    assert len(lines) == 7 and set(out) == {l.name for l in cfg.layers} and len(times) > 10

    def pruned(name, X):
        W = cfg.weights(next(l for l in cfg.layers if l.name == name), device=DEV)
        L.prune_layer(W, X=X.contiguous(), params=params)
        assert torch.equal(W, out[name][0]), name
        return W

    x = cfg.activations("attn_in", device=DEV)
    n = x.shape[0]
    ones = torch.ones(256, dtype=BF, device=DEV)
    x1 = L.rms_norm(x, ones)
    q, k, v = (L.linear(x1, pruned(nm, x1)).view(n, -1, 64) for nm in ("q_proj", "k_proj", "v_proj"))
    pos = (torch.arange(n, device=DEV) % 256).to(torch.int32)
    q, k = L.rotary(q, k, L.rotary_freqs(64, device=DEV), positions=pos)
    a = L.attention(q, k, v, A._i32([0, 256, 512, 768, 1024, 1100])).view(n, -1)
    h = L.linear(a, pruned("o_proj", a), residual=x)
    x2 = L.rms_norm(h, ones)
    f = L.gated_ffn_input(x2, pruned("gate_proj", x2), pruned("up_proj", x2))
    assert torch.equal(hidden, L.linear(f, pruned("down_proj", f), residual=h))
    for W, info in out.values():
        assert torch.all((W.view(W.shape[0], -1, 4) != 0).sum(2) <= 2)


def test_prune_block_whole_refuses_partial_workloads():
    with pytest.raises(ValueError):
        sequential.prune_block_whole(synth.config(3), L.make_params(pattern=(2, 4)))


def test_two_streams_at_once_give_the_serial_results():
    g = torch.Generator().manual_seed(9)
    draw = lambda *s: torch.randn(s, generator=g).to(BF).to(DEV)
    sets = []
    for i in range(2):
        W = draw(1032, 4096)
        X = draw(70 + i, 4096)  # pieces of the contraction, joined through a workspace
        q, k, v = draw(1 + i, 8, 128), draw(9000, 2, 128), draw(9000, 2, 128)  # pieces of the keys
        assert L.linear_workspace_size(*X.shape, W.shape[0]) > 0
        sets.append((X, W, q, k, v))

    def run(X, W, q, k, v):
        starts = [torch.tensor([0, t.shape[0]], dtype=torch.int32).to(DEV) for t in (q, k)]
        return [(L.linear(X, W, act="silu"), L.attention(q, k, v, starts[0], k_start=starts[1]),
                 L.rms_norm(X, W[0])) for _ in range(10)]

    serial = [run(*s)[0] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for s, stream in zip(sets, streams):
        with torch.cuda.stream(stream):
            got.append(run(*s))
    torch.cuda.synchronize()
    for results, want in zip(got, serial):
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
