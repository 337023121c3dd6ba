"""A pruned block as it is served: weights pruned 2:4 and held in 4 bits, the residual stream in
bf16 with 8-bit inputs to the products, a paged cache; prompts in chunks, then single tokens.

Every step is compared with its fp64 definition on the inputs that the library's step before
it gave, within the tolerances of its own tests; the whole against prompts that come at once.
"""
import numpy as np
import pytest
import torch

import oracle as O
from layer_wise_obs_amd import _lib as L
from tests.test_gpu_add_norm import _check as check_norm
from tests.test_gpu_attention import _check as check_attention
from tests.test_gpu_attention import _i32
from tests.test_gpu_mx import _check_product, _check_quantized

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16
HIDDEN, FF, HEADS, KV, D, PAGE = 256, 544, 4, 2, 64, 16


def _randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF)


class Block:
    def __init__(self, rooms, seed=0):
        shapes = {"q": (HEADS * D, HIDDEN), "k": (KV * D, HIDDEN), "v": (KV * D, HIDDEN),
                  "o": (HIDDEN, HEADS * D), "gate": (FF, HIDDEN), "up": (FF, HIDDEN), "down": (HIDDEN, FF)}
        self.w, self.dense = {}, {}
        for i, (name, (c, b)) in enumerate(shapes.items()):
            w = _randn((c, b), seed + i, b ** -0.5).to(DEV)
            x = _randn((4 * b, b), seed + 50 + i).to(DEV)
            L.prune_layer(w, X=x, params=L.make_params(pattern=(2, 4), block=32))
            self.dense[name] = w
            self.w[name] = L.mx_quantize(w, "e2m1")
        self.norms = [(1 + _randn((HIDDEN,), seed + 90 + i, 0.1).float()).to(BF).to(DEV) for i in range(2)]
        self.freqs = L.rotary_freqs(D, device=DEV)
        pages = sum(-(-r // PAGE) for r in rooms)
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(pages, generator=g).int()
        self.table = torch.zeros(len(rooms), max(-(-r // PAGE) for r in rooms), dtype=torch.int32)
        at = 0
        for s, r in enumerate(rooms):
            n = -(-r // PAGE)
            self.table[s, :n] = order[at:at + n]
            at += n
        self.pages = self.table.to(DEV)
        # as new memory may be: nothing of it may enter
        self.k, self.v = (torch.full((pages, PAGE, KV, D), float("nan"), dtype=BF, device=DEV) for _ in range(2))
        self.lens = [0] * len(rooms)

    def step(self, hidden, added, counts, check=False):
        """New tokens of every sequence (counts) through the block: hidden is the residual stream,
        added what the layer before it gave. Returns the stream and what is to be added to it."""
        self.lens = [a + b for a, b in zip(self.lens, counts)]
        n = sum(counts)
        starts = [sum(counts[:i]) for i in range(len(counts) + 1)]
        even = len(set(counts)) == 1 and not check
        q_start, k_len = None if even else _i32(starts), _i32(self.lens)
        positions = _i32([ln - c + i for ln, c in zip(self.lens, counts) for i in range(c)])
        h, x = L.add_rms_norm(hidden, self.norms[0], residual=added, out="e4m3")
        q = L.mx_linear(x, self.w["q"]).view(n, HEADS, D)
        k = L.mx_linear(x, self.w["k"]).view(n, KV, D)
        v = L.mx_linear(x, self.w["v"]).view(n, KV, D)
        q, k = L.rotary(q, k, self.freqs, positions, q_out=q, k_out=k)
        L.cache_store(k, v, self.k, self.v, self.pages, k_len, q_start)
        o = L.paged_attention(q, self.k, self.v, self.pages, k_len, q_start)
        ox = L.mx_quantize(o.view(n, -1), "e4m3")
        a = L.mx_linear(ox, self.w["o"])
        h2, y = L.add_rms_norm(h, self.norms[1], residual=a, out="e4m3")
        f = L.mx_linear(y, self.w["gate"], act="silu") * L.mx_linear(y, self.w["up"])
        fx = L.mx_quantize(f, "e4m3")
        out = L.mx_linear(fx, self.w["down"])
        if check:
            both = (hidden.double() + added.double()).to(BF).cpu()
            assert torch.equal(h.cpu(), both)
            check_norm(x, both, self.norms[0].cpu(), 1e-5)
            # v is not turned: the product's own output
            _check_product(v.view(n, -1), x, self.w["v"], None, "none", None)
            Kc, ks = O.paged_keys(self.k.cpu(), self.table, self.lens)
            Vc, _ = O.paged_keys(self.v.cpu(), self.table, self.lens)
            assert np.isfinite(Kc).all()  # every key of every sequence was stored, in its place
            last = np.concatenate([np.arange(ks[s + 1] - c, ks[s + 1]) for s, c in enumerate(counts)])
            assert np.array_equal(Kc[last], k.double().cpu().numpy())
            assert np.array_equal(Vc[last], v.double().cpu().numpy())
            check_attention(o, q.cpu(), torch.from_numpy(Kc).to(BF), torch.from_numpy(Vc).to(BF), starts, ks)
            _check_quantized(o.view(n, -1).cpu(), "e4m3", ox)
            _check_product(a, ox, self.w["o"], None, "none", None)
            assert torch.equal(h2.cpu(), (h.double() + a.double()).to(BF).cpu())
            check_norm(y, h2.cpu(), self.norms[1].cpu(), 1e-5)
            _check_quantized(f.cpu(), "e4m3", fx)
            _check_product(out, fx, self.w["down"], None, "none", None)
        return h2, out


def test_weights_stay_pruned_in_four_bits():
    """Pruned weights are 0 in 4 bits too, and the others off by half a step at most; what that
    costs the layer is read off its reconstruction error."""
    print("[case] serving weights", flush=True)
    c, b = 96, 256
    w = _randn((c, b), 1, b ** -0.5).to(DEV)
    x = _randn((1024, b), 2).to(DEV)
    before = w.clone()
    L.prune_layer(w, X=x, params=L.make_params(pattern=(2, 4), block=32))
    m = L.mx_quantize(w, "e2m1")
    y = L.mx_dequantize(m)
    assert torch.all((y == 0) | (w != 0))
    step = torch.exp2(m.scales.float() - 127).repeat_interleave(32, 1)
    assert torch.all((y.float() - w.float()).abs() <= torch.maximum(w.float().abs() / 4, step / 4))
    whole, pruned = (L.reconstruction_error(before, z, X=x)[1] for z in (y, w))
    assert pruned < whole < pruned + 0.1


def test_a_block_is_served_in_chunks_and_single_tokens():
    print("[case] serving a block", flush=True)
    rooms = [90, 40, 133]
    block = Block(rooms)
    n = sum(rooms)
    hidden, added = _randn((n, HIDDEN), 7, 2.0), _randn((n, HIDDEN), 8)
    starts = [0, rooms[0], rooms[0] + rooms[1]]
    done, out, stream = [0] * 3, torch.zeros(n, HIDDEN, dtype=BF), torch.zeros(n, HIDDEN, dtype=BF)
    # uneven chunks, a sequence that has none, single tokens among a chunk, then single tokens
    for counts in ([30, 17, 64], [25, 0, 1], [1, 1, 60], [33, 21, 7], [1, 1, 1]):
        rows = torch.cat([torch.arange(s + d, s + d + c) for s, d, c in zip(starts, done, counts)])
        h, o = block.step(hidden[rows].to(DEV), added[rows].to(DEV), counts, check=True)
        stream[rows], out[rows] = h.cpu(), o.cpu()
        done = [a + b for a, b in zip(done, counts)]
    assert done == rooms
    # at once: 8-bit inputs that lie next to a border may go either way with the order of sums
    # (a step of 2^-4 of them), so the two ways are near, not equal
    again = Block(rooms)
    h, o = again.step(hidden.to(DEV), added.to(DEV), rooms)
    for a, b in ((h.cpu(), stream), (o.cpu(), out)):
        d = (a.double() - b.double()).norm() / b.double().norm()
        assert d < 2.0 ** -4, float(d)


def test_single_tokens_replayed_from_a_graph():
    """A step of single tokens captured once and replayed as the cache grows, beside the same steps
    run eagerly in a block of their own."""
    print("[case] serving from a graph", flush=True)
    rooms, first = [70, 45], [20, 31]
    blocks = [Block(rooms, seed=3) for _ in range(2)]
    n = sum(first)
    for b in blocks:
        b.step(_randn((n, HIDDEN), 1).to(DEV), _randn((n, HIDDEN), 2).to(DEV), first)
    b = blocks[0]
    hidden, added = torch.zeros(2, HIDDEN, dtype=BF, device=DEV), torch.zeros(2, HIDDEN, dtype=BF, device=DEV)
    k_len, positions = _i32(first), _i32(first)

    def step():
        h, x = L.add_rms_norm(hidden, b.norms[0], residual=added, out="e4m3")
        q = L.mx_linear(x, b.w["q"]).view(2, HEADS, D)
        k, v = (L.mx_linear(x, b.w[w]).view(2, KV, D) for w in "kv")
        q, k = L.rotary(q, k, b.freqs, positions, q_out=q, k_out=k)
        L.cache_store(k, v, b.k, b.v, b.pages, k_len)
        o = L.paged_attention(q, b.k, b.v, b.pages, k_len)
        a = L.mx_linear(L.mx_quantize(o.view(2, -1), "e4m3"), b.w["o"])
        h, y = L.add_rms_norm(h, b.norms[1], residual=a, out="e4m3")
        f = L.mx_linear(y, b.w["gate"], act="silu") * L.mx_linear(y, b.w["up"])
        return h, L.mx_linear(L.mx_quantize(f, "e4m3"), b.w["down"])

    k_len.add_(1)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    k_len.sub_(1)
    for i in range(14):
        x, y = _randn((2, HIDDEN), 100 + i).to(DEV), _randn((2, HIDDEN), 200 + i).to(DEV)
        hidden.copy_(x)
        added.copy_(y)
        k_len.add_(1)
        positions.copy_(k_len - 1)
        g.replay()
        eager = blocks[1].step(x, y, [1, 1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager[0]) and torch.equal(outs[1], eager[1])
        assert torch.equal(b.k.nan_to_num(9.0), blocks[1].k.nan_to_num(9.0))
