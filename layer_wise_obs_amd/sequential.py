"""One transformer block pruned in order, with shared factors and the feed-forward
input propagated from the pruned layers; or, with --whole, every layer's input.

Usage: python -m layer_wise_obs_amd.sequential [--config 4] [--pattern 2:4] [--whole]

"Pruning LLMs with Thanos", section "The layer-reconstruction lens": every linear
layer is reconstructed from its own calibration inputs; layers that read the same
input (q/k/v; gate/up) share one Hessian, so its factor U (H^-1 = U^T U) is
computed once (th_factor) and each of them is pruned from it
(th_prune_layer_factored). down_proj's input is not an independent stream: it is
produced by the pruned gate and up projections through the gated feed-forward
(th_gated_ffn_input, section "The compression target: linear layers"), and down
is pruned on the Hessian of that input. In prune_block the attention output
feeding o_proj and the feed-forward's input stay independent synthetic streams.

prune_block_whole reads one stream, the residual stream before the block, and
forms every layer's input from it with the block's own forward steps: the row norm
(th_rms_norm), q, k and v from their pruned projections (th_linear), rotary
positions (th_rotary), causal attention within each calibration sequence
(th_attention), o_proj added to the residual stream, and the same for the
feed-forward. It returns the residual stream behind the pruned block, which is the
next block's input.

Every step runs in the HIP library; this module only orders the calls, owns the
tensors and prints one JSON line per layer plus a summary.
"""
from __future__ import annotations

import argparse
import json
import time

import torch

from . import _lib as L
from . import synth

DEV = "cuda:0"


def _sync_ms(t0):
    torch.cuda.synchronize()
    return (time.perf_counter() - t0) * 1e3


def _params(cfg, pattern):
    if pattern is None:
        p = cfg.patterns[0]
        if p[0] == "unstructured":
            return L.make_params(sparsity=p[1], block=cfg.block, lam=cfg.lambda_rel)
        return L.make_params(pattern=(p[1], p[2]), block=cfg.block, lam=cfg.lambda_rel)
    return L.make_params(pattern=pattern, block=cfg.block, lam=cfg.lambda_rel)


def _stream_x(cfg, name):
    s = cfg.streams[name]
    X = torch.empty((s.n, s.b), dtype=cfg.xdtype, device=DEV)
    cfg.activations(name, device=DEV, out=X)
    torch.cuda.synchronize()  # generation is not part of any timed phase
    return X


def _group_pruner(cfg, params, out, times, report):
    """prune_group(X, names, tag): the named layers pruned on the one input X."""
    layers = {l.name: l for l in cfg.layers}

    def prune_group(X, names, tag):
        t0 = time.perf_counter()
        U, lam = L.factor(X=X, lam=cfg.lambda_rel, relative=True)
        times[f"factor {tag}"] = round(_sync_ms(t0), 3)
        for nm in names:
            W = cfg.weights(layers[nm], device=DEV)
            W0 = W.clone()
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            info = L.prune_layer_factored(W, U, params=params)
            times[nm] = round(_sync_ms(t0), 3)
            _, er = L.reconstruction_error(W0, W, X=X)
            out[nm] = (W, info)
            report(json.dumps({"layer": nm, "c": W.shape[0], "b": W.shape[1],
                               "input": tag, "E_rel": er, "pruned": info["pruned"],
                               "ms": times[nm]}))
        del U

    return prune_group


def prune_block(cfg, params, propagate=True, report=print):
    """Prune the block's layers in order. Returns {layer: (W_hat bf16, info)} and the
    timing of each phase in ms."""
    layers = {l.name: l for l in cfg.layers}
    out, times = {}, {}
    prune_group = _group_pruner(cfg, params, out, times, report)
    X = _stream_x(cfg, "attn_in")
    prune_group(X, [n for n in ("q_proj", "k_proj", "v_proj") if n in layers], "attn_in")
    del X
    X = _stream_x(cfg, "o_in")
    prune_group(X, ["o_proj"], "o_in")
    del X
    X = _stream_x(cfg, "mlp_in")
    prune_group(X, ["gate_proj", "up_proj"], "mlp_in")
    if propagate:
        t0 = time.perf_counter()
        Xd = L.gated_ffn_input(X, out["gate_proj"][0], out["up_proj"][0])
        times["gated ffn"] = round(_sync_ms(t0), 3)
        tag = "gated(mlp_in)"
    else:
        Xd, tag = _stream_x(cfg, "down_in"), "down_in"
    del X
    prune_group(Xd, ["down_proj"], tag)
    return out, times


def attention_output(X, Wq, Wk, Wv, head, starts, freqs):
    """What o_proj reads, [n, hq * head], from the (normed) block input X [n, b] and the three
    projections: heads of `head` elements at rotary positions counted within each sequence,
    sequences at starts (int32, device), causal attention."""
    n = X.shape[0]
    q, k, v = (L.linear(X, W).view(n, -1, head) for W in (Wq, Wk, Wv))
    rows = torch.arange(n, dtype=torch.int32, device=X.device)
    seq = torch.searchsorted(starts[1:], rows, right=True).clamp_(max=starts.numel() - 2)
    L.rotary(q, k, freqs, positions=rows - starts[seq], q_out=q, k_out=k)
    return L.attention(q, k, v, starts).view(n, -1)


def prune_block_whole(cfg, params, head=128, tokens=2048, eps=1e-5, report=print):
    """Prune the block's seven layers in order, each on the input that the block's own
    forward steps and its pruned predecessors produce from the stream "attn_in", taken as
    the residual stream before the block (calibration sequences of `tokens` tokens, the
    last one shorter where they do not divide it; unit norm weights; rotary base 10000).
    Returns {layer: (W_hat bf16, info)}, the residual stream behind the block and the
    timing of each phase in ms."""
    names = [l.name for l in cfg.layers]
    needed = ("q_proj", "k_proj", "v_proj", "o_proj", "gate_proj", "up_proj", "down_proj")
    if any(nm not in names for nm in needed):
        raise ValueError(f"the workload lacks layers of a whole block: has {names}")
    if cfg.xdtype != torch.bfloat16 or cfg.wdtype != torch.bfloat16:
        raise ValueError("the forward steps take bf16 weights and activations")
    out, times = {}, {}
    prune_group = _group_pruner(cfg, params, out, times, report)

    def timed(tag, fn, *args, **kw):
        t0 = time.perf_counter()
        y = fn(*args, **kw)
        times[tag] = round(_sync_ms(t0), 3)
        return y

    def weight(nm):
        return out[nm][0]

    hidden = _stream_x(cfg, "attn_in")
    n, b = hidden.shape
    ones = torch.ones(b, dtype=hidden.dtype, device=DEV)
    starts = torch.tensor([*range(0, n, tokens), n], dtype=torch.int32, device=DEV)
    freqs = L.rotary_freqs(head, device=DEV)

    X = timed("attention norm", L.rms_norm, hidden, ones, eps=eps)
    prune_group(X, ["q_proj", "k_proj", "v_proj"], "norm(hidden)")
    A = timed("attention", attention_output, X, weight("q_proj"), weight("k_proj"),
              weight("v_proj"), head, starts, freqs)
    prune_group(A, ["o_proj"], "attention")
    timed("o_proj product", L.linear, A, weight("o_proj"), residual=hidden, Y=hidden)
    del A
    timed("feed-forward norm", L.rms_norm, hidden, ones, eps=eps, Y=X)
    prune_group(X, ["gate_proj", "up_proj"], "norm(hidden + o)")
    X = timed("gated ffn", L.gated_ffn_input, X, weight("gate_proj"), weight("up_proj"))
    prune_group(X, ["down_proj"], "gated")
    timed("down_proj product", L.linear, X, weight("down_proj"), residual=hidden, Y=hidden)
    return out, hidden, times


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--config", type=int, default=4)
    ap.add_argument("--pattern", default=None, help="n:m (default: the workload's own)")
    ap.add_argument("--independent", action="store_true",
                    help="down_proj on its independent synthetic stream instead")
    ap.add_argument("--whole", action="store_true",
                    help="every layer on the input that the block's forward steps produce")
    args = ap.parse_args()
    assert torch.cuda.is_available(), "needs a GPU"
    cfg = synth.config(args.config)
    pattern = tuple(int(v) for v in args.pattern.split(":")) if args.pattern else None
    if args.whole:
        if args.independent:
            ap.error("--whole and --independent exclude each other")
        _, _, times = prune_block_whole(cfg, _params(cfg, pattern))
    else:
        _, times = prune_block(cfg, _params(cfg, pattern), propagate=not args.independent)
    print(json.dumps({"config": args.config, "times_ms": times,
                      "total_ms": round(sum(times.values()), 1)}))


if __name__ == "__main__":
    main()
