"""Plain fp64 definitions of the block's forward steps between the pruned layers:
a linear layer with its epilogue, row norms, rotary positions and causal attention
over packed sequences. Loops and dense matrices; no code of the library.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["forward_linear", "rms_norm", "rotary_freqs", "rotary", "attention"]


def _f64(x) -> np.ndarray:
    if hasattr(x, "detach"):
        x = x.detach().cpu().double().numpy()
    return np.asarray(x, dtype=np.float64)


def forward_linear(X, W, bias=None, act="none", residual=None) -> np.ndarray:
    """act(X W^T + bias) + residual."""
    z = _f64(X) @ _f64(W).T
    if bias is not None:
        z = z + _f64(bias)
    if act == "relu":
        z = np.maximum(z, 0.0)
    elif act == "silu":
        z = z * 0.5 * (1.0 + np.tanh(0.5 * z))
    elif act == "gelu":
        z = 0.5 * z * np.vectorize(math.erfc, otypes=[np.float64])(-z / math.sqrt(2.0))
    elif act != "none":
        raise ValueError(act)
    return z if residual is None else z + _f64(residual)


def rms_norm(X, weight, eps) -> np.ndarray:
    X = _f64(X)
    return X / np.sqrt(np.mean(X * X, axis=-1, keepdims=True) + eps) * _f64(weight)


def rotary_freqs(rot, base=10000.0, divide=1.0, bands=None) -> np.ndarray:
    out = []
    for i in range(rot // 2):
        f = 1.0 / base ** (2 * i / rot)
        if bands is None:
            out.append(f / divide)
            continue
        length, slow, fast = bands
        turns = length / (2 * math.pi / f)
        if turns >= fast:
            out.append(f)
        elif turns <= slow:
            out.append(f / divide)
        else:
            part = (turns - slow) / (fast - slow)
            out.append(part * f + (1 - part) * f / divide)
    return np.array(out)


def rotary(x, positions, freqs, layout="half", amplitude=1.0, norm=None, eps=1e-6) -> np.ndarray:
    """x [n, heads, d]: normed heads, then the first 2 len(freqs) elements turned."""
    y = _f64(x).copy() if norm is None else rms_norm(x, norm, eps)
    half = len(freqs)
    # the angle in extended precision: positions up to 2^31 leave fp64 few bits of the turn
    angle = (np.asarray(positions, dtype=np.longdouble)[:, None]
             * np.asarray(freqs, dtype=np.longdouble)[None, :])
    z = amplitude * (np.cos(angle).astype(np.float64) + 1j * np.sin(angle).astype(np.float64))
    ia = np.arange(half) if layout == "half" else 2 * np.arange(half)
    ib = ia + half if layout == "half" else ia + 1
    turned = (y[:, :, ia] + 1j * y[:, :, ib]) * z[:, None, :]
    y[:, :, ia], y[:, :, ib] = turned.real, turned.imag
    return y


def attention(Q, K, V, q_start, k_start, causal=True, scale=None) -> np.ndarray:
    """Q [nq, hq, d], K and V [nk, hk, d]. Sequence s has queries q_start[s] .. q_start[s+1]
    and keys k_start[s] .. k_start[s+1]; with causal its last query sees its last key. A
    query that sees no key gets zeros; rows of no sequence stay NaN here. Sums run over the
    visible keys only, so what hidden rows hold never enters."""
    Q, K, V = _f64(Q), _f64(K), _f64(V)
    nq, hq, d = Q.shape
    g = hq // K.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out = np.full((nq, hq, V.shape[2]), np.nan)
    for s in range(len(q_start) - 1):
        q0, q1, k0, k1 = q_start[s], q_start[s + 1], k_start[s], k_start[s + 1]
        for h in range(hq):
            for i in range(q0, q1):
                end = k1 if not causal else k0 + max(0, min(k1 - k0, (i - q0) + 1 + (k1 - k0) - (q1 - q0)))
                if end <= k0:
                    out[i, h] = 0.0
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    z = K[k0:end, h // g] @ Q[i, h] * scale
                    p = np.exp(z - np.max(z))
                    out[i, h] = (p / np.sum(p)) @ V[k0:end, h // g]
    return out
