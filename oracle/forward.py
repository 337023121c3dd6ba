"""Plain fp64 definitions of the block's forward steps between the pruned layers:
a linear layer with its epilogue, row norms, rotary positions and causal attention
over packed sequences. Loops and dense matrices; no code of the library.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["forward_linear", "rms_norm", "rotary_freqs", "rotary", "attention", "mx_numbers",
           "mx_quantize", "mx_values", "paged_keys", "paged_store"]


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


def mx_numbers(form) -> list:
    """The form's numbers from 0 up, in the order of their codes, and the one that would follow."""
    bits, bias, last = {"e4m3": (3, 7, 126), "e2m1": (1, 1, 7)}[form]
    out = []
    for code in range(last + 2):
        e, m = code >> bits, code & ((1 << bits) - 1)
        out.append(math.ldexp(m, 1 - bias - bits) if e == 0
                   else math.ldexp((1 << bits) + m, e - bias - bits))
    return out


def _mx_nearest(v, numbers):
    """Code of the number nearest to each of v >= 0 (a tie: the even code)."""
    n = np.array(numbers)
    i = np.clip(np.searchsorted(n, v, side="right") - 1, 0, len(n) - 2)
    up, down = n[i + 1] - v, v - n[i]
    return i + ((up < down) | ((up == down) & (i % 2 == 1)))


def mx_quantize(X, form):
    """(codes [n, b], scales [n, b / 32]) of X: exponents are tried from the lowest that can be
    until the block's largest number is rounded to one of the form's."""
    X = _f64(X)
    n, b = X.shape
    numbers = mx_numbers(form)
    last = len(numbers) - 2
    top = int(math.log2(numbers[last]))
    x = X.reshape(n, b // 32, 32)
    codes = np.zeros(x.shape, dtype=np.int64)
    scales = np.zeros((n, b // 32), dtype=np.int64)
    for t in range(n):
        for j in range(b // 32):
            v = np.abs(x[t, j])
            if not np.isfinite(v).all():
                scales[t, j] = 255
                continue
            big = float(v.max())
            e = -127 if big == 0 else max(-127, math.frexp(big)[1] - 1 - top - 1)
            while e < 127 - top and _mx_nearest(math.ldexp(big, -e), numbers) > last:
                e += 1
            codes[t, j] = np.minimum(_mx_nearest(np.ldexp(v, -e), numbers), last)
            codes[t, j] += np.signbit(x[t, j]) * (last + (2 if form == "e4m3" else 1))
            scales[t, j] = e + 127
    return codes.reshape(n, b), scales


def mx_values(codes, scales, form) -> np.ndarray:
    """The numbers that codes [n, b] stand for with their blocks' scales."""
    numbers = mx_numbers(form)
    half = 128 if form == "e4m3" else 8
    table = np.array(numbers[:half - 1] + [np.nan] if form == "e4m3" else numbers[:8])
    codes, scales = np.asarray(codes), np.asarray(scales)
    v = np.where(codes >= half, -1.0, 1.0) * table[codes % half]
    power = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(power, 32, axis=1)


def paged_keys(cache, pages, k_len):
    """Keys (or values) of every sequence of a paged cache [pages, page, hk, d], packed, and
    their starts."""
    cache = _f64(cache)
    page = cache.shape[1]
    rows, starts = [], [0]
    for row, n in zip(np.asarray(pages), k_len):
        rows += [cache[row[x // page], x % page] for x in range(n)]
        starts.append(starts[-1] + n)
    return np.array(rows).reshape(starts[-1], *cache.shape[2:]), starts


def paged_store(cache, new, pages, k_len, q_start):
    """The cache with the new rows as the last keys of their sequences."""
    out = _f64(cache).copy()
    new, page = _f64(new), out.shape[1]
    for s in range(len(q_start) - 1):
        for t in range(q_start[s], q_start[s + 1]):
            key = k_len[s] - (q_start[s + 1] - t)
            p = pages[s][key // page] if 0 <= key < page * len(pages[s]) else -1
            if 0 <= p < out.shape[0]:
                out[p, key % page] = new[t]
    return out
