"""fp64 oracle of the operators that give the step its gradients: the 8-bit form of
activations, the weight gradient from it, the fused norm and the embedding, with their
gradients.  Plain NumPy, written from the formulas; nothing is shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 e4m3 bytes (sign, 4 exponent bits of bias 7, 3 fraction
    bits; no infinities, both all-ones magnitudes are NaN)."""
    out = np.empty(256)
    for b in range(256):
        sign, e, f = (-1.0 if b & 128 else 1.0), (b >> 3) & 15, b & 7
        if e == 15 and f == 7:
            out[b] = math.nan
        elif e == 0:
            out[b] = sign * f * 2.0 ** -9
        else:
            out[b] = sign * (8 + f) * 2.0 ** (e - 10)
    return out


def act_exponent(top: float) -> int:
    """The smallest e in [-117, 119] with top <= 448 * 2^e, or 119."""
    for e in range(-117, 120):
        if top <= 448.0 * 2.0 ** e:
            return e
    return 119


def act_round(x: np.ndarray):
    """(values, exponent bytes): what 8 bits keep of x [t, d].  The nearest e4m3 value is
    looked up among all of them, ties to the even fraction."""
    t, d = x.shape
    nb = -(-d // BLOCK)
    grid = e4m3_values()[:127]                # 0 .. 448, ascending; index parity = fraction's
    out = np.full((t, d), math.nan)
    scale = np.full((t, nb), 255, np.uint8)
    for i in range(t):
        for b in range(nb):
            v = x[i, b * BLOCK:(b + 1) * BLOCK].astype(np.float64)
            if not np.all(np.isfinite(v)):
                continue
            e = act_exponent(float(np.max(np.abs(v))))
            a = np.minimum(np.abs(v) * 2.0 ** -e, 448.0)
            hi = np.clip(np.searchsorted(grid, a), 0, 126)
            lo = np.maximum(hi - 1, 0)
            up, down = grid[hi] - a, a - grid[lo]
            pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
            out[i, b * BLOCK:(b + 1) * BLOCK] = np.sign(v) * grid[pick] * 2.0 ** e
            scale[i, b] = e + 127
    return out, scale


def act_value(q: np.ndarray, scale: np.ndarray, d: int) -> np.ndarray:
    """The values that bytes q [t, ld] with exponent bytes scale [t, ld / 32] stand for."""
    f = np.where(scale == 255, math.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return (e4m3_values()[q] * np.repeat(f, BLOCK, axis=1))[:, :d]


def weight_grad(a: np.ndarray, d: np.ndarray, transposed: bool = False) -> np.ndarray:
    return d.T @ a if transposed else a.T @ d


def _rms(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def _ones(g, d):
    return np.ones(d) if g is None else g


def norm_forward(x, y=None, *, pre_gain=None, post_gain=None, gate=None, residual_scale=1.0,
                 eps=1e-6, post_norm=None):
    """(h, u) of include/dion.h's dion_norm_forward."""
    d = x.shape[1]
    post_norm = post_gain is not None if post_norm is None else post_norm
    h = x
    if y is not None:
        z = _ones(post_gain, d) * y * _rms(y, eps) if post_norm else y
        h = x + residual_scale * _ones(gate, d) * z
    return h, _ones(pre_gain, d) * h * _rms(h, eps)


def norm_backward(h, y=None, *, du=None, dh=None, pre_gain=None, post_gain=None, gate=None,
                  residual_scale=1.0, eps=1e-6, post_norm=None):
    """Gradients {dx, dy, dpre_gain, dpost_gain, dgate} at h and y."""
    d = h.shape[1]
    post_norm = post_gain is not None if post_norm is None else post_norm
    out = {}
    g = np.zeros_like(h) if dh is None else dh.copy()
    if du is not None:
        r = _rms(h, eps)
        w = _ones(pre_gain, d) * du
        g = g + r * w - h * r ** 3 * np.mean(w * h, axis=1, keepdims=True)
        out["dpre_gain"] = np.sum(du * h * r, axis=0)
    out["dx"] = g
    if y is not None:
        c = residual_scale * _ones(gate, d) * g          # gradient of z
        if post_norm:
            ry = _rms(y, eps)
            out["dpost_gain"] = np.sum(c * y * ry, axis=0)
            w = c * _ones(post_gain, d)
            out["dy"] = ry * w - y * ry ** 3 * np.mean(w * y, axis=1, keepdims=True)
            z = _ones(post_gain, d) * y * ry
        else:
            out["dy"] = c
            z = y
        out["dgate"] = residual_scale * np.sum(g * z, axis=0)
    return out


def embed_lookup(table, ids, scale=1.0):
    out = np.zeros((len(ids), table.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < table.shape[0]:
            out[t] = scale * table[i]
    return out


def embed_grad(ids, dout, vocab, scale=1.0):
    out = np.zeros((vocab, dout.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < vocab:
            out[i] += scale * dout[t]
    return out
