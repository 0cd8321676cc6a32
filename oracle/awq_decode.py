"""CPU oracle of the decode-step operators around the W4A16 products — TEST INFRASTRUCTURE ONLY.

The RMS norm with the residual's addition (its weight carries the inverse scales, AWQ-P1 §6),
the position rotation, the places of a paged cache and the attention of one new token, each
from its formula in fp64. Arrays are numpy; 8-bit caches come as the values they hold.

Pins: tests/test_oracle_decode_pins.py.
"""
from __future__ import annotations

import numpy as np

__all__ = ["E4M3_MAX", "rms_norm", "row_scales", "frequencies", "rotate", "places", "attention"]

E4M3_MAX = 448.0


def rms_norm(X, residual, weight, eps: float):
    """(y, h): h = X + residual, y = h weight / sqrt(mean(h^2) + eps) per row."""
    h = np.asarray(X, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    return h * np.asarray(weight, dtype=np.float64) / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps), h


def row_scales(y) -> np.ndarray:
    """Scale of each row's e4m3 codes: max|y| / 448, 1 for a row of zeros."""
    s = np.max(np.abs(y), axis=1) / E4M3_MAX
    return np.where(s == 0, 1.0, s)


def frequencies(rotary_dim: int, base: float = 10000.0, scaling=None, factor: float = 1.0, original_len: float = 0.0,
                low: float = 1.0, high: float = 4.0):
    """(freqs, magnitude) of the rotation, pair by pair."""
    freqs = []
    for i in range(rotary_dim // 2):
        f = base ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "base":
            f = (base * factor ** (rotary_dim / (rotary_dim - 2.0))) ** (-2.0 * i / rotary_dim)
        elif scaling == "bands":
            turns = original_len * f / (2 * np.pi)
            if turns <= low:
                f /= factor
            elif turns < high:
                share = (turns - low) / (high - low)
                f = (1 - share) * f / factor + share * f
        elif scaling == "ramp":
            at = lambda turns: rotary_dim * np.log(original_len / (turns * 2 * np.pi)) / (2 * np.log(base))  # noqa: E731
            first, end = max(0.0, np.floor(at(high))), min(rotary_dim - 1.0, np.ceil(at(low)))
            if i >= end:
                f /= factor
            elif i > first:
                share = (i - first) / max(end - first, 1e-3)
                f = f / factor * share + f * (1 - share)
        freqs.append(f)
    return np.array(freqs), 0.1 * np.log(factor) + 1.0 if scaling == "ramp" else 1.0


def rotate(x, positions, freqs, interleaved: bool, magnitude: float = 1.0) -> np.ndarray:
    """x (T, heads, D) with the pairs of its first 2 len(freqs) dims turned by position x frequency."""
    out = np.array(x, dtype=np.float64)
    R = 2 * len(freqs)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        theta = (np.asarray(positions, dtype=np.float64) * f)[:, None]
        c, s = magnitude * np.cos(theta), magnitude * np.sin(theta)
        xa, xb = np.array(x[..., a], dtype=np.float64), np.array(x[..., b], dtype=np.float64)
        out[..., a], out[..., b] = xa * c - xb * s, xa * s + xb * c
    return out


def places(block_table, page_size: int, num_pages: int, positions, seqs=None):
    """(page, slot) of each token, (-1, -1) where it has none (padded, or outside)."""
    found = []
    for t, p in enumerate(positions):
        b = t if seqs is None else int(seqs[t])
        at = (-1, -1)
        if p >= 0 and 0 <= b < block_table.shape[0] and p // page_size < block_table.shape[1]:
            page = int(block_table[b, p // page_size])
            if 0 <= page < num_pages:
                at = (page, int(p) % page_size)
        found.append(at)
    return found


def attention(q, k, v, scale: float) -> np.ndarray:
    """One token's queries (Hq, D) over keys and values (len, heads, D): softmax(scale q k^T) v,
    zeros without tokens; (Hq, D)."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    Hq, D = q.shape
    n, heads, _ = k.shape
    if n == 0:
        return np.zeros((Hq, D))
    out = np.empty((Hq, D))
    for h in range(Hq):
        kv = h // (Hq // heads)
        s = scale * (k[:, kv] @ q[h])
        p = np.exp(s - np.max(s))
        out[h] = p @ v[:, kv] / np.sum(p)
    return out
