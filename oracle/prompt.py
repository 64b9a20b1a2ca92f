"""The prompt path in fp64: rotary positions, RMS norm, attention of one prompt -- TEST INFRASTRUCTURE ONLY.

Plain definitions over one stream's rows (the chunked-prefill note, section 1: a chunk of queries against its
prefix and itself).  Frequencies for long contexts follow YaRN (Peng et al., 2023).
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(dim: int, base: float, scaling: str = "plain", factor: float = 1.0, original: float = 0.0,
                fast: float = 32.0, slow: float = 1.0):
    """(radians a position of each pair [dim / 2], amplitude)."""
    f = np.array([base ** (-2.0 * i / dim) for i in range(dim // 2)])
    if scaling == "plain":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    assert scaling == "yarn"
    where = [dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (fast, slow)]
    lo, hi = max(0, math.floor(where[0])), min(dim - 1, math.ceil(where[1]))
    ramp = np.array([min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(dim // 2)])
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def rotate(x: np.ndarray, positions, freq: np.ndarray, amplitude: float, half: bool) -> np.ndarray:
    """x [rows][heads][dim], row i turned to positions[i]."""
    x = np.asarray(x, np.float64)
    out = np.empty_like(x)
    d = x.shape[-1]
    for r, p in enumerate(positions):
        for i in range(d // 2):
            a, b = (i, i + d // 2) if half else (2 * i, 2 * i + 1)
            t = math.fmod(int(p) * freq[i], 2 * math.pi)
            c, s = amplitude * math.cos(t), amplitude * math.sin(t)
            out[r, :, a] = x[r, :, a] * c - x[r, :, b] * s
            out[r, :, b] = x[r, :, b] * c + x[r, :, a] * s
    return out


def rms_norm(x: np.ndarray, gain: np.ndarray, eps: float) -> np.ndarray:
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, causal: bool):
    """One stream: q [nq][H][d], k [nk][Hkv][d], v [nk][Hkv][dv] -> (out [nq][H][dv], lse [nq][H]).  A row that
    sees no key gives zeros and -inf."""
    nq, H = q.shape[:2]
    nk, Hkv = k.shape[:2]
    out, lse = np.zeros((nq, H, v.shape[-1])), np.full((nq, H), -np.inf)
    for h in range(H):
        g = h // (H // Hkv)
        for i in range(nq):
            n = min(nk, max(0, nk - nq + i + 1)) if causal else nk
            if n == 0:
                continue
            s = scale * (k[:n, g].astype(np.float64) @ q[i, h].astype(np.float64))
            m = s.max()
            e = np.exp(s - m)
            out[i, h] = e @ v[:n, g].astype(np.float64) / e.sum()
            lse[i, h] = m + math.log(e.sum())
    return out, lse
