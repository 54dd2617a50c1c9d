"""Rotary positions, per-head norms and page tables, float64.

The StreamingLLM + KIVI page leaves the rotation to the model and keeps keys
at their absolute position ("RoPE caveat"); these are the rotation's own
definitions.  Pair i of a head turns by position * f_i radians.  Frequency
scalings: linear interpolation (Chen et al. 2023), NTK-aware base change,
YaRN's ramp over pair indices with its magnitude (Peng et al. 2023), the
Llama 3.1 ramp over turns within the trained length, and one factor per pair
(LongRoPE, Ding et al. 2024).
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np


def frequencies(rot_dim: int, base: float, scaling: str = "none", factor: float = 1.0,
                original_max_position: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                low_freq_factor: float = 1.0, high_freq_factor: float = 4.0, factors=None):
    """(radians per position of each pair, magnitude of sines and cosines)."""
    mag = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = np.array([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], dtype=np.float64)
    if scaling == "linear":
        f = f / factor
    elif scaling == "factors":
        f = f / np.asarray(factors, dtype=np.float64)
    elif scaling == "yarn":
        def pair(beta):
            return rot_dim * math.log(original_max_position / (beta * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot_dim - 1)
        r = np.clip((np.arange(rot_dim // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        f, mag = f * (1 - r) + f / factor * r, 0.1 * math.log(factor) + 1
    elif scaling == "llama3":
        turns = original_max_position * f / (2 * math.pi)
        keep = np.clip((turns - low_freq_factor) / (high_freq_factor - low_freq_factor), 0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f, mag


def table_entry(radians: float) -> int:
    """round(radians / 2 pi modulo 1 turn * 2^64), modulo 2^64, by rational arithmetic on a 64-bit pi."""
    turn = Fraction(radians) / (2 * Fraction(math.pi))
    return round((turn - math.floor(turn)) * 2 ** 64) % 2 ** 64


def head_norm(x: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    """x * weight / sqrt(mean(x^2) + eps) over the last axis."""
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def rotate(x: np.ndarray, positions: np.ndarray, freqs: np.ndarray, mag: float = 1.0,
           interleaved: bool = False) -> np.ndarray:
    """x [T, H, D] with the pairs of its first 2 len(freqs) channels turned by positions [T] * freqs."""
    y = np.array(x, dtype=np.float64)
    rot = 2 * len(freqs)
    ang = np.asarray(positions, dtype=np.float64)[:, None, None] * freqs
    c, s = np.cos(ang) * mag, np.sin(ang) * mag
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def page_rows(table: np.ndarray, n: int, page_size: int):
    """(page ids, rows) of tokens 0 .. n - 1 of a sequence with page table `table` [max_pages]."""
    j = np.arange(n)
    return np.asarray(table)[j // page_size], j % page_size
