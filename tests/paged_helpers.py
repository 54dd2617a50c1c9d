"""Pools, page tables and float64 references of the paged-cache tests."""
from __future__ import annotations

import numpy as np
import torch

from kvq_helpers import host
from oracle import positions as opos
from oracle import quantize as oq

FORMATS = {"fp16": ("fp16", 16), "aff8": ("affine_token", 8), "aff4": ("affine_token", 4)}


def make_pool(kvq, fmt, H, D, page, n_pages, kgroup=64, vgroup=64, seed=0, fill=True):
    """A pool whose every row (used or not) holds ordinary codes and metadata."""
    f, bits = FORMATS[fmt]
    kg, vg = (0, 0) if fmt == "fp16" else (min(kgroup, D), min(vgroup, D))
    c = kvq.PagedKVCache(H, D, page, n_pages, f, bits, kg, f, bits, vg)
    if fill:
        g = torch.Generator().manual_seed(seed)
        for side in "kv":
            x = c.plane(side + "_codes")
            if fmt == "fp16":
                x.copy_(torch.randn(x.shape, generator=g))
            else:
                x.copy_(torch.randint(0, 256, x.shape, generator=g).to(torch.uint8))
                m = c.plane(side + "_meta")
                w = torch.rand(m.shape[:-1], generator=g) * 3 + 3
                m.copy_(torch.stack((w / (2 ** bits - 1), -w * torch.rand(m.shape[:-1], generator=g)), -1))
    return c


def values(cache, side) -> np.ndarray:
    """float64 [n_pages, H, page, D]: the values every row of the pool stands for."""
    x = cache.plane(side + "_codes").cpu().numpy()
    if x.dtype == np.float16:
        return x.astype(np.float64)
    bits, D = cache.cfg.k_bits, cache.head_dim
    u = oq.int8_to_codes(x.view(np.int8)) if bits == 8 else np.stack((x & 15, x >> 4), -1).reshape(*x.shape[:-1], D)
    m = cache.plane(side + "_meta").cpu().numpy().astype(np.float64)
    g = D // m.shape[-2]
    u = u.astype(np.float64).reshape(*u.shape[:-1], D // g, g)
    return (u * m[..., 0:1] + m[..., 1:2]).reshape(*x.shape[:-1], D)


def tables(lens, prefix, page, seed=0, extra=2, spare_cols=1):
    """(page_table [B, cols] with -1 past each sequence's pages, prefix pages, pages in the pool)."""
    need = [-(-n // page) for n in lens]
    npre = -(-prefix // page)
    total = sum(need) + npre + extra
    order = np.random.default_rng(seed).permutation(total).astype(np.int32)
    cols = max(need, default=0) + spare_cols
    t = np.full((len(lens), cols), -1, dtype=np.int32)
    at = npre
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, order[:npre].copy(), total


def gather(vals, table_row, n, page) -> np.ndarray:
    """[H, n, D] of a sequence's first n tokens."""
    ids, rows = opos.page_rows(table_row, n, page)
    return vals[ids, :, rows].transpose(1, 0, 2) if n else np.zeros((vals.shape[1], 0, vals.shape[3]))


def reference(q, kv, vv, table, lens, pre, prefix, page, scale=None):
    """(float64 out [B, Hq, D], worst max |v| of a row, worst sum |q||k| scale of a row) of attention."""
    q = host(q).astype(np.float64)
    B, Hq, D = q.shape
    H = kv.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros_like(q)
    vmax, smax = np.zeros((B, Hq, 1)), np.zeros((B, Hq, 1))
    for b in range(B):
        k = np.concatenate((gather(kv, pre, prefix, page), gather(kv, table[b], lens[b], page)), 1)
        v = np.concatenate((gather(vv, pre, prefix, page), gather(vv, table[b], lens[b], page)), 1)
        if not k.shape[1]:
            continue
        for h in range(Hq):
            g = h // (Hq // H)
            s = k[g] @ q[b, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[b, h] = p @ v[g]
            vmax[b, h], smax[b, h] = np.abs(v[g]).max(), (np.abs(k[g]) @ np.abs(q[b, h])).max() * scale
    return out, vmax, smax


def check_attention(got, want, vmax, smax, what=""):
    """Two bounds.  Every element: keys, values and softmax weights may each enter the products rounded to
    fp16 (half a step, u = 2^-11).  Keys move a score by at most u * sum |q||k| scale, so each weight by twice
    that relative; weights and values add u each, the sums' 32 bits far less; so the output, a mean of values,
    moves by at most vmax * (2 u smax + 3 u), and is rounded once to its type.  Altogether (2-norm): roundings
    are as often up as down, so the whole is at most the root mean square of those parts' worst cases, of
    which half is allowed."""
    u = 2.0 ** -11
    half = torch.finfo(got.dtype).eps / 2
    g = host(got).astype(np.float64)
    assert np.all(np.isfinite(g)), f"{what}: non-finite output"
    inner = vmax * (2 * u * smax + 3 * u)
    tol = half * (np.abs(want) + inner) + inner + torch.finfo(got.dtype).tiny
    err = np.abs(g - want)
    assert np.all(err <= tol), f"{what}: {(err > tol).sum()} off, worst {(err / tol).max():.2f} of the tolerance"
    assert np.linalg.norm(err) <= 0.5 * np.linalg.norm(tol), f"{what}: 2-norm {np.linalg.norm(err):.3e}"
