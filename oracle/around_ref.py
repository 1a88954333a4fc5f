"""fp64 CPU oracle for the operators around the decode: rotary positions,
cache append, attention weights and their accumulation, eviction.

TEST INFRASTRUCTURE ONLY (see sparse_mla_ref).  Each function is the plain
definition in float64; none shares code with the CUDA library.  Pinned by
``tests/test_oracle_around.py`` against closed forms, complex arithmetic,
brute force and planted mistakes.
"""
from __future__ import annotations

import math

import numpy as np

from .sparse_mla_ref import gather_rows_f64, resolve_rows


def rope_frequencies(dim: int, *, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_ctx: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0) -> np.ndarray:
    """Radians per position of the dim / 2 pairs."""
    f = np.array([base ** (-2.0 * i / dim) for i in range(dim // 2)])
    if scaling is None:
        return f
    if scaling == "linear":
        return f / factor
    turn = [dim * math.log(original_ctx / (2 * math.pi * t)) / (2 * math.log(base)) for t in (beta_fast, beta_slow)]
    lo, hi = max(math.floor(turn[0]), 0), min(math.ceil(turn[1]), dim - 1)
    r = np.clip((np.arange(dim // 2) - lo) / max(hi - lo, 0.001), 0.0, 1.0)
    return (1 - r) * f + r * f / factor


def rope(x: np.ndarray, positions: np.ndarray, freq: np.ndarray, *, offset: int, interleaved: bool,
         mscale: float = 1.0, transpose: bool = False) -> np.ndarray:
    """x [..., heads, dim] (positions [...]) with its rotary dims turned."""
    y = np.array(x, dtype=np.float64)
    half = len(freq)
    a_at = offset + (2 * np.arange(half) if interleaved else np.arange(half))
    b_at = a_at + (1 if interleaved else half)
    angle = np.asarray(positions, dtype=np.float64)[..., None, None] * freq
    if transpose:
        angle = -angle
    a, b = y[..., a_at].copy(), y[..., b_at].copy()
    y[..., a_at] = mscale * (a * np.cos(angle) - b * np.sin(angle))
    y[..., b_at] = mscale * (a * np.sin(angle) + b * np.cos(angle))
    return y


def append_rows(x: np.ndarray, *, norm_weight=None, eps: float = 1e-6, freq=None, positions=None,
                interleaved: bool = True, mscale: float = 1.0) -> np.ndarray:
    """The rows a cache append encodes: x [n, d] normed over its first 512
    dims, its last 64 turned."""
    y = np.array(x, dtype=np.float64)
    if norm_weight is not None:
        latent = y[:, :512]
        y[:, :512] = latent / np.sqrt((latent ** 2).mean(axis=1, keepdims=True) + eps) * norm_weight
    if freq is not None:
        y = rope(y[:, None, :], positions, freq, offset=y.shape[1] - 64, interleaved=interleaved, mscale=mscale)[:, 0]
    return y


def group_exponent(amax: float) -> int:
    """The smallest e >= -126 with amax <= 448 * 2^e."""
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def slot_rows(slots, seq, page_table) -> np.ndarray:
    """Physical row of each token (-1: skipped); flat where page_table is None."""
    out = []
    for i, s in enumerate(slots):
        if s < 0:
            out.append(-1)
        elif page_table is None:
            out.append(int(s))
        else:
            out.append(int(page_table[seq[i], s // 64]) * 64 + int(s) % 64)
    return np.array(out, dtype=np.int64)


def attention_weights(q: np.ndarray, rows: np.ndarray, lse: np.ndarray, scale: float) -> np.ndarray:
    """q [H, d], rows [n, d], lse [H] -> [n]: sum over heads of exp(scale q.k - lse)."""
    s = scale * (q @ rows.T)
    w = np.zeros(rows.shape[0])
    for h in range(q.shape[0]):
        if lse[h] != -np.inf:
            w += np.exp(s[h] - lse[h])
    return w


def list_weights(q, kv, indices, lse, scale, *, kv_format, kv_row_scale=None, page_table_row=None, page_size=0):
    """attention_weights over one index list: [k], 0 for padding; also the
    rows and the mask of valid entries."""
    valid = indices >= 0
    num = kv.shape[0] * (64 if kv_format == "dsv4_paged" else 1)
    phys = resolve_rows(indices[valid], page_table_row=page_table_row, page_size=page_size, num_rows=num)
    rows = gather_rows_f64(kv, phys, kv_format=kv_format, row_scale=kv_row_scale)
    w = np.zeros(indices.shape[0])
    w[valid] = attention_weights(q, rows, lse, scale)
    return w, rows, valid


def accumulate(acc: np.ndarray, indices: np.ndarray, weights: np.ndarray, decay: float) -> np.ndarray:
    """acc [B, n], indices and weights [B, e]."""
    out = decay * acc.astype(np.float64)
    for b in range(acc.shape[0]):
        for p, w in zip(indices[b], weights[b]):
            if 0 <= p < acc.shape[1]:
                out[b, p] += float(w)
    return out


def evict_select(acc_row: np.ndarray, n: int, budget: int, sinks: int, recent: int) -> list[int]:
    """Kept positions of one sequence, ascending."""
    if n <= budget:
        return list(range(n))
    fixed = [i for i in range(n) if i < sinks or i >= n - recent]
    rest = [i for i in range(n) if sinks <= i < n - recent]
    rest.sort(key=lambda i: (np.isnan(acc_row[i]), -acc_row[i] if not np.isnan(acc_row[i]) else 0.0, i))
    return sorted(fixed + rest[:budget - len(fixed)])
