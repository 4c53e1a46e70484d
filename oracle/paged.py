"""fp64 oracle of the per-head norms with rotation, the paged cache, its decode and
its page selection.  Test infrastructure only; plain numpy, no code shared with the
CUDA library.

Layouts: keys [page][kv head][d/16][slot][16] (pairs interleaved), values
[page][kv head][slot][d], bounds [page][kv head][2][d], page tables [batch][max_pages].
"""
from __future__ import annotations

import math

import numpy as np

import oracle


def f64(x) -> np.ndarray:
    """A torch tensor's values as fp64."""
    return x.detach().double().cpu().numpy()


def norm_rope(x, weight, eps, pos, pair_axis, theta, pairing):
    """x [T][H][d] normed over d (weight None: not) and turned: pair i by
    pos[pair_axis[i]][t] * theta^(-2i/d).  Returns (y, size), pairs interleaved, size
    the sum of the pair's magnitudes before the turn (the scale of its rounding)."""
    T, H, d = x.shape
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight if weight is not None else x
    a, b = (y[..., : d // 2], y[..., d // 2:]) if pairing == oracle.ROTATE_HALF else (y[..., 0::2], y[..., 1::2])
    ang = np.stack([pos[pair_axis[i]].astype(np.float64) * theta ** (-2.0 * i / d) for i in range(d // 2)], -1)[:, None]
    out, size = np.empty_like(y), np.empty_like(y)
    out[..., 0::2] = a * np.cos(ang) - b * np.sin(ang)
    out[..., 1::2] = a * np.sin(ang) + b * np.cos(ang)
    size[..., 0::2] = size[..., 1::2] = np.abs(a) + np.abs(b)
    return out, size


def page_rows(k_pages, v_pages, page_table, b, kv_head, logical):
    """Keys [n * slots][d] and values of the given logical pages of one sequence and head."""
    pages = [int(page_table[b][i]) for i in logical]
    k = np.concatenate([np.moveaxis(k_pages[p, kv_head], 0, 1).reshape(k_pages.shape[3], -1) for p in pages])
    return k, np.concatenate([v_pages[p, kv_head] for p in pages])


def decode(q, k_pages, v_pages, page_table, kv_len, theta, alpha, selected=None):
    """Returns (out, lse, weight, spread): out [B][Hq][d]; weight, the softmax-weighted
    |v|, and spread [B][Hq], the largest sum of |q k| / sqrt(d), the scales of the
    kernel's roundings."""
    B, Hq, d = q.shape
    Hkv, ps = k_pages.shape[1], k_pages.shape[3]
    W = np.repeat(oracle.windows(d, theta, alpha)[0], 2)
    out, weight = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    lse, spread = np.full((B, Hq), -math.inf), np.zeros((B, Hq))
    for b in range(B):
        n = int(kv_len[b])
        if n <= 0:
            continue
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            logical = range(-(-n // ps)) if selected is None else [
                int(i) for i in selected[b][hk][: -(-n // ps)] if i >= 0]
            key = np.concatenate([np.arange(i * ps, i * ps + ps) for i in logical] or [np.empty(0, int)])
            live = key < n
            if not live.any():
                continue
            k, v = page_rows(k_pages, v_pages, page_table, b, hk, logical)
            k, v, key = k[live], v[live], key[live]
            prod = np.where((n - 1 - key)[:, None] <= W, k * q[b, h], 0.0) / math.sqrt(d)
            x = prod.sum(-1)
            p = np.exp(x - x.max())
            lse[b, h] = x.max() + math.log(p.sum())
            p /= p.sum()
            out[b, h], weight[b, h] = p @ v, p @ np.abs(v)
            spread[b, h] = np.abs(prod).sum(-1).max()
    return out, lse, weight, spread


def select(q, bounds, page_table, kv_len, page_size, n_select, theta, alpha, n_first, n_last):
    """[B][Hkv][n_select] int: the pages kept, ascending, -1 behind the last."""
    B, Hq, d = q.shape
    Hkv = bounds.shape[1]
    G = Hq // Hkv
    W = np.repeat(oracle.windows(d, theta, alpha)[0], 2)
    kept = np.full((B, Hkv, n_select), -1, dtype=np.int64)
    for b in range(B):
        n = max(0, int(kv_len[b]))
        pages = -(-n // page_size)
        for hk in range(Hkv):
            score = []
            for i in range(pages):
                on = n - 1 - min(n, (i + 1) * page_size) + 1 <= W
                mn, mx = bounds[int(page_table[b][i]), hk]
                best = max(math.fsum(np.maximum(q[b, hk * G + g] * mn, q[b, hk * G + g] * mx)[on]) for g in range(G))
                score.append(math.inf if i < n_first or i >= pages - n_last else best)
            order = sorted(range(pages), key=lambda i: (-score[i], i))[:n_select]
            kept[b, hk, : len(order)] = sorted(order)
    return kept
