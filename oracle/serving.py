"""The operators around an attention step, plain numpy in 64 bits (CPU oracle).

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py): rotary positions with
several axes, the attention weight of each page, the choice of the pages that
stay, and the verification of drafted tokens, each from its definition.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def pair_axes(half, sections, interleaved):
    """Axis of each rotary pair."""
    n = len(sections)
    if not interleaved:
        return [x for x in range(n) for _ in range(sections[x])]
    return [i % n if i // n < sections[i % n] else 0 for i in range(half)]


def rope(x, pos, rotary_dim, sections, theta=10000.0, inv_freq=None, interleaved=False, adjacent=False):
    """x [T][H][d] float64, pos [axes][T]: pair i turns by pos[axis(i)] * f_i."""
    x = np.asarray(x, np.float64).copy()
    half = rotary_dim // 2
    f = theta ** (-2.0 * np.arange(half) / rotary_dim) if inv_freq is None else np.asarray(inv_freq, np.float64)
    axes = pair_axes(half, sections, interleaved)
    for i in range(half):
        angle = np.asarray(pos, np.float64)[axes[i]] * f[i]
        z = np.exp(1j * angle)[:, None]
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        y = (x[:, :, a] + 1j * x[:, :, b]) * z
        x[:, :, a], x[:, :, b] = y.real, y.imag
    return x


def decode_weights(q, k_pages, v_pages, block_table, seq_len, scale):
    """q [S][Hq][d]; k_pages, v_pages [pages][Hkv][P][d] values (float64).
    (o [S][Hq][d], w [S][max_pages]): softmax attention over keys [0, L) and
    the weight of each page, summed over query heads."""
    S, hq, d = q.shape
    hkv, P = k_pages.shape[1:3]
    o, w = np.zeros((S, hq, d)), np.zeros(block_table.shape)
    for s in range(S):
        L = int(seq_len[s])
        if L <= 0:
            continue
        n = -(-L // P)
        table = block_table[s, :n]
        there = np.repeat(table >= 0, P)[:L]  # a page that a table does not name is left out
        k = k_pages[np.maximum(table, 0)].transpose(1, 0, 2, 3).reshape(hkv, n * P, d)[:, :L]
        v = v_pages[np.maximum(table, 0)].transpose(1, 0, 2, 3).reshape(hkv, n * P, d)[:, :L]
        if not there.any():
            continue
        for h in range(hq):
            g = h * hkv // hq
            x = np.where(there, k[g] @ np.asarray(q[s, h], np.float64) * scale, -np.inf)
            e = np.exp(x - x.max())
            e /= e.sum()
            o[s, h] = e @ np.where(there[:, None], v[g], 0)
            w[s, :n] += np.pad(e, (0, n * P - L)).reshape(n, P).sum(1)
    return o, w


def evict_select(seq_len, weight, budget, page_size, sink_pages, recent_tokens):
    """The pages that stay of each sequence, ascending."""
    out = []
    for L, w, b in zip(seq_len, weight, budget):
        n = -(-max(int(L), 0) // page_size)
        fixed = [p for p in range(n) if p < sink_pages or (p + 1) * page_size > L - recent_tokens]
        rest = sorted((p for p in range(n) if p not in set(fixed)),
                      key=lambda p: (0, -float(w[p]), p) if w[p] == w[p] else (1, 0, p))
        out.append(sorted(fixed + rest[:max(0, int(b) - len(fixed))]))
    return out


def steps(row, bits):
    """Probabilities as whole steps of 2^-bits: clamped to [0, 1], NaN as 0."""
    x = np.asarray(row, np.float64)
    return np.rint(np.clip(np.where(np.isnan(x), 0, x), 0, 1) * 2.0 ** bits).astype(np.int64)


def verify(p, q, draft, n_draft, u, bits=50):
    """p [S][n][V], q [S][n - 1][V] or None, draft [S][n - 1], u [S][n]:
    (accepted [S], tokens [S][n]). bits: 50 for fp32 values, 45 for bf16."""
    S, n, V = p.shape
    accepted, tokens = np.zeros(S, np.int32), np.full((S, n), -1, np.int32)
    for s in range(S):
        last = n - 1 if n_draft is None else min(max(int(n_draft[s]), 0), n - 1)
        a = 0
        while a < last:
            x = int(draft[s, a])
            if not 0 <= x < V:
                break
            px, qx, ux = float(p[s, a, x]), 1.0 if q is None else float(q[s, a, x]), float(u[s, a])
            left = Fraction(ux) * Fraction(qx) if np.isfinite(ux) and np.isfinite(qx) else ux * qx
            if not left < px:  # exact for finite values; NaN is below nothing
                break
            a += 1
        target = steps(p[s, a], bits)
        weight = target
        if a < last:
            if q is None:
                weight = target.copy()
                if 0 <= draft[s, a] < V:
                    weight[int(draft[s, a])] = 0
            else:
                weight = np.maximum(target - steps(q[s, a], bits), 0)
            if not weight.any():
                weight = target
        accepted[s] = a
        if a:
            tokens[s, :a] = draft[s, :a]
        if weight.any():
            cum = np.cumsum(weight.astype(object)) if weight.sum(dtype=np.float64) > 2.0 ** 62 else np.cumsum(weight)
            ux = float(u[s, n - 1])
            ux = min(max(0.0 if ux != ux else ux, 0.0), 1 - 2.0 ** -24)
            at = int(Fraction(ux) * int(cum[-1]))  # floor
            tokens[s, a] = int(np.searchsorted(cum, at, side="right"))
    return accepted, tokens
