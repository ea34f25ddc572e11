"""Packed sequences, the paged cache and rotary positions in float64 on the CPU: the definitions, written out.

TEST INFRASTRUCTURE ONLY (see the package docstring). Packed tensors are ``[T, H, d]``; sequence b is rows
``cu[b]:cu[b + 1]``. Paged tensors are ``[n_pages, Hkv, page, d]``; key j of sequence b is slot ``j % page`` of page
``table[b, j // page]``. Query head h reads KV head ``h // (Hq // Hkv)``. The n new tokens of a paged sequence are the
last of its ``lens[b]`` cached ones. A row that sees no key has O = 0 and L = -inf.

Every function also returns what the tests' error bounds are made of: sums of the magnitudes that a rounding of the
softmax weights (or of dS) multiplies.
"""

from __future__ import annotations

import numpy as np


def _rows(q, k, v, first, causal, scale):
    """One sequence and head: weights P [n, m], O, L; query i sits at place first + i."""
    n, m = q.shape[0], k.shape[0]
    s = scale * (q @ k.T) if m else np.zeros((n, 0))
    seen = np.ones((n, m), dtype=bool)
    if causal:
        seen = np.arange(m)[None] <= (first + np.arange(n))[:, None]
    p = np.zeros((n, m))
    lse = np.full(n, -np.inf)
    for i in range(n):
        z = s[i, seen[i]]
        if z.size:
            top = z.max()
            e = np.exp(z - top)
            p[i, seen[i]] = e / e.sum()
            lse[i] = top + np.log(e.sum())
    return p, p @ v if m else np.zeros((n, v.shape[1])), lse


def packed_fwd_ref(q, k, v, cu, causal, scale):
    """O [T, Hq, d], L [Hq, T] and sum_j P_ij |v_j| like O; NaN in rows outside every sequence."""
    T, hq, d = q.shape
    r = hq // k.shape[1]
    O, A, L = np.full((T, hq, d), np.nan), np.full((T, hq, d), np.nan), np.full((hq, T), np.nan)
    for b in range(len(cu) - 1):
        at = slice(cu[b], cu[b + 1])
        for h in range(hq):
            p, O[at, h], L[h, at] = _rows(q[at, h], k[at, h // r], v[at, h // r], 0, causal, scale)
            A[at, h] = p @ np.abs(v[at, h // r])
    return O, L, A


def packed_bwd_ref(q, k, v, dout, cu, causal, scale, c):
    """dQ, dK, dV and for each a bound on what errors of relative size c of the weights, of dS and of O make of it.

    dV = P^T dO; dS = P o (dO V^T - D), D_i = sum_c dO_ic O_ic; dQ = scale dS K, dK = scale dS^T Q.
    """
    T, hq, d = q.shape
    r = hq // k.shape[1]
    out = [np.full(x.shape, np.nan) for x in (q, k, v)] + [np.zeros(x.shape) for x in (q, k, v)]
    dq, dk, dv, eq, ek, ev = out
    for b in range(len(cu) - 1):
        at = slice(cu[b], cu[b + 1])
        dk[at] = dv[at] = 0.0
        for h in range(hq):
            g = h // r
            qs, ks, vs, do = q[at, h], k[at, g], v[at, g], dout[at, h]
            p, o, _ = _rows(qs, ks, vs, 0, causal, scale)
            ds = p * (do @ vs.T - (do * o).sum(1, keepdims=True))
            d_err = (np.abs(do) * (p @ np.abs(vs))).sum(1, keepdims=True)
            s_err = c * (np.abs(ds) + p * d_err)
            dv[at, g] += p.T @ do
            ev[at, g] += c * (p.T @ np.abs(do))
            dq[at, h] = scale * ds @ ks
            eq[at, h] = scale * s_err @ np.abs(ks)
            dk[at, g] += scale * ds.T @ qs
            ek[at, g] += scale * s_err.T @ np.abs(qs)
    return dq, dk, dv, eq, ek, ev


def paged_keys(pages, table_row, n):
    """The first n keys [n, Hkv, d] of a sequence."""
    page = pages.shape[2]
    return np.stack([pages[table_row[j // page], :, j % page] for j in range(n)]) if n else \
        np.zeros((0, pages.shape[1], pages.shape[3]))


def paged_ref(q, k_pages, v_pages, table, lens, cu, causal, scale):
    """As packed_fwd_ref, for new tokens over a paged cache."""
    T, hq, d = q.shape
    r = hq // k_pages.shape[1]
    O, A, L = np.full((T, hq, d), np.nan), np.full((T, hq, d), np.nan), np.full((hq, T), np.nan)
    for b in range(len(cu) - 1):
        at = slice(cu[b], cu[b + 1])
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        k, v = (paged_keys(x, table[b], lens[b]) for x in (k_pages, v_pages))
        for h in range(hq):
            p, O[at, h], L[h, at] = _rows(q[at, h], k[:, h // r], v[:, h // r], lens[b] - n, causal, scale)
            A[at, h] = p @ np.abs(v[:, h // r])
    return O, L, A


def rope_ref(x, positions, inv_freq, sections, interleaved, inverse):
    """Pair i of every head turned by positions[axis of i] * inv_freq[i]; x [T, H, d], positions [axes, T]."""
    y = np.array(x)
    pairs = sum(sections)
    i = 0
    for axis, n in enumerate(sections):
        for _ in range(n):
            t = positions[axis].astype(np.float64) * inv_freq[i] * (-1.0 if inverse else 1.0)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
            cos, sin = np.cos(t)[:, None], np.sin(t)[:, None]
            y[:, :, a] = x[:, :, a] * cos - x[:, :, b] * sin
            y[:, :, b] = x[:, :, b] * cos + x[:, :, a] * sin
            i += 1
    return y


def places(lens, cu, T):
    """(sequence, place) of each of T tokens, (-1, 0) outside every sequence."""
    out = [(-1, 0)] * T
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            out[cu[b] + i] = (b, int(lens[b]) - n + i)
    return out


def append_ref(pages, x, table, lens, cu):
    """Pages with x [T, Hkv, d] written to the tokens' places; places below 0 are left out."""
    out = np.array(pages)
    page = pages.shape[2]
    for t, (b, at) in enumerate(places(lens, cu, x.shape[0])):
        if b >= 0 and at >= 0:
            out[table[b, at // page], :, at % page] = x[t]
    return out
