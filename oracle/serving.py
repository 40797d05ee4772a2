"""fp64 CPU oracle for the serving cache, attention of drafted tokens over it, and causal
attention with a sliding window and sinks (forward and gradients).

TEST INFRASTRUCTURE ONLY, like the rest of this package. Everything is written from the
definitions, row by row, in numpy.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import kv_head

# element formats: mantissa bits, bias, largest finite value, number of non-negative codes
_ELEMENT = {"mxfp8": (3, 7, 448.0, 127), "mxfp4": (1, 1, 6.0, 8)}


def element_values(fmt: str) -> np.ndarray:
    """The value of every non-negative code, in code order (e4m3 without its NaN, e2m1)."""
    bits, bias, top, n = _ELEMENT[fmt]
    out = []
    for code in range(n):
        e, m = code >> bits, code & ((1 << bits) - 1)
        frac = m / (1 << bits)
        out.append(frac * 2.0 ** (1 - bias) if e == 0 else (1 + frac) * 2.0 ** (e - bias))
    assert out[-1] == top
    return np.array(out)


def quantise(x: np.ndarray, fmt: str):
    """x [..., D] fp64 -> (codes [..., D] int with the sign in the top bit, scale bytes [..., D/32],
    the values they stand for). Blocks of 32; the scale is the smallest power of two (not below
    2^-127) with max|x| <= top * scale; nearest code, ties to the even one."""
    bits, _, top, n = _ELEMENT[fmt]
    table = element_values(fmt)
    mid = (table[:-1] + table[1:]) / 2
    shape = x.shape
    blocks = np.asarray(x, dtype=np.float64).reshape(-1, 32)
    codes = np.zeros(blocks.shape, dtype=np.int64)
    bytes_ = np.zeros(blocks.shape[0], dtype=np.int64)
    values = np.zeros(blocks.shape)
    for r, blk in enumerate(blocks):
        if not np.isfinite(blk).all():
            bytes_[r] = 255
            values[r] = np.nan
            continue
        k = -127
        big = np.abs(blk).max()
        if big > 0:
            k = max(-127, math.frexp(big / top)[1] - 1)  # 2^k <= big/top < 2^(k+1), then up unless exact
            if math.ldexp(top, k) < big:
                k += 1
        y = np.abs(blk) * 2.0 ** -k
        c = np.searchsorted(mid, y, side="left")       # ties land below: move the odd ones up
        tie = (c < n - 1) & (np.take(np.append(mid, np.inf), c) == y) & (c % 2 == 1)
        c = c + tie
        bytes_[r] = k + 127
        sign = np.signbit(blk)
        codes[r] = c + sign * (1 << (bits + (4 if fmt == "mxfp8" else 2)))
        values[r] = np.where(sign, -1.0, 1.0) * table[c] * 2.0 ** k
    return codes.reshape(shape), bytes_.reshape(*shape[:-1], shape[-1] // 32), values.reshape(shape)


def tree_visible(n: int, parents, T: int, window: int, sinks: int) -> np.ndarray:
    """[T, n + T] truth: drafted node t (at position n + its depth) sees cache row u."""
    ok = np.zeros((T, n + T), dtype=bool)
    depth = []
    for t in range(T):
        p = t - 1 if parents is None else int(parents[t])
        depth.append(0 if p < 0 else depth[p] + 1)
    for t in range(T):
        pos = n + depth[t]

        def sees(u):
            return window <= 0 or u > pos - window or u < sinks

        for u in range(n):
            ok[t, u] = sees(u)
        j = t
        while j >= 0:
            ok[t, n + j] = sees(n + depth[j])
            j = j - 1 if parents is None else int(parents[j])
    return ok


def window_visible(S: int, window: int, sinks: int) -> np.ndarray:
    """[S, S] truth: token t sees u <= t in its last `window` tokens or among the first `sinks`."""
    t = np.arange(S)[:, None]
    u = np.arange(S)[None]
    return (u <= t) & ((u > t - window) | (u < sinks))


def masked_attention(q, K, V, ok, scale: float):
    """Rows q [n, D] over K, V [L, D] where ok [n, L]. Returns (O, lse, A, E): A = sum p |v| and E =
    the largest scale * sum |q k| of each row, the magnitudes that rounding errors scale with.
    A row that sees nothing: O = 0, lse = -inf."""
    n, D = q.shape
    O, A = np.zeros((n, D)), np.zeros((n, D))
    lse, E = np.full(n, -np.inf), np.zeros(n)
    for i in range(n):
        sel = np.nonzero(ok[i])[0]
        if sel.size == 0:
            continue
        s = scale * (K[sel] @ q[i])
        m = s.max()
        p = np.exp(s - m)
        l = p.sum()
        p /= l
        O[i], A[i], lse[i] = p @ V[sel], p @ np.abs(V[sel]), m + math.log(l)
        E[i] = (scale * (np.abs(K[sel]) @ np.abs(q[i]))).max()
    return O, lse, A, E


def tree_reference(q, k, v, lengths, parents, counts, window: int, sinks: int, scale: float):
    """q [B,Hq,T,D]; k, v [B,Hkv,C,D] the cache's values; lengths, counts per sequence (counts None: T);
    parents [B,T] or None. Returns (O, lse, A, E) shaped like the output."""
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    O, A = np.zeros((B, Hq, T, D)), np.zeros((B, Hq, T, D))
    lse, E = np.full((B, Hq, T), -np.inf), np.zeros((B, Hq, T))
    for b in range(B):
        n, cnt = int(lengths[b]), T if counts is None else int(counts[b])
        if cnt == 0:
            continue
        ok = tree_visible(n, None if parents is None else parents[b], cnt, window, sinks)
        for h in range(Hq):
            g = kv_head(h, Hq, Hkv)
            O[b, h, :cnt], lse[b, h, :cnt], A[b, h, :cnt], E[b, h, :cnt] = masked_attention(
                q[b, h, :cnt], k[b, g, :n + cnt], v[b, g, :n + cnt], ok, scale)
    return O, lse, A, E


def window_reference(q, k, v, window: int, sinks: int, scale: float):
    """Causal attention with a sliding window and sinks: (O, lse, A, E)."""
    B, Hq, S, D = q.shape
    ok = window_visible(S, window, sinks)
    O, A = np.zeros((B, Hq, S, D)), np.zeros((B, Hq, S, D))
    lse, E = np.zeros((B, Hq, S)), np.zeros((B, Hq, S))
    for b in range(B):
        for h in range(Hq):
            g = kv_head(h, Hq, k.shape[1])
            O[b, h], lse[b, h], A[b, h], E[b, h] = masked_attention(q[b, h], k[b, g], v[b, g], ok, scale)
    return O, lse, A, E


def window_backward_reference(q, k, v, out, lse, dout, window: int, sinks: int, scale: float):
    """Gradients from the given out and lse, and the magnitudes that their rounding errors scale with:
    (dq, dk, dv, mq, mk, mv)."""
    B, Hq, S, D = q.shape
    Hkv = k.shape[1]
    ok = window_visible(S, window, sinks)
    dq, mq = np.zeros(q.shape), np.zeros(q.shape)
    dk, dv, mk, mv = (np.zeros(k.shape) for _ in range(4))
    for b in range(B):
        for h in range(Hq):
            g = kv_head(h, Hq, Hkv)
            Q, K, V, dO = q[b, h], k[b, g], v[b, g], dout[b, h]
            P = np.where(ok, np.exp(np.where(ok, scale * (Q @ K.T), 0.0) - lse[b, h][:, None]), 0.0)
            delta = (dO * out[b, h]).sum(1)[:, None]
            dS = P * (dO @ V.T - delta)
            # what dS is computed from, in magnitude: P (|dO||V| + |dO||O|)
            mS = P * (np.abs(dO) @ np.abs(V).T + (np.abs(dO) * np.abs(out[b, h])).sum(1)[:, None])
            dq[b, h], mq[b, h] = scale * (dS @ K), scale * (mS @ np.abs(K))
            dk[b, g] += scale * (dS.T @ Q)
            mk[b, g] += scale * (mS.T @ np.abs(Q))
            dv[b, g] += P.T @ dO
            mv[b, g] += P.T @ np.abs(dO)
    return dq, dk, dv, mq, mk, mv
