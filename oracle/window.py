"""Plain fp64 oracle of sliding-window attention with sinks, of RMS norms with rotary positions, and of the cache's pages.

Test infrastructure only, as ``oracle.attention``: no code in common with the library.

* ``visible`` -- query i of N at position p = Nk - N + i sees key j when j <= p and (p - j < W or j < S).
* ``window_attention`` / ``window_backward`` -- softmax over the visible keys and its derivatives, as ``oracle.cross``.
* ``norm_rope`` / ``norm_rope_backward`` -- y = R(w x / sqrt(mean x^2 + eps)) and its derivatives.
* ``pages_extend`` -- the cache's pages on Python lists.

The attention and norm functions also return the sums of absolute values that bound the kernels' rounding (see the tests).
"""

from __future__ import annotations

import numpy as np

from .cross import _f64, _softmax, rope


def visible(N, Nk, window, sinks):
    """[N, Nk] of bool."""
    p, j = np.arange(Nk - N, Nk)[:, None], np.arange(Nk)[None]
    return (j <= p) & ((p - j < window) | (j < sinks))


def _heads(q, k):
    for b in range(q.shape[0]):
        for h in range(q.shape[1]):
            yield b, h, h // (q.shape[1] // k.shape[1])


def _shown(k, v, see):
    """k and v with zeros in place of keys that no query sees (which may hold anything)."""
    keep = see.any(0)[:, None]
    return np.where(keep, k, 0.0), np.where(keep, v, 0.0)


def window_attention(q, k, v, scale, window, sinks=0):
    """O, lse, and P |V| (like O) and the largest scale |q| |k|^T of any pair."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    see = visible(q.shape[2], k.shape[2], window, sinks)
    o, pv, lse, big = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:3]), 0.0
    for b, h, j in _heads(q, k):
        kk, vv = _shown(k[b, j], v[b, j], see)
        p, lse[b, h] = _softmax(np.where(see, scale * q[b, h] @ kk.T, -np.inf))
        o[b, h], pv[b, h] = p @ vv, p @ np.abs(vv)
        big = max(big, scale * float((np.abs(q[b, h]) @ np.abs(kk).T).max()))
    return o, lse, pv, big


def window_backward(q, k, v, do, scale, window, sinks=0, rel=0.0, o_err=None):
    """dQ, dK, dV, and bounds as oracle.cross.cross_backward's."""
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(do)
    see = visible(q.shape[2], k.shape[2], window, sinks)
    g = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    e = {n: np.zeros_like(x) for n, x in g.items()}
    for b, h, j in _heads(q, k):
        kk, vv = _shown(k[b, j], v[b, j], see)
        qq, dd = q[b, h], do[b, h]
        p, _ = _softmax(np.where(see, scale * qq @ kk.T, -np.inf))
        o, dp = p @ vv, dd @ vv.T
        D = (o * dd).sum(-1, keepdims=True)
        ds = p * (dp - D)
        g["dq"][b, h] = scale * ds @ kk
        g["dk"][b, j] += scale * ds.T @ qq
        g["dv"][b, j] += p.T @ dd
        D_err = (np.abs(dd) * (0 if o_err is None else o_err[b, h])).sum(-1, keepdims=True)
        dp_abs, D_abs = np.abs(dd) @ np.abs(vv).T, (np.abs(o) * np.abs(dd)).sum(-1, keepdims=True)
        ds_err = rel * np.abs(ds) + p * (D_err + rel / 16 * (np.abs(dp - D) + dp_abs / 64 + D_abs / 64))
        e["dq"][b, h] = scale * ds_err @ np.abs(kk)
        e["dk"][b, j] += scale * ds_err.T @ np.abs(qq)
        e["dv"][b, j] += rel * (p.T @ np.abs(dd))
    return g, e


def window_decode(q, k, v, lens, scale, window, sinks=0):
    """One token of each sequence: q [B, Hq, d] against the first lens[b] keys of k, v [B, Hkv, L, d]."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Hq, d = q.shape
    o, pv, lse, big = np.zeros_like(q), np.zeros_like(q), np.full((B, Hq), -np.inf), 0.0
    for b, n in enumerate(min(max(int(x), 0), k.shape[2]) for x in lens):
        if n:
            x = window_attention(q[b][None, :, None], k[b:b + 1, :, :n], v[b:b + 1, :, :n], scale, window, sinks)
            o[b], lse[b], pv[b], big = x[0][0, :, 0], x[1][0, :, 0], x[2][0, :, 0], max(big, x[3])
    return o, lse, pv, big


def _norm(x, w, eps):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return r, x * r, x * r * (1.0 if w is None else _f64(w))


def norm_rope(x, w, pos, axis, rates, interleaved=False, eps=1e-6):
    """y, and |a| + |b| of each element's pair of the normed row, like x."""
    return rope(_norm(_f64(x), w, eps)[2], pos, axis, rates, interleaved)


def norm_rope_backward(x, w, dy, pos, axis, rates, interleaved=False, eps=1e-6, far=0.0, rel=0.0):
    """dx [B, H, N, d], dw [d], and bounds on what an implementation may be off by whose turned gradient g is off by ``far``
    of |a| + |b| of its pair and whose norms and sums are off by ``rel`` of their terms' absolute values."""
    x = _f64(x)
    g, size = rope(dy, pos, axis, rates, interleaved, inverse=True)
    r, n, _ = _norm(x, None, eps)
    weight = np.ones(x.shape[-1]) if w is None else _f64(w)
    h, h_err = g * weight, far * size * np.abs(weight)
    dx = r * (h - n * (h * n).mean(-1, keepdims=True))
    mean = np.abs(h * n).mean(-1, keepdims=True)
    dx_err = r * (h_err + np.abs(n) * (h_err * np.abs(n)).mean(-1, keepdims=True) + rel * (np.abs(h) + np.abs(n) * mean))
    dw, dw_abs = (g * n).sum((0, 1, 2)), np.abs(g * n).sum((0, 1, 2))
    dw_err = (far * size * np.abs(n)).sum((0, 1, 2)) + rel * dw_abs
    return dx, dw, dx_err, dw_err, dw_abs


def pages_extend(table, lens, new, stack, n_free, page_size, N=0):
    """The state after a call, on lists: table, lens, stack, n_free, granted, slots [B][N]."""
    table, lens, stack = [list(row) for row in table], list(lens), list(stack)
    free, granted, slots, back, short = min(max(n_free, 0), len(stack)), [], [], [], False
    for b, m in enumerate(new):
        room = len(table[b]) * page_size
        n = min(max(lens[b], 0), room)
        m = max(m, -n)
        had, want = -(-n // page_size), -(-(n + m) // page_size)
        if n + m > room:
            m = 0
        elif want > had:
            short = short or want - had > free
            if short:
                m = 0
            for i in range(had, want if m else had):
                free -= 1
                table[b][i] = stack[free]
        for i in range(want, had):
            back.append(table[b][i])
            table[b][i] = -1
        slots.append([table[b][(n + t) // page_size] * page_size + (n + t) % page_size
                      if t < m and 0 <= table[b][(n + t) // page_size] < len(stack) else -1 for t in range(N)])
        granted.append(m)
        lens[b] = n + m
    for p in reversed(back):
        stack[free] = p
        free += 1
    return table, lens, stack, free, granted, slots
