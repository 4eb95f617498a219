"""Plain fp64 oracle of cross attention and of rotary positions with several axes.

Test infrastructure only, as ``oracle.attention``: no code in common with the library.

* ``cross_head`` / ``cross_attention`` -- S = scale q K^T over a sequence's own keys, P = softmax(S),
  O = P V, lse = ln sum exp S; query head h reads key head h // (Hq / Hkv).  A sequence without keys
  gets O = 0, lse = -inf.
* ``cross_backward`` -- dV = P^T dO, dS = P * (dO V^T - rowsum(O dO)), dQ = scale dS K,
  dK = scale dS^T Q, summed over the query heads of a key head.
* ``rope_rates`` / ``rope`` -- pair i turned by pos[axis_i] * rate_i.

``cross_attention`` and ``cross_backward`` also return, from the same matrices, the sums of absolute
values that bound the kernels' rounding (see tests/test_gpu_cross.py).
"""

from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x.detach().cpu().double().numpy() if hasattr(x, "detach") else x, dtype=np.float64)


def _softmax(s):
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    t = e.sum(-1, keepdims=True)
    return e / t, (m + np.log(t))[..., 0]


def _lens(kv_lens, B, Nk):
    return [Nk] * B if kv_lens is None else [min(max(int(n), 0), Nk) for n in kv_lens]


def cross_attention(q, k, v, scale, kv_lens=None):
    """O, lse, and P |V| (like O) and the largest scale |q| |k|^T of any pair."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Hq, Nq, d = q.shape
    G, Nk = Hq // k.shape[1], k.shape[2]
    o, pv, lse, big = np.zeros_like(q), np.zeros_like(q), np.full((B, Hq, Nq), -np.inf), 0.0
    for b, n in enumerate(_lens(kv_lens, B, Nk)):
        for h in range(Hq if n else 0):
            kk, vv = k[b, h // G, :n], v[b, h // G, :n]
            p, lse[b, h] = _softmax(scale * q[b, h] @ kk.T)
            o[b, h], pv[b, h] = p @ vv, p @ np.abs(vv)
            big = max(big, scale * float((np.abs(q[b, h]) @ np.abs(kk).T).max()))
    return o, lse, pv, big


def cross_backward(q, k, v, do, scale, kv_lens=None, rel=0.0, o_err=None):
    """dQ, dK, dV, and bounds on what an implementation may be off by whose P and dS are each off by
    ``rel`` of themselves, whose dP - D is off by ``rel`` / 16 of itself (P's share of it) and by ``rel`` / 1024
    of the sums of dP's and D's terms' absolute values, and whose O is off by ``o_err``."""
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(do)
    B, Hq, Nq, d = q.shape
    G, Nk = Hq // k.shape[1], k.shape[2]
    g = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    e = {n: np.zeros_like(x) for n, x in g.items()}
    for b, n in enumerate(_lens(kv_lens, B, Nk)):
        for h in range(Hq if n else 0):
            j = h // G
            qq, kk, vv, dd = q[b, h], k[b, j, :n], v[b, j, :n], do[b, h]
            p, _ = _softmax(scale * qq @ kk.T)
            o, dp = p @ vv, dd @ vv.T
            D = (o * dd).sum(-1, keepdims=True)
            ds = p * (dp - D)
            g["dq"][b, h] = scale * ds @ kk
            g["dk"][b, j, :n] += scale * ds.T @ qq
            g["dv"][b, j, :n] += p.T @ dd
            D_err = (np.abs(dd) * (0 if o_err is None else o_err[b, h])).sum(-1, keepdims=True)
            dp_abs, D_abs = np.abs(dd) @ np.abs(vv).T, (np.abs(o) * np.abs(dd)).sum(-1, keepdims=True)
            ds_err = rel * np.abs(ds) + p * (D_err + rel / 16 * (np.abs(dp - D) + dp_abs / 64 + D_abs / 64))
            e["dq"][b, h] = scale * ds_err @ np.abs(kk)
            e["dk"][b, j, :n] += scale * ds_err.T @ np.abs(qq)
            e["dv"][b, j, :n] += rel * (p.T @ np.abs(dd))
    return g, e


def rope_rates(d, sections, base=10000.0, per_axis=False, cyclic=False):
    """(axis, rate) of each of the d / 2 pairs, by the definition."""
    n, left, order = d // 2, list(sections), []
    while any(left):
        for a in range(len(left)):
            take = min(1, left[a]) if cyclic else left[a]
            order += [a] * take
            left[a] -= take
    assert len(order) == n
    seen = [0] * len(sections)
    rates = []
    for i, a in enumerate(order):
        x = np.longdouble(seen[a]) / sections[a] if per_axis else np.longdouble(i) / n
        seen[a] += 1
        rates.append(np.longdouble(base) ** -x)
    return order, np.array(rates, dtype=np.longdouble)


def rope(x, pos, axis, rates, interleaved=False, inverse=False):
    """x [B, H, N, d] turned by pos [axes, B, N]; also |a| + |b| of each element's pair, like x."""
    x, pos = _f64(x), np.asarray(pos.cpu().numpy() if hasattr(pos, "cpu") else pos).astype(np.longdouble)
    angle = np.stack([pos[a] * r for a, r in zip(axis, rates)], -1)[:, None]  # [B, 1, N, d/2]
    angle = np.remainder(angle, 2 * np.longdouble("3.14159265358979323846264338327950288"))
    c, s = np.cos(angle).astype(np.float64), np.sin(angle).astype(np.float64)
    if inverse:
        s = -s
    n = x.shape[-1] // 2
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, n), slice(n, None))
    a, b = x[..., first], x[..., second]
    y, size = np.empty_like(x), np.empty_like(x)
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    size[..., first] = size[..., second] = np.abs(a) + np.abs(b)
    return y, size
