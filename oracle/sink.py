"""Sliding-window attention with sink tokens and the query/key norm with rotation,
float64, written from their definitions.

Test infrastructure only (see the package docstring).

The window follows the reading of ``swa``: w keys including the query's own. The
first ``sinks`` tokens stay visible to every later query. Query head h reads
key/value head h // (Hq // Hkv). ``lengths`` are the tokens per sequence of a padded
batch; padding rows are zeros (lse: -inf).
"""

from __future__ import annotations

import numpy as np


def sink_visible(n: int, w: int, sinks: int) -> np.ndarray:
    """visible[i, j]: j <= i and (j > i - w or j < sinks)."""
    i = np.arange(n)[:, None]
    j = np.arange(n)[None, :]
    return (j <= i) & ((j > i - w) | (j < sinks))


def _weights(q, k, w, sinks, scale):
    s = np.where(sink_visible(q.shape[0], w, sinks), scale * (q @ k.T), -np.inf)
    m = s.max(axis=1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(axis=1, keepdims=True)
    return e / l, (m + np.log(l))[:, 0]


def _lengths(lengths, B, N):
    return [N] * B if lengths is None else [int(n) for n in lengths]


def swa_sink(q, k, v, w: int, sinks: int, scale: float, lengths=None):
    """(y, lse, mass): mass_i = sum_j p_ij |v_j|, the scale of the rounding error of p."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    B, Hq, N, d = q.shape
    G = Hq // k.shape[1]
    y = np.zeros_like(q)
    mass = np.zeros_like(q)
    lse = np.full((B, Hq, N), -np.inf)
    for b, n in enumerate(_lengths(lengths, B, N)):
        for h in range(Hq if n else 0):
            p, ls = _weights(q[b, h, :n], k[b, h // G, :n], w, sinks, scale)
            y[b, h, :n] = p @ v[b, h // G, :n]
            mass[b, h, :n] = p @ np.abs(v[b, h // G, :n])
            lse[b, h, :n] = ls
    return y, lse, mass


def swa_sink_backward(q, k, v, dy, w: int, sinks: int, scale: float, lengths=None, y_error=None, rel: float = 0.0):
    """(dq, dk, dv) of swa_sink for dy, and the bounds (eq, ek, ev) of their errors when
    p and dS are off by at most `rel` of their size and y by at most y_error:
        |d dS_ij| <= rel |dS_ij| + scale p_ij sum_c |dy_ic| y_error_ic.
    """
    q, k, v, dy = (np.asarray(x, dtype=np.float64) for x in (q, k, v, dy))
    B, Hq, N, d = q.shape
    G = Hq // k.shape[1]
    out = [np.zeros_like(x) for x in (q, k, v, q, k, v)]
    dq, dk, dv, eq, ek, ev = out
    for b, n in enumerate(_lengths(lengths, B, N)):
        for h in range(Hq if n else 0):
            qh, gh = q[b, h, :n], dy[b, h, :n]
            kh, vh = k[b, h // G, :n], v[b, h // G, :n]
            p, _ = _weights(qh, kh, w, sinks, scale)
            dp = gh @ vh.T
            ds = scale * p * (dp - (p * dp).sum(axis=1, keepdims=True))
            dq[b, h, :n] = ds @ kh
            dk[b, h // G, :n] += ds.T @ qh
            dv[b, h // G, :n] += p.T @ gh
            err = rel * np.abs(ds)
            if y_error is not None:
                err = err + scale * p * (np.abs(gh) * y_error[b, h, :n]).sum(axis=1, keepdims=True)
            eq[b, h, :n] = err @ np.abs(kh)
            ek[b, h // G, :n] += err.T @ np.abs(qh)
            ev[b, h // G, :n] += rel * (p.T @ np.abs(gh))
    return tuple(out)


def swa_sink_cache(x, w: int, sinks: int, lengths=None) -> np.ndarray:
    """[B, H, sinks + w, d]: slot t < sinks holds token t, slot sinks + (t - sinks) mod w
    the latest token t >= sinks; zeros where no token went."""
    x = np.asarray(x, dtype=np.float64)
    B, H, N, d = x.shape
    out = np.zeros((B, H, sinks + w, d))
    for b, n in enumerate(_lengths(lengths, B, N)):
        for t in range(n):
            out[b, :, t if t < sinks else sinks + (t - sinks) % w] = x[b, :, t]
    return out


def swa_sink_decode_step(k_cache, v_cache, positions, q, k, v, w: int, sinks: int, scale: float):
    """One token per sequence; (y, k_cache', v_cache', mass). positions[b] < 0: idle."""
    kc, vc = (np.array(x, dtype=np.float64) for x in (k_cache, v_cache))
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    y = np.zeros_like(q)
    mass = np.zeros_like(q)
    G = q.shape[1] // k.shape[1]
    for b, t in enumerate(int(p) for p in positions):
        if t < 0:
            continue
        slot = t if t < sinks else sinks + (t - sinks) % w
        kc[b, :, slot] = k[b]
        vc[b, :, slot] = v[b]
        n = min(t + 1, sinks + w)
        for h in range(q.shape[1]):
            s = scale * (kc[b, h // G, :n] @ q[b, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            y[b, h] = p @ vc[b, h // G, :n]
            mass[b, h] = p @ np.abs(vc[b, h // G, :n])
    return y, kc, vc, mass


def rope_angles(positions, rot: int, base: float) -> np.ndarray:
    """[..., rot / 2]: position * base^(-2 i / rot)."""
    return np.asarray(positions, dtype=np.float64)[..., None] * base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))


def _pairs(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def norm_rope(x, weight, angles, rot: int, eps: float, interleaved: bool):
    """x [B, H, N, d], angles [B, N, rot / 2]; (out, size): size bounds the terms of each output."""
    x = np.asarray(x, dtype=np.float64)
    n = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * weight
    out, size = n.copy(), np.abs(n)
    if rot:
        a, b = _pairs(rot, interleaved)
        c, s = np.cos(angles)[:, None], np.sin(angles)[:, None]
        out[..., a] = n[..., a] * c - n[..., b] * s
        out[..., b] = n[..., a] * s + n[..., b] * c
        size[..., a] = np.abs(n[..., a] * c) + np.abs(n[..., b] * s)
        size[..., b] = np.abs(n[..., a] * s) + np.abs(n[..., b] * c)
    return out, size


def norm_rope_backward(x, weight, angles, dout, rot: int, eps: float, interleaved: bool):
    """(dx, dweight, dx_size, dweight_size): the sizes bound the terms of each sum."""
    x, g = np.asarray(x, dtype=np.float64), np.asarray(dout, dtype=np.float64)
    dn, dn_size = g.copy(), np.abs(g)
    if rot:
        a, b = _pairs(rot, interleaved)
        c, s = np.cos(angles)[:, None], np.sin(angles)[:, None]
        dn[..., a] = g[..., a] * c + g[..., b] * s
        dn[..., b] = g[..., b] * c - g[..., a] * s
        dn_size[..., a] = np.abs(g[..., a] * c) + np.abs(g[..., b] * s)
        dn_size[..., b] = np.abs(g[..., b] * c) + np.abs(g[..., a] * s)
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    xh = x * r
    dh = dn * weight
    dx = r * (dh - xh * (dh * xh).mean(axis=-1, keepdims=True))
    hs = dn_size * np.abs(weight)
    dx_size = r * (hs + np.abs(xh) * (hs * np.abs(xh)).mean(axis=-1, keepdims=True))
    return dx, (dn * xh).sum(axis=(0, 1, 2)), dx_size, (dn_size * np.abs(xh)).sum(axis=(0, 1, 2))
