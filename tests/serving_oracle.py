"""Plain float64 forms of the operators around the attention of a serving
step: head norms with rotation, the tree of drafted tokens, scored decode and
eviction.  Test infrastructure only; written from the definitions in
include/gqa.h, one row at a time, sharing nothing with the library.

Each attention function also returns the absolute mix sum_j p_j |v_j| of every
output, in which the rounding bounds are stated."""
import numpy as np


def norm_rope(x, Hq, Hkv, d, qw, kw, eps, inv_freq, positions, axes, interleaved):
    """x [B,T,(Hq+2Hkv)d] -> q, k, v, and per output the sum |u| + |v| of the
    pair it was made from (itself where it is not rotated)."""
    B, T, _ = x.shape
    x = x[:, :, :(Hq + 2 * Hkv) * d].reshape(B, T, Hq + 2 * Hkv, d)
    half = 0 if inv_freq is None else len(inv_freq)
    outs, mags = [], []
    for h in range(Hq + 2 * Hkv):
        y = x[:, :, h].copy()
        w = qw if h < Hq else (kw if h < Hq + Hkv else None)
        if w is not None:
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
        z, m = y.copy(), np.abs(y)
        if h < Hq + Hkv:
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                ang = positions[axes[i]].astype(np.float64) * inv_freq[i]
                z[..., a] = y[..., a] * np.cos(ang) - y[..., b] * np.sin(ang)
                z[..., b] = y[..., b] * np.cos(ang) + y[..., a] * np.sin(ang)
                m[..., a] = m[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
        outs.append(z)
        mags.append(m)
    def pick(lst, a, b):
        return np.stack(lst[a:b], axis=1)
    cut = (0, Hq, Hq + Hkv, Hq + 2 * Hkv)
    return [pick(outs, cut[i], cut[i + 1]) for i in range(3)], \
        [pick(mags, cut[i], cut[i + 1]) for i in range(3)]


def line_of(parents, i):
    """Node i and its ancestors from the node up; None for padding, "bad" for
    a node whose line meets an invalid parent."""
    out = []
    at = i
    while True:
        out.append(at)
        up = -1 if parents is None and at == 0 else (at - 1 if parents is None else int(parents[at]))
        if up == -1:
            return out
        if up == -2 and at == i:
            return None
        if up < 0 or up >= at:
            return "bad"
        at = up


def _mix(q, ks, vs, scale):
    """softmax over rows ks, mix of vs: (o, absolute mix, weights)."""
    s = ks @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ vs, p @ np.abs(vs), p


def tree(q, kc, vc, kd, vd, parents, lens, window=None, scale=None):
    """-> o, absolute mix; a refused sequence or node is zero."""
    B, Hq, t, d = q.shape
    Hkv, C = kc.shape[1], kc.shape[2]
    r = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        n = lens[b]
        if not 0 <= n <= C:
            continue
        for i in range(t):
            line = line_of(None if parents is None else parents[b], i)
            if line is None or line == "bad":
                continue
            depth = len(line) - 1
            lo = 0 if window is None else max(0, n + depth - (window - 1))
            if window is not None:
                line = line[:window]
            for h in range(Hq):
                g = h // r
                ks = np.concatenate([kc[b, g, lo:n], kd[b, g, line]])
                vs = np.concatenate([vc[b, g, lo:n], vd[b, g, line]])
                o[b, h, i], mag[b, h, i], _ = _mix(q[b, h, i], ks, vs, scale)
    return o, mag


def scored(q, kc, vc, lens, scale=None):
    """-> o, absolute mix, weights received by each cell, and the largest
    scale * sum |q| |k| (which bounds a score's rounding)."""
    B, Hq, t, d = q.shape
    Hkv, C = kc.shape[1], kc.shape[2]
    r = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    o, mag, w, big = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, Hkv, C)), 0.0
    for b in range(B):
        n = lens[b]
        if not t <= n <= C:
            continue
        for h in range(Hq):
            g = h // r
            for i in range(t):
                z = n - t + i + 1
                o[b, h, i], mag[b, h, i], p = _mix(q[b, h, i], kc[b, g, :z], vc[b, g, :z], scale)
                w[b, g, :z] += p
                big = max(big, float((np.abs(kc[b, g, :z]) @ np.abs(q[b, h, i])).max() * abs(scale)))
    return o, mag, w, big


def survivors(w, n, budget, recent):
    """Cells of a lane of n cells that stay, ascending."""
    if n <= budget:
        return list(range(n))
    order = sorted(range(n - recent), key=lambda j: (-w[j] if w[j] == w[j] else np.inf, j))
    return sorted(order[:budget - recent]) + list(range(n - recent, n))
