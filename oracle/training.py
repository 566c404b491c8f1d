"""Plain fp64 reference of the operators around the HiMuon update in a training step: the
clipped policy loss with its gradient, the gradient norm and AdamW with fp32 or 8-bit
states.  numpy only, elementwise from the formulas, no code shared with the GPU path."""
from __future__ import annotations

import numpy as np

BLOCK = 256
E4M3_MAX = 448.0
TINY = 2.0 ** -100
MULT = (0x9E3779B1, 0x85EBCA6B)


def policy_loss(logits, label, weight, advantage, old_logp=None, ref_logp=None, clip=(0.2, 0.2), kl_coef=0.0,
                temperature=1.0, grad_scale=1.0):
    """(stats (4), logp (N), dlogits (N, V)) of the clipped policy loss, row by row."""
    z = np.asarray(logits, np.float64)
    N, V = z.shape
    stats, logp, grad = np.zeros(4), np.zeros(N), np.zeros((N, V))
    for i in range(N):
        y, w = int(label[i]), float(weight[i])
        if w == 0 or not 0 <= y < V:
            continue
        with np.errstate(all="ignore"):
            row = z[i] / temperature
            top = row.max()
            e = np.exp(row - top)
            lp = row[y] - top - np.log(e.sum())
            A = float(advantage[i])
            rho = 1.0 if old_logp is None else np.exp(lp - float(old_logp[i]))
            if old_logp is None and np.isnan(lp):
                rho = lp
            u, c = rho * A, np.clip(rho, 1 - clip[0], 1 + clip[1]) * A
            d = 0.0 if ref_logp is None else float(ref_logp[i]) - lp
            kl = np.expm1(d) - d
            clipped = u > c
            surrogate = c if clipped else u
            logp[i] = lp
            count = (kl_coef * kl, kl_coef * np.expm1(d)) if kl_coef else (0.0, 0.0)
            stats += w * np.array([count[0] - surrogate, -surrogate, kl, float(clipped)])
            dlp = (0.0 if clipped else -u) - count[1]
            grad[i] = -dlp * (e / e.sum())
            grad[i, y] += dlp
            grad[i] *= grad_scale * w / temperature
    return stats, logp, grad


def grad_norm(grads, max_norm):
    """(norm, factor): the 2-norm over all arrays and min(1, max_norm / (norm + 1e-6)) (NaN if not finite)."""
    with np.errstate(all="ignore"):
        total = sum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads)
    norm = np.sqrt(total)
    return norm, min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(total) else np.nan


def adamw(w, g, m, v, t, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, scale=1.0):
    """(w, m, v) after step t; a NaN scale changes nothing."""
    w, g, m, v = (np.asarray(x, np.float64) for x in (w, g, m, v))
    if np.isnan(scale):
        return w, m, v
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    hat = (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return w - lr * (hat + weight_decay * w), m, v


def e4m3_values():
    """The value of every e4m3 byte (OCP: no infinities, 0x7f and 0xff are NaN)."""
    out = np.empty(256)
    for b in range(256):
        e, f = b >> 3 & 15, b & 7
        x = (8 + f) * 2.0 ** (e - 10) if e else f * 2.0 ** -9
        out[b] = np.nan if b & 127 == 127 else -x if b & 128 else x
    return out


def unpack8(code, scale):
    """fp64 values that e4m3 bytes and their per-block scales stand for."""
    unit = np.repeat(np.asarray(scale, np.float64), BLOCK)[:code.size]
    return e4m3_values()[code] * unit


def pack8(x, kind, dither):
    """x (fp64, flat) in the 8-bit state format: (values, scale, margin).  kind 0: first moment, 1: root of the
    second.  values are in units of the scale; margin is the distance, in units of the neighbours' gap, of the
    dithered magnitude to the nearest point where the rounding turns over (rounding errors of another computation
    smaller than that leave the value unchanged).  Elements that are not finite have the value NaN and no part in
    their block's scale."""
    x = np.asarray(x, np.float64)
    lost = ~np.isfinite(x)
    x = np.where(lost, 0.0, x)
    n = x.size
    i = np.arange(n, dtype=np.uint64)
    u = (((i * MULT[kind] + dither) % 2 ** 32) >> np.uint64(16)).astype(np.float64)
    u = (u + 0.5) / 65536
    blocks = -(-n // BLOCK)
    values, scale, margin = np.zeros(n), np.zeros(blocks), np.full(n, np.inf)
    for b in range(blocks):
        s = slice(b * BLOCK, min(n, (b + 1) * BLOCK))
        peak = np.abs(x[s]).max()
        if peak < TINY:
            continue
        y = np.abs(x[s]) * (E4M3_MAX / peak)
        gap = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
        at = y / gap + u[s]
        q = np.floor(at) * gap
        margin[s] = np.where(x[s] == 0, np.inf, np.minimum(at - np.floor(at), 1 - (at - np.floor(at))))
        q = np.clip(q, 2.0 ** -9 if kind else 0.0, E4M3_MAX)
        values[s] = np.where(x[s] == 0, 0.0, np.sign(x[s]) * q)
        scale[b] = peak / E4M3_MAX
    values[lost] = np.nan
    return values, scale, margin


def distill_loss(logits, value, index, weight, rest=None, temperature=1.0, grad_scale=1.0):
    """(loss, kl (N), dlogits (N, V)) of the distillation loss on a teacher's entries, row by row."""
    z = np.asarray(logits, np.float64)
    N, V = z.shape
    kl, grad = np.zeros(N), np.zeros((N, V))
    for i in range(N):
        w = float(weight[i])
        if w == 0:
            continue
        with np.errstate(all="ignore"):
            counts = [j for j in range(len(index[i])) if 0 <= index[i][j] < V]
            token = np.array([int(index[i][j]) for j in counts], np.int64)
            t = np.array([float(value[i][j]) for j in counts]) / temperature
            if rest is not None:
                t = np.append(t, float(rest[i]))
            if not (t != -np.inf).any():
                continue
            q = np.exp(t - t.max())
            q /= q.sum()
            logq = t - t.max() - np.log(np.exp(t - t.max()).sum())
            row = z[i] / temperature
            lse = row.max() + np.log(np.exp(row - row.max()).sum())
            others = np.ones(V, bool)
            others[token] = False
            lp = row[token] - lse
            share = np.zeros(V)
            if rest is not None:
                top = row[others].max() if others.any() else -np.inf
                e = np.exp(row[others] - top) if np.isfinite(top) else np.zeros(others.sum())
                if np.isnan(row).any():
                    e = e * np.nan
                lp = np.append(lp, top + np.log(e.sum()) - lse)
                if q[-1] != 0 and e.sum() != 0:
                    share[others] = q[-1] * (e / e.sum())
            kl[i] = sum(a * (b - c) for a, b, c in zip(q, logq, lp) if a != 0)
            grad[i] = np.exp(row - lse) - share
            for v, a in zip(token, q):
                grad[i, v] -= a
            if np.isnan(q).any():
                grad[i] = np.nan
            grad[i] *= grad_scale * w / temperature
    return float(sum(w * d for w, d in zip(np.asarray(weight, np.float64), kl) if d != 0)), kl, grad
