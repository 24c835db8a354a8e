"""fp64 reference of the operators around the attention calls: the head norm with the
position rotation (and its gradient), the append to a paged cache, 8-bit pages.

Plain numpy loops over rows and pages; it shares nothing with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import sas_oracle as O

BLOCK = O.BLOCK
E4M3_MAX = 448.0
MIN_SCALE_EXP = -64


def f64(x):
    if isinstance(x, torch.Tensor):
        x = x.detach().cpu()
        return x.float().double().numpy() if x.dtype != torch.float64 else x.numpy()
    return np.asarray(x, dtype=np.float64)


def norm(x, w, eps):
    """x [..., D] -> x / rms * w (x itself without weights)."""
    x = f64(x)
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * f64(w)


def rotate(n, table, pos, sign=1.0):
    """n [T, H, D] by the angles of table[pos] (cosines, then sines)."""
    D = n.shape[-1]
    row = f64(table)[np.asarray(pos)][:, None, :]
    c, s = row[..., :D // 2], sign * row[..., D // 2:]
    a, b = n[..., :D // 2], n[..., D // 2:]
    return np.concatenate((a * c - b * s, b * c + a * s), axis=-1)


def norm_rope(x, w, table, pos, eps):
    """x [T, H, D]. Returns y and, for tolerances, |a| + |b| of each rotation pair."""
    n = norm(x, w, eps)
    half = n.shape[-1] // 2
    pair = np.abs(n[..., :half]) + np.abs(n[..., half:])
    return rotate(n, table, pos), np.concatenate((pair, pair), axis=-1)


def norm_rope_bwd(dy, x, w, table, pos, eps):
    """Returns dx, dw (None without weights) and the magnitudes their rounding errors scale with."""
    x, dy = f64(x), f64(dy)
    D = x.shape[-1]
    gn = rotate(dy, table, pos, sign=-1.0)
    pair = np.abs(dy[..., :D // 2]) + np.abs(dy[..., D // 2:])
    pair = np.concatenate((pair, pair), axis=-1)
    if w is None:
        return gn, None, pair, None
    w = f64(w)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    g = gn * w
    dx = r * (g - xh * (g * xh).mean(-1, keepdims=True))
    G = pair * np.abs(w)
    mag = r * (G + np.abs(xh) * (G * np.abs(xh)).mean(-1, keepdims=True))
    return dx, (gn * xh).reshape(-1, D).sum(0), mag, (pair * np.abs(xh)).reshape(-1, D).sum(0)


def scale_of(amax):
    """Least power of two s (not under 2^-64) with amax <= 448 s."""
    if amax == 0.0:
        return 2.0 ** MIN_SCALE_EXP
    m, e = math.frexp(amax)                      # amax = m 2^e, 448 = 0.875 * 2^9
    return 2.0 ** max(MIN_SCALE_EXP, e - 9 + (1 if m > 0.875 else 0))


def new_rows(kv_len, cu_new, T):
    """(sequence, token row, position) of every new token."""
    out = []
    for n in range(len(kv_len)):
        if cu_new is None:
            lo, hi = n, n + (1 if kv_len[n] else 0)
        else:
            lo, hi = int(cu_new[n]), int(cu_new[n + 1])
        for t in range(lo, hi):
            out.append((n, t, int(kv_len[n]) - (hi - t)))
    return out


def page_items(kv_len, cu_new, T, page_table):
    """{page: [(row in page, token row, position), ...]} of one append."""
    items = {}
    for n, t, pos in new_rows(kv_len, cu_new, T):
        items.setdefault(int(page_table[n][pos // BLOCK]), []).append((pos % BLOCK, t, pos))
    return items


def decode_q8(q, k_codes, v_codes, k_scale, v_scale, page_table, kv_len, idx, cnt, log_gate, sm_scale):
    """o, lse and their error bounds for fp32 logits and probabilities of two fp16 numbers (see the body)."""
    q, kc, vc = f64(q), f64(k_codes), f64(v_codes)
    ks, vs = f64(k_scale), f64(v_scale)
    pt, kv_len = page_table.cpu().numpy(), kv_len.cpu().numpy()
    idx, cnt, gate = idx.cpu().numpy(), cnt.cpu().numpy(), f64(log_gate)
    N, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    o, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    o_tol, lse_tol = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    u = 2.0 ** -24
    for n in range(N):
        if kv_len[n] == 0:
            continue
        c = (int(kv_len[n]) - 1) // BLOCK
        for h in range(Hkv):
            # a gate of -inf leaves its block out (its weight is 0, and so is its part of the bound)
            blocks = [(int(pt[n, j]), BLOCK, gate[n, h, i]) for i, j in enumerate(idx[n, h, :cnt[n, h]])
                      if gate[n, h, i] != -np.inf]
            blocks.append((int(pt[n, c]), int(kv_len[n]) - c * BLOCK, 0.0))
            kcode = np.concatenate([kc[p, h, :r] for p, r, _ in blocks])
            vcode = np.concatenate([vc[p, h, :r] for p, r, _ in blocks])
            kscale = np.concatenate([np.full(r, ks[p, h]) for p, r, _ in blocks])
            vscale = np.concatenate([np.full(r, vs[p, h]) for p, r, _ in blocks])
            bias = np.concatenate([np.full(r, g) for _, r, g in blocks])
            for hq in range(h * G, (h + 1) * G):
                x = sm_scale * kscale * (kcode @ q[n, hq]) + bias
                m = x.max()
                e = np.exp(x - m)
                z = e.sum()
                p = e / z
                o[n, hq] = p @ (vscale[:, None] * vcode)
                lse[n, hq] = m + math.log(z)
                # logits: D + 8 roundings of the dot product's terms, and eight of the
                # sum's size (scale, gate, maximum, exp2)
                dx = (D + 8) * u * sm_scale * kscale * (np.abs(kcode) @ np.abs(q[n, hq])) + \
                    8 * u * (np.abs(x) + np.abs(m) + 1)
                # probabilities: exp of such a logit; the sum and the value product add n + 8
                # roundings; weights, the largest of which is 2^15, as two fp16 numbers are 2^-21
                # off, or 2^-25 for each number in the subnormal range (2^-39 of the largest; 2^-38
                # where 15 itself is rounded)
                # the blocks' products are added times 2^-36: scales below 2^-90 are
                # subnormal then, half a step of 2^-149 off; so are the smallest sums
                rel = dx + dx.max() + (len(x) + 8) * u + np.where(vscale < 2.0 ** -90, 2.0 ** -150 / (vscale * 2.0 ** -36), 0)
                w_err = p * vscale * (rel + 2.0 ** -21) + 2.0 ** -38 * vscale / z
                o_tol[n, hq] = w_err @ np.abs(vcode) + 2.0 ** -8 * np.abs(o[n, hq]) + len(blocks) * 2.0 ** -126
                # the sum is of weights up to 2^15: exponents of that size (half a step, 8 u, times
                # ln 2) and a logarithm of up to 31 (a step of it, 32 u, times ln 2)
                lse_tol[n, hq] = dx.max() + (len(x) + 8) * u + 8 * u * abs(lse[n, hq]) + 28 * u
    return o, lse, o_tol * 1.01, lse_tol * 1.01
