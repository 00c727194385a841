"""Plain 64-bit references of the serving-step operators (numpy, CPU),
written from the definitions in ``include/kda_block_tables.h``,
``include/kda_qk_rope.h`` and ``include/kda_verify.h``, one element, request
or row at a time."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3_MAX = 448.0
SEQLENS, CAPACITY, SLOT_RANGE, TOKEN_RANGE = 4, 8, 1, 32


def block_tables(cached, new, table, free, head, bs, num_blocks, T, held=None):
    """Returns (table, cu, seq_lens, positions, slot_map, head_out, held_out, error bits)."""
    table, err = np.array(table), 0
    B, M = table.shape
    cu, lens, pos, slot, held_out = [0], [], [0] * T, [-1] * T, []
    at, t = head, 0
    for i in range(B):
        c, n = int(cached[i]), int(new[i])
        if c < 0 or n < 0 or c + n > 2 ** 31 - 1:
            err |= SEQLENS
            c, n = max(c, 0), 0
        first, end = -(-c // bs), -(-(c + n) // bs)
        if held is not None:
            first = max(first, int(held[i]))
        has = min(first, M)
        if n > 0 and end > M:
            err |= CAPACITY
        got = {}
        for k in range(first, min(end, M)):
            if 0 <= at < len(free):
                got[k] = int(free[at])
                has += has == k
                if not 0 <= got[k] < num_blocks:
                    got[k], err = -1, err | SLOT_RANGE
            else:
                got[k], err = -1, err | CAPACITY
            at += 1
        for p in range(c, c + n):
            k = p // bs
            if t < T:
                if k < M and k in got:
                    b = got[k]
                    if p % bs == 0:
                        table[i, k] = b
                elif k < M:
                    b = int(table[i, k])
                    if not 0 <= b < num_blocks:
                        b, err = -1, err | SLOT_RANGE
                else:
                    b = -1
                pos[t] = p
                slot[t] = -1 if b < 0 else b * bs + p % bs
            t += 1
        cu.append(t)
        lens.append(c + n)
        held_out.append(has)
    if t > T:
        err |= CAPACITY
    return table, cu, lens, pos, slot, min(at, max(len(free), head)), held_out, err


def norm_rotate(x, w, pos, inv_freq, interleaved, eps):
    """x [..., 128] fp64 of one token at position pos"""
    x = np.array(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    y = x.copy()
    half = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = math.cos(pos * f), math.sin(pos * f)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def inv_freqs(rot, base):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)] if rot else []


def fit_scale(amax):
    if amax == 0:
        return 2.0 ** -64
    e = -64
    while e < 119 and amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def e4m3_values():
    """The value of each of the 256 codes."""
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def e4m3_nearest(x):
    """Codes of fp64 values: nearest, ties to the even code, saturating; brute force over the table."""
    vals = e4m3_values()
    pos = vals[:127]
    x = np.asarray(x, np.float64)
    out = np.zeros(x.shape, np.uint8)
    flat, o = x.reshape(-1), out.reshape(-1)
    for i, v in enumerate(flat):
        if np.isnan(v):
            o[i] = 127
            continue
        m = min(abs(v), E4M3_MAX)
        k = int(np.searchsorted(pos, m))
        if k > 0 and (k == 127 or pos[k] != m):
            lo, hi = pos[k - 1], pos[k]
            k = k - 1 if m - lo < hi - m or (m - lo == hi - m and (k - 1) % 2 == 0) else k
        o[i] = k | (128 if np.signbit(v) else 0)
    return out


def write_cache(codes, scale, x, slot, bs):
    """codes uint8 [nb, H, bs, 128] and scale [nb, H] of one cache, x fp64 [T, H, 128].  Returns (codes, scale,
    {(block, h): list of (row, x row)}): the older rows' codes rescaled, the new rows left to the caller to compare."""
    codes, scale, vals = codes.copy(), scale.astype(np.float64).copy(), e4m3_values()
    blocks = {}
    for t, s in enumerate(slot):
        if s >= 0:
            blocks.setdefault(int(s) // bs, []).append((int(s) % bs, t))
    new = {}
    for b, rows in blocks.items():
        first = min(r for r, _ in rows)
        for h in range(codes.shape[1]):
            v = np.stack([x[t, h] for _, t in rows])
            fin = np.abs(v[np.isfinite(v)])
            fit = fit_scale(fin.max() if fin.size else 0.0)
            s = fit if first == 0 else max(scale[b, h], fit)
            if first and s != scale[b, h]:
                codes[b, h, :first] = e4m3_nearest(vals[codes[b, h, :first]] * (scale[b, h] / s))
            scale[b, h] = s
            new[b, h] = [(r, x[t, h]) for r, t in rows]
    return codes, scale, new


def verify(draft, p, u, su, q=None, src=None, slots=None):
    """Lists of tokens, accepted counts, next slots, and the error bits; exact integers and fractions."""
    N, T, V = p.shape
    tokens, acc, nxt, err = [], [], [], 0

    def fixed(x):
        x = np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=1.0, neginf=0.0)
        return (np.clip(x, 0, 1) * 2.0 ** 60).astype(np.uint64)

    for n in range(N):
        if src is not None and src[n] <= 0:
            tokens.append([-1] * T), acc.append(0), nxt.append(0)
            continue
        err |= TOKEN_RANGE if (np.asarray(draft[n]) >= V).any() else 0
        k, refused = 0, False
        while k < T - 1:
            d = int(draft[n][k])
            if not 0 <= d < V:
                break
            qd = 1.0 if q is None else float(q[n, k, d])
            if not float(u[n][k]) * qd < float(p[n, k, d]):
                refused = True
                break
            k += 1
        full = fixed(p[n, k])
        w = full
        if refused:
            if q is None:
                w = full.copy()
                w[int(draft[n][k])] = 0
            else:
                Q = fixed(q[n, k])
                w = np.where(full > Q, full - Q, np.uint64(0))
            if int(w.sum()) == 0:
                w = full
        total = int(w.sum())
        x = float(su[n])
        r = 0 if not x > 0 else min(int(x * 2.0 ** 31), 2 ** 31 - 1) if x < 1 else 2 ** 31 - 1
        c = np.cumsum(w, dtype=np.uint64)
        tok = V - 1 if total == 0 else int(np.searchsorted(c, np.uint64(r * total // 2 ** 31), side="right"))
        tokens.append([int(v) for v in draft[n][:k]] + [tok] + [-1] * (T - 1 - k))
        acc.append(k)
        nxt.append(int(slots[n][k]) if slots is not None else 0)
    return tokens, acc, nxt, err
