"""Plain 64-bit implementations of the serving calls (numpy / torch on the host), written from their definitions in
include/trellis.h, and input helpers.  No code of the product path is used."""
from __future__ import annotations

import math

import numpy as np
import torch

F8 = torch.float8_e4m3fn


def f64(t):
    return t.detach().cpu().to(torch.float32).double().numpy() if t.dtype != torch.float64 else t.detach().cpu().numpy()


def bf16_round(x):
    """float64 to the nearest bf16 number (ties to even) in one rounding, as float64; finite inputs."""
    _, e = np.frexp(x)
    unit = np.ldexp(1.0, np.maximum(e, -125) - 8)  # 8 significant bits; fixed below the smallest normal number
    return np.rint(x / unit) * unit


def in_bf16_band(got, want, tol):
    """Every number is the rounding of one within tol of the wanted one."""
    return bool(np.all((got >= bf16_round(want - tol)) & (got <= bf16_round(want + tol))))


def norm_rope(x, w, rope_rows, rot, interleaved, eps, offset):
    """x [n, heads, dim] float64, rope_rows [n, rot]; returns the rotated norms and, per number, the size of its pair
    (what its rounding errors scale with)."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (w + offset)
    size = np.abs(y).copy()
    if rot:
        half = rot // 2
        c, s = rope_rows[:, None, :half], rope_rows[:, None, half:]
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        size[..., a] = size[..., b] = np.abs(ya) + np.abs(yb)
    return y, size


def attention(q, k, v, seen, scale):
    """One head: q [t, dim], k and v [len, dim], seen [t, len]; float64.  Returns out, lse, sum w|v|, max scale sum|qk|."""
    t, n = q.shape[0], k.shape[0]
    out, lse = np.zeros((t, q.shape[1])), np.full(t, -np.inf)
    mass, size = np.zeros((t, q.shape[1])), np.zeros(t)
    for i in range(t):
        at = np.flatnonzero(seen[i])
        if at.size == 0:
            continue
        x = k[at] @ q[i] * scale
        m = x.max()
        if m == -np.inf:
            continue
        e = np.exp(x - m)
        out[i], lse[i] = e @ v[at] / e.sum(), m + math.log(e.sum())
        mass[i] = e @ np.abs(v[at]) / e.sum()
        size[i] = (np.abs(k[at]) @ np.abs(q[i])).max() * abs(scale)
    return out, lse, mass, size


def fork(table, lens, refs, parent, child, page, room):
    """numpy int arrays, sequential; returns new table, lens, refs, status and the list of (src, dst) page copies."""
    old, old_len, old_refs = table.copy(), lens.copy(), refs.copy()
    table, lens, refs = table.copy(), lens.copy(), refs.copy()
    rows, width = table.shape
    free = [p for p in range(len(refs)) if old_refs[p] == 0]
    status, copies, asked, at = [], [], 0, 0
    held_of = lambda r: next((i for i in range(width) if old[r, i] < 0), width)  # noqa: E731
    for par, ch in zip(parent, child):
        if not (0 <= ch < rows and -1 <= par < rows):
            status.append(2)
            continue
        held = held_of(ch)
        used = -(-int(old_len[par]) // page) if par >= 0 else 0
        if par >= 0 and not 0 <= old_len[par] <= width * page:
            status.append(2)
            continue
        if any(old[ch, i] >= len(refs) for i in range(held)) or \
                (par not in (-1, ch) and any(not 0 <= old[par, i] < len(refs) for i in range(used))):
            status.append(2)
            continue
        grow, drop = par == ch, par == -1
        full = 0 if drop else held if grow else int(old_len[par]) // page
        need = 0 if drop else max(full, -(-(int(old_len[par]) + room) // page))
        fresh = need - full if need <= width else 0
        take = list(range(at, at + fresh))
        at += fresh
        ok = need <= width and (fresh == 0 or at <= len(free))
        status.append(0 if ok else 1)
        if grow:
            if ok:
                for i, f in enumerate(take):
                    table[ch, full + i] = free[f]
                    refs[free[f]] += 1
            continue
        for i in range(held):
            refs[old[ch, i]] -= 1
        table[ch], lens[ch] = -1, 0
        if drop or not ok:
            continue
        for i in range(full):
            table[ch, i] = old[par, i]
            refs[old[par, i]] += 1
        for i, f in enumerate(take):
            table[ch, full + i] = free[f]
            refs[free[f]] += 1
        if old_len[par] % page:
            copies.append((old[par, full], table[ch, full]))
        lens[ch] = old_len[par]
    return table, lens, refs, np.array(status), copies


def compact(table, refs):
    n = int((refs > 0).sum())
    high = [p for p in range(n, len(refs)) if refs[p] > 0]
    holes = [p for p in range(n) if refs[p] <= 0]
    to = {p: p for p in range(len(refs))}
    to.update(zip(high, holes))
    out = np.zeros_like(refs)
    for p in range(len(refs)):
        if refs[p] > 0:
            out[to[p]] = refs[p]
    return np.vectorize(lambda e: to.get(int(e), int(e)))(table).astype(table.dtype), out, list(zip(high, holes))


def logprobs(x, tokens, top, temp):
    """x [n, vocab] float64 (the logits as they are), tokens [n, c]; returns lp, lse, entropy, ids, top_lp."""
    n, vocab = x.shape
    lp, lse, ent = np.full(tokens.shape, -np.inf), np.zeros(n), np.zeros(n)
    ids, tlp = np.zeros((n, top), dtype=np.int64), np.zeros((n, top))
    for r in range(n):
        z = x[r] / temp
        nan = np.isnan(z)
        # NaN before every number, then descending, equal numbers by index
        order = np.lexsort((np.arange(vocab), -np.where(nan, 0, z), ~nan))[:top]
        ids[r] = order
        with np.errstate(invalid="ignore"):
            m = z.max()
            if m == -np.inf:
                lse[r], ent[r], tlp[r] = -np.inf, 0.0, -np.inf
                continue
            e = np.exp(z - m)
            lse[r] = m + np.log(e.sum())
            p = e / e.sum()
            ent[r] = np.log(e.sum()) - np.sum(np.where(p > 0, p * np.where(p > 0, z - m, 0), np.where(np.isnan(p), np.nan, 0)))
            tlp[r] = z[order] - lse[r]
            for c, t in enumerate(tokens[r]):
                if 0 <= t < vocab:
                    lp[r, c] = z[t] - lse[r]
    return lp, lse, ent, ids, tlp
