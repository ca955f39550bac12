"""Plain forms of the operators of include/qmv_serve.h in 64 bits (or whole
numbers), row by row from the definitions in the header, shared by the tests.
Nothing here is used by the library."""
import math

import numpy as np

EPS32 = 2.0 ** -24  # half a step of float32, relative
PAGES, ROWS, LENGTH, STACK = 1, 2, 4, 8
BLOCK = {"q8_0": (32, 34), "q4_0": (32, 18), "q4_k": (256, 144), "q6_k": (256, 210)}


# ---- plan

def pages(x, page):
    return -(-x // page)


def plan(table, stack, count, kv_len, keep, n_new, page, T):
    """What kv_plan leaves: a dict of its outputs, tables and stack as lists;
    position and slot as dicts by row."""
    B, width = table.shape
    table, kv_len, n_new = table.copy(), [int(v) for v in kv_len], [int(v) for v in n_new]
    keep = kv_len if keep is None else [int(v) for v in keep]
    most = width * page
    status = lacking = 0
    if any(not (0 <= k <= l <= most and 0 <= n <= most - k) for l, k, n in zip(kv_len, keep, n_new)):
        status |= LENGTH
    good = [0 <= k <= l <= most and 0 <= n <= most - k for l, k, n in zip(kv_len, keep, n_new)]
    old = [pages(l, page) if g else 0 for l, g in zip(kv_len, good)]
    new = [pages(k + n, page) if g else 0 for k, n, g in zip(keep, n_new, good)]
    back = sum(max(0, o - w) for o, w in zip(old, new))
    taken = sum(max(0, w - o) for o, w in zip(old, new))
    if not 0 <= count <= len(stack) or count + back > len(stack):
        status |= STACK
    if sum(n for n, g in zip(n_new, good) if g) > T:
        status |= ROWS
    if not status & STACK and taken > count + back:
        status |= PAGES
        lacking = taken - count - back
    out = {"status": [status, lacking], "table": table, "position": {}, "slot": {}}
    if status:
        return out | {"new_len": kv_len, "count": count, "row_start": [0] * (B + 1), "stack": list(stack[:max(count, 0)])}
    free = [int(v) for v in stack[:count]]
    for b in range(B):
        free += [int(v) for v in table[b, new[b]:old[b]]]
    for b in range(B):
        for j in range(old[b], new[b]):
            table[b, j] = free.pop()
    start = [0]
    for b in range(B):
        for i in range(n_new[b]):
            p = keep[b] + i
            out["position"][start[-1] + i] = p
            g = int(table[b, p // page])
            out["slot"][start[-1] + i] = g * page + p % page if 0 <= g < len(stack) else -1
        start.append(start[-1] + n_new[b])
    return out | {"new_len": [k + n for k, n in zip(keep, n_new)], "count": len(free), "row_start": start, "stack": free}


# ---- embedding rows

def weights(fmt, rows):
    """float64 weights [M][K] of rows of blocks, uint8 [M][bytes], as the float32 steps of the header give them."""
    n, size = BLOCK[fmt]
    w = rows.reshape(rows.shape[0], -1, size)
    half = lambda at: w[:, :, at:at + 2].copy().view(np.float16).astype(np.float64)  # noqa: E731
    out = np.zeros(w.shape[:2] + (n,))
    for e in range(n):
        if fmt == "q8_0":
            out[:, :, e] = w[:, :, 2 + e].astype(np.int8) * half(0)[:, :, 0]
        elif fmt == "q4_0":
            c = w[:, :, 2 + e % 16]
            out[:, :, e] = ((c >> 4 if e >= 16 else c & 15).astype(np.float64) - 8) * half(0)[:, :, 0]
        elif fmt == "q4_k":
            s = e // 32
            c = w[:, :, 16 + 32 * (s // 2) + e % 32]
            q = (c >> 4 if s % 2 else c & 15).astype(np.float64)
            p = w[:, :, 4:16].astype(int)
            if s < 4:
                sc, mn = p[:, :, s] & 63, p[:, :, s + 4] & 63
            else:
                sc = (p[:, :, s + 4] & 15) | ((p[:, :, s - 4] >> 6) << 4)
                mn = (p[:, :, s + 4] >> 4) | ((p[:, :, s] >> 6) << 4)
            out[:, :, e] = half(0)[:, :, 0] * sc * q - half(2)[:, :, 0] * mn
        else:
            h, g, l = e // 128, e // 32 % 4, e % 32
            c = w[:, :, 64 * h + 32 * (g % 2) + l]
            q = (c >> 4 if g >= 2 else c & 15) | (((w[:, :, 128 + 32 * h + l] >> (2 * g)) & 3) << 4)
            out[:, :, e] = half(208)[:, :, 0] * w[:, :, 192 + e // 16].astype(np.int8) * (q.astype(np.float64) - 32)
    return out.reshape(rows.shape[0], -1)


def embed(fmt, table, tokens, scale):
    """float32 as defined: the weight rounded to float32, then one product."""
    ok = (tokens >= 0) & (tokens < table.shape[0])
    w = weights(fmt, table[np.where(ok, tokens, 0)]).astype(np.float32) * np.float32(scale)
    return np.where(ok[:, None], w, np.float32(0.0))


# ---- adapters

def lora(A, Bm, scale, rank, adapter, row_start, x, base):
    """y and a bound on a float32 evaluation's error, float64; rows of no sequence are NaN.

    A sum of n float32 products in any fixed order that splits them over lanes
    is off by a random walk of half steps of its partial sums: 4 sqrt(n) eps
    sum|terms| is four standard deviations, and 8 eps covers the few roundings
    of the operands, the lane sums and the scale.  The ranks' errors pass
    through |Bm|; base and result are rounded once each."""
    slots, R, K = A.shape
    y = np.full((x.shape[0], Bm.shape[1]), np.nan)
    tol = np.full_like(y, 1e-30)
    x = x.astype(np.float64)
    for b in range(len(row_start) - 1):
        rows = slice(row_start[b], row_start[b + 1])
        y[rows] = 0.0 if base is None else base[rows]
        s = adapter[b]
        if not 0 <= s < slots:
            continue
        r = R if rank is None else int(np.clip(rank[s], 0, R))
        a, m, sc = A[s, :r].astype(np.float64), Bm[s, :, :r].astype(np.float64), float(scale[s])
        v = x[rows] @ a.T
        dv = (4 * math.sqrt(K) + 8) * EPS32 * (np.abs(x[rows]) @ np.abs(a).T)
        d = sc * (v @ m.T)
        tol[rows] += abs(sc) * (dv @ np.abs(m).T) + (4 * math.sqrt(r) + 8) * EPS32 * abs(sc) * (np.abs(v) @ np.abs(m).T)
        tol[rows] += 2 * EPS32 * (np.abs(y[rows]) + np.abs(d))
        y[rows] += d
    return y, tol


# ---- the draw

def draw_row(z, temperature, top_k, top_p, min_p, u, softcap):
    """token, kept and whether every decision was far enough from its border
    to be decided: the header's accuracy of an exponential (and of tanh, whose
    error counts softcap / temperature times) and of whole multiples of 2^-q,
    half a unit an element of a sum, twice each."""
    z = np.asarray(z, dtype=np.float32)
    ok = np.nonzero(z > -np.inf)[0]
    if not len(ok):
        return -1, 0, True
    y = np.minimum(z[ok], np.float32(3.4028234663852886e38))
    order = np.lexsort((ok, -y))
    ok, y = ok[order], y[order].astype(np.float64)
    if not temperature > 0:
        return int(ok[0]), 1, True
    if softcap:
        y = softcap * np.tanh(y / softcap)
    w = np.exp((y - y[0]) / np.float64(np.float32(temperature)))
    run = np.cumsum(w)
    q = min(51, 62 - max(0, math.ceil(math.log2(len(z)))))
    of_w = 2.0 ** -40 * (1.0 + softcap / max(float(np.float32(temperature)), 1e-300))
    of_sum = of_w + len(z) * 2.0 ** -q
    far = True
    n = len(w)
    if top_k is not None and top_k > 0:
        n = min(n, int(top_k))
    if top_p is not None and top_p < 1:
        border = max(float(np.float32(top_p)), 0.0) * run[n - 1]
        c = int(np.searchsorted(run[:n], border, side="left")) + 1
        far &= all(abs(run[i] - border) > of_sum * run[n - 1] for i in (c - 2, c - 1) if 0 <= i < n)
        n = min(n, c)
    if min_p is not None and min_p > 0:
        m = float(np.float32(min_p))
        c = int((w >= m).sum())
        # weights of 1 are exact, and so is a border of 1
        far &= all(abs(w[i] - m) > of_w * m or w[i] == m == 1 for i in (c - 1, c) if 0 <= i < len(w))
        n = min(n, c)
    n = max(n, 1)
    point = min(max(float(np.float32(u)), 0.0), 1.0) * run[n - 1]
    at = min(int(np.searchsorted(run[:n], point, side="right")), n - 1)
    if point > 0:
        far &= all(abs(run[i] - point) > of_sum * run[n - 1] for i in (at - 1, at) if 0 <= i < n - 1)
    return int(ok[at]), n, bool(far)
