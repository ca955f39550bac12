"""Plain 64-bit forms of the decode-step operators (include/qmv_step.h) and
builders of paged caches, shared by the tests.  Written from the definitions
in the header, row by row; nothing here is used by the library."""
import math

import numpy as np
import torch

EPS32 = 2.0 ** -24  # half a step of float32, relative


def quantize_rows(x):
    """int8 codes and float32 scales of the last axis: float32 division, half away from zero."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        d = (np.abs(x).max(axis=-1) / np.float32(127.0)).astype(np.float32)
        r = (x / d[..., None]).astype(np.float32).astype(np.float64)
        q = np.clip(np.trunc(r + np.copysign(0.5, r)), -127, 127)
    q = np.where(np.abs(x).max(axis=-1, keepdims=True) == 0, 0.0, q)
    bad = ~np.isfinite(x).all(axis=-1)
    d = np.where(bad, np.float32(np.nan), d)
    return np.where(bad[..., None], 0, q).astype(np.int8), d


class Pages:
    """A paged cache on the host with sequences scattered over it.

    lens: cached positions of each sequence.  Free pages, the tails of last
    pages and unused table entries hold what must never matter: codes of 127
    with NaN scales (float16: NaN), and page numbers outside the cache."""

    def __init__(self, lens, heads, dim, page, fmt, rng, extra_pages=2, max_pages=None, spread=1.0):
        self.lens, self.heads, self.dim, self.page, self.fmt = list(lens), heads, dim, page, fmt
        need = [-(-n // page) for n in lens]
        self.max_pages = max_pages or max(max(need), 1) + 1
        self.num = sum(need) + extra_pages
        order = rng.permutation(self.num)
        bad = np.array([-1, self.num, 2 ** 31 - 1, -2 ** 31])
        self.table = bad[rng.integers(0, 4, (len(need), self.max_pages))].astype(np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.num, heads, page, dim)
        if fmt == "q8":
            self.k = np.full(shape, 127, np.int8)
            self.v = np.full(shape, 127, np.int8)
            self.ks = np.full(shape[:3], np.nan, np.float32)
            self.vs = np.full(shape[:3], np.nan, np.float32)
        else:
            self.k = np.full(shape, np.nan, np.float16)
            self.v = np.full(shape, np.nan, np.float16)
            self.ks = self.vs = None
        for b, n in enumerate(lens):
            for j in range(need[b]):
                m = min(page, n - j * page)
                pg = self.table[b, j]
                if fmt == "q8":
                    for c, s in ((self.k, self.ks), (self.v, self.vs)):
                        c[pg, :, :m] = np.clip(np.rint(rng.normal(0, 45, (heads, m, dim))), -127, 127)
                        s[pg, :, :m] = (rng.random((heads, m)) + 0.5) * (spread * 3.0 / 127)
                else:
                    for c in (self.k, self.v):
                        c[pg, :, :m] = rng.normal(0, spread, (heads, m, dim))

    def rows(self, which, b, count=None):
        """[count][heads][dim] float64 of sequence b's first positions."""
        n = self.lens[b] if count is None else count
        c, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        out = np.zeros((n, self.heads, self.dim))
        for p in range(n):
            pg, at = self.table[b, p // self.page], p % self.page
            out[p] = c[pg, :, at].astype(np.float64)
            if s is not None:
                out[p] *= s[pg, :, at].astype(np.float64)[:, None]
        return out

    def to_gpu(self, dev):
        from quantized_dequant_matrix_amd import qmv
        t = [None if a is None else torch.from_numpy(a).to(dev) for a in (self.k, self.v, self.ks, self.vs)]
        return qmv.KVCache(*t), torch.from_numpy(self.table).to(dev)


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def attention(q, k, v, positions, scale, window):
    """Rows q [n][Hq][D] at `positions` over one sequence's k, v [L][H][D], all
    float64.  Returns the output and a bound on a float32 evaluation's error:

    a score is a sum whose query is held to 2^-22 of the row's largest
    magnitude (21 bits in three 7-bit parts, or two float16 terms) and that is
    rounded a few times in float32: |ds| <= 2^-21 max|q| sum|k| + 8 eps
    sum|q k|.  A relative error e^ds - 1 of every weight moves the result by at
    most 2 max|ds| sum p|v|.  exp2, the scale and the split of p into two
    float16 terms cost a few roundings each (16 eps), and a running sum of L
    terms a random walk of half steps (4 sqrt(L) eps).

    A weight is held as p c with c such that p = 1 at the largest value scale
    is 2^10 (float16 caches: c = 2^10), and its second float16 term ends at
    float16's smallest step 2^-24: a weight is off by at most 2^-34 of the
    largest one however small it is.  The sum of the weights is at least 1, so
    the result is off by at most L 2^-34 max|v| more, with max|v| at most
    twice the largest element (127 codes of the largest scale; every row here
    has a code of 64 or more)."""
    n, Hq, D = q.shape
    L, H, _ = k.shape
    out = np.zeros((n, Hq, D))
    tol = np.full((n, Hq, D), 1e-30)
    for i in range(n):
        p = positions[i]
        hi = min(p + 1, L)
        lo = max(0, p - window + 1) if window else 0
        if hi <= lo:
            continue
        for h in range(Hq):
            kk, vv = k[lo:hi, h // (Hq // H)], v[lo:hi, h // (Hq // H)]
            s = scale * (kk @ q[i, h])
            ds = abs(scale) * (2.0 ** -21 * np.abs(q[i, h]).max() * np.abs(kk).sum(axis=1)
                               + 8 * EPS32 * (np.abs(kk) @ np.abs(q[i, h])))
            e = np.exp(s - s.max())
            e /= e.sum()
            out[i, h] = e @ vv
            tol[i, h] += (e @ np.abs(vv)) * (2 * ds.max() + (16 + 4 * math.sqrt(hi - lo)) * EPS32)
            tol[i, h] += (hi - lo) * 2.0 ** -34 * 2 * np.abs(vv).max()
    return out, tol


def norm(x, r, w, eps):
    """z float32, and y by the definition's float32 steps with the mean in 64 bits."""
    z = x if r is None else (x + r).astype(np.float32)
    z64 = z.astype(np.float64)
    rstd = (1.0 / np.sqrt((z64 * z64).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))).astype(np.float32)
    return z, ((z * rstd).astype(np.float32) * w).astype(np.float32)


def softmax64(y, temperature, softcap):
    y = np.asarray(y, dtype=np.float32)
    dead = np.isnan(y) | (y == -np.inf)
    v = np.minimum(np.where(dead, 0.0, y), np.float32(3.4028234663852886e38)).astype(np.float64)
    if softcap:
        v = softcap * np.tanh(v / softcap)
    v = v / temperature
    if dead.all():
        return np.zeros_like(v)
    e = np.where(dead, 0.0, np.exp(v - v[~dead].max()))
    return e / e.sum()


def draft_verify(target, draft, tokens, n_draft, u, temperature, softcap):
    """accepted, tokens and, for each sequence, how far the nearest decision was
    from its border (relative): decisions closer than the sums' rounding are
    not decided."""
    B, G1, V = target.shape
    G = G1 - 1
    acc, out, margin = np.zeros(B, np.int32), np.full((B, G1), -1, np.int32), np.ones(B)
    for b in range(B):
        n = G if n_draft is None else int(np.clip(n_draft[b], 0, G))
        a = n
        q = None
        for i in range(n):
            p, q = softmax64(target[b, i], temperature, softcap), softmax64(draft[b, i], temperature, softcap)
            t = int(tokens[b, i])
            if not 0 <= t < V:
                a = i
                break
            left, right = np.float64(np.float32(u[b, i])) * q[t], p[t]
            margin[b] = min(margin[b], abs(left - right) / max(right, left, 1e-300))
            if not left < right:
                a = i
                break
        p = softmax64(target[b, a], temperature, softcap)
        w = np.maximum(p - q, 0.0) if a < n else p
        if not w.sum() > 0:
            w = p
        run = np.cumsum(w)
        acc[b] = a
        out[b, :a] = tokens[b, :a]
        if run[-1] > 0:
            point = np.float64(np.float32(u[b, G])) * run[-1]
            past = np.nonzero((run > point) & (w > 0))[0]
            at = past[0] if len(past) else np.nonzero(w > 0)[0][-1]
            out[b, a] = at
            lower = run[at] - w[at]
            margin[b] = min(margin[b], (run[at] - point) / run[-1], (point - lower) / run[-1] if point > 0 else 1.0)
        else:
            out[b, a] = -1
    return acc, out, margin
