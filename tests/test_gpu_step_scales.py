"""attn_paged over 8-bit values whose scales differ by many decades, with the
weight on the small ones: a value that weighs nothing must take no accuracy
from the others, however large it is.

The bound is step_ref.attention's with its last term made relative to what the
values weigh.  A weight times its value's scale is held to 2^-34 of the largest
such product of the row (the second float16 term ends at 2^-24 where the
largest product is 2^10 or more), so L of them are off by at most
L 2^-34 max_j (p_j s_j) 127, and every row of codes here has one of 64 or more:
L 2^-34 2 max_j (p_j max|v_j|).  A weight below 2^-114 of the largest may
vanish: it is held from 2^80 down to 2^-34 whatever the values' scales."""
import math

import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import DEV, assert_within, dev, host, say

pytestmark = pytest.mark.gpu


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def _tolerance(q, k, v, positions, scale):
    """step_ref.attention's terms, the last one by weighted values."""
    n, Hq, D = q.shape
    group = Hq // k.shape[1]
    out, tol = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    for i in range(n):
        hi = min(positions[i] + 1, k.shape[0])
        for h in range(Hq):
            kk, vv = k[:hi, h // group], v[:hi, h // group]
            s = scale * (kk @ q[i, h])
            ds = abs(scale) * (2.0 ** -21 * np.abs(q[i, h]).max() * np.abs(kk).sum(axis=1)
                               + 8 * R.EPS32 * (np.abs(kk) @ np.abs(q[i, h])))
            e = np.exp(s - s.max())
            e /= e.sum()
            out[i, h] = e @ vv
            tol[i, h] = (e @ np.abs(vv)) * (2 * ds.max() + (16 + 4 * math.sqrt(hi)) * R.EPS32)
            tol[i, h] += hi * (2.0 ** -34 * 2 * (e * np.abs(vv).max(axis=1)).max() + 2.0 ** -114 * np.abs(vv).max())
    return out, tol


class Case:
    """Keys of one direction: the score of position j is peak x gain[j] (nats) for a query head of
    sign +, its negative for one of sign -."""

    def __init__(self, lens, new, Hq, heads, dim, gain, vscale, max_pages=None, seed=0, page=16):
        rng = np.random.default_rng(seed)
        self.P = P = R.Pages(lens, heads, dim, page, "q8", rng, max_pages=max_pages)
        for b, L in enumerate(lens):
            for j in range(L):
                pg, at = P.table[b, j // page], j % page
                code = int(round(127 * gain(j, L)))
                P.k[pg, :, at] = 0
                P.k[pg, :, at, 0] = code
                P.ks[pg, :, at] = 1 / 127
                P.vs[pg, :, at] = vscale(j, L) / 127
        self.lens, self.new, self.Hq, self.dim, self.T = lens, new, Hq, dim, sum(new)
        self.q = np.zeros((self.T, Hq, dim), np.float32)
        self.sign = np.where(np.arange(Hq) % 2 == 0, 1.0, -1.0)

    def check(self, peak, what):
        say(what)
        qmv = _qmv()
        self.q[:, :, 0] = peak * self.sign
        cache, table = self.P.to_gpu(DEV)
        batch = qmv.KVBatch(table, _ints(R.starts(self.new)), _ints(self.lens), self.T)
        width = self.Hq * self.dim
        out = torch.empty(self.T, width, device=DEV)
        wsb = qmv.attn_paged_ws_bytes(cache, batch, self.Hq)
        ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
        qmv.attn_paged(cache, batch, dev(self.q.reshape(self.T, width)), width, out, width, self.Hq, 1.0, 0, ws, wsb)
        got = host(out).reshape(self.q.shape)
        at = 0
        for b, (n, L) in enumerate(zip(self.new, self.lens)):
            rows = slice(at, at + n)
            ref, tol = _tolerance(self.q[rows].astype(np.float64), self.P.rows("k", b), self.P.rows("v", b),
                                  [L - n + i for i in range(n)], 1.0)
            assert_within(got[rows], ref, tol, f"{what}, sequence {b}")
            at += n


TABLES = pytest.mark.parametrize("max_pages", [None, 640 // 16 + 1, 10000 // 16], ids=["whole", "eight", "pieces"])
# where the small values that take the weight lie
PLACES = {"first": lambda j, L: j < 20, "last": lambda j, L: j >= L - 20, "middle": lambda j, L: 100 <= j < 140,
          "scattered": lambda j, L: j % 37 == 5, "one": lambda j, L: j == 3}


@TABLES
@pytest.mark.parametrize("ratio,peak", [(1e-4, 14.0), (1e-8, 24.0), (1e-10, 30.0), (1e-12, 34.0), (1e-18, 48.0)])
@pytest.mark.parametrize("place", list(PLACES))
def test_small_values_that_take_the_attention(place, ratio, peak, max_pages):
    """Heads of sign + give all weight to small values beside large ones, heads of sign - the reverse."""
    f = PLACES[place]
    Case([400, 170], [1, 2], 4, 2, 64, lambda j, L: 1.0 if f(j, L) else 0.0, lambda j, L: ratio if f(j, L) else 1.0,
         max_pages=max_pages).check(peak, f"{place} ratio {ratio} peak {peak}")


@pytest.mark.parametrize("dim", [64, 128, 256])
@TABLES
def test_scales_that_fall_as_the_scores_rise(dim, max_pages):
    """Each position has a higher score and a smaller value than the one before: the largest weighted value stays or
    falls while the maximum rises (and, for heads of sign -, rises faster than the score falls)."""
    for rate in (0.5, 1.0, 2.0):
        Case([384], [1], 4, 2, dim, lambda j, L: j / L, lambda j, L: math.exp(-40.0 * rate * j / L),
             max_pages=max_pages).check(40.0, f"D {dim} rate {rate}")


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_chunks_of_many_rows(dim):
    """Two row tiles a workgroup at head size 128."""
    Case([300], [280], 32, 16, dim, lambda j, L: 1.0 if j % 9 == 0 else 0.0, lambda j, L: 1e-9 if j % 9 == 0 else 1.0,
         page=32).check(26.0, f"chunk D {dim}")


@TABLES
def test_values_of_zero_that_take_the_attention(max_pages):
    """The result is what the other positions weigh: 2^-72 of the sum."""
    Case([500], [2], 4, 2, 128, lambda j, L: 1.0 if j % 50 == 7 else 0.0, lambda j, L: 0.0 if j % 50 == 7 else 1.0,
         max_pages=max_pages).check(50.0, "zeros")


@TABLES
def test_small_and_large_values_within_the_stated_range(max_pages):
    """Values of 2^-66 that take the attention beside values of 2^95 that do not."""
    Case([300], [1], 2, 1, 64, lambda j, L: 1.0 if j == 120 else 0.0, lambda j, L: 2.0 ** -66 if j == 120 else 2.0 ** 95,
         max_pages=max_pages).check(122.0, "2^-66 beside 2^95")


SIGNALLING = np.array([0x7FA00000, 0xFFA00001, 0x7F800001, 0xFFBFFFFF], np.uint32).view(np.float32)


def _fill_tails(P, lens):
    """Scales behind the last positions: signalling NaN of both signs."""
    for b, L in enumerate(lens):
        for j in range(L, -(-L // P.page) * P.page):
            for s in (P.ks, P.vs):
                s[P.table[b, j // P.page], :, j % P.page] = SIGNALLING[j % 4]


@TABLES
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("L", [33, 34, 35, 36, 49, 50, 145, 161, 273, 289, 297])
def test_a_large_value_beside_places_that_hold_signalling_nan(L, dim, max_pages):
    """The last position's value is 2^33 times the others', so the weights' reference has to move in the tile whose
    other places nobody sees, whatever is in them."""
    c = Case([L, 5], [1, 1], 4, 2, dim, lambda j, n: 0.5, lambda j, n: 1e4 if j == n - 1 else 1e-6, max_pages=max_pages)
    _fill_tails(c.P, [L, 5])
    c.check(2.0, f"length {L}, D {dim}")


@TABLES
@pytest.mark.parametrize("heads,group,dim", [(2, 2, 64), (2, 2, 128), (2, 2, 256), (16, 16, 128)])
def test_a_signalling_nan_that_only_later_rows_see(heads, group, dim, max_pages):
    """Rows before it are as without it, though their own last value moves the reference; rows from it on are NaN."""
    L, n = 149, 64 if heads == 16 else 8
    first = L - n
    c = Case([L], [n], heads * group, heads, dim, lambda j, m: 0.5, lambda j, m: 1e4 if j in (first, first + 4) else 1e-6,
             max_pages=max_pages if heads == 2 else None)
    bad = first + 5
    c.P.vs[c.P.table[0, bad // 16], :, bad % 16] = SIGNALLING[0]
    qmv = _qmv()
    c.q[:, :, 0] = 2.0 * c.sign
    cache, table = c.P.to_gpu(DEV)
    batch = qmv.KVBatch(table, _ints([0, n]), _ints([L]), n)
    width = c.Hq * dim
    out = torch.empty(n, width, device=DEV)
    wsb = qmv.attn_paged_ws_bytes(cache, batch, c.Hq)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    qmv.attn_paged(cache, batch, dev(c.q.reshape(n, width)), width, out, width, c.Hq, 1.0, 0, ws, wsb)
    got = host(out).reshape(c.q.shape)
    ref, tol = _tolerance(c.q[:5].astype(np.float64), c.P.rows("k", 0)[:bad], c.P.rows("v", 0)[:bad],
                          [first + i for i in range(5)], 1.0)
    assert_within(got[:5], ref, tol, "rows before it")
    assert np.isnan(got[5:]).all()
