"""Calls at the edges of the documented ranges: they are computed, not refused."""
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


@pytest.mark.parametrize("T,heads,dim,fmt,length", [(1, 255, 128, "q8", 1024), (2, 130, 64, "f16", 700)])
def test_attention_of_few_rows_among_very_many_sequences(T, heads, dim, fmt, length):
    """65,535 sequences of which one or two have rows: few items, and a workgroup for every sequence and head."""
    qmv = _qmv()
    say(f"attn T {T}, 65535 sequences, {heads} heads of {dim} {fmt}")
    rng = np.random.default_rng(heads)
    B, page = 65535, 16
    P = R.Pages([length], heads, dim, page, fmt, rng, max_pages=64)
    t = [None if a is None else dev(a) for a in (P.k, P.v, P.ks, P.vs)]
    cache = qmv.KVCache(*t)
    at = 40000  # the sequence that has the rows
    table = np.full((B, 64), -1, np.int32)
    table[at] = P.table[0]
    start, lens = np.zeros(B + 1, np.int32), np.zeros(B, np.int32)
    start[at + 1:] = T
    lens[at] = length
    batch = qmv.KVBatch(_ints(table), _ints(start), _ints(lens), T)
    q = rng.normal(0, 1.2, (T, heads * dim)).astype(np.float32)
    out = torch.full((T, heads * dim), 9.5, device=DEV)
    wsb = qmv.attn_paged_ws_bytes(cache, batch, heads)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    qmv.attn_paged(cache, batch, dev(q), heads * dim, out, heads * dim, heads, dim ** -0.5, 0, ws, wsb)
    ref, tol = R.attention(q.astype(np.float64).reshape(T, heads, dim), P.rows("k", 0), P.rows("v", 0),
                           [length - T + i for i in range(T)], dim ** -0.5, 0)
    assert_within(host(out).reshape(ref.shape), ref, tol, "few rows, many sequences")


@pytest.mark.parametrize("scale,q_scale", [(1e-38, 1e37), (3e-39, 1e38), (1e-30, 1e30), (3.4e38, 1e-39), (2.5e38, 4e-39),
                                           (-3e38, 3e-39), (1e20, 1e-20), (1.2e-38, 2e37)])
@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_scales_at_the_ends_of_float32(fmt, scale, q_scale):
    """Scale and query are far from 1, their product is not: neither may overflow or lose bits by itself.  (Queries
    below 2^-126 have fewer bits, which the plain form is given too.)"""
    qmv = _qmv()
    say(f"attn {fmt} scale {scale} queries {q_scale}")
    rng = np.random.default_rng(7)
    heads, Hq, dim, lens, new = 2, 4, 64, [200, 33], [2, 1]
    P = R.Pages(lens, heads, dim, 16, fmt, rng)
    q = (rng.uniform(0.5, 1.0, (3, Hq, dim)) * np.where(rng.random((3, Hq, dim)) < 0.5, -1, 1) * q_scale).astype(np.float32)
    cache, table = P.to_gpu(DEV)
    batch = qmv.KVBatch(table, _ints(R.starts(new)), _ints(lens), 3)
    out = torch.empty(3, Hq * dim, device=DEV)
    wsb = qmv.attn_paged_ws_bytes(cache, batch, Hq)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    qmv.attn_paged(cache, batch, dev(q.reshape(3, -1)), Hq * dim, out, Hq * dim, Hq, scale, 0, ws, wsb)
    got, at = host(out).reshape(q.shape), 0
    for b, (n, L) in enumerate(zip(new, lens)):
        rows = slice(at, at + n)
        ref, tol = R.attention(q[rows].astype(np.float64), P.rows("k", b), P.rows("v", b), [L - n + i for i in range(n)],
                               float(np.float32(scale)), 0)
        assert_within(got[rows], ref, tol, f"scale {scale}, sequence {b}")
        at += n


@pytest.mark.parametrize("fmt,window", [("q8", 0), ("f16", 0), ("q8", 300)])
def test_units_of_more_than_one_step(fmt, window):
    """So many items and so long a table that units of 128 keys could not be numbered in 31 bits: 1100 sequences
    that share their first page, 16 heads, tables of 2^24 positions."""
    qmv = _qmv()
    say(f"attn {fmt} 1100 sequences, tables of 2^24 positions, window {window}")
    rng = np.random.default_rng(9)
    B, heads, dim, page, longest = 1100, 16, 64, 1024, 900
    P = R.Pages([longest], heads, dim, page, fmt, rng)
    cache, _ = P.to_gpu(DEV)
    table = torch.full((B, 16384), -1, dtype=torch.int32, device=DEV)
    table[:, 0] = int(P.table[0, 0])
    lens = rng.integers(1, longest + 1, B)
    lens[[0, 500, B - 1]] = [longest, 0, 257]
    batch = qmv.KVBatch(table, _ints(np.arange(B + 1)), _ints(lens), B)
    q = rng.normal(0, 1.2, (B, heads, dim)).astype(np.float32)
    out = torch.full((B, heads * dim), 9.5, device=DEV)
    wsb = qmv.attn_paged_ws_bytes(cache, batch, heads)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    qmv.attn_paged(cache, batch, dev(q.reshape(B, -1)), heads * dim, out, heads * dim, heads, 0.1, window, ws, wsb)
    got, k, v = host(out).reshape(q.shape), P.rows("k", 0), P.rows("v", 0)
    assert np.isfinite(got).all() and (got[500] == 0).all() and not (got == 9.5).any()
    for b in [0, 1, 77, 500, 801, B - 1]:
        n = int(lens[b])
        ref, tol = R.attention(q[b:b + 1].astype(np.float64), k[:n], v[:n], [n - 1], 0.1, window)
        assert_within(got[b:b + 1], ref, tol, f"sequence {b} of {n}")
