"""kv_write and kv_read against the plain forms: codes and scales bit for bit,
untouched cells untouched, rows without a place, tables that lie."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import DEV, dev, host, say

pytestmark = pytest.mark.gpu


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def _bits(a):
    return a.view({1: np.uint8, 2: np.uint16, 4: np.uint32}[a.dtype.itemsize])


CASES = [  # heads, dim, page, fmt, cached before, new rows, ld padding, misaligned rows
    (16, 128, 16, "q8", [776], [1], 0, False),
    (1, 64, 16, "q8", [0, 5, 40], [3, 0, 17], 0, False),
    (3, 64, 32, "f16", [0, 31, 32, 100], [1, 2, 33, 7], 12, False),
    (2, 256, 64, "q8", [63, 0], [66, 1], 7, False),
    (5, 128, 128, "q8", [1, 2, 3], [1, 1, 1], 4, True),
    (2, 256, 16, "f16", [15, 16, 17], [18, 1, 30], 0, True),
    (4, 64, 1024, "q8", [1000], [200], 0, False),
    (1, 128, 16, "f16", [0], [300], 0, False),
    # from 1024 rows on a workgroup takes several: four wide ones, sixteen narrow ones
    (8, 128, 128, "q8", [3, 0, 700], [1021, 1, 30], 0, False),
    (5, 256, 64, "f16", [0, 20], [1000, 45], 3, True),
    (17, 64, 256, "q8", [1, 1], [700, 324], 8, False),
    (3, 64, 32, "f16", [7, 0, 0, 31], [500, 0, 1, 601], 4, True),
    (1, 64, 16, "q8", [0, 100], [1030, 17], 0, True),
    (7, 128, 64, "q8", [50], [1100], 0, False),
    (3, 256, 16, "f16", [0, 0, 9], [1, 1050, 2], 0, False),
]


def _inputs(T, width, pad, off, rng, scale):
    ld = width + pad
    buf = rng.normal(0, scale, T * ld + 4).astype(np.float32)
    t = dev(buf)
    view = buf[off:off + T * ld].reshape(T, ld)[:, :width]
    return t[off:], view, ld


@pytest.mark.parametrize("heads,dim,page,fmt,before,new,pad,off", CASES)
def test_write_then_read(heads, dim, page, fmt, before, new, pad, off):
    qmv = _qmv()
    rng = np.random.default_rng(1)
    say(f"kv {heads}x{dim} page {page} {fmt} before {before} new {new}")
    total = [a + b for a, b in zip(before, new)]
    P = R.Pages(total, heads, dim, page, fmt, rng)
    cache, table = P.to_gpu(DEV)
    T, width = sum(new), heads * dim
    kt, kh, ld = _inputs(T, width, pad, 1 if off else 0, rng, 1.5)
    vt, vh, _ = _inputs(T, width, pad, 1 if off else 0, rng, 1e-3)
    kh[0, :dim] = 0.0                     # an all-zero row
    kh[-1, :4] = [2.5, -2.5, 127.0, 0.5]  # ties at unit scale (row maximum 127 or its own)
    kt[: T * ld].copy_(dev(np.ascontiguousarray(_restore(kt, kh, ld, T))))
    batch = qmv.KVBatch(table, _ints(R.starts(new)), _ints(total), T)
    qmv.kv_write(cache, batch, kt, ld, vt, ld)
    got = [host(t) for t in cache.tensors]
    # the cache by the definition: only the new rows' cells change
    want = [a.copy() for a in (P.k, P.v, P.ks, P.vs) if a is not None]
    r = 0
    for b in range(len(new)):
        for i in range(new[b]):
            p = before[b] + i
            pg, at = P.table[b, p // page], p % page
            for x, codes, scales in ((kh, 0, 2), (vh, 1, 3)):
                row = x[r].reshape(heads, dim)
                if fmt == "q8":
                    want[codes][pg, :, at], want[scales][pg, :, at] = R.quantize_rows(row)
                else:
                    want[codes][pg, :, at] = row.astype(np.float16)
            r += 1
    for g, w in zip(got, want):
        assert np.array_equal(_bits(g), _bits(w))
    # read back: the new rows, with the write's batch
    back = torch.full((T + 2, ld), 7.25, device=DEV)
    back2 = torch.full((T + 2, ld), 7.25, device=DEV)
    qmv.kv_read(cache, batch, back, ld, back2, ld)
    for t, codes, scales in ((back, 0, 2), (back2, 1, 3)):
        h = host(t)
        assert (h[T:] == 7.25).all() and (h[:, width:] == 7.25).all()
        r = 0
        for b in range(len(new)):
            for i in range(new[b]):
                p = before[b] + i
                pg, at = P.table[b, p // page], p % page
                x = want[codes][pg, :, at].astype(np.float32)
                if fmt == "q8":
                    x = x * want[scales][pg, :, at][:, None]
                assert np.array_equal(h[r, :width], x.reshape(-1))
                r += 1
    # and whole sequences, with row_start the running sum of kv_len
    n = sum(total)
    whole = qmv.KVBatch(table, _ints(R.starts(total)), _ints(total), n)
    a, c = torch.empty(n, width, device=DEV), torch.empty(n, width, device=DEV)
    qmv.kv_read(cache, whole, a, width, c, width)
    P.k, P.v = want[0], want[1]
    if fmt == "q8":
        P.ks, P.vs = want[2], want[3]
    for t, which in ((a, "k"), (c, "v")):
        ref = np.concatenate([P.rows(which, b) for b in range(len(new))])
        assert np.array_equal(host(t), ref.reshape(n, width).astype(np.float32))


def _restore(t, view, ld, T):
    full = host(t)[: T * ld].reshape(T, ld).copy()
    full[:, : view.shape[1]] = view
    return full.reshape(-1)


@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_rows_without_a_place(fmt):
    """Negative positions, positions behind the table, pages outside the cache, rows behind
    the last sequence: nothing is written, and they read as zeros or stay."""
    qmv = _qmv()
    rng = np.random.default_rng(2)
    heads, dim, page = 2, 64, 16
    P = R.Pages([20, 32, 8], heads, dim, page, fmt, rng, max_pages=2)
    P.table[2, 0] = P.num  # the third sequence's page does not exist
    cache, table = P.to_gpu(DEV)
    before = [host(t).copy() for t in cache.tensors]
    # 4 rows for 2 positions; 3 rows ending at 34 of at most 32 positions; 2 rows on no page
    new, lens = [4, 3, 2], [2, 34, 8]
    T, width = 12, heads * dim
    k = torch.ones(T, width, device=DEV)
    batch = qmv.KVBatch(table, _ints(R.starts(new)), _ints(lens), T)
    qmv.kv_write(cache, batch, k, width, k, width)
    after = [host(t) for t in cache.tensors]
    places = {(int(P.table[0, 0]), 0), (int(P.table[0, 0]), 1), (int(P.table[1, 1]), 15)}
    for x, y in zip(before, after):
        for pg in range(P.num):
            for at in range(page):
                same = np.array_equal(_bits(x[pg, :, at].copy()), _bits(y[pg, :, at].copy()))
                assert same == ((pg, at) not in places)
    a, c = torch.full((T, width), 3.0, device=DEV), torch.full((T, width), 3.0, device=DEV)
    qmv.kv_read(cache, batch, a, width, c, width)
    for t in (a, c):
        h = host(t)
        assert (h[9:] == 3.0).all()
        assert (h[[0, 1, 5, 6, 7, 8]] == 0.0).all()
        assert np.allclose(h[[2, 3, 4]], 1.0, rtol=2e-3)


def test_row_starts_out_of_order_are_harmless():
    qmv = _qmv()
    rng = np.random.default_rng(3)
    P = R.Pages([16, 16, 16], 1, 64, 16, "q8", rng)
    cache, table = P.to_gpu(DEV)
    k = torch.ones(8, 64, device=DEV)
    for start in ([0, 5, 2, 8], [-7, 2, 4, 90], [3, 3, 3, 3], [9, 8, 7, 6]):
        for lens in ([16, 16, 16], [-5, 0, 2 ** 31 - 1]):
            batch = qmv.KVBatch(table, _ints(start), _ints(lens), 8)
            qmv.kv_write(cache, batch, k, 64, k, 64)
            qmv.kv_read(cache, batch, k.clone(), 64, k.clone(), 64)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_rows_that_are_not_finite_become_nan(fmt):
    qmv = _qmv()
    rng = np.random.default_rng(4)
    P = R.Pages([6], 2, 64, 16, fmt, rng)
    cache, table = P.to_gpu(DEV)
    x = rng.normal(0, 1, (6, 128)).astype(np.float32)
    x[1, 3], x[2, 70], x[3, 0] = np.nan, np.inf, -np.inf
    x[4, 5] = 1e30 if fmt == "f16" else 3e38  # float16 has no such number; the codes do
    batch = qmv.KVBatch(table, _ints([0, 6]), _ints([6]), 6)
    a, c = torch.empty(6, 128, device=DEV), torch.empty(6, 128, device=DEV)
    qmv.kv_write(cache, batch, dev(x), 128, dev(x), 128)
    qmv.kv_read(cache, batch, a, 128, c, 128)
    bad = np.zeros((6, 2), bool)
    bad[1, 0] = bad[2, 1] = bad[3, 0] = True
    bad[4, 0] = fmt == "f16"
    for t in (a, c):
        h = host(t).reshape(6, 2, 64)
        assert np.array_equal(np.isnan(h).all(axis=2), bad) and np.array_equal(np.isnan(h).any(axis=2), bad)


def test_rows_without_a_place_among_many():
    """More rows than positions, positions behind the table, rows behind the last sequence, with the
    rows shared by workgroups: zeros, and rows as they were."""
    qmv = _qmv()
    rng = np.random.default_rng(6)
    for heads in (1, 16):  # sixteen rows a workgroup, four
        P = R.Pages([640, 640, 640], heads, 64, 64, "q8", rng, max_pages=10)
        cache, table = P.to_gpu(DEV)
        new, lens = [500, 451, 300], [397, 1001, 640]
        T, width = 1260, heads * 64
        x = rng.normal(0, 1, (T, width)).astype(np.float32)
        batch = qmv.KVBatch(table, _ints(R.starts(new)), _ints(lens), T)
        qmv.kv_write(cache, batch, dev(x), width, dev(-x), width)
        a, c = torch.full((T, width), 3.0, device=DEV), torch.full((T, width), 3.0, device=DEV)
        qmv.kv_read(cache, batch, a, width, c, width)
        want = np.full((T, width), 3.0, np.float32)
        codes, d = R.quantize_rows(x.reshape(T, heads, 64))
        back = (codes.astype(np.float32) * d[..., None]).reshape(T, width)
        r = 0
        for n, L in zip(new, lens):
            for i in range(n):
                want[r] = back[r] if 0 <= L - n + i < 640 else 0.0
                r += 1
        assert np.array_equal(host(a), want)
        want[:1251] *= -1.0
        assert np.array_equal(host(c), want)


def test_subnormal_rows():
    """Rows whose scale has no reciprocal in float32 (below 2^-128)."""
    qmv = _qmv()
    rng = np.random.default_rng(7)
    P = R.Pages([8], 2, 64, 16, "q8", rng)
    cache, table = P.to_gpu(DEV)
    x = rng.uniform(0.01, 1.0, (8, 2, 64)) * np.where(rng.random((8, 2, 64)) < 0.5, -1, 1)
    x *= 10.0 ** -np.array([35.0, 36, 37, 38, 38.5, 39, 40, 41])[:, None, None]
    x = x.astype(np.float32)
    assert (x != 0).all()
    qmv.kv_write(cache, qmv.KVBatch(table, _ints([0, 8]), _ints([8]), 8), dev(x.reshape(8, 128)), 128,
                 dev(x.reshape(8, 128)), 128)
    codes, d = R.quantize_rows(x)
    assert (d > 0).all()
    for got, want in zip([host(t) for t in cache.tensors], (codes, codes, d, d)):
        assert np.array_equal(got[P.table[0, 0]][:, :8].swapaxes(0, 1), want)


def test_many_sequences():
    """The search for a row's sequence: more than 64 * 64 sequences, empty ones among them."""
    qmv = _qmv()
    rng = np.random.default_rng(5)
    B = 5000
    new = rng.integers(0, 3, B)
    new[:70] = 0
    new[-3:] = [2, 0, 0]
    T = int(new.sum())
    table = np.arange(B, dtype=np.int32)[:, None]
    k = torch.zeros(B, 1, 16, 64, dtype=torch.float16, device=DEV)
    cache = qmv.KVCache(k, torch.zeros_like(k))
    x = np.tile(np.arange(T, dtype=np.float32)[:, None] % 1000, (1, 64))
    batch = qmv.KVBatch(_ints(table), _ints(R.starts(new)), _ints(np.full(B, 7)), T)
    qmv.kv_write(cache, batch, dev(x), 64, dev(x), 64)
    h = host(k)[:, 0, :, 0].astype(np.float32)
    want = np.zeros((B, 16), np.float32)
    r = 0
    for b in range(B):
        for i in range(new[b]):
            want[b, 7 - new[b] + i] = r % 1000
            r += 1
    assert np.array_equal(h, want)
