"""attn_paged with many rows a sequence and many items, which are computed an
item a workgroup, two row tiles at once where heads are 128 wide: head layouts,
row tiles that end anywhere, windows, rows that see nothing, pages that do not
exist, what masked places may hold, strides, graphs.  Many heads make few
tokens enough."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import assert_within, say
from test_gpu_step_attn import Call, _ints

pytestmark = pytest.mark.gpu


def _chunk(c):
    """The batch has 64 rows a sequence or more, and two rounds of items of 32 rows."""
    seqs, group = min(len(c.new), c.T), c.Hq // c.P.heads
    rows = c.T * group
    assert rows >= 64 * seqs
    assert min(c.T * -(-group // 32), (rows + 31 * seqs) // 32) * c.P.heads >= 512
    return c


def _heads(c):
    """Some key/value heads, the first and the last among them, and their query heads."""
    group, heads = c.Hq // c.P.heads, c.P.heads
    kv = [0, heads - 1, heads // 2, 7, 5, 30][: max(2, 12 // group)]
    return kv, [h * group + g for h in kv for g in range(group)]


def _reference(c):
    """[rows][_heads][dim] and its error bound."""
    kv, qh = _heads(c)
    out, tol, at = [], [], 0
    for b, (n, L) in enumerate(zip(c.new, c.lens)):
        if n:
            q = c.q[at:at + n, : c.width].astype(np.float64).reshape(n, c.Hq, c.dim)[:, qh]
            o, t = R.attention(q, c.P.rows("k", b)[:, kv], c.P.rows("v", b)[:, kv], [L - n + i for i in range(n)],
                               c.scale, c.window)
            out.append(o)
            tol.append(t)
        at += n
    return np.concatenate(out), np.concatenate(tol)


def _result(c):
    """Like _reference; what lies behind rows and heads is as it was, and no element is left out."""
    n = sum(c.new)
    got = c.result()
    assert (got[n:] == 9.5).all() and (got[:, c.width:] == 9.5).all() and not (got[:n, : c.width] == 9.5).any()
    return got[:n, : c.width].reshape(n, c.Hq, c.dim)[:, _heads(c)[1]]


def _check(c, what):
    say(f"attn {what}")
    c.upload()
    c.enqueue()
    ref, tol = _reference(c)
    assert_within(_result(c), ref, tol, what)


@pytest.mark.parametrize("lens,new,heads,group,dim,page,window", [
    ([300], [300], 128, 1, 64, 16, 0),
    ([513, 130], [200, 100], 96, 1, 128, 64, 0),
    ([420], [100], 90, 3, 64, 32, 0),
    ([257], [33], 90, 8, 128, 16, 0),          # 264 rows: the last tile has 8
    ([1000, 90, 129], [8, 3, 5], 100, 64, 64, 128, 0),
    ([129, 64], [129, 64], 90, 1, 128, 1024, 0),
    ([160], [160], 150, 1, 64, 16, 1),
    ([300], [150], 130, 1, 128, 16, 40),
    ([640, 33], [70, 33], 70, 4, 64, 32, 129),
    ([700], [64], 90, 6, 128, 16, 320),
    ([500], [64], 90, 6, 128, 16, 2 ** 31 - 1),
    ([128, 96, 160, 32], [64, 64, 64, 32], 64, 2, 64, 16, 64),
])
def test_chunks(lens, new, heads, group, dim, page, window):
    _check(_chunk(Call(lens, new, heads * group, heads, dim, page, "q8", seed=sum(lens), window=window)),
           f"{heads} x {group} heads of {dim}, {new} of {lens}, window {window}")


@pytest.mark.parametrize("pad,off", [(4, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("dim", [64, 128])
def test_strides_alignment_and_rows_behind_the_last(pad, off, dim):
    _check(_chunk(Call([150, 0, 90], [140, 0, 70], 100, 100, dim, 16, "q8", seed=2, pad=pad, off=off, tail=3)),
           f"ld + {pad}, base + {off}")


@pytest.mark.parametrize("window", [0, 20])
def test_rows_that_see_nothing(window):
    """More rows than positions: the first rows' positions are negative."""
    lens, new = [40, 70], [150, 70]
    c = _chunk(Call(lens, new, 128, 128, 64, 16, "q8", seed=3, window=window)).upload()
    say("rows without positions")
    c.enqueue()
    got = _result(c)
    assert (got[:110] == 0.0).all()
    d = Call(lens, [40, 70], 128, 128, 64, 16, "q8", seed=3, window=window)
    d.P, d.q = c.P, c.q[110:]
    ref, tol = _reference(d)
    assert_within(got[110:], ref, tol, "the others")


@pytest.mark.parametrize("dim", [64, 128])
def test_pages_outside_the_cache_are_not_seen(dim):
    lens, new, heads = [200], [130], 140
    c = _chunk(Call(lens, new, heads, heads, dim, 16, "q8", seed=4))
    k, v = c.P.rows("k", 0), c.P.rows("v", 0)
    for j, page in ((0, -1), (3, c.P.num), (7, -2 ** 31), (8, 2 ** 31 - 1)):
        c.P.table[0, j] = page
    c.upload()
    say("holes in the table")
    c.enqueue()
    got = _result(c)
    kv, qh = _heads(c)
    there = np.ones(200, bool)
    for j in (0, 3, 7, 8):
        there[16 * j:16 * j + 16] = False
    q = c.q.astype(np.float64).reshape(130, heads, dim)[:, qh]
    k, v = k[:, kv], v[:, kv]
    for r in (0, 1, 57, 58, 73, 74, 129):
        keep = there & (np.arange(200) <= 70 + r)
        ref, tol = R.attention(q[r:r + 1], k[keep], v[keep], [keep.sum() - 1], c.scale, 0)
        assert_within(got[r:r + 1], ref, tol, f"row {r}")


def test_what_masked_places_hold():
    lens, new, window, heads = [260], [130], 50, 140
    args = dict(seed=5, window=window)
    clean = _chunk(Call(lens, new, heads, heads, 64, 16, "q8", **args))
    ref, tol = _reference(clean)
    kv = _heads(clean)[0]
    for j in (81, 100, 128, 131, 160, 201, 259):
        c = Call(lens, new, heads, heads, 64, 16, "q8", **args)
        pg, at = c.P.table[0, j // 16], j % 16
        (c.P.vs if j % 2 else c.P.ks)[pg, kv[j % 4], at] = np.nan
        c.upload()
        c.enqueue()
        got = _result(c)
        pos = np.arange(130, 260)
        sees = (j <= pos) & (j > pos - window)
        broken = np.zeros(ref.shape[:2], bool)
        broken[sees, j % 4] = True
        assert np.isnan(got[broken]).all(), j
        assert_within(got[~broken], ref[~broken], tol[~broken], f"NaN at {j}")


def test_queries_that_are_not_finite():
    c = _chunk(Call([200], [130], 140, 140, 128, 16, "q8", seed=6))
    ref, tol = _reference(c)
    broken = np.zeros(ref.shape[:2], bool)
    for r, i, x in ((0, 0, np.nan), (31, 3, np.inf), (32, 1, -np.inf), (129, 2, np.nan)):
        h = _heads(c)[1][i]
        c.q[r, h * 128 + 7 * h % 128] = x
        broken[r, i] = True
    c.upload()
    c.enqueue()
    got = _result(c)
    assert np.isnan(got[broken]).all()
    assert_within(got[~broken], ref[~broken], tol[~broken], "beside broken queries")


@pytest.mark.parametrize("q_scale,scale,spread", [(30.0, 1.0, 1.0), (1e-4, 1.0, 1.0), (1.2, 0.0, 1.0), (1.2, -0.3, 1.0),
                                                  (1e4, 1e-4, 100.0), (0.0, 1.0, 1.0)])
@pytest.mark.parametrize("dim", [64, 128])
def test_magnitudes(dim, q_scale, scale, spread):
    _check(_chunk(Call([300], [130], 140, 140, dim, 16, "q8", seed=7, q_scale=q_scale, scale=scale, spread=spread)),
           f"q {q_scale} scale {scale} kv {spread}")


@pytest.mark.parametrize("first,then", [(1e-36, 1.0), (0.0, 1.0), (1e30, 1.0), (1e-28, 1e28)])
def test_value_scales_far_apart(first, then):
    c = Call([400], [130], 140, 140, 64, 16, "q8", seed=8)
    rng = np.random.default_rng(9)
    fine = ~np.isnan(c.P.vs)
    c.P.vs[fine] *= 10.0 ** rng.uniform(-6, 0, fine.sum()).astype(np.float32)
    for j in range(25):
        c.P.vs[c.P.table[0, j]] *= np.float32(first if j < 12 else then)
    _check(_chunk(c), f"values times {first}, then times {then}")


def test_rising_scores():
    """Every block of keys moves the running maximum."""
    c = Call([500], [130], 140, 140, 64, 16, "q8", seed=10)
    for j in range(500):
        c.P.ks[c.P.table[0, j // 16], :, j % 16] *= np.float32(0.05 + j / 100)
    _check(_chunk(c), "rising scores")


def test_lengths_near_the_largest_integer():
    c = _chunk(Call([64], [130], 140, 140, 64, 16, "q8", seed=11, window=40, max_pages=4)).upload()
    for lens in ([2 ** 31 - 1], [2 ** 31 - 97]):
        c.out.fill_(9.5)
        c.len.copy_(_ints(lens))
        c.enqueue()
        assert (c.result() == 0.0).all()


def test_row_starts_out_of_order_are_harmless():
    c = _chunk(Call([130, 130], [65, 65], 140, 140, 64, 16, "q8", seed=12)).upload()
    for start in ([0, 140, 3], [-5, -2, 100], [130, 1, 0], [0, 0, 0], [70, 20, 130]):
        for lens in ([-3, 2 ** 31 - 1], [130, 0]):
            c.start.copy_(_ints(start))
            c.len.copy_(_ints(lens))
            c.enqueue()
    torch.cuda.synchronize()


def test_captured_replayed_and_the_same_every_time():
    c = _chunk(Call([400, 200], [90, 60], 140, 140, 128, 16, "q8", seed=13)).upload()
    ref, tol = _reference(c)
    c.enqueue()
    first = c.result().copy()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.enqueue()
    for _ in range(3):
        c.out.fill_(9.5)
        g.replay()
        assert np.array_equal(first.view(np.uint32), c.result().view(np.uint32))
    assert_within(_result(c), ref, tol, "eager and replayed")


@pytest.mark.parametrize("fmt,heads,group,dim,new", [("q8", 33, 8, 256, 70), ("f16", 33, 8, 256, 70), ("f16", 24, 4, 128, 180),
                                                     ("f16", 33, 8, 64, 70), ("q8", 33, 8, 64, 70)])
def test_long_sequences_the_other_ways(fmt, heads, group, dim, new):
    """Chunks over float16 caches, of 256-wide heads, of fewer rows: many tiles of keys a wave."""
    _check(Call([1300], [new], heads * group, heads, dim, 32, fmt, seed=28), f"{fmt} {heads} x {group} heads of {dim}")
    if fmt == "q8":
        c = Call([1300], [new], heads * group, heads, dim, 32, fmt, seed=29)
        c.P.vs[c.P.table[0, :10]] *= np.float32(0.0)
        _check(c, f"{heads} x {group} heads of {dim} after 320 rows of zeros")
