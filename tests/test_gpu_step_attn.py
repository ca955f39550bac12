"""attn_paged against the plain form in 64 bits, with the error bound that
step_ref.attention derives: head layouts, page sizes, ragged batches, windows,
rows that see nothing, what masked places may hold, strides, graphs, streams.

A batch whose table is short is computed an item (sequence, rows, head) a
workgroup, with eight waves where the table is not quite so short (`wide`: 640
positions) and items are few; one whose table is long (10,000 positions) in
pieces that a second kernel joins.  The lengths in the table do not matter for
that, so all ways are run on the same sequences."""
import math

import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import DEV, assert_within, dev, host, say

pytestmark = pytest.mark.gpu
both = pytest.mark.parametrize("wide", [False, 640, True], ids=["whole", "eight", "pieces"])


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


class Call:
    """A batch over a paged cache on both sides."""

    def __init__(self, lens, new, Hq, heads, dim, page, fmt, seed=0, window=0, pad=0, off=0, tail=0, q_scale=1.2,
                 scale=None, spread=1.0, max_pages=None, wide=False):
        rng = np.random.default_rng(seed)
        if wide is True:
            max_pages = 10000 // page
        elif wide:
            max_pages = max(wide, max(lens)) // page + 1
        self.P = R.Pages(lens, heads, dim, page, fmt, rng, spread=spread, max_pages=max_pages)
        self.lens, self.new, self.Hq, self.dim, self.window = lens, new, Hq, dim, window
        self.T, self.width, self.ld, self.off = sum(new) + tail, Hq * dim, Hq * dim + pad, off
        self.q = rng.normal(0, q_scale, (self.T, self.ld)).astype(np.float32)
        self.scale = 1.0 / math.sqrt(dim) if scale is None else scale

    def upload(self):
        qmv = _qmv()
        self.cache, self.table = self.P.to_gpu(DEV)
        self.start, self.len = _ints(R.starts(self.new)), _ints(self.lens)
        self.batch = qmv.KVBatch(self.table, self.start, self.len, self.T)
        flat = np.concatenate([np.zeros(self.off, np.float32), self.q.reshape(-1)])
        self.tq = dev(flat)[self.off:]
        self.out = torch.full((self.T * self.ld + self.off,), 9.5, device=DEV)[self.off:]
        self.wsb = qmv.attn_paged_ws_bytes(self.cache, self.batch, self.Hq)
        self.ws = torch.full((self.wsb,), 0xff, dtype=torch.uint8, device=DEV)
        return self

    def enqueue(self, stream=None):
        _qmv().attn_paged(self.cache, self.batch, self.tq, self.ld, self.out, self.ld, self.Hq, self.scale, self.window,
                          self.ws, self.wsb, stream=stream)

    def result(self):
        return host(self.out).reshape(self.T, self.ld)

    def reference(self):
        out = np.zeros((sum(self.new), self.Hq, self.dim))
        tol = np.zeros_like(out)
        at = 0
        for b, (n, L) in enumerate(zip(self.new, self.lens)):
            q = self.q[at:at + n, : self.width].astype(np.float64).reshape(n, self.Hq, self.dim)
            pos = [L - n + i for i in range(n)]
            if n:
                out[at:at + n], tol[at:at + n] = R.attention(q, self.P.rows("k", b), self.P.rows("v", b), pos,
                                                             self.scale, self.window)
            at += n
        return out, tol

    def check(self, what):
        say(f"attn {what}")
        self.upload()
        self.enqueue()
        got = self.result()
        ref, tol = self.reference()
        n = sum(self.new)
        assert (got[n:] == 9.5).all() and (got[:, self.width:] == 9.5).all()
        return assert_within(got[:n, : self.width].reshape(ref.shape), ref, tol, what)


@both
@pytest.mark.parametrize("fmt", ["q8", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 700])
def test_single_token(fmt, dim, length, wide):
    Call([length], [1], 4, 2, dim, 16, fmt, seed=length, wide=wide).check(f"{fmt} D {dim} length {length}")


@both
@pytest.mark.parametrize("Hq,heads", [(1, 1), (2, 1), (3, 1), (7, 1), (8, 1), (16, 1), (17, 1), (64, 1), (32, 16),
                                      (24, 8), (5, 5), (33, 3)])
@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_head_layouts(Hq, heads, fmt, wide):
    Call([200, 3], [1, 2], Hq, heads, 64, 32, fmt, seed=Hq, wide=wide).check(f"{fmt} {Hq} over {heads} heads")


@both
@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
@pytest.mark.parametrize("fmt,dim", [("q8", 128), ("f16", 64)])
def test_page_sizes(page, fmt, dim, wide):
    Call([300, 16, 1, 129], [1, 4, 1, 1], 4, 2, dim, page, fmt, seed=page, wide=wide).check(f"{fmt} page {page}")


@both
@pytest.mark.parametrize("new,lens", [([8, 8], [8, 700]), ([1, 5, 16, 17], [900, 64, 16, 100]), ([40], [1000]),
                                      ([33, 1, 0, 64], [33, 500, 77, 64]), ([150, 2], [300, 2]), ([300], [300])])
@pytest.mark.parametrize("fmt,dim", [("q8", 128), ("q8", 64), ("q8", 256), ("f16", 128), ("f16", 256)])
def test_chunks(new, lens, fmt, dim, wide):
    Call(lens, new, 4, 2, dim, 32, fmt, seed=sum(new), wide=wide).check(f"{fmt} D {dim} chunks {new} over {lens}")


@pytest.mark.parametrize("window", [1, 2, 16, 31, 64, 100, 513, 5000])
@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_windows(window, fmt):
    Call([600, 70, 3], [5, 70, 1], 4, 2, 64, 16, fmt, seed=window, window=window).check(f"{fmt} window {window}")


@pytest.mark.parametrize("fmt", ["q8", "f16"])
@pytest.mark.parametrize("window", [1000, 2047])
def test_long_windows(fmt, window):
    Call([3000, 90, 2500], [3, 2, 1], 4, 2, 64, 16, fmt, seed=window, window=window).check(f"{fmt} window {window}")


@pytest.mark.parametrize("fmt,heads,group", [("q8", 16, 4), ("f16", 16, 4), ("q8", 20, 3)])
def test_chunks_of_many_rows(fmt, heads, group):
    """Two row tiles a workgroup (head size 128, many rows a sequence)."""
    Call([330, 71, 40], [270, 71, 5], heads * group, heads, 128, 32, fmt, seed=heads).check(f"{fmt} {heads} x {group} heads")


@pytest.mark.parametrize("dim", [64, 256])
def test_many_items(dim):
    """More items than two rounds of workgroups, not of the two-tile kind."""
    Call([150, 60], [130, 30], 64, 16, dim, 16, "q8", seed=dim).check(f"D {dim}")


@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_long_context(fmt):
    Call([20011], [1], 4, 2, 128, 64, fmt, seed=1).check(f"{fmt} 20011 positions")
    Call([9000, 40], [3, 3], 2, 1, 128, 64, fmt, seed=2).check(f"{fmt} 9000 and 40 positions")


@both
@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_many_short_sequences(fmt, wide):
    """More sequences than a workgroup has threads, empty ones among them."""
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 60, 600).tolist()
    new = [int(n > 0) for n in rng.integers(0, 4, 600)]
    Call(lens, new, 2, 1, 64, 16, fmt, seed=4, wide=wide).check(f"{fmt} 600 sequences")


@both
@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_empty_sequences_and_rows_behind_the_last(fmt, wide):
    """No new tokens, no cached tokens, and rows that belong to nobody."""
    Call([5, 0, 90, 0, 33], [1, 0, 0, 0, 2], 4, 2, 64, 16, fmt, tail=3, wide=wide).check(f"{fmt} empty sequences")


@both
def test_rows_that_see_nothing(wide):
    """More new rows than positions: the first rows' positions are negative.  Their output is zero."""
    c = Call([3, 20], [6, 1], 4, 2, 64, 16, "q8", seed=5, wide=wide)
    c.check("negative positions")
    assert (c.result()[:3, : c.width] == 0).all()
    c = Call([0, 20], [2, 1], 4, 2, 64, 16, "f16", seed=6, wide=wide)
    c.check("no positions")
    assert (c.result()[:2, : c.width] == 0).all()


@both
@pytest.mark.parametrize("pad,off", [(4, 0), (3, 0), (0, 1), (5, 3)])
def test_strides_and_alignment(pad, off, wide):
    Call([100, 33], [2, 1], 4, 2, 128, 16, "q8", seed=7, pad=pad, off=off, wide=wide).check(f"ld + {pad}, base + {off}")


@both
@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_what_masked_places_hold(fmt, wide):
    """Later tokens of the chunk and tokens before the window hold NaN: rows that do not see them
    are as without, rows that see them are NaN in whole heads."""
    lens, new, window = [90], [40], 30
    clean = Call(lens, new, 2, 1, 64, 16, fmt, seed=8, window=window, wide=wide)
    ref, tol = clean.reference()
    for j in (10, 55, 70, 89):
        c = Call(lens, new, 2, 1, 64, 16, fmt, seed=8, window=window, wide=wide)
        pg, at = c.P.table[0, j // 16], j % 16
        if fmt == "q8":
            (c.P.vs if j % 2 else c.P.ks)[pg, 0, at] = np.nan
        else:
            (c.P.v if j % 2 else c.P.k)[pg, 0, at] = np.nan
        c.upload()
        c.enqueue()
        got = c.result()[:, : c.width].reshape(ref.shape)
        pos = np.arange(50, 90)
        sees = (j <= pos) & (j > pos - window)
        assert np.isnan(got[sees]).all(), j
        assert_within(got[~sees], ref[~sees], tol[~sees], f"{fmt} NaN at {j}")


@both
@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_infinite_values_in_masked_places(fmt, wide):
    c = Call([64], [20], 2, 1, 64, 16, fmt, seed=18, wide=wide)
    ref, tol = c.reference()
    pg, at = c.P.table[0, 3], 63 % 16
    if fmt == "q8":
        c.P.vs[pg, 0, at] = np.inf
        c.P.ks[pg, 0, at] = -np.inf
    else:
        c.P.v[pg, 0, at] = np.inf
        c.P.k[pg, 0, at] = -np.inf
    c.upload()
    c.enqueue()
    got = c.result()[:, : c.width].reshape(ref.shape)
    assert_within(got[:19], ref[:19], tol[:19], "rows before the infinite one")


@both
def test_queries_that_are_not_finite(wide):
    c = Call([50], [3], 4, 2, 64, 16, "q8", seed=9, wide=wide)
    ref, tol = c.reference()
    c.q[1, 5] = np.nan           # head 0 of row 1
    c.q[1, 3 * 64 + 1] = np.inf  # head 3
    c.upload()
    c.enqueue()
    got = c.result()[:, : c.width].reshape(ref.shape)
    assert np.isnan(got[1, 0]).all() and np.isnan(got[1, 3]).all()
    got[1, [0, 3]] = ref[1, [0, 3]]
    assert_within(got, ref, tol, "heads beside broken ones")


@both
@pytest.mark.parametrize("fmt", ["q8", "f16"])
@pytest.mark.parametrize("q_scale,scale,spread", [(30.0, 1.0, 1.0), (1e-4, 1.0, 1.0), (1.2, 0.0, 1.0), (1.2, -0.3, 1.0),
                                                  (1.2, 0.1, 1e-3), (1e4, 1e-4, 100.0), (0.0, 1.0, 1.0)])
def test_magnitudes(fmt, q_scale, scale, spread, wide):
    """Sharp and flat softmaxes, tiny and large keys and values, a zero query."""
    Call([500, 40], [2, 1], 4, 2, 128, 16, fmt, seed=10, q_scale=q_scale, scale=scale,
         spread=spread, wide=wide).check(f"{fmt} q {q_scale} scale {scale} kv {spread}")


@both
def test_scales_far_apart(wide):
    """Values whose scales differ by 10^6 from token to token (a token with tiny values that takes the
    attention, beside tokens with large ones)."""
    c = Call([300], [2], 4, 2, 64, 16, "q8", seed=11, wide=wide)
    rng = np.random.default_rng(12)
    fine = ~np.isnan(c.P.vs)
    c.P.vs[fine] *= 10.0 ** rng.uniform(-6, 0, fine.sum()).astype(np.float32)
    c.check("value scales over six decades")
    c = Call([300], [2], 4, 2, 64, 16, "q8", seed=11, wide=wide)
    fine = ~np.isnan(c.P.vs)
    c.P.vs[fine] = 0.0
    c.check("all values zero")


@both
@pytest.mark.parametrize("first", [1e-36, 1e-30, 0.0, 1e30])
def test_first_values_of_another_magnitude(first, wide):
    """A sequence that opens with rows of tiny, zero or huge values, in all waves' tiles."""
    c = Call([700], [2], 4, 2, 128, 16, "q8", seed=25, wide=wide)
    for j in range(20):
        c.P.vs[c.P.table[0, j]] *= np.float32(first)
    c.check(f"320 rows of values times {first}")


@pytest.mark.parametrize("first", [1e-36, 0.0, 1e30])
def test_first_values_of_another_magnitude_in_one_pass(first):
    """... where a wave goes over several of a row's tiles."""
    c = Call([500], [2], 4, 2, 128, 16, "q8", seed=27)
    for j in range(20):
        c.P.vs[c.P.table[0, j]] *= np.float32(first)
    c.check(f"320 rows of values times {first}")


@both
def test_values_from_the_smallest_to_the_largest(wide):
    """Tiny values whose weights must still count when huge ones follow."""
    c = Call([700], [2], 4, 2, 128, 16, "q8", seed=26, wide=wide)
    for j in range(44):
        c.P.vs[c.P.table[0, j]] *= np.float32(1e-28 if j < 20 else 1e28)
    c.check("values over 56 decades")


@both
def test_rising_scores(wide):
    """The running maximum rises at every run of keys, and the weights of the first keys vanish."""
    for sign in (1.0, -1.0):
        c = Call([800], [1], 1, 1, 64, 16, "f16", seed=13, scale=1.0, wide=wide)
        for j in range(800):
            c.P.k[c.P.table[0, j // 16], 0, j % 16] = np.float16(sign * j / 64.0)
        c.q[:] = 0.2
        c.check(f"scores rising {sign}")


@both
def test_pages_outside_the_cache_are_not_seen(wide):
    """Positions on a page number outside [0, num_pages) hold nothing."""
    c = Call([64, 20], [1, 1], 2, 1, 64, 16, "q8", seed=14, wide=wide)
    hole = list(range(16, 32))
    k, v = c.P.rows("k", 0), c.P.rows("v", 0)
    c.P.table[0, 1] = c.P.num
    c.upload()
    c.enqueue()
    got = c.result()[:, : c.width].reshape(2, 2, 64)
    keep = [j for j in range(64) if j not in hole]
    q = c.q[:1, : c.width].astype(np.float64).reshape(1, 2, 64)
    ref, tol = R.attention(q, k[keep], v[keep], [len(keep) - 1], c.scale, 0)
    assert_within(got[:1], ref, tol, "without the hole")


def test_lengths_that_lie_are_harmless():
    """Positions behind the table do not exist; the visible ones end with it.  Row starts out of order."""
    c = Call([32, 32], [2, 1], 2, 1, 64, 16, "q8", seed=15, max_pages=2)
    c.upload()
    c.len.copy_(_ints([50, 32]))
    c.enqueue()
    got = c.result()[:, : c.width].reshape(3, 2, 64)
    q = c.q[:, : c.width].astype(np.float64).reshape(3, 2, 64)
    for r, b, pos in ((0, 0, 48), (1, 0, 49), (2, 1, 31)):
        ref, tol = R.attention(q[r:r + 1], c.P.rows("k", b), c.P.rows("v", b), [pos], c.scale, 0)
        assert_within(got[r:r + 1], ref, tol, f"row {r}")
    for start in ([0, 9, 3], [-5, -2, 100], [2, 1, 0], [0, 0, 0]):
        for lens in ([-3, 2 ** 31 - 1], [32, 0]):
            c.start.copy_(_ints(start))
            c.len.copy_(_ints(lens))
            c.enqueue()
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt,dim,group,window", [("q8", 128, 1, 0), ("q8", 128, 4, 300), ("f16", 128, 2, 0), ("q8", 64, 2, 0),
                                                  ("f16", 64, 1, 1000), ("q8", 64, 16, 0), ("q8", 256, 1, 0), ("f16", 256, 1, 0)])
def test_eight_waves_over_long_sequences(fmt, dim, group, window):
    """Few items of up to 17 steps: whole, some waves with several tiles and some with none."""
    rng = np.random.default_rng(dim + group)
    lens = rng.integers(1, 2100, 20).tolist()
    lens[3], lens[11] = 2100, 0
    new = [min(n, 1 + i % 3) for i, n in enumerate(lens)]
    Call(lens, new, 8 * group, 8, dim, 64, fmt, seed=group, window=window, tail=2).check(
        f"{fmt} 20 sequences, {group} x 8 heads of {dim}, window {window}")


def test_row_starts_that_make_too_much_work_are_harmless():
    """Every second sequence claims all rows: more pieces than 31 bits can number, and none is computed."""
    qmv = _qmv()
    heads, T, B, pages = 64, 60, 65535, 64
    k = torch.zeros(1, heads, 1024, 64, dtype=torch.float16, device=DEV)
    cache = qmv.KVCache(k, k.clone())
    start = np.zeros(B + 1, np.int32)
    start[1::2] = T
    batch = qmv.KVBatch(torch.zeros(B, pages, dtype=torch.int32, device=DEV), _ints(start),
                        _ints(np.full(B, 2 ** 31 - 1)), T)
    q = torch.zeros(T, heads * 64, device=DEV)
    out = torch.empty_like(q)
    wsb = qmv.attn_paged_ws_bytes(cache, batch, heads)
    assert wsb > 2 ** 24  # computed in pieces
    ws = torch.zeros(wsb, dtype=torch.uint8, device=DEV)
    say("rows claimed by 32768 sequences")
    qmv.attn_paged(cache, batch, q, heads * 64, out, heads * 64, heads, 0.1, 0, ws, wsb)
    torch.cuda.synchronize()


@both
@pytest.mark.parametrize("window", [1, 40, 2 ** 31 - 1])
def test_lengths_near_the_largest_integer(window, wide):
    """Positions far behind the table: a window there sees nothing, no window (or one of 2^31 - 1) the whole table."""
    c = Call([64, 64], [1, 3], 4, 2, 64, 16, "q8", seed=24, window=window, max_pages=4, wide=wide)
    if wide is True:  # the table's other pages do not exist
        assert c.P.max_pages * 16 == 10000
    c.upload()
    for lens in ([2 ** 31 - 1, 2 ** 31 - 1], [2 ** 31 - 97, 2 ** 31 - 33]):
        c.out.fill_(9.5)
        c.len.copy_(_ints(lens))
        c.enqueue()
        got = c.result()[:, : c.width].reshape(4, 4, 64)
        if window < 2 ** 31 - 1:
            assert (got == 0.0).all()
            continue
        q = c.q[:, : c.width].astype(np.float64).reshape(4, 4, 64)
        for r, b, back in ((0, 0, 1), (1, 1, 3), (2, 1, 2), (3, 1, 1)):
            ref, tol = R.attention(q[r:r + 1], c.P.rows("k", b), c.P.rows("v", b), [lens[b] - back], c.scale, window)
            assert_within(got[r:r + 1], ref, tol, f"row {r}")


def test_cache_beyond_32_bit_offsets():
    """A cache of more than 2^31 elements, with the sequence's pages at its end."""
    qmv = _qmv()
    rng = np.random.default_rng(16)
    heads, dim, page, L = 8, 128, 64, 130
    num = 2 ** 31 // (heads * page * dim) + 40
    small = R.Pages([L], heads, dim, page, "q8", rng)
    k = torch.zeros(num, heads, page, dim, dtype=torch.int8, device=DEV)
    v = torch.zeros_like(k)
    ks = torch.zeros(num, heads, page, device=DEV)
    vs = torch.zeros_like(ks)
    table = np.full((1, 4), -1, np.int32)
    for j in range(3):
        table[0, j] = num - 1 - 3 * j
        for dst, src in ((k, small.k), (v, small.v), (ks, small.ks), (vs, small.vs)):
            dst[int(table[0, j])] = dev(src[small.table[0, j]])
    cache = qmv.KVCache(k, v, ks, vs)
    batch = qmv.KVBatch(_ints(table), _ints([0, 1]), _ints([L]), 1)
    q = rng.normal(0, 1, (1, heads * dim)).astype(np.float32)
    out = torch.empty(1, heads * dim, device=DEV)
    wsb = qmv.attn_paged_ws_bytes(cache, batch, heads)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    qmv.attn_paged(cache, batch, dev(q), heads * dim, out, heads * dim, heads, 0.09, 0, ws, wsb)
    ref, tol = R.attention(q.astype(np.float64).reshape(1, heads, dim), small.rows("k", 0), small.rows("v", 0), [L - 1],
                           0.09, 0)
    assert_within(host(out).reshape(1, heads, dim), ref, tol, "far pages")


@both
def test_same_bits_every_time(wide):
    c = Call([3000, 100, 900], [4, 1, 9], 8, 2, 128, 32, "q8", seed=17, wide=wide).upload()
    c.enqueue()
    first = c.result().copy()
    for _ in range(3):
        c.ws.random_(0, 255)
        c.out.fill_(9.5)
        c.enqueue()
        assert np.array_equal(first.view(np.uint32), c.result().view(np.uint32))


def test_two_streams_with_workspaces_of_their_own():
    a = Call([2000, 64], [1, 3], 4, 2, 128, 16, "q8", seed=20).upload()
    b = Call([700, 1500], [2, 1], 4, 2, 64, 32, "f16", seed=21).upload()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.enqueue(s1)
        b.enqueue(s2)
    for c in (a, b):
        ref, tol = c.reference()
        assert_within(c.result()[:, : c.width].reshape(ref.shape), ref, tol, "on its stream")


def test_captured_and_replayed_as_the_sequence_grows():
    """The graph holds addresses, not lengths: replays follow kv_len, row_start and the table."""
    c = Call([40, 9], [1, 1], 4, 2, 128, 16, "q8", seed=22, max_pages=40)
    more = R.Pages([600, 300], 2, 128, 16, "q8", np.random.default_rng(23), max_pages=40)
    c.P = more
    c.upload()
    c.enqueue()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.enqueue()
    for lens in ([40, 9], [41, 10], [600, 0], [1, 300], [599, 299]):
        c.len.copy_(_ints(lens))
        c.out.fill_(9.5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = c.result().copy()
        c.out.fill_(9.5)
        c.enqueue()
        assert np.array_equal(replayed.view(np.uint32), c.result().view(np.uint32))
        got = replayed[:, : c.width].reshape(2, 4, 128)
        q = c.q[:, : c.width].astype(np.float64).reshape(2, 4, 128)
        for b in range(2):
            ref, tol = R.attention(q[b:b + 1], more.rows("k", b, lens[b]), more.rows("v", b, lens[b]), [lens[b] - 1],
                                   c.scale, 0)
            assert_within(got[b:b + 1], ref, tol, f"length {lens[b]}")
