"""lora_add against the adapters' products in 64 bits."""
import numpy as np
import pytest
import torch

import serve_ref as R
from gpu_util import DEV, assert_within, say

pytestmark = pytest.mark.gpu

UNTOUCHED = -77.0


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def strided(a, ld, offset=0):
    """Rows of a, ld apart, `offset` floats into a buffer of UNTOUCHED."""
    T, n = a.shape
    buf = torch.full((offset + T * ld + 4,), UNTOUCHED, device=DEV)
    rows = buf[offset:offset + T * ld].view(T, ld)
    rows[:, :n] = torch.from_numpy(a).to(DEV)
    return buf, rows


class Adapters:
    def __init__(self, slots, max_rank, K, N, fmt, ragged, seed):
        rng = np.random.default_rng(seed)
        self.dtype = torch.bfloat16 if fmt == "bf16" else torch.float16
        f = lambda a: torch.from_numpy(a.astype(np.float32)).to(self.dtype)  # noqa: E731
        self.A, self.Bm = f(rng.normal(0, K ** -0.5, (slots, max_rank, K))), f(rng.normal(0, 0.3, (slots, N, max_rank)))
        self.scale = (rng.random(slots) + 0.5).astype(np.float32) * np.where(rng.random(slots) < 0.3, -1, 1).astype(np.float32)
        self.rank = None
        if ragged:
            self.rank = rng.integers(0, max_rank + 1, slots).astype(np.int32)
            self.rank[:3] = [max_rank + 5, 0, -2][:slots]
            for s in range(slots):  # what no rank reaches must not matter
                r = int(np.clip(self.rank[s], 0, max_rank))
                self.A[s, r:], self.Bm[s, :, r:] = float("nan"), float("inf")
        self.K, self.N = K, N

    def gpu(self):
        return _qmv().Lora(self.A.to(DEV), self.Bm.to(DEV), torch.from_numpy(self.scale).to(DEV),
                           None if self.rank is None else ints(self.rank))

    def ref(self, adapter, start, x, base):
        A = torch.nan_to_num(self.A.double(), 0, 0, 0).numpy()
        Bm = torch.nan_to_num(self.Bm.double(), 0, 0, 0).numpy()
        return R.lora(A, Bm, self.scale, self.rank, adapter, start, x, base)


def check(L, adapter, rows, spare=3, base="other", ldx=0, ldb=0, ldy=0, offset=0, seed=0, lora=None):
    qmv = _qmv()
    rng = np.random.default_rng(seed)
    start = np.concatenate([[0], np.cumsum(rows)]).astype(int)
    T, B = int(start[-1]) + spare, len(rows)
    x = rng.normal(0, 1, (T, L.K)).astype(np.float32)
    b = rng.normal(0, 1, (T, L.N)).astype(np.float32)
    ldx, ldb, ldy = ldx or L.K, ldb or L.N, ldy or L.N
    _, xs = strided(x, ldx, offset)
    bbuf, bs = strided(b, ldb, offset)
    ybuf, ys = strided(np.full((T, L.N), UNTOUCHED, np.float32), ldy, offset)
    before = None
    if base == "y":
        ybuf, ys, ldy = bbuf, bs, ldb
        before = bs.clone()
    d = lora or L.gpu()
    size = qmv.lora_add_ws_bytes(d, B, T)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN everywhere
    qmv.lora_add(d, ints(adapter), ints(start), xs, ldx, None if base is None else bs, ldb, ys, ldy, B, T, ws, size)
    torch.cuda.synchronize()
    want, tol = L.ref(adapter, start, x, None if base is None else b)
    n = int(start[-1])
    got = ys.cpu().numpy()
    if n:
        assert_within(got[:n, :L.N], want[:n], tol[:n], "rows")
    rest = np.full((spare, L.N), UNTOUCHED) if before is None else b[n:]
    assert np.array_equal(got[n:, :L.N], rest)
    assert (got[:, L.N:] == UNTOUCHED).all()
    full = ybuf.cpu().numpy()
    assert (full[:offset] == UNTOUCHED).all() and (full[offset + T * ldy:] == UNTOUCHED).all()
    return got[:n, :L.N]


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("max_rank,K,N", [(8, 64, 32), (16, 512, 300), (16, 5376, 1000), (24, 104, 77), (32, 2048, 513),
                                          (64, 1376, 640), (128, 512, 200), (256, 264, 130)])
@pytest.mark.parametrize("rows", [[1], [1, 1, 1, 1, 1], [0, 7, 1, 0, 33, 2], [130, 0, 1, 64, 16]])
def test_ranks_widths_and_rows(fmt, max_rank, K, N, rows):
    say(f"lora_add {fmt} R={max_rank} K={K} N={N} rows={rows}")
    for ragged in (False, True):
        L = Adapters(4, max_rank, K, N, fmt, ragged, K + max_rank)
        adapter = np.arange(len(rows)) * 3 % 4 + (0 if ragged else 0)
        if len(rows) > 2:
            adapter[2] = -1
        check(L, adapter, rows)


@pytest.mark.parametrize("base", [None, "y", "other"])
@pytest.mark.parametrize("adapter", [[0, 1, 2, 1], [-1, 3, 5, 2 ** 31 - 1], [-1, -1, -2 ** 31, -1], [2, 2, 2, 2]])
def test_bases_and_adapters_outside(base, adapter):
    say(f"lora_add base={base} adapter={adapter}")
    L = Adapters(3, 16, 256, 270, "bf16", False, 1)
    for rows in ([1, 2, 1, 1], [5, 40, 0, 21]):
        check(L, adapter, rows, base=base, seed=3)


@pytest.mark.parametrize("offset,ldx,ldb,ldy", [(1, 0, 0, 0), (0, 259, 301, 333), (2, 264, 304, 304), (3, 257, 0, 0)])
def test_strides_and_alignment(offset, ldx, ldb, ldy):
    say(f"lora_add offset={offset} ld={ldx, ldb, ldy}")
    for fmt in ("bf16", "f16"):
        L = Adapters(3, 16, 256, 300, fmt, True, 2)
        for rows in ([1, 1, 1], [3, 50, 18]):
            check(L, [0, 1, 2], rows, offset=offset, ldx=ldx, ldb=ldb, ldy=ldy)
            check(L, [2, -1, 0], rows, offset=offset, ldx=ldx, ldb=ldb, ldy=ldy, base="y")


def test_many_sequences_and_empty_ones():
    rng = np.random.default_rng(5)
    L = Adapters(7, 16, 128, 96, "bf16", True, 5)
    for B in (300, 5000):
        say(f"lora_add B={B}")
        rows = rng.integers(0, 3, B) * (rng.random(B) < 0.5)
        check(L, rng.integers(-1, 8, B), rows)
    say("lora_add no rows at all")
    check(L, [0, 1, 2], [0, 0, 0], spare=5)


def test_a_long_chunk():
    say("lora_add 1500 rows")
    check(Adapters(2, 16, 1024, 1100, "f16", False, 6), [1, 0, 1], [1200, 3, 300], seed=6)


def test_large_and_small_numbers():
    """float16 weights near their ends, x from 1e-30 to 1e30."""
    say("lora_add large and small numbers")
    L = Adapters(3, 16, 256, 64, "f16", False, 7)
    L.A[0] *= 1e4
    L.Bm[1] = (L.Bm[1].double() * 2.0 ** -20).half()  # subnormal
    qmv = _qmv()
    d = L.gpu()
    rng = np.random.default_rng(7)
    for T in (4, 60):
        x = (rng.normal(0, 1, (T, 256)) * 10.0 ** np.linspace(-30, 30, T)[:, None]).astype(np.float32)
        start = [0, T // 3, T // 2, T]
        size = qmv.lora_add_ws_bytes(d, 3, T)
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        y = torch.empty(T, 64, device=DEV)
        qmv.lora_add(d, ints([0, 1, 2]), ints(start), torch.from_numpy(x).to(DEV), 256, None, 64, y, 64, 3, T, ws, size)
        want, tol = L.ref([0, 1, 2], start, x, None)
        # results below float32's normal numbers are off by half a step of the smallest ones, as are the ranks
        floor = 2.0 ** -149 * (1 + 16 * 64.0)
        assert_within(y.cpu().numpy(), want, tol + floor, "rows")


def test_rows_are_independent():
    """NaN and infinity in one row stay there."""
    say("lora_add NaN in a row")
    L = Adapters(2, 16, 256, 64, "bf16", False, 8)
    qmv = _qmv()
    d = L.gpu()
    rng = np.random.default_rng(8)
    for T in (6, 50):
        x = rng.normal(0, 1, (T, 256)).astype(np.float32)
        out = []
        for bad in (False, True):
            z = x.copy()
            if bad:
                z[2, 7], z[4, 200] = np.nan, np.inf
            size = qmv.lora_add_ws_bytes(d, 2, T)
            ws = torch.empty(size, dtype=torch.uint8, device=DEV)
            y = torch.empty(T, 64, device=DEV)
            qmv.lora_add(d, ints([0, 1]), ints([0, 3, T]), torch.from_numpy(z).to(DEV), 256, None, 64, y, 64, 2, T, ws, size)
            out.append(y.cpu().numpy())
        ok = np.ones(T, bool)
        ok[[2, 4]] = False
        assert np.array_equal(out[0][ok], out[1][ok]) and not np.isfinite(out[1][~ok]).any()


def test_row_starts_out_of_order_touch_nothing_else():
    say("lora_add row starts out of order")
    qmv = _qmv()
    L = Adapters(2, 16, 64, 32, "bf16", False, 9)
    d = L.gpu()
    for T in (5, 80):
        for start in ([0, 9, 3], [-5, -2, 100], [5, 1, 0], [0, 2 ** 31 - 1, -2 ** 31], [3, 3, 5], [0, T + 50, T + 90]):
            buf = torch.full((T + 40, 32), UNTOUCHED, device=DEV)
            x = torch.randn(T, 64, device=DEV)
            size = qmv.lora_add_ws_bytes(d, 2, T)
            full = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
            qmv.lora_add(d, ints([0, 1]), ints(start), x, 64, None, 32, buf[20:20 + T], 32, 2, T, full[:size], size)
            torch.cuda.synchronize()
            assert (buf[:20] == UNTOUCHED).all() and (buf[20 + T:] == UNTOUCHED).all() and (full[size:] == 0x5A).all()
