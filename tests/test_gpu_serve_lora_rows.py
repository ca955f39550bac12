"""lora_add on rows that do not begin with the buffer's: the row starts of a
part of a batch.  Rows before the first start belong to no sequence here."""
import numpy as np
import pytest
import torch

import serve_ref as R
from gpu_util import DEV, assert_within, say
from test_gpu_serve_lora import UNTOUCHED, Adapters, ints, strided

pytestmark = pytest.mark.gpu


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def call(L, adapter, start, T, base, seed):
    """y [T][N] before and after, and the definition's rows (NaN: of no sequence)."""
    qmv = _qmv()
    rng = np.random.default_rng(seed)
    B = len(start) - 1
    x, b = (rng.normal(0, 1, (T, n)).astype(np.float32) for n in (L.K, L.N))
    _, xs = strided(x, L.K)
    _, bs = strided(b, L.N)
    _, ys = strided(np.full((T, L.N), UNTOUCHED, np.float32), L.N)
    if base == "y":
        ys = bs
    before = ys.cpu().numpy()
    d = L.gpu()
    size = qmv.lora_add_ws_bytes(d, B, T)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    qmv.lora_add(d, ints(adapter), ints(start), xs, L.K, None if base is None else bs, L.N, ys, L.N, B, T, ws, size)
    torch.cuda.synchronize()
    want, tol = L.ref(adapter, start, x, None if base is None else b)
    return before, ys.cpu().numpy(), want, tol


def check(L, adapter, start, spare, base, seed):
    first, end = int(start[0]), int(start[-1])
    before, got, want, tol = call(L, adapter, start, end + spare, base, seed)
    assert np.array_equal(got[:first], before[:first]), "rows before the first sequence"
    assert np.array_equal(got[end:], before[end:]), "rows behind the last sequence"
    if end > first:
        assert_within(got[first:end], want[first:end], tol[first:end], "rows")


@pytest.mark.parametrize("base", [None, "y", "other"])
@pytest.mark.parametrize("first", [1, 3, 15, 16, 32, 35, 100])
def test_rows_before_the_first_sequence(first, base):
    for rows in ([1], [16], [1, 1, 1], [5, 0, 40, 1], [0, 0, 0]):
        say(f"lora_add first={first} rows={rows} base={base}")
        start = first + np.concatenate([[0], np.cumsum(rows)])
        for max_rank in (16, 64):
            L = Adapters(3, max_rank, 256, 300, "bf16", False, first)
            check(L, np.arange(len(rows)) % 3, start, 3, base, seed=first)
            check(L, -1 + np.arange(len(rows)) % 3, start, 0, base, seed=first)


@pytest.mark.parametrize("base", [None, "y", "other"])
@pytest.mark.parametrize("first", [3, 32, 100, 2000])
def test_rows_before_many_sequences(first, base):
    rng = np.random.default_rng(first)
    L = Adapters(5, 16, 128, 96, "f16", True, 5)
    for B in (65, 300):
        say(f"lora_add first={first} B={B} base={base}")
        start = first + np.concatenate([[0], np.cumsum(rng.integers(0, 4, B))])
        check(L, rng.integers(-1, 6, B), start, 5, base, seed=B)


@pytest.mark.parametrize("at", [1, 40, 70])
def test_a_batch_in_two_calls(at):
    """Row starts and adapters from a sequence on, and up to it: together the whole batch, in place."""
    qmv = _qmv()
    rng = np.random.default_rng(at)
    L = Adapters(4, 16, 256, 130, "bf16", False, 1)
    d = L.gpu()
    rows = rng.integers(0, 20, 100)
    start = np.concatenate([[0], np.cumsum(rows)])
    T, adapter = int(start[-1]), rng.integers(-1, 4, 100)
    x, b = (rng.normal(0, 1, (T, n)).astype(np.float32) for n in (L.K, L.N))
    y, xs = torch.from_numpy(b).to(DEV), torch.from_numpy(x).to(DEV)
    say(f"lora_add in two calls at {at}")
    s, a = ints(start), ints(adapter)
    for lo, hi in ((at, 100), (0, at)):
        size = qmv.lora_add_ws_bytes(d, hi - lo, T)
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        qmv.lora_add(d, a[lo:hi], s[lo:hi + 1], xs, L.K, y, L.N, y, L.N, hi - lo, T, ws, size)
    torch.cuda.synchronize()
    want, tol = L.ref(adapter, start, x, b)
    assert_within(y.cpu().numpy(), want, tol, "rows")
