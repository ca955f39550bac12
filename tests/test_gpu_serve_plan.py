"""kv_plan against a plain plan made of lists: pages, stack, row starts,
positions, slots, refusals.  Everything is whole numbers and has to be equal."""
import numpy as np
import pytest
import torch

import serve_ref as R
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

UNTOUCHED = -77


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def ints(a, dtype=torch.int32):
    return torch.from_numpy(np.asarray(a)).to(dtype).to(DEV)


class Plan:
    """A pool with sequences scattered over it, and one call."""

    def __init__(self, lens, page, width, free, rng, T):
        self.page, self.T, B = page, T, len(lens)
        held = [R.pages(n, page) for n in lens]
        order = rng.permutation(sum(held) + free)
        self.table = np.full((B, width), -5, np.int64)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.stack = np.full(len(order), -6, np.int64)
        self.stack[:free] = order[at:]
        self.count, self.lens = free, np.asarray(lens)

    def call(self, keep, n_new, in_place=False, position=True, slot=True, count=None, lens=None):
        qmv = _qmv()
        count = self.count if count is None else count
        lens = self.lens if lens is None else np.asarray(lens)
        B = len(lens)
        t, st, ln, ct = ints(self.table), ints(self.stack), ints(lens), ints([count])
        kp, nn = None if keep is None else ints(keep), ints(n_new)
        out_len = ln if in_place else ints([UNTOUCHED] * B)
        out_ct = ct if in_place else ints([UNTOUCHED])
        start, status = ints([UNTOUCHED] * (B + 1)), ints([UNTOUCHED] * 2)
        pos = ints([UNTOUCHED] * self.T) if position else None
        sl = ints([UNTOUCHED] * self.T, torch.int64) if slot else None
        pool = qmv.KVPool(t, st, self.page)
        size = qmv.kv_plan_ws_bytes(pool)
        ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV)
        qmv.kv_plan(pool, ln, kp, nn, ct, out_len, out_ct, start, pos, sl, status, self.T, ws, size)
        torch.cuda.synchronize()
        want = R.plan(self.table, self.stack, count, lens, keep, n_new, self.page, self.T)
        assert status.tolist() == want["status"]
        assert out_len.tolist() == want["new_len"] and out_ct.tolist() == [want["count"]]
        assert start.tolist() == want["row_start"]
        assert t.cpu().numpy().tolist() == want["table"].tolist()
        assert st.cpu().numpy()[:max(want["count"], 0)].tolist() == want["stack"]
        if want["status"][0]:
            assert st.cpu().numpy().tolist() == self.stack.tolist()
        for got, ref in ((pos, want["position"]), (sl, want["slot"])):
            if got is not None:
                full = np.full(self.T, UNTOUCHED)
                for r, v in ref.items():
                    full[r] = v
                assert got.cpu().numpy().tolist() == full.tolist()
        return want


def mixed(rng, B, top, page, width):
    """Lengths, kept ones and new rows of sequences that go on, drop, end, begin or do nothing."""
    lens = rng.integers(0, top + 1, B)
    keep, n = lens.copy(), rng.integers(0, 3 * page, B)
    kind = rng.integers(0, 6, B)
    keep[kind == 0], n[kind == 0] = 0, 0                    # ends
    lens[kind == 1], keep[kind == 1] = 0, 0                 # begins
    drop = kind == 2
    keep[drop] = (lens[drop] * rng.random(drop.sum())).astype(int)
    n[kind == 3] = 0                                        # waits
    n[kind == 4] = 1
    n = np.minimum(n, width * page - keep)
    return lens, keep, n


@pytest.mark.parametrize("B,page,width", [(1, 16, 4), (5, 16, 8), (64, 32, 6), (65, 128, 5), (1024, 16, 9), (1025, 16, 7),
                                          (3000, 64, 4), (65535, 16, 3)])
def test_plans(B, page, width):
    rng = np.random.default_rng(B + page)
    for turn in range(2 if B > 10000 else 4):
        say(f"kv_plan B={B} page={page} turn={turn}")
        lens, keep, n = mixed(rng, B, width * page, page, width)
        need = int(np.maximum(0, -(-(keep + n) // page) + (-lens // page)).sum())
        p = Plan(lens, page, width, need + (0, 1, 50, 3)[turn], rng, max(1, int(n.sum()) + (0, 7, 300, 1)[turn]))
        want = p.call(keep, n, in_place=turn % 2 == 1, position=turn != 2, slot=turn != 3)
        assert want["status"] == [0, 0]


def test_keep_missing_means_all():
    rng = np.random.default_rng(1)
    p = Plan([0, 15, 16, 17, 40], 16, 5, 6, rng, 40)
    say("kv_plan keep=None")
    p.call(None, [1, 1, 1, 15, 8])
    p.call(None, [1, 1, 1, 15, 8], in_place=True)


def test_pages_given_back_serve_the_same_step():
    """An empty stack: every page that is taken was just given back, across sequences."""
    rng = np.random.default_rng(2)
    p = Plan([160, 0, 33, 0, 80, 1], 16, 12, 0, rng, 300)
    say("kv_plan through the stack")
    want = p.call([0, 0, 1, 0, 80, 1], [0, 90, 0, 60, 16, 15])
    assert want["status"] == [0, 0] and want["count"] == 10 + 2 - 6 - 4 - 1
    # and with some on it
    p = Plan([160, 0, 33, 0, 80, 1], 16, 12, 3, rng, 300)
    p.call([0, 0, 1, 0, 80, 1], [0, 160, 0, 60, 16, 15])


def test_one_long_sequence():
    rng = np.random.default_rng(3)
    p = Plan([5], 16, 7000, 6999, rng, 100000)
    say("kv_plan one long sequence")
    assert p.call([5], [99995])["count"] == 6999 - 6249
    p = Plan([100000, 0], 16, 7000, 0, rng, 100000)
    p.call([0, 0], [0, 99999])


def test_refusals_leave_everything():
    rng = np.random.default_rng(4)
    say("kv_plan refusals")
    lens = [20, 0, 33]
    for free, keep, n, T, code, lacking in (
            (1, [20, 0, 33], [30, 16, 16], 100, R.PAGES, 3),
            (9, [20, 0, 33], [30, 16, 16], 61, R.ROWS, 0),
            (0, [20, 0, 33], [30, 16, 16], 5, R.PAGES + R.ROWS, 4),
            (9, [21, 0, 33], [0, 0, 0], 100, R.LENGTH, 0),
            (9, [-1, 0, 33], [0, 0, 0], 100, R.LENGTH, 0),
            (9, [20, 0, 33], [0, -1, 0], 100, R.LENGTH, 0),
            (9, [20, 0, 33], [0, 0, 2 ** 31 - 1], 100, R.LENGTH, 0),
            (9, [20, 0, 33], [45, 0, 0], 100, R.LENGTH, 0),
            (9, [20, 0, 33], [44, 0, 0], 44, 0, 0)):
        for in_place in (False, True):
            p = Plan(lens, 16, 4, free, rng, T)
            want = p.call(keep, n, in_place=in_place)
            assert want["status"] == [code, lacking]
    p = Plan(lens, 16, 4, 2, rng, 50)
    for lens2 in ([20, 65, 33], [20, -1, 33], [2 ** 31 - 1, 0, 0], [-2 ** 31, 0, 0]):
        assert p.call(None, [0, 0, 0], lens=lens2)["status"] == [R.LENGTH, 0]
    assert p.call([20, 0, 33], [1, 0, 0], count=-1)["status"] == [R.STACK, 0]
    assert p.call([20, 0, 33], [1, 0, 0], count=len(p.stack) + 1)["status"] == [R.STACK, 0]
    # pages that come back would not fit the stack
    assert p.call([0, 0, 0], [0, 0, 0], count=len(p.stack) - 4)["status"] == [R.STACK, 0]


def test_pages_are_moved_as_they_are():
    """Numbers outside the cache go back and come again, and their rows have no slot."""
    rng = np.random.default_rng(5)
    p = Plan([64, 0], 16, 6, 1, rng, 90)
    p.table[0, :4] = [-1, 2 ** 31 - 1, -2 ** 31, len(p.stack)]
    say("kv_plan pages outside the cache")
    want = p.call([0, 0], [0, 80])
    assert -1 in want["slot"].values()


def test_a_loop_of_steps():
    """Steps in place, one after the other: no page is lost or held twice."""
    qmv = _qmv()
    rng = np.random.default_rng(6)
    B, page, width, num = 40, 16, 10, 200
    t, st = ints(np.full((B, width), -1)), ints(rng.permutation(num))
    ln, ct, start, status = ints([0] * B), ints([num]), ints([0] * (B + 1)), ints([0, 0])
    T = 4000
    pos, sl = ints([0] * T), ints([0] * T, torch.int64)
    pool = qmv.KVPool(t, st, page)
    size = qmv.kv_plan_ws_bytes(pool)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    lens = np.zeros(B, int)
    refused = 0
    for step in range(60):
        say(f"kv_plan step {step}")
        keep = np.maximum(lens - rng.integers(0, 4, B), 0)
        n = rng.integers(0, 30, B)
        ends = rng.random(B) < 0.15
        keep[ends], n[ends] = 0, 0
        n = np.minimum(n, width * page - keep)
        qmv.kv_plan(pool, ln, ints(keep), ints(n), ct, ln, ct, start, pos, sl, status, T, ws, size)
        torch.cuda.synchronize()
        if status.tolist()[0] == 0:
            lens = keep + n
        else:
            refused += 1
            assert status.tolist()[0] == R.PAGES and start.tolist() == [0] * (B + 1)
            drop = rng.random(B) < 0.5  # the server ends half of them
            qmv.kv_plan(pool, ln, ints(np.where(drop, 0, lens)), ints([0] * B), ct, ln, ct, start, pos, sl, status, T, ws, size)
            torch.cuda.synchronize()
            lens = np.where(drop, 0, lens)
            assert status.tolist()[0] == 0
        assert ln.tolist() == lens.tolist()
        table, stack, count = t.cpu().numpy(), st.cpu().numpy(), int(ct)
        held = [int(g) for b in range(B) for g in table[b, :R.pages(int(lens[b]), page)]]
        assert sorted(held + stack[:count].tolist()) == list(range(num))
    assert refused > 0
