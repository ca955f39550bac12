"""logits_draw against the definition in 64 bits: tokens and counts are equal
wherever no decision lies within the documented distance of its border."""
import math

import numpy as np
import pytest
import torch

import serve_ref as R
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

NEG, NAN, INF, LOW = -np.inf, np.nan, np.inf, np.finfo(np.float32).min


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def up(a, dtype):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def run(z, temperature, top_k=None, top_p=None, min_p=None, u=0.5, softcap=0.0, ld=0, offset=0, want_kept=True):
    """z [M][V]; filters are one number or one a row."""
    qmv = _qmv()
    z = np.asarray(z, dtype=np.float32)
    M, V = z.shape
    full = lambda a, t: None if a is None else np.broadcast_to(np.asarray(a, dtype=t), (M,)).copy()  # noqa: E731
    temperature, top_k, top_p, min_p, u = (full(temperature, np.float32), full(top_k, np.int32), full(top_p, np.float32),
                                           full(min_p, np.float32), full(u, np.float32))
    ld = ld or V
    buf = torch.full((offset + M * ld,), 1e30, device=DEV)
    rows = buf[offset:].view(M, ld)
    rows[:, :V] = torch.from_numpy(z).to(DEV)
    token, kept = (torch.full((M,), -9, dtype=torch.int32, device=DEV) for _ in range(2))
    size = qmv.logits_draw_ws_bytes(V, M)
    ws = torch.full((size,), 0xC3, dtype=torch.uint8, device=DEV)
    qmv.logits_draw(rows, ld, up(temperature, torch.float32), up(top_k, torch.int32), up(top_p, torch.float32),
                    up(min_p, torch.float32), up(u, torch.float32), token, kept if want_kept else None, V, M, softcap, ws, size)
    torch.cuda.synchronize()
    return token.cpu().numpy(), kept.cpu().numpy(), (temperature, top_k, top_p, min_p, u)


def check(z, *args, least=0.6, **kw):
    """Compares with the definition; at least this share of the rows is decided."""
    z = np.asarray(z, dtype=np.float32)
    softcap = kw.get("softcap", 0.0)
    token, kept, rows = run(z, *args, **kw)
    M, V = z.shape
    decided = 0
    for m in range(M):
        a = [None if r is None else r[m] for r in rows]
        t, n, far = R.draw_row(z[m], *a, softcap)
        if not far:
            continue
        decided += 1
        assert (token[m], kept[m]) == (t, n), f"row {m} of {M}x{V}, {a}: {token[m], kept[m]}, not {t, n}"
    assert decided >= least * M, (decided, M)
    return token, kept


def logits(rng, M, V, peaks=True):
    z = rng.normal(0, 2.0, (M, V)).astype(np.float32)
    if peaks:
        k = min(48, V)
        for m in range(M):
            z[m, rng.choice(V, k, replace=False)] = rng.random(k) * 9 + 3
    return z


FILTERS = [dict(), dict(top_k=1), dict(top_k=5), dict(top_k=50), dict(top_k=3000), dict(top_p=0.9), dict(top_p=0.3),
           dict(top_p=0.999), dict(min_p=0.05), dict(min_p=1e-6), dict(top_k=40, top_p=0.95), dict(top_k=500, top_p=0.5, min_p=0.01),
           dict(top_k=0, top_p=1.0, min_p=0.0)]


@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 1000, 4096, 4097, 32000, 50257])
def test_filters(V):
    rng = np.random.default_rng(V)
    for i, f in enumerate(FILTERS):
        say(f"logits_draw V={V} {f}")
        for peaks in (True, False):
            check(logits(rng, 6, V, peaks), rng.choice([0.5, 0.8, 1.0, 1.5], 6), u=rng.random(6), **f)


@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_mixed_rows(M):
    rng = np.random.default_rng(M)
    V = 9001
    say(f"logits_draw M={M} mixed")
    check(logits(rng, M, V), rng.choice([0.0, 0.3, 0.7, 1.0, 2.0], M), rng.choice([-3, 0, 1, 7, 64, 900, 20000], M),
          rng.choice([1.0, 1.5, 0.95, 0.5, 0.0, -1.0], M), rng.choice([0.0, -1.0, 0.02, 0.5, 1.0, 3.0], M), u=rng.random(M))


@pytest.mark.parametrize("V,M", [(262144, 1), (262144, 5), (262143, 2), (600001, 2), (128256, 3)])
def test_large_vocabularies(V, M):
    rng = np.random.default_rng(V)
    for f in (dict(), dict(top_k=50, top_p=0.9), dict(top_p=0.95), dict(min_p=0.02), dict(top_k=100000)):
        for softcap in (0.0, 30.0):
            for peaks in (True, False):
                say(f"logits_draw V={V} M={M} {f} softcap={softcap} peaks={peaks}")
                check(logits(rng, M, V, peaks), 0.8, u=rng.random(M), softcap=softcap, least=0.5, **f)


@pytest.mark.parametrize("fill", [NEG, LOW, NAN])
def test_masked_rows(fill):
    """Most of the vocabulary is forbidden, by each of the ways to say so; all of it in one row."""
    rng = np.random.default_rng(1)
    V, M = 20000, 12
    z = logits(rng, M, V)
    z[rng.random((M, V)) < 0.99] = fill
    z[3] = fill
    z[4] = fill
    z[4, 777] = -50.0
    z[5, :] = fill
    z[5, [3, 19999]] = [2.0, 2.0]
    for f in FILTERS:
        say(f"logits_draw masked by {fill} {f}")
        check(z, 1.0, u=rng.random(M), least=0.8, **f)  # rows 3 and 5 have equal weights: half of them is a border
    token, kept, _ = run(z, [1.0, 0.0] * 6)
    if fill is not LOW:
        assert token[3] == -1 and kept[3] == 0 and token[4] == 777 and kept[4] == 1 and kept[5] in (1, 2)
    else:  # one weight for all of them
        assert 0 <= token[3] < V


def test_ties_go_to_the_lowest_index():
    V = 5000
    z = np.zeros((8, V), np.float32)
    say("logits_draw equal logits")
    u = (np.arange(8) + 0.5) / 8
    # V equal weights: the first n by index, and the token is floor(u n)
    for k, p, n in ((0, 1.0, V), (100, 1.0, 100), (0, 0.5, V // 2), (1000, 0.25, 250), (1, 1.0, 1), (4999, 1.0, 4999)):
        token, kept, _ = run(z, 1.0, k, p, u=u)
        assert kept.tolist() == [n] * 8
        assert token.tolist() == np.floor(np.float64(u) * n).astype(int).tolist()
    # pairs of equal logits across the row, and signed zeros
    rng = np.random.default_rng(2)
    z = rng.integers(-6, 7, (8, V)).astype(np.float32) * np.where(rng.random((8, V)) < 0.5, 1, 1).astype(np.float32)
    z[z == 0] = np.where(rng.random((z == 0).sum()) < 0.5, 0.0, -0.0)
    for f in FILTERS:
        check(z, 2.0, u=rng.random(8), **f)
    z = np.full((3, V), -2.0, np.float32)
    z[0, 4001], z[0, 17] = 0.0, -0.0
    token, kept, _ = run(z, 0.0)
    assert token.tolist() == [17, 0, 0] and kept.tolist() == [1, 1, 1]


def test_large_tied_vocabulary():
    V = 262144
    say("logits_draw 262144 equal logits")
    z = np.full((2, V), 3.0, np.float32)
    token, kept, _ = run(z, 1.0, [0, 200000], [1.0, 0.5], u=[0.75, 0.5])
    assert kept.tolist() == [V, 100000] and token.tolist() == [V * 3 // 4, 50000]


def test_infinities():
    V = 3000
    rng = np.random.default_rng(3)
    z = logits(rng, 6, V)
    z[0, [5, 2900]] = INF
    z[1, 100] = INF
    z[1, 50] = np.finfo(np.float32).max
    z[2, :] = INF
    z[3, 7] = NAN
    z[4, :] = NEG
    z[4, 2999] = LOW
    say("logits_draw infinities")
    for t in (0.0, 1.0, 3e38, 1e-30):
        token, kept = check(z, t, u=rng.random(6))
        assert token[0] in (5, 2900) or t > 1e30
    token, kept, _ = run(z, 1.0, u=0.75)
    assert token[0] == 2900 and kept[0] == V and token[1] == 100 and token[4] == 2999 and kept[4] == 1


def test_temperatures():
    """None (the first), the smallest, very large, infinite (every weight 1) and no number."""
    V = 2000
    rng = np.random.default_rng(4)
    z = logits(rng, 1, V)
    say("logits_draw temperatures")
    for t in (0.0, -0.0, -1.0, NAN, NEG):
        token, kept, _ = run(z, t, u=0.9)
        assert token[0] == z[0].argmax() and kept[0] == 1
    for t in (1e-45, 1e-38, 1e-10):
        token, kept, _ = run(z, t, u=0.999)
        assert token[0] == z[0].argmax() and kept[0] == V
    for t in (3e38, INF):
        token, kept, _ = run(z, t, top_k=1000, u=(10 + 0.5) / 1000)
        order = np.lexsort((np.arange(V), -z[0]))
        assert token[0] == order[10] and kept[0] == 1000
    z[0, 0], z[0, 1] = 3e38, -3e38
    for t in (1e-45, 1.0, 1e38, INF):
        check(np.repeat(z, 4, 0), t, u=rng.random(4), softcap=0.0)


def test_random_numbers_at_their_ends():
    V = 777
    rng = np.random.default_rng(5)
    z = logits(rng, 1, V, peaks=False)
    order = np.lexsort((np.arange(V), -z[0]))
    say("logits_draw u at its ends")
    for u, want in ((0.0, 0), (-1.0, 0), (NAN, 0), (1.0, 49), (5.0, 49), (INF, 49), (np.float32(1 - 2.0 ** -24), 49)):
        token, kept, _ = run(z, 1.0, top_k=50, u=u)
        assert token[0] == order[want] and kept[0] == 50, u


def test_strong_caps():
    """Logits far beyond the cap have one weight and keep their order."""
    V = 4000
    rng = np.random.default_rng(6)
    z = logits(rng, 5, V) * 100
    say("logits_draw strong caps")
    for cap in (0.01, 1.0, 50.0, 65536.0):
        check(z, 1.0, u=rng.random(5), softcap=cap, least=0.5)
        check(z, 1.0, top_k=33, u=rng.random(5), softcap=cap, least=0.5)


@pytest.mark.parametrize("spread,shift", [(1e-6, 0.0), (1e-3, 1000.0), (30.0, 0.0), (300.0, -5000.0), (1e20, 0.0)])
def test_spreads(spread, shift):
    """Logits that lie close together, far apart, or far from zero."""
    V = 30000
    rng = np.random.default_rng(7)
    z = (rng.normal(0, 1, (6, V)) * spread + shift).astype(np.float32)
    for f in FILTERS:
        say(f"logits_draw spread={spread} shift={shift} {f}")
        check(z, 1.0, u=rng.random(6), **f)


def test_one_logit_stands_far_out():
    """A single very large or very small logit beside an ordinary row."""
    V = 40000
    rng = np.random.default_rng(8)
    for v in (1e6, -1e6, 3e38, -3e38, 60.0):
        z = logits(rng, 4, V)
        z[:, 12345] = v
        for f in FILTERS:
            say(f"logits_draw one logit {v} {f}")
            check(z, 1.0, u=rng.random(4), **f)


@pytest.mark.parametrize("offset,ld", [(0, 5003), (1, 0), (3, 5001), (2, 5004)])
def test_strides_and_alignment(offset, ld):
    rng = np.random.default_rng(9)
    say(f"logits_draw offset={offset} ld={ld}")
    check(logits(rng, 7, 5000), 0.9, 40, 0.9, 0.01, u=rng.random(7), offset=offset, ld=ld)


def test_no_place_for_the_counts():
    rng = np.random.default_rng(10)
    z = logits(rng, 3, 1000)
    say("logits_draw kept=None")
    a, _, _ = run(z, 1.0, 10, u=0.3)
    b, kept, _ = run(z, 1.0, 10, u=0.3, want_kept=False)
    assert np.array_equal(a, b) and (kept == -9).all()


def test_the_same_every_time():
    rng = np.random.default_rng(11)
    z = logits(rng, 20, 100000)
    say("logits_draw again")
    a = run(z, 1.0, None, 0.9, u=rng.random(20).astype(np.float32))
    for _ in range(5):
        b = run(z, 1.0, None, 0.9, u=a[2][4])
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_frequencies():
    """Tokens come as often as their weights say (a chi-square far below its 1e-9 point)."""
    V, M = 12, 40000
    rng = np.random.default_rng(12)
    z = np.tile(rng.normal(0, 1, V).astype(np.float32), (M, 1))
    say("logits_draw frequencies")
    token, kept, _ = run(z, 0.7, 8, u=rng.random(M))
    w = np.exp(z[0].astype(np.float64) / np.float32(0.7))
    w[np.argsort(-w)[8:]] = 0
    want = M * w / w.sum()
    got = np.bincount(token, minlength=V)
    assert (got[want == 0] == 0).all()
    assert ((got - want)[want > 0] ** 2 / want[want > 0]).sum() < 60
