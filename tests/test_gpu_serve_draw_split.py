"""logits_draw on rows that several workgroups share (long rows): mixed
arguments, masks, equal logits, wide bins, strides, streams and graphs."""
import numpy as np
import pytest
import torch

import serve_ref as R
from gpu_util import DEV, say
from test_gpu_serve_draw import FILTERS, INF, LOW, NAN, NEG, check, logits, run

pytestmark = pytest.mark.gpu


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


@pytest.mark.parametrize("V,M", [(17000, 3), (41000, 40), (70000, 2), (66000, 129), (41000, 257), (41000, 512), (41000, 513)])
def test_mixed_rows(V, M):
    rng = np.random.default_rng(V + M)
    say(f"logits_draw V={V} M={M} mixed")
    z = logits(rng, M, V)
    if M > 2:
        z[rng.integers(0, M, M // 3)] = NEG                       # rows without anything
        z[rng.integers(0, M, M // 3), : V - 50] = NAN             # with little
    check(z, rng.choice([0.0, 0.3, 0.7, 1.0, 2.0], M), rng.choice([-3, 0, 0, 1, 7, 64, 900, 5000, 10 ** 6], M),
          rng.choice([1.0, 1.5, 0.95, 0.5, 0.0, -1.0], M), rng.choice([0.0, -1.0, 0.02, 0.5, 1.0, 3.0], M), u=rng.random(M))


@pytest.mark.parametrize("kind", ["none", "by runs", "counted", "summed"])
@pytest.mark.parametrize("M", [2, 9])
def test_all_rows_of_a_kind(kind, M):
    """The work is shared out by what the rows ask for: all of one kind."""
    rng = np.random.default_rng(M)
    V = 90000
    z = logits(rng, M, V)
    say(f"logits_draw {M} rows {kind}")
    t, k = {"none": (0.0, 5), "by runs": (1.0, 300), "counted": (1.0, 1500), "summed": (1.0, 0)}[kind]
    check(z, t, k, 0.9, 0.01, u=rng.random(M))
    check(z, t, k, u=rng.random(M))


@pytest.mark.parametrize("fill", [NEG, LOW, NAN])
def test_masked_rows(fill):
    rng = np.random.default_rng(1)
    V, M = 60000, 6
    z = logits(rng, M, V)
    z[rng.random((M, V)) < 0.99] = fill
    z[1, rng.random(V) < 0.9] = fill
    z[2] = fill
    z[2, 59999] = 1.0
    z[3] = fill
    z[3, ::1000] = np.arange(60) % 7  # fewer than most top-k
    for f in FILTERS:
        say(f"logits_draw split, masked by {fill} {f}")
        check(z, 1.0, u=rng.random(M), least=0.5, **f)


def test_bins_without_width():
    """Infinite temperature over equal and masked logits: every weight is 1, and what is masked stays out."""
    say("logits_draw infinite temperature")
    for V in (3000, 60000):
        z = np.full((4, V), 2.5, np.float32)
        z[:, ::3] = NEG
        z[1, 1::3] = NAN
        ok = np.flatnonzero(z[0] > NEG)
        for k, p in ((0, 1.0), (0, 0.5), (1000, 1.0), (40, 0.5), (5000, 0.25)):
            token, kept, _ = run(z, [INF, INF, 3e38, 1e30], k, p, u=0.5)
            for m in range(4):
                live = np.flatnonzero(z[m] > NEG)
                n = min(len(live), k or len(live))
                n = int(np.ceil(p * n))
                assert kept[m] == n and token[m] == live[n // 2], (V, k, p, m)
        assert len(ok) == V - -(-V // 3)


@pytest.mark.parametrize("V", [3000, 45000])
def test_far_logits_keep_their_order(V):
    """Logits hundreds of times the mean distance away, which weigh as much as any at such a temperature."""
    say(f"logits_draw far logits V={V}")
    rng = np.random.default_rng(3)
    z = rng.normal(0, 0.1, (6, V)).astype(np.float32)
    far = rng.permutation(V)[:900]
    z[:, far] = -(10.0 ** rng.uniform(1, 5.9, (6, 900)))
    for k in (0, V - 450, V - 100, 2000, 2048):
        check(z, 1e20, k, 1.0, u=rng.random(6), least=0)
        for u in (0.97, 0.99, 0.999):
            token, kept, _ = run(z, INF, k, 1.0, u=u)
            for m in range(6):
                n = k or V
                order = np.lexsort((np.arange(V), -z[m]))
                assert kept[m] == n and token[m] == order[int(np.float64(np.float32(u)) * n)], (k, u, m)


def test_ties():
    say("logits_draw split, ties")
    rng = np.random.default_rng(2)
    V = 100000
    z = rng.integers(-6, 7, (4, V)).astype(np.float32)
    for f in FILTERS:
        # 500 equal weights have a border at their half: those rows are not decided here
        check(z, 2.0, u=rng.random(4), least=0 if f.get("top_p") == 0.5 else 0.5, **f)
    z[:] = -1.0
    u = (np.arange(4) + 0.5) / 4
    for k, p, n in ((0, 1.0, V), (1000, 0.25, 250), (2048, 1.0, 2048), (90000, 0.5, 45000)):
        token, kept, _ = run(z, 1.0, k, p, u=u)
        assert kept.tolist() == [n] * 4 and token.tolist() == np.floor(np.float64(u) * n).astype(int).tolist()


@pytest.mark.parametrize("spread,shift", [(1e-6, 0.0), (1e-3, 1000.0), (300.0, -5000.0), (1e20, 0.0)])
def test_spreads(spread, shift):
    V = 45000
    rng = np.random.default_rng(7)
    z = (rng.normal(0, 1, (3, V)) * spread + shift).astype(np.float32)
    for f in FILTERS:
        say(f"logits_draw split, spread={spread} shift={shift} {f}")
        check(z, 1.0, u=rng.random(3), **f)


@pytest.mark.parametrize("offset,ld", [(0, 50003), (1, 0), (3, 50001), (2, 50004)])
def test_strides_and_alignment(offset, ld):
    rng = np.random.default_rng(9)
    say(f"logits_draw split, offset={offset} ld={ld}")
    z = logits(rng, 5, 50000)
    for k in (0, 40, 1000):
        check(z, 0.9, k, 0.9, 0.01, u=rng.random(5), offset=offset, ld=ld)


def _call(z, k, p, u, ws, size, token, kept):
    M, V = z.shape
    _qmv().logits_draw(z, V, torch.full((M,), 0.9, device=DEV), k, p, None, u, token, kept, V, M, 30.0, ws, size)


def test_two_streams_with_a_workspace_each():
    qmv = _qmv()
    say("logits_draw on two streams")
    g = torch.Generator(device=DEV).manual_seed(5)
    V, M = 131072, 8
    streams = [torch.cuda.Stream() for _ in range(2)]
    state = []
    for i in range(2):
        z = torch.randn(M, V, generator=g, device=DEV) * 3
        size = qmv.logits_draw_ws_bytes(V, M)
        state.append((z, torch.tensor([0, 50] * 4, dtype=torch.int32, device=DEV), torch.full((M,), 0.9, device=DEV),
                      torch.rand(M, generator=g, device=DEV), torch.empty(size, dtype=torch.uint8, device=DEV), size,
                      torch.empty(M, dtype=torch.int32, device=DEV), torch.empty(M, dtype=torch.int32, device=DEV)))
    want = []
    for s in state:
        _call(*s)
        torch.cuda.synchronize()
        want.append((s[6].clone(), s[7].clone()))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, stream in zip(state, streams):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                _call(*s)
    torch.cuda.synchronize()
    for s, w in zip(state, want):
        assert torch.equal(s[6], w[0]) and torch.equal(s[7], w[1])


def test_graph():
    """Replayed with other logits and arguments, which decide on the device how the work is shared out."""
    qmv = _qmv()
    say("logits_draw in a graph")
    rng = np.random.default_rng(6)
    V, M = 50000, 5
    z = torch.empty(M, V, device=DEV)
    k, p, u = torch.zeros(M, dtype=torch.int32, device=DEV), torch.ones(M, device=DEV), torch.rand(M, device=DEV)
    size = qmv.logits_draw_ws_bytes(V, M)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    out = [torch.empty(M, dtype=torch.int32, device=DEV) for _ in range(4)]
    t = torch.full((M,), 0.9, device=DEV)
    z.normal_()

    def call(token, kept):
        qmv.logits_draw(z, V, t, k, p, None, u, token, kept, V, M, 0.0, ws, size)

    call(*out[:2])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(*out[:2])
    for i in range(12):
        z.copy_(torch.from_numpy(logits(rng, M, V)))
        t.copy_(torch.from_numpy(rng.choice([0.0, 0.5, 1.0], M).astype(np.float32)))
        k.copy_(torch.from_numpy(rng.choice([0, 30, 2000], M).astype(np.int32)))
        p.copy_(torch.from_numpy(rng.choice([1.0, 0.9], M).astype(np.float32)))
        u.copy_(torch.from_numpy(rng.random(M, dtype=np.float32)))
        g.replay()
        torch.cuda.synchronize()
        call(*out[2:])
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])


@pytest.mark.parametrize("V,M", [(32000, 20), (90000, 3), (262144, 1)])
@pytest.mark.parametrize("less", [-1, 0, 1, 40])
def test_a_range_is_allowed(V, M, less):
    """As many runs of 64 as top_k have logits at all, or a few more or fewer: most of the range is behind their border."""
    say(f"logits_draw a range of V={V}, runs less {less}")
    rng = np.random.default_rng(11)
    k = min(V // 256, 1000)
    z = np.full((M, V), NEG, np.float32)
    z[:, 640 : 640 + 64 * (k - less)] = rng.normal(0, 2, (M, 64 * (k - less)))
    check(z, 1.0, k, u=rng.random(M))
    check(z, 0.7, k, 0.9, 0.01, u=rng.random(M))


@pytest.mark.parametrize("M", [257, 512])
def test_many_long_rows(M):
    """As many as are shared out by workgroups, of all kinds."""
    rng = np.random.default_rng(M)
    say(f"logits_draw {M} long rows")
    z = logits(rng, M, 66000)
    z[rng.integers(0, M, 40)] = NEG
    check(z, rng.choice([0.0, 0.7, 1.0], M), rng.choice([0, 0, 1, 64, 900, 5000], M), rng.choice([1.0, 0.95, 0.5], M),
          rng.choice([0.0, 0.02], M), u=rng.random(M))


@pytest.mark.parametrize("V,M", [(50257, 16), (80001, 200)])
@pytest.mark.parametrize("masked", [0.0, 0.97])
def test_few_kept_of_long_parts(V, M, masked):
    """Filters on sums that end among few elements: only the runs that reach them are read again."""
    say(f"logits_draw few kept of V={V} M={M} masked={masked}")
    rng = np.random.default_rng(V)
    z = rng.normal(0, 2, (M, V)).astype(np.float32)
    z[np.arange(M)[:, None], rng.integers(0, V, (M, 40))] = rng.uniform(14, 26, (M, 40))
    z[rng.random((M, V)) < masked] = NEG
    z[:, V - 1] = rng.uniform(20, 27, M)
    z[:, 100:200] = NAN
    check(z, rng.choice([0.7, 1.0], M), rng.choice([0, 0, 5000, V // 200], M), rng.choice([0.9, 0.5, 0.999], M),
          rng.choice([0.0, 0.02], M), u=rng.random(M))
    check(z, 1.0, 0, 0.95, u=rng.random(M), offset=1, ld=V + 2)
    check(z, 1.0, u=rng.random(M))


@pytest.mark.parametrize("V", [65536, 262200])
def test_the_same_in_any_batch(V):
    """One workgroup a row for 513 rows, several for 100: sums are exact, so tokens and counts are the same."""
    qmv = _qmv()
    say(f"logits_draw V={V}, 513 rows and 100 at a time")
    M = 513
    g = torch.Generator(device=DEV).manual_seed(V)
    z = torch.randn(M, V, generator=g, device=DEV) * 3
    u = torch.rand(M, generator=g, device=DEV)

    def pick(values, dtype):
        i = torch.randint(0, len(values), (M,), generator=g, device=DEV)
        return torch.tensor(values, dtype=dtype, device=DEV)[i]

    t, p = pick([0.0, 0.5, 1.0, 1.0], torch.float32), pick([1.0, 0.9, 0.3], torch.float32)
    k, low = pick([0, 0, 1, 50, 900, 5000], torch.int32), pick([0.0, 0.05], torch.float32)

    def draw(rows):
        a = [x[rows].contiguous() for x in (z, t, k, p, low, u)]
        n = a[0].shape[0]
        token, kept = (torch.full((n,), -7, dtype=torch.int32, device=DEV) for _ in range(2))
        size = qmv.logits_draw_ws_bytes(V, n)
        qmv.logits_draw(a[0], V, *a[1:], token, kept, V, n, 0.0, torch.empty(size, dtype=torch.uint8, device=DEV), size)
        return torch.stack([token, kept])

    whole = draw(slice(0, M))
    parts = torch.cat([draw(slice(i, min(i + 100, M))) for i in range(0, M, 100)], 1)
    torch.cuda.synchronize()
    assert torch.equal(whole, parts)
