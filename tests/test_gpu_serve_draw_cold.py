"""logits_draw at small temperatures, where most of a row weighs nothing: the
first top_k are the same elements, and take about as long to find, as at any
other temperature."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from test_gpu_serve_draw import LOW, NEG, check, logits, run

pytestmark = pytest.mark.gpu


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


TOP_P, MIN_P = (1.0, 0.9, 1.0, 0.99), (0.0, 0.0, 1e-45, 0.01)


@pytest.mark.parametrize("V,M", [(32000, 4), (32000, 20), (50257, 4), (262144, 4)])
@pytest.mark.parametrize("k", [1, 50, 1000, 2048, 5000])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_small_temperatures(V, M, k, softcap):
    rng = np.random.default_rng(V + k)
    say(f"logits_draw V={V} M={M} top_k={k} softcap={softcap} cold")
    for T in (0.02, 1e-3, 1e-6, 1e-40):
        # a cap's level is known to 2^-42, which the smallest temperatures make much of
        least = 0.6 if softcap == 0.0 or T > 1e-5 else 0.0
        _, kept = check(logits(rng, M, V), T, k, np.resize(TOP_P, M), np.resize(MIN_P, M), u=rng.random(M), softcap=softcap,
                        least=least)
        assert (kept[::4] == k).all()


@pytest.mark.parametrize("V,M", [(30000, 4), (60000, 4)])
def test_equal_largest_logits(V, M):
    """The weights that are left are 1 each: tokens and counts are known exactly."""
    rng = np.random.default_rng(V)
    say(f"logits_draw V={V} equal largest, cold")
    for n in (1, 7, 300, 4000):
        z = np.minimum(logits(rng, M, V), 9.0).astype(np.float32)
        where = [np.sort(rng.permutation(V)[:n]) for _ in range(M)]
        for m in range(M):
            z[m, where[m]] = 10.0
        for T in (1e-3, 1e-6, 1e-30):
            for k in (1, 50, 1000, 2048, 5000):
                u = (np.arange(M) + 0.5) / M
                live = min(n, k)
                token, kept, _ = run(z, T, k, u=u)
                assert kept.tolist() == [k] * M  # what weighs nothing is kept too
                assert token.tolist() == [where[m][int(u[m] * live)] for m in range(M)], (n, T, k)
                token, kept, _ = run(z, T, k, 1.0, 0.5, u=u)
                assert kept.tolist() == [live] * M
                assert token.tolist() == [where[m][int(u[m] * live)] for m in range(M)], (n, T, k)


@pytest.mark.parametrize("V", [30000, 100000])
@pytest.mark.parametrize("fill", [LOW, -1e30, -1e9, NEG])
def test_little_is_allowed(V, fill):
    """Fewer allowed logits than top_k, the others at the type's lowest value or far down."""
    M = 6
    rng = np.random.default_rng(3)
    say(f"logits_draw V={V} masked by {fill}")
    z = np.full((M, V), fill, np.float32)
    for m, n in enumerate((1, 3, 20, 49, 50, 700)):
        z[m, rng.permutation(V)[:n]] = rng.normal(0, 2, n)
    for T in (1.0, 0.5, 1e-3):
        for k in (5, 50, 1000, 5000):
            at = rng.integers(0, 4, M)
            check(z, T, k, np.take(TOP_P, at), np.take(MIN_P, at), u=rng.random(M))


def _time(z, T, k):
    """Microseconds of a call, the smallest of several."""
    qmv = _qmv()
    M, V = z.shape
    t, kk = torch.full((M,), T, device=DEV), torch.full((M,), k, dtype=torch.int32, device=DEV)
    u = torch.full((M,), 0.5, device=DEV)
    token = torch.empty(M, dtype=torch.int32, device=DEV)
    size = qmv.logits_draw_ws_bytes(V, M)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    times = []
    for _ in range(8):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        for _ in range(4):
            qmv.logits_draw(z, V, t, kk, None, None, u, token, None, V, M, 0.0, ws, size)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 250)
    return min(times)


@pytest.mark.parametrize("V,M", [(32000, 16), (262144, 1), (262144, 8)])
@pytest.mark.parametrize("k", [40, 1000, 5000])
def test_no_slower_than_at_one(V, M, k):
    """Five times is far beyond what the two differ by where neither goes digit by digit (which is 10 to 30 times)."""
    z = torch.from_numpy(logits(np.random.default_rng(1), M, V)).to(DEV)
    warm = _time(z, 1.0, k)
    for T in (0.01, 2e-3, 1e-3, 1e-6):
        cold = _time(z, T, k)
        say(f"logits_draw {M} x {V} top_k={k}: {cold:.1f} us at {T}, {warm:.1f} at 1")
        assert cold < 5 * warm
