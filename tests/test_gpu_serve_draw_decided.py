"""logits_draw among equal and far logits with filters and random numbers away
from the borders, so that every row has one right answer."""
import numpy as np
import pytest

from gpu_util import say
from test_gpu_serve_draw import INF, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [5000, 30000, 100000])
def test_equal_logits(V):
    """Whole logits: the first n are of one value, whose weights are 1, so that counts and tokens are whole numbers."""
    say(f"logits_draw V={V} equal logits, decided")
    rng = np.random.default_rng(V)
    M = 8
    z = (rng.integers(-6, 7, (M, V)) * np.where(rng.random((M, V)) < 0.5, 1, -1)).astype(np.float32)
    first = [np.flatnonzero(z[m] == 6) for m in range(M)]
    least = min(len(f) for f in first)
    assert least > 300
    for k in (1, 40, 250, least):
        for p in (1.0, 0.93, 0.5, 0.31):
            # an element inside the border: p k is between two whole numbers
            kept = k if p == 1.0 else int(np.floor(np.float64(np.float32(p)) * k)) + 1
            if p != 1.0 and abs(np.float64(np.float32(p)) * k - round(float(np.float32(p)) * k)) < 1e-3:
                p, kept = (kept - 0.5) / k, kept
            at = rng.integers(0, kept, M)
            u = (at + 0.5) / kept
            token, n, _ = run(z, 2.0, k, p, u=u)
            assert n.tolist() == [kept] * M, (k, p)
            assert token.tolist() == [int(first[m][at[m]]) for m in range(M)], (k, p)


@pytest.mark.parametrize("V", [3000, 45000])
@pytest.mark.parametrize("T", [1e20, INF])
def test_far_logits(V, T):
    """Weights of 1 all of them, over logits up to a million apart: the order alone decides."""
    say(f"logits_draw V={V} far logits at {T}")
    rng = np.random.default_rng(3)
    M = 6
    z = rng.normal(0, 0.1, (M, V)).astype(np.float32)
    z[:, rng.permutation(V)[:900]] = -(10.0 ** rng.uniform(1, 5.9, (M, 900)))
    order = [np.lexsort((np.arange(V), -z[m])) for m in range(M)]
    for k in (0, 7, 900, 2000, 2048, V - 450, V - 100):
        n = k or V
        for at in (0, n // 3, n - 300 if n > 300 else n // 2, n - 1):
            token, kept, _ = run(z, T, k, 1.0, u=np.float32((at + 0.5) / n))
            assert kept.tolist() == [n] * M, (k, at)
            assert token.tolist() == [int(order[m][at]) for m in range(M)], (k, at)
