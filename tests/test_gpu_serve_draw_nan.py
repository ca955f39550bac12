"""logits_draw where NaN, of any kind, stands beside the largest logits: it is
never drawn and moves nothing."""
import numpy as np
import pytest

from gpu_util import say
from test_gpu_serve_draw import check, logits, run

pytestmark = pytest.mark.gpu

MOST = np.finfo(np.float32).max
# quiet and signalling, either sign, smallest and largest payloads
KINDS = (0x7fc00000, 0xffc00000, 0x7f800001, 0xff800001, 0x7fbfffff, 0x7fffffff, 0xffffffff)


def put(z, at, bits):
    z.view(np.uint32)[at] = bits


@pytest.mark.parametrize("V", [8, 1003, 70001])
@pytest.mark.parametrize("top", [np.inf, MOST, 12.0])
def test_nan_beside_the_largest(V, top):
    """The largest logit at each place of its group of four, NaN at the other three or before it."""
    rng = np.random.default_rng(V)
    M = 4 * len(KINDS)
    for base in sorted({0, V // 2 // 4 * 4}):
        z = logits(rng, M, V, peaks=False)
        for m in range(M):
            at, kind = m % 4, KINDS[m // 4]
            for e in range(4):
                if e != at:
                    put(z, (m, base + e), kind)
            z[m, base + at] = top
        want = [base + m % 4 for m in range(M)]
        say(f"logits_draw V={V} top={top} at {base}")
        for T in (0.0, 1.0, 1e-3):
            for k in (0, 1, 20):
                token, kept, _ = run(z, T, k, u=0.0)
                assert token.tolist() == want, (T, k)
                assert k != 1 and T != 0.0 or kept.tolist() == [1] * M
        check(z, 1.0, 30, 0.9, u=rng.random(M))


def test_nan_before_equal_largest():
    """Of equal largest logits the first one, with NaN before each of them."""
    for V in (64, 5000, 50000):
        for top in (np.inf, MOST, 0.0):
            z = np.full((3, V), -1.0, np.float32)
            for m, at in enumerate((1, 18, 39)):
                for p in (at, at + 1, at + 20):
                    z[m, p] = top
                    put(z, (m, p - 1), KINDS[m]) if p != at + 1 else None
            say(f"logits_draw V={V} equal {top}")
            token, kept, _ = run(z, 0.0)
            assert token.tolist() == [1, 18, 39] and kept.tolist() == [1, 1, 1]


def test_rows_of_nan_kinds():
    say("logits_draw rows of NaN")
    for V in (7, 3000, 45000):
        z = np.empty((len(KINDS), V), np.float32)
        for m, k in enumerate(KINDS):
            put(z, (m, slice(None)), k)
        for T in (0.0, 1.0):
            token, kept, _ = run(z, T, 5, 0.9)
            assert token.tolist() == [-1] * len(KINDS) and kept.tolist() == [0] * len(KINDS)
        z[:, V - 2] = -3.0
        for T in (0.0, 1.0):
            token, kept, _ = run(z, T, 5, 0.9)
            assert token.tolist() == [V - 2] * len(KINDS) and kept.tolist() == [1] * len(KINDS)
