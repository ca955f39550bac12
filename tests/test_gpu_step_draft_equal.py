"""draft_verify where the drafter's row is the target's own: max(p - q, 0) is
all zero there, and the token after a rejected draft is drawn from p itself."""
import numpy as np
import pytest

import step_ref as R
from gpu_util import say
from test_gpu_step_draft import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,G,V,T,cap", [(64, 1, 3000, 1.0, 0.0), (64, 1, 3000, 0.7, 30.0), (7, 3, 50257, 1.0, 0.0),
                                         (200, 2, 40000, 1.3, 20.0), (1, 4, 262144, 0.8, 30.0)])
@pytest.mark.parametrize("how", ["outside the vocabulary", "without weight"])
def test_a_draft_rejected_where_both_rows_are_equal(B, G, V, T, cap, how):
    say(f"equal rows, draft {how}: B {B} G {G} V {V} T {T} cap {cap}")
    rng = np.random.default_rng(B + V)
    target = rng.normal(0, 2.0, (B, G + 1, V)).astype(np.float32)
    target[:, :, 11] = -np.inf
    draft = target[:, :G].copy()
    tokens = rng.integers(20, V, (B, G)).astype(np.int32)
    at = np.arange(B) % G  # the drafts before it are accepted: p = q
    tokens[np.arange(B), at] = 11 if how == "without weight" else np.where(np.arange(B) % 2, -1, V)
    u = rng.random((B, G + 1), dtype=np.float32)
    acc, out, _ = R.draft_verify(target, draft, tokens, None, u, T, cap)
    assert np.array_equal(acc, at) and (out[np.arange(B), at] >= 0).all()
    # the margin of the draw from p alone: as the bonus row of a batch without drafts
    sure = np.array([R.draft_verify(target[b:b + 1, at[b]:at[b] + 1].repeat(2, 1), draft[b:b + 1, at[b]:at[b] + 1],
                                    np.zeros((1, 1), np.int32), np.zeros(1, np.int32), u[b:b + 1, [0, G]], T, cap)[2][0]
                     for b in range(B)])
    assert sure.min() > 1e-12  # the draws from p themselves lie off their borders
    got = _run(target, draft, tokens, None, u, T, cap)
    assert np.array_equal(got[0], acc) and np.array_equal(got[1], out)


@pytest.mark.parametrize("B,G,V", [(300, 1, 2), (200, 3, 37), (100, 2, 5000), (8, 1, 60000)])
@pytest.mark.parametrize("T", [0.89, 1.0, 0.3])
def test_rows_that_differ_by_a_constant_are_equal(B, G, V, T):
    """p and q of logits that differ by a constant are the same: a draft rejected there (it is outside the vocabulary)
    is followed by the token that u draws from p, as from a bonus row.  The logits are whole numbers and a constant of
    up to 1000 leaves them so: their differences are exact."""
    say(f"rows apart by a constant: B {B} G {G} V {V} T {T}")
    rng = np.random.default_rng(V)
    target = np.round(rng.normal(0, 3.0, (B, G + 1, V))).astype(np.float32)
    draft = target[:, :G] + rng.integers(-1000, 1001, (B, G, 1)).astype(np.float32)
    tokens = np.full((B, G), V, np.int32)
    u = rng.random((B, G + 1), dtype=np.float32)
    # the same draw as that of a sequence without drafts, in the plain form and in the kernel
    acc, out, margin = R.draft_verify(target, draft, tokens, np.zeros(B, np.int32), u, T, 0.0)
    assert (acc == 0).all() and margin.min() > 1e-12
    for n in (None, np.zeros(B, np.int32)):
        got = _run(target, draft, tokens, n, u, T, 0.0)
        assert np.array_equal(got[0], acc) and np.array_equal(got[1], out)
