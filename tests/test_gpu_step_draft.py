"""draft_verify against the plain form in 64 bits: the same counts and tokens
wherever no decision lies within 1e-12 of its border (none of the seeds used
does: asserted)."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import DEV, dev, empty, host, say

pytestmark = pytest.mark.gpu


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def _run(target, draft, tokens, n_draft, u, T, cap, ldt=None, ldd=None):
    qmv = _qmv()
    B, G1, V = target.shape
    G = G1 - 1

    def padded(a, ld):
        if ld is None:
            return dev(a), V
        out = np.full((a.shape[0], a.shape[1], ld), 1e9, np.float32)
        out[..., :V] = a
        return dev(out), ld

    t, ldt = padded(target, ldt)
    d, ldd = padded(draft, ldd)
    need = qmv.draft_verify_ws_bytes(B, G, V)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    acc, out = empty(B, dtype=torch.int32), empty((B, G + 1), dtype=torch.int32)
    qmv.draft_verify(t, ldt, d, ldd, dev(tokens), None if n_draft is None else dev(n_draft), dev(u), acc, out, B, G, V,
                     T, cap, ws, need)
    return host(acc), host(out)


def _problem(B, G, V, seed, noise=1.0, sharp=2.5):
    rng = np.random.default_rng(seed)
    target = rng.normal(0, sharp, (B, G + 1, V)).astype(np.float32)
    draft = (target[:, :G] + rng.normal(0, noise, (B, G, V))).astype(np.float32)
    tokens = (draft + rng.gumbel(size=draft.shape)).argmax(axis=2).astype(np.int32)
    u = rng.random((B, G + 1), dtype=np.float32)
    return target, draft, tokens, u


def _check(args, T=1.0, cap=0.0, n_draft=None, **kw):
    target, draft, tokens, u = args
    acc, out, margin = R.draft_verify(target, draft, tokens, n_draft, u, T, cap)
    assert margin.min() > 1e-12
    got = _run(target, draft, tokens, n_draft, u, T, cap, **kw)
    assert np.array_equal(got[0], acc) and np.array_equal(got[1], out)
    return acc


@pytest.mark.parametrize("B,G,V,T,cap", [(1, 4, 262144, 0.8, 30.0), (3, 1, 1, 1.0, 0.0), (2, 3, 7, 1.0, 30.0),
                                         (5, 2, 4096, 0.5, 0.0), (4, 5, 4097, 1.3, 20.0), (2, 8, 50257, 1.0, 0.0),
                                         (40, 3, 1000, 0.7, 30.0), (1, 64, 300, 1.0, 5.0), (300, 2, 65, 1.0, 0.0),
                                         # many sequences of many logits: four steps a workgroup of the second kernel
                                         (210, 1, 20001, 0.9, 0.0), (150, 2, 28676, 1.0, 30.0),
                                         # more groups than the draw's threads hold in registers
                                         (6, 1, 700001, 1.0, 0.0), (1, 2, 2000000, 1.5, 30.0)])
def test_plain(B, G, V, T, cap):
    say(f"draft_verify B {B} G {G} V {V} T {T} cap {cap}")
    _check(_problem(B, G, V, B + G + V), T, cap)


@pytest.mark.parametrize("cap", [0.01, 1000.0, 65536.0])
def test_small_and_large_caps(cap):
    """A level cap(y) / T is off by at most 2^-42 cap, so a weight by 2^-42 cap relative to the
    others and p - q by as much of p: decisions are asked for that lie 8 times that far from a border."""
    args = _problem(12, 3, 700, 31)
    acc, out, margin = R.draft_verify(*args[:3], None, args[3], 1.0, cap)
    assert margin.min() > max(1e-12, cap * 2.0 ** -39)
    got = _run(*args[:3], None, args[3], 1.0, cap)
    assert np.array_equal(got[0], acc) and np.array_equal(got[1], out)


def test_some_accept_all_and_some_none():
    acc = _check(_problem(200, 3, 500, 9, noise=0.7))
    assert set(acc.tolist()) == {0, 1, 2, 3}


def test_fewer_drafts_rows_apart_and_unaligned():
    args = _problem(6, 4, 1003, 3)
    n = np.array([0, 4, 2, 1, -3, 99], np.int32)  # clamped to [0, 4]
    _check(args, 0.9, 0.0, n_draft=n)
    _check(args, 0.9, 30.0, n_draft=n, ldt=1010, ldd=1025)


def test_draws_at_the_ends():
    """u = 0 draws the first index that weighs anything, u just below 1 the last that matters."""
    target, draft, tokens, u = _problem(2, 2, 9000, 4)
    target[:, :, :5] = -np.inf
    draft[:, :, :5] = -np.inf
    n = np.zeros(2, np.int32)
    u[0, 2], u[1, 2] = 0.0, 1.0 - 2.0 ** -24
    acc, out = _run(target, draft, tokens, n, u, 1.0, 0.0)
    ref = R.draft_verify(target, draft, tokens, n, u, 1.0, 0.0)
    assert np.array_equal(acc, [0, 0]) and out[0, 0] == 5 == ref[1][0, 0] and out[1, 0] == ref[1][1, 0]


def test_masked_and_broken_logits():
    """-infinity and NaN weigh nothing (with a cap too), +infinity takes all, a row without weight draws -1."""
    target, draft, tokens, u = _problem(6, 2, 5000, 5)
    target[0, :, ::2] = -np.inf
    target[1, :, 1::3] = np.nan
    target[2, 0, 77] = np.inf
    target[3] = -np.inf
    target[4, 0] = np.nan
    draft[5] = -np.inf  # the drafter gives no weight: q = 0
    for cap in (0.0, 30.0):
        acc, out, margin = R.draft_verify(target, draft, tokens, None, u, 1.0, cap)
        got = _run(target, draft, tokens, None, u, 1.0, cap)
        assert np.array_equal(got[0], acc) and np.array_equal(got[1], out)
        assert got[1][3].tolist() == [-1, -1, -1] and got[1][4].tolist() == [-1, -1, -1]
        assert got[0][5] == 2


def test_equal_distributions_accept_everything():
    """p = q: u q < p for every u < 1; and a residual without weight is never drawn from."""
    rng = np.random.default_rng(6)
    target = rng.normal(0, 1, (20, 4, 700)).astype(np.float32)
    draft = target[:, :3].copy()
    tokens = rng.integers(0, 700, (20, 3)).astype(np.int32)
    u = rng.random((20, 4), dtype=np.float32)
    assert (_check((target, draft, tokens, u)) == 3).all()


def test_tokens_outside_the_vocabulary_and_random_numbers_outside_their_range():
    target, draft, tokens, u = _problem(6, 3, 300, 7)
    tokens[0, 0], tokens[1, 1], tokens[2, 0] = -1, 300, 2 ** 31 - 1
    u[3] = np.nan
    u[4] = 2.0
    u[5] = -1.0
    acc, out = _run(target, draft, tokens, None, u, 1.0, 0.0)
    ref = R.draft_verify(target[:3], draft[:3], tokens[:3], None, u[:3], 1.0, 0.0)
    assert np.array_equal(acc[:3], ref[0]) and np.array_equal(out[:3], ref[1])
    # whatever the numbers are, a token of the vocabulary is drawn
    for b in range(3, 6):
        assert 0 <= out[b, acc[b]] < 300 and (out[b, acc[b] + 1:] == -1).all()


def test_extreme_temperatures():
    target, draft, tokens, u = _problem(4, 2, 2000, 8)
    _check((target, draft, tokens, u), T=1e3)
    got = _run(target, draft, tokens, None, u, 1e-30, 0.0)  # the largest logit takes all
    best = target.argmax(axis=2)
    for b in range(4):
        a = got[0][b]
        assert got[1][b, a] == best[b, a]


def test_tokens_are_distributed_as_the_targets():
    """One draft from q, then the rule: the emitted first token follows p.  8 tokens, 60,000 sequences
    with their own random numbers: every frequency within 5 standard deviations of p."""
    rng = np.random.default_rng(10)
    B, V = 60000, 8
    t1, d1 = rng.normal(0, 1, V).astype(np.float32), rng.normal(0, 1, V).astype(np.float32)
    target = np.broadcast_to(t1, (B, 2, V)).copy()
    draft = np.broadcast_to(d1, (B, 1, V)).copy()
    q = R.softmax64(d1, 1.0, 0.0)
    tokens = rng.choice(V, size=(B, 1), p=q).astype(np.int32)
    u = rng.random((B, 2), dtype=np.float32)
    acc, out = _run(target, draft, tokens, None, u, 1.0, 0.0)
    p = R.softmax64(t1, 1.0, 0.0)
    f = np.bincount(out[:, 0], minlength=V) / B
    assert (np.abs(f - p) < 5 * np.sqrt(p * (1 - p) / B)).all(), (f, p)
