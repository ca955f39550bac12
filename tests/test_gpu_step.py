"""The operators together, as a serving loop uses them: norm, projections,
cache, attention, products of codes, logits and verification of drafts, step
after step, eager and captured; every step against the plain forms."""
import math

import numpy as np
import pytest
import torch

import oracle
import step_ref as R
from gpu_util import DEV, assert_within, dev, empty, host, say
from quantized_dequant_matrix_amd import synth

pytestmark = pytest.mark.gpu

E, HQ, HK, D, PAGE, V, B, G = 512, 8, 4, 64, 16, 2000, 3, 2  # a small model's width, heads, vocabulary


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


class Step:
    """Buffers and one step of a loop over B sequences, G + 1 rows each (drafts and their base)."""

    def __init__(self, fmt):
        qmv = _qmv()
        rng = np.random.default_rng(0)
        self.n, self.M = G + 1, B * (G + 1)
        M = self.M
        self.Wq, self.Wk, self.Wv, self.Wo = (synth.q4_0_weights(n, k, s) for n, k, s in
                                              ((HQ * D, E, 1), (HK * D, E, 2), (HK * D, E, 3), (E, HQ * D, 4)))
        self.Wl = synth.problem("q8_0", V, E, 1, 5)[0]
        self.w1, self.w2 = (rng.normal(1, 0.1, E).astype(np.float32) for _ in range(2))
        self.dW = [dev(a) for a in (self.Wq, self.Wk, self.Wv, self.Wo, self.Wl)]
        self.dw = [dev(self.w1), dev(self.w2)]
        pages = 6 * B
        dt = torch.int8 if fmt == "q8" else torch.float16
        shape = (pages, HK, PAGE, D)
        scales = [torch.zeros(shape[:3], device=DEV) for _ in range(2)] if fmt == "q8" else [None, None]
        self.cache = qmv.KVCache(torch.zeros(shape, dtype=dt, device=DEV), torch.zeros(shape, dtype=dt, device=DEV), *scales)
        self.table = _ints(rng.permutation(pages).reshape(B, 6))
        self.start, self.len = _ints(np.arange(B + 1) * self.n), _ints([0] * B)
        self.batch = qmv.KVBatch(self.table, self.start, self.len, M)
        self.x, self.r = empty((M, E)), empty((M, E))
        self.z, self.z2 = empty((M, E)), empty((M, E))
        self.codes, self.scales = empty((M, E), dtype=torch.int8), empty((M, E // 32))
        self.q, self.k, self.v = empty((M, HQ * D)), empty((M, HK * D)), empty((M, HK * D))
        self.o, self.a, self.h, self.y = empty((M, HQ * D)), empty((M, E)), empty((M, E)), empty((M, V))
        self.draft = empty((B * G, V))
        self.tokens, self.u = _ints(np.zeros((B, G))), empty((B, G + 1))
        self.accepted, self.out = empty(B, dtype=torch.int32), empty((B, G + 1), dtype=torch.int32)
        self.ws = {}
        for name, size in (("attn", qmv.attn_paged_ws_bytes(self.cache, self.batch, HQ)),
                           ("q", qmv.qmm_q4_0_q8_ws_bytes(HQ * D, E, M)), ("k", qmv.qmm_q4_0_q8_ws_bytes(HK * D, E, M)),
                           ("o", qmv.qmm_q4_0_f32act_ws_bytes(E, HQ * D, M)), ("d", qmv.draft_verify_ws_bytes(B, G, V))):
            self.ws[name] = (torch.empty(size, dtype=torch.uint8, device=DEV), size)

    def enqueue(self):
        qmv, M = _qmv(), self.M
        qmv.rmsnorm_add_q8(self.x, self.r, self.dw[0], self.z, self.codes, self.scales, E, M, 1e-6)
        qmv.qmm_q4_0_q8(self.dW[0], self.codes, self.scales, self.q, HQ * D, E, M, *self.ws["q"])
        for W, y in ((self.dW[1], self.k), (self.dW[2], self.v)):
            qmv.qmm_q4_0_q8(W, self.codes, self.scales, y, HK * D, E, M, *self.ws["k"])
        qmv.kv_write(self.cache, self.batch, self.k, HK * D, self.v, HK * D)
        qmv.attn_paged(self.cache, self.batch, self.q, HQ * D, self.o, HQ * D, HQ, 1 / math.sqrt(D), 0, *self.ws["attn"])
        qmv.qmm_q4_0_f32act(self.dW[3], self.o, self.a, E, HQ * D, M, *self.ws["o"])
        qmv.rmsnorm_add(self.a, self.z, self.dw[1], self.z2, self.h, E, M, 1e-6)
        qmv.qmv_q8_0(self.dW[4], self.h, self.y, V, E, M)
        qmv.draft_verify(self.y, V, self.draft, V, self.tokens, None, self.u, self.accepted, self.out, B, G, V, 1.0, 30.0,
                         *self.ws["d"])

    def outputs(self):
        return [host(t).copy() for t in (self.z, self.codes, self.scales, self.q, self.k, self.v, self.o, self.a, self.z2,
                                         self.h, self.y, self.accepted, self.out, *self.cache.tensors)]


def _inputs(s, step):
    rng = np.random.default_rng(100 + step)
    s.x.copy_(dev(rng.normal(0, 1, (s.M, E)).astype(np.float32)))
    s.r.copy_(dev(rng.normal(0, 1, (s.M, E)).astype(np.float32)))
    s.draft.copy_(dev(rng.normal(0, 1, (B * G, V)).astype(np.float32)))
    s.tokens.copy_(_ints(rng.integers(0, V, (B, G))))
    s.u.copy_(dev(rng.random((B, G + 1), dtype=np.float32)))
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_steps(fmt):
    """Each stage is checked on the inputs that the stage before really gave it."""
    s = Step(fmt)
    lens = np.zeros(B, int)
    kept = [[np.zeros((0, HK, D)), np.zeros((0, HK, D))] for _ in range(B)]
    for step in range(6):
        say(f"step {step} {fmt}")
        lens += s.n
        s.len.copy_(_ints(lens))
        _inputs(s, step)
        s.enqueue()
        z, codes, scales, q, k, v, o, a, z2, h, y, acc, out = s.outputs()[:13]
        zr, x1 = R.norm(host(s.x), host(s.r), s.w1, 1e-6)
        qr, dr = R.quantize_rows(x1.reshape(s.M, -1, 32))
        assert np.array_equal(z, zr) and np.array_equal(codes, qr.reshape(s.M, E)) and np.array_equal(scales, dr)
        for W, got, n in ((s.Wq, q, HQ * D), (s.Wk, k, HK * D), (s.Wv, v, HK * D)):
            ref, S = oracle.qmm_q4_0_q8(W, n, E, codes, scales, s.M)
            assert_within(got, ref, oracle.float_tol(S), "projection")
        for b in range(B):
            rows = slice(b * s.n, (b + 1) * s.n)
            for i, x in enumerate((k, v)):
                x = x[rows].reshape(s.n, HK, D)
                if fmt == "q8":
                    c, d = R.quantize_rows(x)
                    x = c.astype(np.float64) * d[..., None].astype(np.float64)
                else:
                    x = x.astype(np.float16).astype(np.float64)
                kept[b][i] = np.concatenate([kept[b][i], x])
            ref, tol = R.attention(q[rows].astype(np.float64).reshape(s.n, HQ, D), *kept[b],
                                   [lens[b] - s.n + i for i in range(s.n)], 1 / math.sqrt(D), 0)
            assert_within(o[rows].reshape(ref.shape), ref, tol, "attention")
        z2r, hr = R.norm(a, z, s.w2, 1e-6)
        assert np.array_equal(z2, z2r) and np.array_equal(h, hr)
        ar, tr, margin = R.draft_verify(y.reshape(B, G + 1, V), host(s.draft).reshape(B, G, V), host(s.tokens), None,
                                        host(s.u), 1.0, 30.0)
        assert margin.min() > 1e-12
        assert np.array_equal(acc, ar) and np.array_equal(out, tr)
        # rejected drafts are dropped: their positions are written again in the next step
        for b in range(B):
            drop = G - int(acc[b])
            lens[b] -= drop
            kept[b] = [x[: lens[b]] for x in kept[b]]


@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_captured_steps(fmt):
    """The whole step in a graph, replayed with eager work between, against an eager twin."""
    s, e = Step(fmt), Step(fmt)
    _inputs(s, 0)
    s.len.copy_(_ints([s.n] * B))
    s.enqueue()  # the first launch of every kernel outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.enqueue()
    for t in s.cache.tensors:
        t.zero_()
    lens = np.zeros(B, int)
    for step in range(5):
        lens += np.array([s.n, s.n - 1, s.n])
        for c in (s, e):
            c.len.copy_(_ints(lens))
            _inputs(c, step)
        g.replay()
        torch.cuda.synchronize()
        e.enqueue()
        for x, y in zip(s.outputs(), e.outputs()):
            assert np.array_equal(x.view(np.uint8), y.view(np.uint8))
