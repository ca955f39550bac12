"""A decode loop that never leaves the GPU: plan, embedding of the token just
drawn, norm, projections with adapters, cache, attention, logits, draw; step
after step, eager and captured.  Each stage is checked on what the stage
before really gave it."""
import math

import numpy as np
import pytest
import torch

import oracle
import serve_ref as R
import step_ref
from gpu_util import DEV, assert_within, dev, empty, host, say
from quantized_dequant_matrix_amd import synth

pytestmark = pytest.mark.gpu

E, HQ, HK, D, PAGE, V, B, WIDTH, RANK = 512, 8, 4, 64, 16, 2000, 4, 5, 16  # a small model
MAX_ROWS = 60


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


class Loop:
    """Buffers and one step over B sequences; `rows` of the row buffers (the last one row a sequence is drawn from)."""

    def __init__(self, rows):
        qmv = _qmv()
        rng = np.random.default_rng(0)
        self.T = rows
        self.Wq, self.Wk, self.Wv, self.Wo = (synth.q4_0_weights(n, k, s) for n, k, s in
                                              ((HQ * D, E, 1), (HK * D, E, 2), (HK * D, E, 3), (E, HQ * D, 4)))
        self.We = synth.problem("q8_0", V, E, 1, 5)[0]  # tied: embedding and logits
        self.w1, self.w2 = (rng.normal(1, 0.1, E).astype(np.float32) for _ in range(2))
        self.dW = [dev(a) for a in (self.Wq, self.Wk, self.Wv, self.Wo, self.We)]
        self.dw = [dev(self.w1), dev(self.w2)]
        f = lambda a: torch.from_numpy(a.astype(np.float32)).bfloat16()  # noqa: E731
        self.A, self.Bm = f(rng.normal(0, E ** -0.5, (3, RANK, E))), f(rng.normal(0, 0.3, (3, HQ * D, RANK)))
        self.rank, self.scale = np.array([16, 5, 9], np.int32), rng.random(3).astype(np.float32) + 0.5
        self.lora = qmv.Lora(self.A.to(DEV), self.Bm.to(DEV), dev(self.scale), ints(self.rank))
        self.adapter = ints([1, -1, 0, 2])
        pages = 14
        shape = (pages, HK, PAGE, D)
        self.cache = qmv.KVCache(*(torch.zeros(shape, dtype=torch.int8, device=DEV) for _ in range(2)),
                                 *(torch.zeros(shape[:3], device=DEV) for _ in range(2)))
        self.table, self.stack = ints(np.full((B, WIDTH), -1)), ints(rng.permutation(pages))
        self.len, self.keep, self.n = ints([0] * B), ints([0] * B), ints([0] * B)
        self.count, self.status, self.start = ints([pages]), ints([0, 0]), ints([0] * (B + 1))
        self.position, self.slot = ints([-1] * rows), torch.full((rows,), -1, dtype=torch.int64, device=DEV)
        self.pool = qmv.KVPool(self.table, self.stack, PAGE)
        self.batch = qmv.KVBatch(self.table, self.start, self.len, rows)
        self.tokens = ints([0] * rows)
        self.x, self.z, self.z2, self.a, self.h = (empty((rows, E)) for _ in range(5))
        self.codes, self.scales = empty((rows, E), dtype=torch.int8), empty((rows, E // 32))
        self.q0, self.q, self.k, self.v = (empty((rows, w)) for w in (HQ * D, HQ * D, HK * D, HK * D))
        self.o, self.y = torch.zeros((rows, HQ * D), device=DEV), empty((rows, V))
        self.temperature, self.u = dev(np.array([1.0, 0.7, 0.0, 1.2], np.float32)), empty(B)
        self.top_k, self.top_p = ints([0, 50, 0, 20]), dev(np.array([0.9, 1.0, 1.0, 0.95], np.float32))
        self.min_p = dev(np.array([0.0, 0.05, 0.0, 0.02], np.float32))
        self.token, self.kept = empty(B, dtype=torch.int32), empty(B, dtype=torch.int32)
        self.ws = {}
        for name, size in (("plan", qmv.kv_plan_ws_bytes(self.pool)), ("lora", qmv.lora_add_ws_bytes(self.lora, B, rows)),
                           ("attn", qmv.attn_paged_ws_bytes(self.cache, self.batch, HQ)),
                           ("q", qmv.qmm_q4_0_q8_ws_bytes(HQ * D, E, rows)), ("k", qmv.qmm_q4_0_q8_ws_bytes(HK * D, E, rows)),
                           ("o", qmv.qmm_q4_0_f32act_ws_bytes(E, HQ * D, rows)), ("draw", qmv.logits_draw_ws_bytes(V, B))):
            self.ws[name] = (torch.empty(size, dtype=torch.uint8, device=DEV), size)

    def enqueue(self, last):
        """last: row of each sequence's last new token, on the GPU."""
        qmv, T = _qmv(), self.T
        qmv.kv_plan(self.pool, self.len, self.keep, self.n, self.count, self.len, self.count, self.start, self.position,
                    self.slot, self.status, T, *self.ws["plan"])
        qmv.embed_q8_0(self.dW[4], self.tokens, self.x, V, E, T, math.sqrt(E))
        qmv.rmsnorm_add_q8(self.x, None, self.dw[0], self.z, self.codes, self.scales, E, T, 1e-6)
        qmv.qmm_q4_0_q8(self.dW[0], self.codes, self.scales, self.q0, HQ * D, E, T, *self.ws["q"])
        qmv.lora_add(self.lora, self.adapter, self.start, self.z, E, self.q0, HQ * D, self.q, HQ * D, B, T, *self.ws["lora"])
        for W, y in ((self.dW[1], self.k), (self.dW[2], self.v)):
            qmv.qmm_q4_0_q8(W, self.codes, self.scales, y, HK * D, E, T, *self.ws["k"])
        qmv.kv_write(self.cache, self.batch, self.k, HK * D, self.v, HK * D)
        qmv.attn_paged(self.cache, self.batch, self.q, HQ * D, self.o, HQ * D, HQ, 1 / math.sqrt(D), 0, *self.ws["attn"])
        qmv.qmm_q4_0_f32act(self.dW[3], self.o, self.a, E, HQ * D, T, *self.ws["o"])
        qmv.rmsnorm_add(self.a, self.z, self.dw[1], self.z2, self.h, E, T, 1e-6)
        qmv.qmv_q8_0(self.dW[4], self.h[:B] if last is None else self.h[last], self.y, V, E, B)
        qmv.logits_draw(self.y, V, self.temperature, self.top_k, self.top_p, self.min_p, self.u, self.token, self.kept, V, B,
                        20.0, *self.ws["draw"])

    def outputs(self):
        return [host(t).copy() for t in (self.len, self.count, self.start, self.status, self.table, self.position, self.slot,
                                         self.x, self.z, self.q0, self.q, self.k, self.v, self.o, self.y, self.token, self.kept,
                                         *self.cache.tensors)]


def cached(s, lens):
    """Keys and values of each sequence as the tables say they lie, float64."""
    k, v, ks, vs = (host(t) for t in s.cache.tensors)
    table = host(s.table)
    out = []
    for b, n in enumerate(lens):
        at = [(table[b, p // PAGE], p % PAGE) for p in range(n)]
        pick = lambda c, d: np.array([c[g, :, i].astype(np.float64) * d[g, :, i, None] for g, i in at]).reshape(n, HK, D)  # noqa: E731
        out.append((pick(k, ks), pick(v, vs)))
    return out


def check_step(s, lens_before, keep, n, stack, table):
    lens = np.asarray(keep) + n
    want = R.plan(table, stack, len(stack), lens_before, keep, n, PAGE, s.T)
    assert host(s.status).tolist() == want["status"] == [0, 0]
    assert host(s.len).tolist() == lens.tolist() and host(s.start).tolist() == want["row_start"]
    assert host(s.table).tolist() == want["table"].tolist()
    start = want["row_start"]
    rows = start[-1]
    assert host(s.position)[:rows].tolist() == [want["position"][r] for r in range(rows)]
    x = host(s.x)
    assert np.array_equal(x, R.embed("q8_0", s.We.reshape(V, -1), host(s.tokens), math.sqrt(E)))
    z, _ = step_ref.norm(x, None, s.w1, 1e-6)
    q0, q, k, v, o, y = (host(t) for t in (s.q0, s.q, s.k, s.v, s.o, s.y))
    ref, tol = R.lora(s.A.double().numpy(), s.Bm.double().numpy(), s.scale, s.rank, host(s.adapter), start, z, q0)
    assert_within(q[:rows], ref[:rows], tol[:rows], "projection with adapters")
    held = cached(s, lens)
    kc, kd = step_ref.quantize_rows(k.reshape(s.T, HK, D))
    for b in range(B):
        mine = slice(start[b], start[b + 1])
        # the new rows lie where the plan says
        assert np.array_equal(held[b][0][lens[b] - n[b]:], kc[mine].astype(np.float64) * kd[mine][..., None])
        ref, tol = step_ref.attention(q[mine].astype(np.float64).reshape(-1, HQ, D), *held[b],
                                      list(range(lens[b] - n[b], lens[b])), 1 / math.sqrt(D), 0)
        assert_within(o[mine].reshape(ref.shape), ref, tol, "attention")
    a = [host(t) for t in (s.temperature, s.top_k, s.top_p, s.min_p, s.u)]
    token, kept = host(s.token), host(s.kept)
    for b in range(B):
        t, c, far = R.draw_row(y[b], *(r[b] for r in a), 20.0)
        assert not far or (token[b], kept[b]) == (t, c)


def test_a_prompt_and_decoding():
    """Prompts of odd lengths, then tokens one by one, each step fed by the last draw; one sequence ends and begins again."""
    rng = np.random.default_rng(1)
    s = Loop(MAX_ROWS)
    lens = np.zeros(B, int)
    for step in range(8):
        n = np.array([17, 1, 20, 9]) if step == 0 else np.ones(B, int)
        keep = lens.copy()
        if step == 4:
            keep[2], n[2] = 0, 20  # another request in its place
        if step == 6:
            keep[0] -= 2           # two tokens taken back
        say(f"serving step {step}")
        stack, table = host(s.stack)[:int(s.count)].copy(), host(s.table).copy()
        s.keep.copy_(ints(keep)), s.n.copy_(ints(n))
        start = np.concatenate([[0], np.cumsum(n)])
        tokens = rng.integers(0, V, s.T)
        if step:
            for b in range(B):
                if n[b] == 1:
                    tokens[start[b]] = int(s.token[b])
        s.tokens.copy_(ints(tokens))
        s.u.copy_(dev(rng.random(B, dtype=np.float32)))
        s.enqueue(ints(start[1:] - 1).long())
        torch.cuda.synchronize()
        check_step(s, lens, keep, n, stack, table)
        lens = keep + n


def test_captured_decoding():
    """One token a sequence in a graph, drawn tokens fed back inside it; replayed with eager work between, against an eager twin."""
    s, e = Loop(B), Loop(B)

    def step(c):
        c.enqueue(None)
        c.tokens.copy_(c.token)
        c.keep.copy_(c.len)

    def begin(c):
        c.len.zero_(), c.keep.zero_(), c.table.fill_(-1), c.count.fill_(14)
        c.n.fill_(1)
        c.stack.copy_(ints(np.random.default_rng(3).permutation(14)))
        c.tokens.copy_(ints([5, 6, 7, 8]))
        c.o.zero_()
        for t in c.cache.tensors:
            t.zero_()

    for c in (s, e):
        begin(c)
        c.u.fill_(0.5)
    step(s)  # the first launch of every kernel outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(s)
    begin(s)
    for i in range(60):
        u = dev(np.random.default_rng(i).random(B, dtype=np.float32))
        s.u.copy_(u), e.u.copy_(u)
        g.replay()
        torch.cuda.synchronize()
        step(e)
        torch.cuda.synchronize()
        for x, y in zip(s.outputs(), e.outputs()):
            assert np.array_equal(x.view(np.uint8), y.view(np.uint8))
    # 4 sequences share 14 pages: the graph went on to where they ran out and stopped there
    assert host(s.status).tolist() == [R.PAGES, 4 - 2] and host(s.len).tolist() == [48] * B
