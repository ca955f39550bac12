"""The decode-step entry points write only their outputs and the workspace they
asked for, and leave their inputs bit-identical: sentinels before and behind
every buffer, on every way that a call can take (the plan of attn_paged, the
layouts of qmm_q4_0_q8, the two second kernels of draft_verify), and also where
row starts are out of order, lengths lie and pages do not exist."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import DEV, dev, say
from quantized_dequant_matrix_amd import synth

pytestmark = pytest.mark.gpu

GUARD = 4096        # bytes before and behind
SENT = 0x7FBADBAD   # a NaN pattern no kernel produces


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


class Buffers:
    """Guarded device buffers: `out` may change, `keep` may not, and nothing may around either."""

    def __init__(self):
        self.all = []

    def _make(self, nbytes):
        words = -(-nbytes // 4) + 2 * GUARD // 4
        full = torch.full((words,), SENT, dtype=torch.int32, device=DEV)
        return full, full.view(torch.uint8)[GUARD:GUARD + nbytes]

    def out(self, shape, dtype=torch.float32):
        shape = (shape,) if isinstance(shape, int) else tuple(shape)
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        full, view = self._make(n)
        self.all.append((full, n, None))
        return view.view(dtype).view(shape)

    def keep(self, a):
        t = torch.from_numpy(np.ascontiguousarray(a))
        n = t.numel() * t.element_size()
        full, view = self._make(n)
        view.copy_(t.view(-1).view(torch.uint8))
        self.all.append((full, n, view.clone()))
        return view.view(t.dtype).view(t.shape)

    def check(self, what):
        torch.cuda.synchronize()
        sent = np.frombuffer(np.int32(SENT).tobytes(), np.uint8)
        for i, (full, n, before) in enumerate(self.all):
            b = full.view(torch.uint8)
            head, tail = b[:GUARD].cpu().numpy(), b[GUARD + n:].cpu().numpy()
            assert (head.reshape(-1, 4) == sent).all(), f"{what}: bytes before buffer {i}"
            want = np.tile(sent, GUARD // 4 + 1)[n % 4:][:len(tail)]
            assert (tail == want).all(), f"{what}: bytes behind buffer {i}"
            if before is not None:
                assert torch.equal(before, b[GUARD:GUARD + n]), f"{what}: input {i} changed"


def _cache(B, P, writable=False):
    f = (lambda a: None if a is None else B.keep(a))
    if writable:
        f = (lambda a: None if a is None else B.out(a.shape, torch.from_numpy(a).dtype))
    return _qmv().KVCache(*(f(a) for a in (P.k, P.v, P.ks, P.vs)))


def _batch(B, P, start, lens, T):
    as_int = lambda a: B.keep(np.asarray(a, dtype=np.int32))
    return _qmv().KVBatch(as_int(P.table), as_int(start), as_int(lens), T)


DISORDER = [[0, 9, 3], [-5, -2, 100], [5, 1, 0], [0, 0, 0], [0, 2 ** 31 - 1, -2 ** 31], [3, 3, 5]]
LENGTHS = [[-3, 2 ** 31 - 1], [20, 0], [0, 20], [5000, 5000]]


def _lies(good_start, good_lens):
    yield good_start, good_lens
    for start in DISORDER:
        for lens in LENGTHS:
            yield start, lens
    for lens in LENGTHS:
        yield good_start, lens


@pytest.mark.parametrize("fmt,heads,dim", [("q8", 3, 64), ("q8", 16, 128), ("f16", 5, 256), ("f16", 2, 64)])
@pytest.mark.parametrize("page", [16, 64])
def test_cache_calls(fmt, heads, dim, page):
    qmv = _qmv()
    say(f"guards kv {fmt} {heads} x {dim}, page {page}")
    rng = np.random.default_rng(1)
    lens, new = [37, 20], [4, 1]
    P = R.Pages(lens, heads, dim, page, fmt, rng, max_pages=5)
    width, T = heads * dim, 5
    x = rng.normal(0, 1, (T, width)).astype(np.float32)
    for start, length in _lies([0, 4, 5], lens):
        B = Buffers()
        cache, batch = _cache(B, P, writable=True), _batch(B, P, start, length, T)
        k, v = B.keep(x), B.keep(2 * x)
        qmv.kv_write(cache, batch, k, width, v, width)
        B.check(f"kv_write {start} {length}")
        B = Buffers()
        cache, batch = _cache(B, P), _batch(B, P, start, length, T)
        k, v = B.out((T, width)), B.out((T, width))
        qmv.kv_read(cache, batch, k, width, v, width)
        B.check(f"kv_read {start} {length}")


@pytest.mark.parametrize("T,heads,dim", [(1030, 3, 64), (1100, 16, 128)])
@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_cache_calls_of_several_rows_a_workgroup(fmt, T, heads, dim):
    qmv = _qmv()
    say(f"guards kv {fmt}, {T} rows of {heads} x {dim}")
    rng = np.random.default_rng(2)
    P = R.Pages([T + 3], heads, dim, 64, fmt, rng)
    width = heads * dim
    for start, length in (([0, T], [T + 3]), ([0, T - 5], [T + 3]), ([7, T], [T + 3]), ([0, T], [9]), ([T, 0], [T])):
        B = Buffers()
        cache, batch = _cache(B, P, writable=True), _batch(B, P, start, length, T)
        qmv.kv_write(cache, batch, B.keep(rng.normal(0, 1, (T, width)).astype(np.float32)), width,
                     B.keep(rng.normal(0, 1, (T, width)).astype(np.float32)), width)
        B.check(f"kv_write {start} {length}")
        B = Buffers()
        cache, batch = _cache(B, P), _batch(B, P, start, length, T)
        qmv.kv_read(cache, batch, B.out((T, width)), width, B.out((T, width)), width)
        B.check(f"kv_read {start} {length}")


# (T, new, lens, query heads, heads, head size, table positions): an item a workgroup of four and of
# eight waves, runs with a second kernel, two row tiles a workgroup
WAYS = {"whole": (5, [4, 1], [37, 20], 4, 2, 80), "eight": (5, [4, 1], [37, 20], 4, 2, 640),
        "pieces": (5, [4, 1], [37, 20], 4, 2, 10000)}


@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("fmt", ["q8", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("way", list(WAYS))
def test_attention(way, dim, fmt, window):
    qmv = _qmv()
    T, new, lens, Hq, heads, positions = WAYS[way]
    say(f"guards attn {way} {fmt} D {dim} window {window}")
    rng = np.random.default_rng(3)
    P = R.Pages(lens, heads, dim, 16, fmt, rng, max_pages=positions // 16)
    width = Hq * dim
    q = rng.normal(0, 1, (T, width)).astype(np.float32)
    for start, length in _lies([0, 4, 5], lens):
        B = Buffers()
        cache, batch = _cache(B, P), _batch(B, P, start, length, T)
        tq, out = B.keep(q), B.out((T, width))
        need = qmv.attn_paged_ws_bytes(cache, batch, Hq)
        ws = B.out(need, torch.uint8)
        qmv.attn_paged(cache, batch, tq, width, out, width, Hq, 0.1, window, ws, need)
        B.check(f"attn {way} {start} {length}")


@pytest.mark.parametrize("fmt,heads,group,dim", [("q8", 16, 4, 128), ("f16", 16, 4, 128), ("q8", 16, 4, 64), ("q8", 8, 8, 256)])
def test_attention_of_chunks(fmt, heads, group, dim):
    qmv = _qmv()
    say(f"guards attn chunk {fmt} {heads} x {group} D {dim}")
    rng = np.random.default_rng(4)
    lens, new = [330, 71], [270, 71]
    P = R.Pages(lens, heads, dim, 32, fmt, rng)
    Hq, T = heads * group, 345
    width = Hq * dim
    q = rng.normal(0, 1, (T, width)).astype(np.float32)
    for start, length in (([0, 270, 341], lens), ([0, 270, 341], [400, -1]), ([100, 20, 345], lens), ([-9, 400, 341], lens)):
        B = Buffers()
        cache, batch = _cache(B, P), _batch(B, P, start, length, T)
        tq, out = B.keep(q), B.out((T, width))
        need = qmv.attn_paged_ws_bytes(cache, batch, Hq)
        qmv.attn_paged(cache, batch, tq, width, out, width, Hq, 0.1, 0, B.out(need, torch.uint8), need)
        B.check(f"attn chunk {start} {length}")


@pytest.mark.parametrize("M,K", [(1, 32), (3, 5376), (2, 1056), (5, 33), (2, 4099), (2, 40000), (700, 96), (1, 1)])
def test_norms(M, K):
    qmv = _qmv()
    say(f"guards norm M {M} K {K}")
    rng = np.random.default_rng(5)
    x, r = (rng.normal(0, 1, (M, K)).astype(np.float32) for _ in range(2))
    w = rng.normal(1, 0.1, K).astype(np.float32)
    for residual in (True, False):
        for keep_z in (True, False):
            B = Buffers()
            args = B.keep(x), B.keep(r) if residual else None, B.keep(w), B.out((M, K)) if keep_z else None
            qmv.rmsnorm_add(*args, B.out((M, K)), K, M, 1e-6)
            B.check(f"rmsnorm_add residual {residual} z {keep_z}")
            if K % 32 == 0:
                B = Buffers()
                args = B.keep(x), B.keep(r) if residual else None, B.keep(w), B.out((M, K)) if keep_z else None
                qmv.rmsnorm_add_q8(*args, B.out((M, K), torch.int8), B.out((M, K // 32)), K, M, 1e-6)
                B.check(f"rmsnorm_add_q8 residual {residual} z {keep_z}")


@pytest.mark.parametrize("N,K,M", [(77, 5376, 1), (300, 2048, 16), (70, 96, 3), (41, 256, 2), (97, 512, 33), (129, 256, 70),
                                   (300, 512, 512), (1000, 1056, 130), (5, 16384, 7)])
def test_product_of_codes(N, K, M):
    qmv = _qmv()
    say(f"guards qmm_q4_0_q8 N {N} K {K} M {M}")
    rng = np.random.default_rng(6)
    B = Buffers()
    W = B.keep(synth.q4_0_weights(N, K, 1))
    q = B.keep(rng.integers(-127, 128, (M, K)).astype(np.int8))
    d = B.keep((rng.random((M, K // 32)) + 0.5).astype(np.float32))
    y = B.out((M, N))
    need = qmv.qmm_q4_0_q8_ws_bytes(N, K, M)
    qmv.qmm_q4_0_q8(W, q, d, y, N, K, M, B.out(need, torch.uint8), need)
    B.check("qmm_q4_0_q8")
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("B_,G,V", [(1, 4, 4097), (3, 1, 1), (5, 2, 8191), (2, 64, 300), (210, 1, 20001), (150, 2, 28676),
                                    (1, 3, 262145)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_draft_verification(B_, G, V, cap):
    qmv = _qmv()
    say(f"guards draft_verify B {B_} G {G} V {V} cap {cap}")
    rng = np.random.default_rng(7)
    for ragged in (False, True):
        B = Buffers()
        target = B.keep(rng.normal(0, 2, (B_, G + 1, V)).astype(np.float32))
        draft = B.keep(rng.normal(0, 2, (B_, G, V)).astype(np.float32))
        tokens = rng.integers(0, V, (B_, G)).astype(np.int32)
        tokens[0, 0] = -7
        tokens[-1, -1] = 2 ** 31 - 1
        n = B.keep(rng.integers(-2, G + 3, B_).astype(np.int32)) if ragged else None
        tokens, u = B.keep(tokens), B.keep(rng.random((B_, G + 1), dtype=np.float32))
        acc, out = B.out(B_, torch.int32), B.out((B_, G + 1), torch.int32)
        need = qmv.draft_verify_ws_bytes(B_, G, V)
        qmv.draft_verify(target, V, draft, V, tokens, n, u, acc, out, B_, G, V, 0.9, cap, B.out(need, torch.uint8), need)
        B.check(f"draft_verify ragged {ragged}")
        assert (acc >= 0).all() and (acc <= G).all() and (out >= -1).all() and (out < V).all()


def test_the_guard_sees_a_changed_byte():
    """The check itself finds a change of either kind."""
    for where in ("before", "behind", "input"):
        B = Buffers()
        B.keep(np.arange(7, dtype=np.int8))
        B.out(3, torch.float32).fill_(1.0)
        full = B.all[0][0].view(torch.uint8)
        B.check("untouched")
        full[{"before": GUARD - 1, "behind": GUARD + 7, "input": GUARD + 3}[where]] += 1
        with pytest.raises(AssertionError):
            B.check(where)
