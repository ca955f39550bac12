"""NaN of either kind: a signalling one (memory never written, masks made of bit
patterns) means to the decode-step operators what a quiet one does."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import DEV, dev, empty, host, say
from test_gpu_step_draft import _problem

pytestmark = pytest.mark.gpu

PATTERNS = np.array([0x7FA00000, 0xFFA00001, 0x7F800001, 0xFFBFFFFF, 0x7FC00000, 0xFFFFFFFF], np.uint32)


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def _bits(a, pattern):
    """A copy of float32 `a` on the GPU with NaN replaced by the pattern (moved as integers, so that no
    conversion quiets it)."""
    b = np.ascontiguousarray(a).view(np.uint32).copy()
    b[np.isnan(a)] = pattern
    return torch.from_numpy(b.view(np.int32)).to(DEV).view(torch.float32)


@pytest.mark.parametrize("pattern", PATTERNS, ids=lambda p: f"{p:08x}")
@pytest.mark.parametrize("V", [37, 5000])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_logits(cap, V, pattern):
    say(f"draft_verify with NaN {pattern:08x}, V {V}, cap {cap}")
    qmv = _qmv()
    B, G = 6, 2
    target, draft, tokens, u = _problem(B, G, V, 5)
    target[0, :, 1::3] = np.nan
    draft[1, :, ::2] = np.nan
    target[2, 0] = np.nan
    draft[3] = np.nan
    target[4, :, :-1] = np.nan
    acc, out, margin = R.draft_verify(target, draft, tokens, None, u, 1.0, cap)
    assert margin.min() > 1e-12
    need = qmv.draft_verify_ws_bytes(B, G, V)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    a, o = empty(B, dtype=torch.int32), empty((B, G + 1), dtype=torch.int32)
    qmv.draft_verify(_bits(target, pattern), V, _bits(draft, pattern), V, dev(tokens), None, dev(u), a, o, B, G, V, 1.0, cap,
                     ws, need)
    assert np.array_equal(host(a), acc) and np.array_equal(host(o), out)


@pytest.mark.parametrize("pattern", PATTERNS, ids=lambda p: f"{p:08x}")
@pytest.mark.parametrize("fmt", ["q8", "f16"])
def test_cache_rows_and_queries(fmt, pattern):
    """Rows with a NaN are stored as NaN in whole, rows that see them are NaN, the others untouched; the same of queries."""
    say(f"cache and attention with NaN {pattern:08x}, {fmt}")
    qmv = _qmv()
    rng = np.random.default_rng(8)
    n, heads, dim, page = 40, 2, 64, 16
    k, v = (rng.normal(0, 1, (n, heads, dim)).astype(np.float32) for _ in range(2))
    q = rng.normal(0, 1, (n, heads, dim)).astype(np.float32)
    results = []
    for broken in (False, True):
        if broken:
            k[20, 0, 5], v[30, 1, 63], q[10, 1, 0] = np.nan, np.nan, np.nan
        dt = torch.int8 if fmt == "q8" else torch.float16
        planes = [torch.zeros(3, heads, page, dim, dtype=dt, device=DEV) for _ in range(2)]
        # what is behind the last position is a signalling NaN too
        scales = [_bits(np.full((3, heads, page), np.nan, np.float32), pattern) for _ in range(2)] if fmt == "q8" else [None] * 2
        if fmt == "f16":
            for p in planes:
                p.view(torch.int16).fill_(0x7D00)
        cache = qmv.KVCache(*planes, *scales)
        batch = qmv.KVBatch(_ints([[2, 0, 1]]), _ints([0, n]), _ints([n]), n)
        width = heads * dim
        qmv.kv_write(cache, batch, _bits(k.reshape(n, width), pattern), width, _bits(v.reshape(n, width), pattern), width)
        back = [empty((n, width)) for _ in range(2)]
        qmv.kv_read(cache, batch, back[0], width, back[1], width)
        out, need = empty((n, width)), qmv.attn_paged_ws_bytes(cache, batch, heads)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        qmv.attn_paged(cache, batch, _bits(q.reshape(n, width), pattern), width, out, width, heads, 0.125, 0, ws, need)
        results.append([host(t).reshape(n, heads, dim) for t in (*back, out)])
    (k0, v0, o0), (k1, v1, o1) = results
    bad = [np.zeros((n, heads), bool) for _ in range(3)]
    bad[0][20, 0] = bad[1][30, 1] = bad[2][10, 1] = True
    bad[2][20:, 0] = bad[2][30:, 1] = True
    for a, b, m in ((k0, k1, bad[0]), (v0, v1, bad[1]), (o0, o1, bad[2])):
        assert np.isfinite(a).all() and np.isnan(b[m]).all()
        assert np.array_equal(a[~m].view(np.uint32), b[~m].view(np.uint32))


@pytest.mark.parametrize("pattern", PATTERNS, ids=lambda p: f"{p:08x}")
@pytest.mark.parametrize("K", [64, 70016])
def test_norm(K, pattern):
    say(f"norm with NaN {pattern:08x}, K {K}")
    qmv = _qmv()
    rng = np.random.default_rng(9)
    x, r = (rng.normal(0, 1, (3, K)).astype(np.float32) for _ in range(2))
    w = rng.normal(1, 0.1, K).astype(np.float32)
    x[1, 33] = np.nan
    w[5] = np.nan  # only the first block of a row
    z, q, d, y = empty((3, K)), empty((3, K), dtype=torch.int8), empty((3, K // 32)), empty((3, K))
    args = _bits(x, pattern), _bits(r, pattern), _bits(w, pattern)
    qmv.rmsnorm_add_q8(*args, z, q, d, K, 3, 1e-6)
    zr, yr = R.norm(x, r, w, 1e-6)
    qr, dr = R.quantize_rows(yr.reshape(3, -1, 32))
    assert np.array_equal(host(z), zr, equal_nan=True) and np.array_equal(host(d), dr, equal_nan=True)
    assert np.array_equal(host(q).reshape(3, -1, 32), qr) and np.isnan(dr[1]).all() and np.isnan(dr[:, 0]).all()
    qmv.rmsnorm_add(*args, z, y, K, 3, 1e-6)
    assert np.array_equal(host(y), yr, equal_nan=True)
