"""Rows and blocks so small that max|x| / 127 is 0 in float32: their codes are 0,
zeros among them included, in the cache and behind the norm, and a product of
such blocks is what qmm_q4_0_q8act makes of the same activations."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, dev, empty, host, say
from quantized_dequant_matrix_amd import synth

pytestmark = pytest.mark.gpu

ULP = np.float32(2.0 ** -149)


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def _ints(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).to(DEV)


def _tiny(rng, shape, top):
    """Multiples of float32's smallest step up to `top` of them, zeros among them."""
    x = (rng.integers(-top, top + 1, shape) * (rng.random(shape) < 0.7)).astype(np.float32) * ULP
    x[..., 0] = top * ULP
    x[..., 1] = 0.0
    return x


def _codes(x, top):
    """float32 division by the scale; a scale of 0 has codes 0."""
    d = np.float32(0.0) if top < 64 else np.float32(np.round(top / 127)) * ULP
    if d == 0:
        return np.zeros(x.shape, np.int8), d
    r = x.astype(np.float64) / np.float64(d)
    return np.clip(np.trunc(r + np.copysign(0.5, r)), -127, 127).astype(np.int8), d


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("top", [1, 7, 63, 64, 100])
@pytest.mark.parametrize("T", [3, 1500])
def test_cache_rows(dim, top, T):
    qmv = _qmv()
    say(f"cache rows of up to {top} steps, dim {dim}, {T} rows")
    rng = np.random.default_rng(top)
    heads, page, pages = 2, 16, -(-T // 16)
    x = _tiny(rng, (T, heads, dim), top)
    cache = qmv.KVCache(*(torch.full((pages, heads, page, dim), 99, dtype=torch.int8, device=DEV) for _ in range(2)),
                        *(torch.full((pages, heads, page), 9.0, device=DEV) for _ in range(2)))
    batch = qmv.KVBatch(_ints(np.arange(pages)[None]), _ints([0, T]), _ints([T]), T)
    width = heads * dim
    qmv.kv_write(cache, batch, dev(x.reshape(T, width)), width, dev(x.reshape(T, width)), width)
    want, d = _codes(x, top)
    for i in (0, 1):
        got = host(cache.tensors[i]).swapaxes(1, 2).reshape(-1, heads, dim)[:T]
        assert np.array_equal(got, want)
        assert (host(cache.tensors[2 + i]).swapaxes(1, 2).reshape(-1, heads)[:T] == d).all()
    back = torch.full((2, T, width), 9.0, device=DEV)
    qmv.kv_read(cache, batch, back[0], width, back[1], width)
    values = (want.astype(np.float32) * d).reshape(T, width)
    assert np.array_equal(host(back[0]), values) and np.array_equal(host(back[1]), values)


@pytest.mark.parametrize("top", [1, 63, 64])
@pytest.mark.parametrize("M,K,N", [(1, 512, 40), (3, 256, 70), (16, 256, 96), (512, 256, 64), (2, 35200, 32)])
def test_norm_blocks(M, K, N, top):
    """z = 1 and eps = 0: y is the weight, whose blocks are tiny in turn with ordinary ones."""
    qmv = _qmv()
    say(f"norm blocks of up to {top} steps, M {M} K {K}")
    rng = np.random.default_rng(K + top)
    w = _tiny(rng, (K // 32, 32), top)
    w[1::3] = rng.normal(0, 1, w[1::3].shape).astype(np.float32)
    x = np.ones((M, K), np.float32)
    q, d, y = empty((M, K), dtype=torch.int8), empty((M, K // 32)), empty((M, K))
    tx, tw = dev(x), dev(w.reshape(K))
    qmv.rmsnorm_add_q8(tx, None, tw, None, q, d, K, M, 0.0)
    qmv.rmsnorm_add(tx, None, tw, None, y, K, M, 0.0)
    got, scales = host(q).reshape(M, K // 32, 32), host(d)
    tiny = np.ones(K // 32, bool)
    tiny[1::3] = False
    want, scale = _codes(w[tiny], top)
    assert np.array_equal(host(y), np.broadcast_to(w.reshape(K), (M, K)))
    assert (got[:, tiny] == want).all() and (scales[:, tiny] == scale).all()
    W = dev(synth.q4_0_weights(N, K, 3))
    need = qmv.qmm_q4_0_q8_ws_bytes(N, K, M)
    a, b = empty((M, N)), empty((M, N))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    qmv.qmm_q4_0_q8(W, q, d, a, N, K, M, ws, need)
    qmv.qmm_q4_0_q8act(W, y, b, N, K, M, ws, need)
    assert np.array_equal(host(a).view(np.uint32), host(b).view(np.uint32)) and np.isfinite(host(a)).all()
