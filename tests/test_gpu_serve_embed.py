"""Embedding rows bit for bit against the formats' definitions."""
import numpy as np
import pytest
import torch

import serve_ref as R
from gpu_util import DEV, dev, host, say

pytestmark = pytest.mark.gpu


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


def table(fmt, V, K, rng):
    """Blocks of random bytes: every code and sub-scale, float16 scales that are finite."""
    n, size = R.BLOCK[fmt]
    w = rng.integers(0, 256, (V, K // n, size), dtype=np.uint8)
    for at in {"q8_0": (0,), "q4_0": (0,), "q4_k": (0, 2), "q6_k": (208,)}[fmt]:
        d = (rng.random((V, K // n)) * 2.0 ** rng.integers(-20, 3, (V, K // n))).astype(np.float16)
        w[:, :, at:at + 2] = d.view(np.uint8).reshape(V, K // n, 2)
    return w.reshape(V, -1)


def run(fmt, W, tokens, K, scale, offset=0):
    M = len(tokens)
    buf = torch.full((M * K + 8,), -3.0, device=DEV)
    y = buf[offset:offset + M * K].view(M, K)
    f = getattr(_qmv(), "embed_" + fmt)
    f(dev(W), torch.from_numpy(np.asarray(tokens, dtype=np.int32)).to(DEV), y, W.shape[0], K, M, scale)
    got = host(y)
    rest = host(buf)
    assert (rest[:offset] == -3.0).all() and (rest[offset + M * K:] == -3.0).all()
    return got


@pytest.mark.parametrize("fmt,blocks", [(f, b) for f in R.BLOCK for b in (1, 2, 7, 21)] + [("q8_0", 168), ("q4_0", 171),
                                                                                          ("q8_0", 2500), ("q6_k", 300)])
@pytest.mark.parametrize("M", [1, 5])
def test_rows(fmt, blocks, M):
    rng = np.random.default_rng(blocks + M)
    K = R.BLOCK[fmt][0] * blocks
    V = 37
    say(f"embed_{fmt} K={K} M={M}")
    W = table(fmt, V, K, rng)
    for scale in (1.0, float(np.float32(np.sqrt(K))), -0.3):
        tokens = rng.integers(0, V, M)
        got = run(fmt, W, tokens, K, scale)
        want = R.embed(fmt, W, tokens, scale)
        assert np.array_equal(got.view(np.uint32) & 0x7FFFFFFF, want.view(np.uint32) & 0x7FFFFFFF)
        assert np.array_equal(got, want)


@pytest.mark.parametrize("fmt", list(R.BLOCK))
def test_tokens_outside_and_repeated(fmt):
    rng = np.random.default_rng(1)
    K = 512
    W = table(fmt, 9, K, rng)
    tokens = np.array([0, 8, 9, -1, 2 ** 31 - 1, -2 ** 31, 8, 8, 3])
    say(f"embed_{fmt} tokens outside the table")
    for offset in (0, 1, 3):  # outputs that are not 16-byte aligned
        got = run(fmt, W, tokens, K, 2.0, offset)
        assert np.array_equal(got, R.embed(fmt, W, tokens, 2.0))
        assert (got[2:6] == 0).all()


def test_many_rows():
    rng = np.random.default_rng(2)
    W = table("q4_k", 1000, 768, rng)
    tokens = rng.integers(0, 1000, 5000)
    say("embed_q4_k M=5000")
    assert np.array_equal(run("q4_k", W, tokens, 768, 1.0), R.embed("q4_k", W, tokens, 1.0))


def test_rows_past_32_bits():
    """A row whose bytes start beyond 4 GiB."""
    K, V = 8192, 600000
    size = K // 32 * 34
    assert (V - 1) * size > 2 ** 32
    say("embed_q8_0 rows beyond 4 GiB")
    rng = np.random.default_rng(3)
    few = table("q8_0", 3, K, rng)
    W = torch.zeros((V, size), dtype=torch.uint8, device=DEV)
    tokens = [0, V // 2 + 1, V - 1]
    for t, row in zip(tokens, few):
        W[t].copy_(torch.from_numpy(row))
    y = torch.empty((3, K), device=DEV)
    _qmv().embed_q8_0(W, torch.tensor(tokens, dtype=torch.int32, device=DEV), y, V, K, 3, 1.0)
    assert np.array_equal(host(y), R.embed("q8_0", few, np.arange(3), 1.0))
