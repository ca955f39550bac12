"""qmm_q4_0_q8 on codes that no quantizer of this library makes: -128, scales
that are NaN, zero or far apart; on every tiling."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import DEV, assert_within, dev, empty, host, say
from quantized_dequant_matrix_amd import synth

pytestmark = pytest.mark.gpu

SHAPES = [(300, 2048, 1), (70, 96, 3), (300, 2048, 16), (33, 512, 5), (97, 512, 33), (129, 256, 70), (300, 512, 512),
          (70, 1056, 200)]


def _product(W, q, d, N, K, M):
    from quantized_dequant_matrix_amd import qmv
    need = qmv.qmm_q4_0_q8_ws_bytes(N, K, M)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    y = empty((M, N))
    qmv.qmm_q4_0_q8(dev(W), dev(q), dev(d), y, N, K, M, ws, need)
    return host(y)


@pytest.mark.parametrize("N,K,M", SHAPES)
def test_codes_over_the_whole_range(N, K, M):
    say(f"product of codes down to -128, N {N} K {K} M {M}")
    rng = np.random.default_rng(N + M)
    W = synth.q4_0_weights(N, K, 2)
    q = rng.integers(-128, 128, (M, K)).astype(np.int8)
    q[0] = -128
    d = (10.0 ** rng.uniform(-8, 8, (M, K // 32))).astype(np.float32)
    d[:, ::3] = 0.0
    ref, S = oracle.qmm_q4_0_q8(W, N, K, q, d, M)
    assert_within(_product(W, q, d, N, K, M), ref, oracle.float_tol(S), "codes")


@pytest.mark.parametrize("N,K,M", SHAPES)
def test_a_block_that_is_not_a_number_stays_in_its_row(N, K, M):
    say(f"product with NaN scales, N {N} K {K} M {M}")
    rng = np.random.default_rng(N * M)
    W = synth.q4_0_weights(N, K, 3)
    q = rng.integers(-127, 128, (M, K)).astype(np.int8)
    d = (rng.random((M, K // 32)) + 0.5).astype(np.float32)
    clean = _product(W, q, d, N, K, M)
    bad = np.unique([0, M // 2, M - 1])
    d[bad, np.arange(len(bad)) % (K // 32)] = np.nan
    q[bad[0], :32] = 0
    got = _product(W, q, d, N, K, M)
    assert np.isnan(got[bad]).all()
    rest = np.setdiff1d(np.arange(M), bad)
    assert np.array_equal(got[rest].view(np.uint32), clean[rest].view(np.uint32))
