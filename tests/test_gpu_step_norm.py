"""rmsnorm_add, rmsnorm_add_q8 and qmm_q4_0_q8: bit for bit against the
definition (the mean in 64 bits makes every later step one float32 operation)
and against the entry points whose steps they share."""
import numpy as np
import pytest
import torch

import oracle
import step_ref as R
from gpu_util import DEV, dev, empty, host, say
from quantized_dequant_matrix_amd import synth

pytestmark = pytest.mark.gpu


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


SHAPES = [(1, 5376), (1, 32), (3, 64), (2, 96), (5, 4096), (17, 5376), (700, 352), (2, 21504), (1, 40000 - 40000 % 32),
          (1, 70016), (600, 5376), (4, 8192), (1030, 32)]


def _problem(M, K, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (M, K)).astype(np.float32)
    r = rng.normal(0, 3, (M, K)).astype(np.float32)
    w = rng.normal(1, 0.3, K).astype(np.float32)
    return x, r, w


@pytest.mark.parametrize("M,K", SHAPES + [(1, 1), (2, 5), (3, 1001), (1, 5377), (9, 66), (1, 70001)])
@pytest.mark.parametrize("with_r", [True, False])
def test_f32(M, K, with_r):
    qmv = _qmv()
    x, r, w = _problem(M, K, M * 7 + K)
    say(f"rmsnorm_add {M} x {K}")
    z, y = empty((M, K)), empty((M, K))
    qmv.rmsnorm_add(dev(x), dev(r) if with_r else None, dev(w), z, y, K, M, 1e-5)
    zr, yr = R.norm(x, r if with_r else None, w, 1e-5)
    assert np.array_equal(host(z), zr) and np.array_equal(host(y), yr)


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("with_r", [True, False])
def test_q8(M, K, with_r):
    qmv = _qmv()
    x, r, w = _problem(M, K, M + K * 3)
    x[0, :min(K, 32)] = 0.0
    r[0, :min(K, 32)] = 0.0  # an all-zero block
    say(f"rmsnorm_add_q8 {M} x {K}")
    z, q, d = empty((M, K)), empty((M, K), dtype=torch.int8), empty((M, K // 32))
    qmv.rmsnorm_add_q8(dev(x), dev(r) if with_r else None, dev(w), z, q, d, K, M, 1e-5)
    zr, yr = R.norm(x, r if with_r else None, w, 1e-5)
    qr, dr = R.quantize_rows(yr.reshape(M, K // 32, 32))
    assert np.array_equal(host(z), zr)
    assert np.array_equal(host(d), dr) and np.array_equal(host(q), qr.reshape(M, K))
    # the same codes as the activation quantizer gives for the float32 output
    q2, d2 = empty((M, K), dtype=torch.int8), empty((M, K // 32))
    qmv.qmvdbg_quantize_q8(dev(yr), q2, d2, K, M)
    assert np.array_equal(host(q2), host(q)) and np.array_equal(host(d2), host(d))


@pytest.mark.parametrize("K", [64, 5376, 70016])
def test_in_place_and_without_z(K):
    qmv = _qmv()
    M = 3
    x, r, w = _problem(M, K, 5)
    zr, yr = R.norm(x, r, w, 1e-6)
    for alias in ("x", "r", "none"):
        tx, tr, y = dev(x), dev(r), empty((M, K))
        z = {"x": tx, "r": tr, "none": None}[alias]
        qmv.rmsnorm_add(tx, tr, dev(w), z, y, K, M, 1e-6)
        assert np.array_equal(host(y), yr)
        if z is not None:
            assert np.array_equal(host(z), zr)
        tx, tr, q, d = dev(x), dev(r), empty((M, K), dtype=torch.int8), empty((M, K // 32))
        z = {"x": tx, "r": tr, "none": None}[alias]
        qmv.rmsnorm_add_q8(tx, tr, dev(w), z, q, d, K, M, 1e-6)
        qr, dr = R.quantize_rows(yr.reshape(M, -1, 32))
        assert np.array_equal(host(q), qr.reshape(M, K)) and np.array_equal(host(d), dr)
        if z is not None:
            assert np.array_equal(host(z), zr)


@pytest.mark.parametrize("K", [96, 5376])
def test_unaligned_rows(K):
    """Buffers that are only 4-byte aligned."""
    qmv = _qmv()
    M = 4
    x, r, w = _problem(M, K, 6)
    zr, yr = R.norm(x, r, w, 1e-6)
    shift = lambda a: torch.cat([torch.zeros(1, device=DEV), dev(a).reshape(-1)])[1:]
    z, y = empty(M * K + 3)[3:], empty(M * K + 1)[1:]
    qmv.rmsnorm_add(shift(x), shift(r), shift(w), z, y, K, M, 1e-6)
    assert np.array_equal(host(z).reshape(M, K), zr) and np.array_equal(host(y).reshape(M, K), yr)
    q, d = empty(M * K + 4, dtype=torch.int8)[4:], empty(M * K // 32 + 1)[1:]
    qmv.rmsnorm_add_q8(shift(x), shift(r), shift(w), z, q, d, K, M, 1e-6)
    qr, dr = R.quantize_rows(yr.reshape(M, -1, 32))
    assert np.array_equal(host(q), qr.reshape(-1)) and np.array_equal(host(d), dr.reshape(-1))


def test_values_at_the_edges():
    """Zero rows, tiny and huge rows, rows that are not finite: the rows beside them stay right."""
    qmv = _qmv()
    K = 128
    x, r, w = _problem(8, K, 7)
    x[0], r[0] = 0.0, 0.0
    x[1] *= 1e-30
    r[1] = 0.0
    x[2] *= 1e18  # the squares' mean is above float32's square root range, not above float64's
    r[2] = 0.0
    x[3, 5] = np.nan
    x[4, 40] = np.inf
    y, q, d = empty((8, K)), empty((8, K), dtype=torch.int8), empty((8, K // 32))
    qmv.rmsnorm_add(dev(x), dev(r), dev(w), None, y, K, 8, 1e-6)
    qmv.rmsnorm_add_q8(dev(x), dev(r), dev(w), None, q, d, K, 8, 1e-6)
    with np.errstate(invalid="ignore"):
        zr, yr = R.norm(x, r, w, 1e-6)
        qr, dr = R.quantize_rows(yr.reshape(8, -1, 32))
    got = host(y)
    assert np.array_equal(np.isnan(got), np.isnan(yr))
    assert np.array_equal(got[~np.isnan(got)], yr[~np.isnan(yr)])
    assert np.array_equal(np.isnan(host(d)), np.isnan(dr))
    fine = ~np.isnan(dr)
    assert np.array_equal(host(d)[fine], dr[fine])
    assert np.array_equal(host(q).reshape(8, -1, 32)[fine], qr[fine])


@pytest.mark.parametrize("N,K,M", [(300, 2048, 1), (70, 96, 3), (65, 128, 1), (300, 2048, 16), (33, 512, 5),
                                   (4096, 256, 512), (2112, 768, 1000), (21504, 512, 2), (129, 5376, 40)])
def test_product_of_given_codes(N, K, M):
    """The same bits as qmm_q4_0_q8act on the activations, and the oracle's value."""
    qmv = _qmv()
    say(f"qmm_q4_0_q8 {N} x {K}, {M} rows")
    W, x = synth.problem("q4_0", N, K, M, 31)
    wsb = qmv.qmm_q4_0_q8_ws_bytes(N, K, M)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    tW, tx, y, y2 = dev(W), dev(x), empty((M, N)), empty((M, N))
    qmv.qmm_q4_0_q8act(tW, tx, y, N, K, M, ws, wsb)
    q, d = empty((M, K), dtype=torch.int8), empty((M, K // 32))
    qmv.qmvdbg_quantize_q8(tx, q, d, K, M)
    ws.fill_(0xff)
    qmv.qmm_q4_0_q8(tW, q, d, y2, N, K, M, ws, wsb)
    assert np.array_equal(host(y2), host(y))
    if M <= 40:
        qx, dx = oracle.quantize_q8(x, M, K)
        yr, S = oracle.qmm_q4_0_q8(W, N, K, qx, dx, M)
        assert (np.abs(host(y2) - yr) <= oracle.float_tol(S)).all()
