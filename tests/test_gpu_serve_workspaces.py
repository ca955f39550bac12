"""One workspace, allocated for the largest batch, serves calls of every
smaller one."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from test_gpu_serve_draw import logits

pytestmark = pytest.mark.gpu


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


@pytest.mark.parametrize("V,M", [(32000, 40), (50257, 130), (262144, 20)])
def test_draw(V, M):
    qmv = _qmv()
    rng = np.random.default_rng(V)
    size = qmv.logits_draw_ws_bytes(V, M)
    full = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    z = torch.from_numpy(logits(rng, M, V)).to(DEV)
    t, p, u = (torch.from_numpy(a.astype(np.float32)).to(DEV) for a in (rng.choice([0.0, 0.7, 1.0], M), rng.choice([1.0, 0.9], M),
                                                                      rng.random(M)))
    k = torch.from_numpy(rng.choice([0, 40, 1000], M).astype(np.int32)).to(DEV)

    def draw(m, ws, ws_bytes):
        token, kept = (torch.full((m,), -7, dtype=torch.int32, device=DEV) for _ in range(2))
        qmv.logits_draw(z, V, t, k, p, None, u, token, kept, V, m, 0.0, ws, ws_bytes)
        return torch.stack([token, kept])

    whole = draw(M, full[:size], size)
    for m in (1, 2, 7, 15, 16, 17, 39, 127, 128, M):
        if m <= M:
            say(f"logits_draw V={V}, {m} rows with the workspace of {M}")
            assert torch.equal(draw(m, full[:size], size), whole[:, :m])
    assert (full[size:] == 0x5A).all()
