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


@pytest.mark.parametrize("K,N,max_rank", [(5376, 600, 64), (1024, 96, 16)])
def test_adapters(K, N, max_rank):
    from test_gpu_serve_lora import Adapters, check, ints
    qmv = _qmv()
    L = Adapters(4, max_rank, K, N, "bf16", True, K)
    d = L.gpu()
    B, T = 40, 3000
    size = qmv.lora_add_ws_bytes(d, B, T)
    full = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(K)
    x, base = (torch.randn(T, n, generator=g, device=DEV) for n in (K, N))
    for b, t in ((1, 1), (1, 16), (3, 17), (32, 32), (40, 40), (2, 512), (4, 1000), (1, 1500), (40, 2999), (B, T)):
        say(f"lora_add K={K}, {t} rows of {b} with the workspace of {T}")
        start = ints(np.linspace(0, t, b + 1).astype(int))
        adapter = ints(np.arange(b) % 4)
        out = []
        for ws, n in ((full[:size], size), (torch.empty(qmv.lora_add_ws_bytes(d, b, t), dtype=torch.uint8, device=DEV), None)):
            y = torch.full((t, N), -77.0, device=DEV)
            qmv.lora_add(d, adapter, start, x, K, base, N, y, N, b, t, ws, n or ws.numel())
            out.append(y)
        assert torch.equal(*out) and (full[size:] == 0x5A).all()
        check(L, np.arange(b) % 4, np.diff(np.linspace(0, t, b + 1).astype(int)), spare=0, lora=d) if t < 100 else None
