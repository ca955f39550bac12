"""Workspaces of include/qmv_serve.h: one that serves a batch serves every
smaller one, as a program that allocates once for its largest needs it."""
import ctypes

import pytest

from quantized_dequant_matrix_amd import qmv

MANY = (1, 2, 3, 7, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 512, 513, 600, 4096, 65535)


def falls(sizes):
    """Neighbours of which the second is smaller."""
    return [(a, b) for a, b in zip(sizes, sizes[1:]) if b[1] < a[1]]


@pytest.mark.parametrize("V", [1, 4096, 20480, 20481, 32000, 40960, 40961, 50257, 65536, 65537, 128256, 262144, 262145, 2 ** 24])
def test_draw_in_the_rows(V):
    sizes = [(M, qmv.logits_draw_ws_bytes(V, M)) for M in MANY]
    assert all(n > 0 for _, n in sizes) and not falls(sizes), falls(sizes)


@pytest.mark.parametrize("M", MANY)
def test_draw_in_the_vocabulary(M):
    sizes = [(V, qmv.logits_draw_ws_bytes(V, M)) for V in (1, 64, 4097, 20480, 20481, 30000, 40960, 40961, 65536, 65537, 90000,
                                                          262144, 262145, 10 ** 6, 2 ** 31 - 1)]
    assert not falls(sizes), falls(sizes)


def lora_bytes(B, T, K=5376, N=21504, max_rank=64):
    l = qmv._Lora(None, None, None, None, K, N, 8, max_rank, 0)
    return qmv.lora_add_ws_bytes(type("D", (), {"ref": ctypes.addressof(l)}), B, T)


@pytest.mark.parametrize("K", [8, 128, 512, 520, 4096, 5376, 21504, 100000, 2 ** 23])
@pytest.mark.parametrize("max_rank", [8, 16, 64, 256])
def test_adapters_in_rows_and_sequences(K, max_rank):
    rows = sorted(set(MANY) | {1000, 1500, 1501, 2000, 3001, 8192, 16384, 16385, 2 ** 20, 2 ** 24 - 1})
    for B in (1, 4, 32, 300, 65535):
        sizes = [(T, lora_bytes(B, T, K, 21504, max_rank)) for T in rows]
        assert all(n > 0 for _, n in sizes) and not falls(sizes), (B, falls(sizes))
    for T in rows:
        sizes = [(B, lora_bytes(B, T, K, 21504, max_rank)) for B in MANY]
        assert not falls(sizes), (T, falls(sizes))


def test_adapters_in_widths():
    for B, T in ((1, 1), (32, 32), (4, 1611), (6, 8192)):
        for vary, values in (("K", (8, 512, 1024, 4096, 5376, 21504, 65536)), ("N", (1, 300, 5376, 21504, 2 ** 23)),
                             ("max_rank", (8, 16, 24, 64, 128, 256))):
            sizes = [(v, lora_bytes(B, T, **{vary: v})) for v in values]
            assert not falls(sizes), (vary, falls(sizes))


def test_plan_in_the_sequences():
    def size(B):
        p = qmv._KVPool(None, None, 100, B, 8, 16)
        return qmv.kv_plan_ws_bytes(type("D", (), {"ref": ctypes.addressof(p)}))

    sizes = [(B, size(B)) for B in MANY]
    assert all(n > 0 for _, n in sizes) and not falls(sizes)
