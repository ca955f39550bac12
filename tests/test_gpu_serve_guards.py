"""The entry points of qmv_serve.h write only their outputs and the workspace
they asked for, and leave their inputs bit-identical: sentinels before and
behind every buffer, also where row starts are out of order, lengths lie and
tokens, adapters and pages do not exist."""
import numpy as np
import pytest
import torch

import serve_ref as R
from gpu_util import say
from test_gpu_serve_embed import table as embed_table
from test_gpu_step_guards import DISORDER, Buffers

pytestmark = pytest.mark.gpu

i32 = lambda a: np.asarray(a, dtype=np.int32)  # noqa: E731
f32 = lambda a: np.asarray(a, dtype=np.float32)  # noqa: E731


def _qmv():
    from quantized_dequant_matrix_amd import qmv
    return qmv


@pytest.mark.parametrize("B,T", [(3, 70), (70, 5000), (1500, 40000)])
def test_plan(B, T):
    qmv = _qmv()
    rng = np.random.default_rng(B)
    width, page, num = 6, 16, 6 * B + 5
    lens = rng.integers(0, 96, B)
    keep = np.where(rng.random(B) < 0.3, 0, lens)
    n = np.minimum(rng.integers(0, 30, B), 96 - keep)
    wild = rng.integers(-2 ** 31, 2 ** 31, B)
    for lens2, keep2, n2, count in ((lens, keep, n, num - 6 * B), (lens, keep, n, 6 * B), (lens, keep, n, 0), (lens, keep, n, -5),
                                    (lens, keep, n, num + 9), (wild, keep, n, 5), (lens, wild, n, 5), (lens, keep, wild, 5),
                                    (lens, None, n, 6 * B)):
        for rows in (T, 1):
            G = Buffers()
            table = G.out((B, width), torch.int32)
            stack = G.out(num, torch.int32)
            table.copy_(torch.from_numpy(i32(rng.integers(-2, num + 2, (B, width)))))
            stack.copy_(torch.from_numpy(i32(rng.permutation(num))))
            pool = qmv.KVPool(table, stack, page)
            size = qmv.kv_plan_ws_bytes(pool)
            k = None if keep2 is None else G.keep(i32(keep2))
            qmv.kv_plan(pool, G.keep(i32(lens2)), k, G.keep(i32(n2)), G.keep(i32([count])), G.out(B, torch.int32),
                        G.out(1, torch.int32), G.out(B + 1, torch.int32), G.out(rows, torch.int32), G.out(rows, torch.int64),
                        G.out(2, torch.int32), rows, G.out(size, torch.uint8), size)
            G.check(f"kv_plan {B} {count} {rows}")
    say(f"guards kv_plan B={B}")


@pytest.mark.parametrize("fmt", list(R.BLOCK))
def test_embed(fmt):
    qmv = _qmv()
    rng = np.random.default_rng(1)
    for K, M in ((256, 1), (1280, 7), (5376, 40)):
        say(f"guards embed_{fmt} K={K} M={M}")
        G = Buffers()
        tokens = rng.integers(-2, 13, M)
        getattr(qmv, "embed_" + fmt)(G.keep(embed_table(fmt, 11, K, rng)), G.keep(i32(tokens)), G.out((M, K)), 11, K, M, 1.5)
        G.check("embed")


@pytest.mark.parametrize("max_rank,K,N", [(8, 64, 33), (16, 1024, 300), (64, 520, 129), (256, 128, 70)])
@pytest.mark.parametrize("T", [2, 5, 90, 400])
def test_lora(max_rank, K, N, T):
    qmv = _qmv()
    rng = np.random.default_rng(T)
    A, Bm = (torch.from_numpy(f32(rng.normal(0, 0.1, s))).bfloat16() for s in ((3, max_rank, K), (3, N, max_rank)))
    for start in [[0, T - 1, T], [0, 0, T - 1], [0, T, T], [0, T // 2, T + 70]] + DISORDER:
        for adapter in ([0, 2], [-1, 3]):
            say(f"guards lora_add R={max_rank} T={T} {start} {adapter}")
            G = Buffers()
            keep = lambda t: G.keep(t.view(torch.int16).numpy()).view(torch.bfloat16)  # noqa: E731
            L = qmv.Lora(keep(A), keep(Bm), G.keep(f32([1, 2, 3])), G.keep(i32([5, 999, -3])))
            size = qmv.lora_add_ws_bytes(L, 2, T)
            qmv.lora_add(L, G.keep(i32(adapter)), G.keep(i32(start)), G.keep(f32(rng.normal(0, 1, (T, K)))), K,
                         G.keep(f32(rng.normal(0, 1, (T, N)))), N, G.out((T, N)), N, 2, T, G.out(size, torch.uint8), size)
            G.check("lora_add")


@pytest.mark.parametrize("V", [1, 100, 5000, 40001, 262144])
def test_draw(V):
    qmv = _qmv()
    rng = np.random.default_rng(V)
    for M in (1, 3, 50):
        if M * V > 10 ** 6:
            continue
        say(f"guards logits_draw V={V} M={M}")
        for fill in (None, 0.0, np.nan):
            z = f32(rng.normal(0, 3, (M, V)) if fill is None else np.full((M, V), fill))
            G = Buffers()
            size = qmv.logits_draw_ws_bytes(V, M)
            qmv.logits_draw(G.keep(z), V, G.keep(f32(rng.choice([0.0, 0.5, 1.0], M))), G.keep(i32(rng.choice([-1, 0, 3, 10 ** 6], M))),
                            G.keep(f32(rng.choice([0.0, 0.5, 0.99, 2.0], M))), G.keep(f32(rng.choice([0.0, 0.1], M))),
                            G.keep(f32(rng.random(M))), G.out(M, torch.int32), G.out(M, torch.int32), V, M, 0.0,
                            G.out(size, torch.uint8), size)
            G.check("logits_draw")
