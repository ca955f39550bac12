"""kv_plan with its new lengths where the kept ones were, as the header allows:
one launch and two, steps that are done and steps that are refused."""
import numpy as np
import pytest
import torch

import serve_ref as R
from gpu_util import say
from test_gpu_serve_plan import Plan, ints, mixed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,page,width", [(1, 16, 4), (40, 16, 8), (64, 32, 6), (65, 16, 7), (2000, 16, 5)])
@pytest.mark.parametrize("lacking", [0, 1])
def test_new_lengths_over_the_kept_ones(B, page, width, lacking):
    from quantized_dequant_matrix_amd import qmv
    rng = np.random.default_rng(B)
    lens, keep, n = mixed(rng, B, width * page, page, width)
    n[0] = width * page - keep[0]  # some pages at least
    had, has = -(-lens // page), -(-(keep + n) // page)
    need, back = int(np.maximum(0, has - had).sum()), int(np.maximum(0, had - has).sum())
    free = max(need - back - lacking, 0)
    P = Plan(lens, page, width, free, rng, int(n.sum()) + 2)
    t, st, ln, kp, ct = ints(P.table), ints(P.stack), ints(lens), ints(keep), ints([free])
    start, status, pos, sl = ints([-7] * (B + 1)), ints([-7] * 2), ints([-7] * P.T), ints([-7] * P.T, torch.int64)
    pool = qmv.KVPool(t, st, page)
    size = qmv.kv_plan_ws_bytes(pool)
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device=t.device)
    say(f"kv_plan B={B}, new lengths over the kept ones, lacking {lacking}")
    qmv.kv_plan(pool, ln, kp, ints(n), ct, kp, ct, start, pos, sl, status, P.T, ws, size)
    torch.cuda.synchronize()
    want = R.plan(P.table, P.stack, free, lens, keep, n, page, P.T)
    assert status.tolist() == want["status"] and kp.tolist() == want["new_len"] and ct.tolist() == [want["count"]]
    assert start.tolist() == want["row_start"] and ln.tolist() == lens.tolist()
    assert t.cpu().numpy().tolist() == want["table"].tolist()
    assert st.cpu().numpy()[:want["count"]].tolist() == want["stack"]
    rows = int(want["row_start"][-1])
    assert pos.tolist() == [want["position"][r] for r in range(rows)] + [-7] * (P.T - rows)
    assert sl.tolist() == [want["slot"][r] for r in range(rows)] + [-7] * (P.T - rows)
