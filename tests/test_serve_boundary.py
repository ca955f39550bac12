"""The entry points of include/qmv_serve.h are exported and bound, and bad
arguments are rejected on the host.  No compute call is made: EVERY call
below must fail argument checking (the fake addresses are never valid device
memory)."""
import ctypes
import os
import re

import pytest
import torch

from quantized_dequant_matrix_amd import qmv

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qmv_serve.h")

OK, NUL, SHAPE, ALIGN, WS, LAUNCH, ARG = range(7)
FAKE = 1 << 20
S = None
BIG = 2 ** 62
NAN, INF = float("nan"), float("inf")


def call(name, *args):
    return getattr(qmv.lib, name)(*args)


def ref(s):
    return None if s is None else ctypes.byref(s)


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^(?:int|size_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))
    assert len(names) == 10 and "kv_plan" in names
    for n in names:
        assert hasattr(qmv.lib, n), n
    assert sorted(qmv.SERVE_EXPORTS) == names


def test_structs_have_the_sizes_of_the_header():
    # 8-byte members first, then int32, padded to 8
    assert ctypes.sizeof(qmv._KVPool) == 2 * 8 + 8 + 3 * 4 + 4
    assert ctypes.sizeof(qmv._Lora) == 4 * 8 + 2 * 8 + 3 * 4 + 4


def pool(**kw):
    f = dict(page_table=FAKE, free_pages=FAKE, num_pages=8, B=2, max_pages=4, page_size=16)
    f.update(kw)
    return qmv._KVPool(*[f[n] for n, _ in qmv._KVPool._fields_])


def plan(p, **kw):
    f = dict(kv_len=FAKE, keep=FAKE, n_new=FAKE, free_count=FAKE, new_len=FAKE, new_count=FAKE, row_start=FAKE,
             position=FAKE, slot=FAKE, status=FAKE, T=8, ws=FAKE, ws_bytes=BIG)
    f.update(kw)
    return call("kv_plan", ref(p), *f.values(), S)


def test_plan_arguments():
    assert plan(None) == NUL and call("kv_plan_ws_bytes", None) == 0
    assert plan(pool(page_table=None)) == NUL and plan(pool(free_pages=None)) == NUL
    for k in ("kv_len", "n_new", "free_count", "new_len", "new_count", "row_start", "status", "ws"):
        assert plan(pool(), **{k: None}) == NUL, k
    for kw in (dict(num_pages=0), dict(num_pages=2 ** 31), dict(B=0), dict(B=65536), dict(max_pages=0), dict(max_pages=-1),
               dict(max_pages=2 ** 26 + 1), dict(page_size=8), dict(page_size=24), dict(page_size=2048), dict(page_size=0)):
        assert plan(pool(**kw)) == SHAPE, kw
        assert call("kv_plan_ws_bytes", ref(pool(**kw))) == 0
    for T in (0, -1, 2 ** 24):
        assert plan(pool(), T=T) == SHAPE
    for k in ("kv_len", "keep", "n_new", "free_count", "new_len", "new_count", "row_start", "position", "status"):
        assert plan(pool(), **{k: FAKE + 2}) == ALIGN, k
    assert plan(pool(), slot=FAKE + 4) == ALIGN and plan(pool(), ws=FAKE + 8) == ALIGN
    assert plan(pool(page_table=FAKE + 2)) == ALIGN and plan(pool(free_pages=FAKE + 1)) == ALIGN
    need = call("kv_plan_ws_bytes", ref(pool()))
    assert need > 0 and plan(pool(), ws_bytes=need - 1) == WS


@pytest.mark.parametrize("fmt,block", [("q8_0", 32), ("q4_0", 32), ("q4_k", 256), ("q6_k", 256)])
def test_embed_arguments(fmt, block):
    good = [FAKE, FAKE, FAKE, 100, 512, 3, 1.0, S]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return call("embed_" + fmt, *a)

    for i in range(3):
        assert with_(i, None) == NUL
    for i, vals in ((3, (0, -1, 2 ** 31)), (4, (0, -block, block // 2, block + 8, 2 ** 31)), (5, (0, -1, 2 ** 24))):
        for v in vals:
            assert with_(i, v) == SHAPE
    for v in (NAN, INF, -INF):
        assert with_(6, v) == ARG
    assert with_(0, FAKE + 8) == ALIGN and with_(1, FAKE + 2) == ALIGN and with_(2, FAKE + 1) == ALIGN


def lora(**kw):
    f = dict(A=FAKE, Bm=FAKE, rank=FAKE, scale=FAKE, K=64, N=100, slots=3, max_rank=16, format=1)
    f.update(kw)
    return qmv._Lora(*[f[n] for n, _ in qmv._Lora._fields_])


def add(l, **kw):
    f = dict(adapter=FAKE, row_start=FAKE, x=FAKE, ldx=64, base=2 * FAKE, ldb=100, y=FAKE, ldy=100, B=2, T=5, ws=FAKE,
             ws_bytes=BIG)
    f.update(kw)
    return call("lora_add", ref(l), *f.values(), S)


def test_lora_arguments():
    assert add(None) == NUL and call("lora_add_ws_bytes", None, 1, 1) == 0
    for k in ("A", "Bm", "scale"):
        assert add(lora(**{k: None})) == NUL
    for k in ("adapter", "row_start", "x", "y", "ws"):
        assert add(lora(), **{k: None}) == NUL
    for kw, want in ((dict(K=0), SHAPE), (dict(K=60), SHAPE), (dict(K=2 ** 24), SHAPE), (dict(N=0), SHAPE),
                     (dict(N=2 ** 24), SHAPE), (dict(max_rank=0), SHAPE), (dict(max_rank=12), SHAPE),
                     (dict(max_rank=264), SHAPE), (dict(slots=0), SHAPE), (dict(slots=2 ** 20), SHAPE),
                     (dict(format=2), ARG), (dict(format=-1), ARG)):
        assert add(lora(**kw)) == want, kw
        assert call("lora_add_ws_bytes", ref(lora(**kw)), 2, 5) == 0
    for kw in (dict(B=0), dict(B=65536), dict(T=0), dict(T=2 ** 24), dict(ldx=63), dict(ldb=99), dict(ldy=99),
               dict(ldx=2 ** 61), dict(ldy=-100)):
        assert add(lora(), **kw) == SHAPE, kw
    assert add(lora(), base=FAKE, ldb=101) == ARG  # in place, rows apart
    for kw in (dict(adapter=FAKE + 2), dict(row_start=FAKE + 1), dict(x=FAKE + 2), dict(base=FAKE + 2), dict(y=FAKE + 2),
               dict(ws=FAKE + 8)):
        assert add(lora(), **kw) == ALIGN, kw
    for kw in (dict(A=FAKE + 8), dict(Bm=FAKE + 4), dict(rank=FAKE + 2), dict(scale=FAKE + 2)):
        assert add(lora(**kw)) == ALIGN, kw
    need = call("lora_add_ws_bytes", ref(lora()), 2, 5)
    assert need > 0 and add(lora(), ws_bytes=need - 1) == WS
    assert call("lora_add_ws_bytes", ref(lora()), 0, 5) == 0 and call("lora_add_ws_bytes", ref(lora()), 2, 2 ** 24) == 0


def test_draw_arguments():
    need = call("logits_draw_ws_bytes", 1000, 4)
    assert need > 0
    #        logits ld    T     k     p     min   u     tok   kept  V     M  cap  ws    bytes
    good = [FAKE, 1000, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1000, 4, 0.0, FAKE, need, S]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return call("logits_draw", *a)

    for i in (0, 2, 6, 7, 12):
        assert with_(i, None) == NUL
    assert with_(1, 999) == SHAPE and with_(1, 2 ** 61) == SHAPE
    for i, vals in ((9, (0, -1, 2 ** 31)), (10, (0, -1, 65536))):
        for v in vals:
            assert with_(i, v) == SHAPE
    for v in (-1.0, NAN, INF, 65537.0):
        assert with_(11, v) == ARG
    for i in (0, 2, 3, 4, 5, 6, 7, 8):
        assert with_(i, FAKE + 2) == ALIGN
    assert with_(12, FAKE + 8) == ALIGN
    assert with_(13, need - 1) == WS
    assert call("logits_draw_ws_bytes", 0, 4) == 0 and call("logits_draw_ws_bytes", 1000, 65536) == 0


def test_binding_refuses_tensors_of_the_host():
    t, i = torch.zeros(64), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        qmv.embed_q8_0(t, i, t, 1, 32, 1, 1.0, stream=0)
    with pytest.raises(ValueError):
        qmv.logits_draw(t, 64, t, None, None, None, t, i, None, 64, 1, 0.0, t, 256, stream=0)
    with pytest.raises(ValueError):
        qmv.KVPool(torch.zeros(1, 2, dtype=torch.int32), i, 16)
    with pytest.raises(ValueError):
        qmv.Lora(torch.zeros(2, 8, 16).half(), torch.zeros(2, 5, 8).half(), torch.zeros(2))


def test_binding_checks_descriptors():
    t, i = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for args in ((t.long(), i), (t, i.long()), (t[0], i), (t, t)):
        with pytest.raises(ValueError, match="int32"):
            qmv.KVPool(*args, 16)
    A, Bm, s, r = torch.zeros(2, 8, 16).half(), torch.zeros(2, 5, 8).half(), torch.zeros(2), torch.zeros(2, dtype=torch.int32)
    for args in ((A, Bm.bfloat16(), s), (A.float(), Bm.float(), s), (A[0], Bm, s), (A, Bm[:1], s), (A, Bm[:, :, :4], s),
                 (A, Bm, s.double()), (A, Bm, s[:1]), (A, Bm, s, r.long()), (A, Bm, s, r[:1])):
        with pytest.raises(ValueError, match="float16|slots|rank"):
            qmv.Lora(*args)


def test_binding_refuses_descriptors_of_another_gpu(monkeypatch):
    monkeypatch.setattr(qmv, "_device", lambda: 0)
    for cls, f in ((qmv.KVPool, lambda o: qmv.kv_plan(o, *[FAKE] * 10, 8, FAKE, 256, stream=0)),
                   (qmv.Lora, lambda o: qmv.lora_add(o, FAKE, FAKE, FAKE, 64, None, 0, FAKE, 64, 1, 1, FAKE, 256, stream=0))):
        o = cls.__new__(cls)
        o.ref, o.device = FAKE, 1
        with pytest.raises(ValueError, match="another GPU"):
            f(o)
