"""The entry points of include/qmv_step.h are exported and bound, and bad
arguments are rejected on the host.  No compute call is made: EVERY call
below must fail argument checking (the fake addresses are never valid device
memory)."""
import ctypes
import os
import re

import pytest
import torch

from quantized_dequant_matrix_amd import qmv

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qmv_step.h")

OK, NUL, SHAPE, ALIGN, WS, LAUNCH, ARG = range(7)
FAKE = 1 << 20
S = None
BIG = 2 ** 62


def call(name, *args):
    return getattr(qmv.lib, name)(*args)


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^(?:int|size_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))
    assert len(names) == 10 and "attn_paged" in names
    for n in names:
        assert hasattr(qmv.lib, n), n
    assert sorted(qmv.STEP_EXPORTS) == names


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=8, kv_heads=4, head_dim=128, page_size=16, format=0)
    f.update(kw)
    return qmv._KVCache(*[f[n] for n, _ in qmv._KVCache._fields_])


def batch(**kw):
    f = dict(page_table=FAKE, row_start=FAKE, kv_len=FAKE, T=3, B=2, max_pages=4)
    f.update(kw)
    return qmv._KVBatch(*[f[n] for n, _ in qmv._KVBatch._fields_])


def ref(s):
    return None if s is None else ctypes.byref(s)


BAD_CACHE = [(dict(k=None), NUL), (dict(v=None), NUL), (dict(k_scale=None), NUL), (dict(v_scale=None), NUL),
             (dict(num_pages=0), SHAPE), (dict(num_pages=-1), SHAPE), (dict(num_pages=2 ** 31), SHAPE),
             (dict(kv_heads=0), SHAPE), (dict(kv_heads=65536), SHAPE), (dict(head_dim=96), SHAPE),
             (dict(head_dim=0), SHAPE), (dict(head_dim=512), SHAPE), (dict(page_size=8), SHAPE),
             (dict(page_size=48), SHAPE), (dict(page_size=2048), SHAPE), (dict(page_size=-16), SHAPE),
             (dict(format=2), ARG), (dict(format=-1), ARG), (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 4), ALIGN),
             (dict(k_scale=FAKE + 4), ALIGN), (dict(v_scale=FAKE + 8), ALIGN)]
BAD_BATCH = [(dict(page_table=None), NUL), (dict(row_start=None), NUL), (dict(kv_len=None), NUL), (dict(T=0), SHAPE),
             (dict(T=-1), SHAPE), (dict(T=2 ** 24), SHAPE), (dict(B=0), SHAPE), (dict(B=65536), SHAPE),
             (dict(max_pages=0), SHAPE), (dict(max_pages=2 ** 26 + 1), SHAPE), (dict(page_table=FAKE + 2), ALIGN),
             (dict(row_start=FAKE + 1), ALIGN), (dict(kv_len=FAKE + 2), ALIGN)]


def kv_calls(c, b):
    return [call("kv_write", ref(c), ref(b), FAKE, 512, FAKE, 512, S),
            call("kv_read", ref(c), ref(b), FAKE, 512, FAKE, 512, S),
            call("attn_paged", ref(c), ref(b), FAKE, 4096, FAKE, 4096, 8, 0.1, 0, FAKE, BIG, S)]


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_cache_descriptor(kw, want):
    c = cache(**kw)
    assert kv_calls(c, batch()) == [want] * 3
    if want in (SHAPE, ARG):
        assert call("attn_paged_ws_bytes", ref(c), ref(batch()), 8) == 0


@pytest.mark.parametrize("kw,want", BAD_BATCH)
def test_batch_descriptor(kw, want):
    b = batch(**kw)
    assert kv_calls(cache(), b) == [want] * 3
    if want == SHAPE:
        assert call("attn_paged_ws_bytes", ref(cache()), ref(b), 8) == 0


def test_float16_cache_needs_no_scales_but_its_planes():
    c = cache(format=1, k_scale=None, v_scale=None, v=None)
    assert kv_calls(c, batch()) == [NUL] * 3


def test_descriptors_missing():
    assert kv_calls(None, batch()) == [NUL] * 3
    assert kv_calls(cache(), None) == [NUL] * 3
    assert call("attn_paged_ws_bytes", None, ref(batch()), 8) == 0
    assert call("attn_paged_ws_bytes", ref(cache()), None, 8) == 0


@pytest.mark.parametrize("name", ["kv_write", "kv_read"])
def test_kv_rows(name):
    c, b = cache(), batch()
    assert call(name, ref(c), ref(b), None, 512, FAKE, 512, S) == NUL
    assert call(name, ref(c), ref(b), FAKE, 512, None, 512, S) == NUL
    assert call(name, ref(c), ref(b), FAKE, 511, FAKE, 512, S) == SHAPE
    assert call(name, ref(c), ref(b), FAKE, 512, FAKE, -512, S) == SHAPE
    assert call(name, ref(c), ref(b), FAKE, 2 ** 61, FAKE, 512, S) == SHAPE
    assert call(name, ref(c), ref(b), FAKE + 2, 512, FAKE, 512, S) == ALIGN
    assert call(name, ref(c), ref(b), FAKE, 512, FAKE + 1, 512, S) == ALIGN


def test_attn_arguments():
    c, b = cache(), batch()
    need = call("attn_paged_ws_bytes", ref(c), ref(b), 8)
    assert need > 0
    good = [ref(c), ref(b), FAKE, 1024, FAKE, 1024, 8, 0.1, 0, FAKE, need, S]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return call("attn_paged", *a)

    assert with_(2, None) == NUL and with_(4, None) == NUL and with_(9, None) == NUL
    assert with_(3, 1023) == SHAPE and with_(5, 1023) == SHAPE
    assert with_(6, 0) == SHAPE and with_(6, 6) == SHAPE and with_(6, 4 * 65) == SHAPE and with_(6, -8) == SHAPE
    assert with_(7, float("nan")) == ARG and with_(7, float("inf")) == ARG and with_(8, -1) == ARG
    assert with_(2, FAKE + 2) == ALIGN and with_(4, FAKE + 2) == ALIGN and with_(9, FAKE + 8) == ALIGN
    assert with_(10, need - 1) == WS
    big = cache(kv_heads=64)
    assert call("attn_paged_ws_bytes", ref(big), ref(batch(T=2 ** 23, B=2)), 4096) == 0  # too many workgroups
    assert call("attn_paged", ref(big), ref(batch(T=2 ** 23, B=2)), FAKE, 2 ** 19, FAKE, 2 ** 19, 4096, 0.1, 0, FAKE, BIG,
                S) == SHAPE
    for heads in (0, 6, 4 * 65, -4):
        assert call("attn_paged_ws_bytes", ref(c), ref(b), heads) == 0


def test_attn_workspace_is_bounded():
    """It holds partial results of a bounded number of workgroups, not of positions."""
    small = call("attn_paged_ws_bytes", ref(cache()), ref(batch(T=1, B=1, max_pages=4)), 8)
    long = call("attn_paged_ws_bytes", ref(cache(num_pages=2 ** 20)), ref(batch(T=1, B=1, max_pages=2 ** 20)), 8)
    assert 0 < small <= long < 256 << 20


def test_norm_arguments():
    n = lambda *a: call("rmsnorm_add", *a)
    q = lambda *a: call("rmsnorm_add_q8", *a)
    assert n(None, FAKE, FAKE, FAKE, FAKE, 64, 1, 1e-6, S) == NUL
    assert n(FAKE, FAKE, None, FAKE, FAKE, 64, 1, 1e-6, S) == NUL
    assert n(FAKE, FAKE, FAKE, FAKE, None, 64, 1, 1e-6, S) == NUL
    assert q(FAKE, FAKE, FAKE, FAKE, None, FAKE, 64, 1, 1e-6, S) == NUL
    assert q(FAKE, FAKE, FAKE, FAKE, FAKE, None, 64, 1, 1e-6, S) == NUL
    for K, M in ((0, 1), (-64, 1), (64, 0), (64, 65536), (2 ** 31, 1)):
        assert n(FAKE, FAKE, FAKE, FAKE, FAKE, K, M, 1e-6, S) == SHAPE
        assert q(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, K, M, 1e-6, S) == SHAPE
    assert q(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 48, 1, 1e-6, S) == SHAPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert n(FAKE, FAKE, FAKE, FAKE, FAKE, 64, 1, eps, S) == ARG
        assert q(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 64, 1, eps, S) == ARG
    for i in (0, 1, 2, 3, 4):
        a = [FAKE] * 5 + [64, 1, 1e-6, S]
        a[i] = FAKE + 2
        assert n(*a) == ALIGN
    for i in range(6):
        a = [FAKE] * 6 + [64, 1, 1e-6, S]
        a[i] = FAKE + 2
        assert q(*a) == ALIGN


def test_qmm_q8_arguments():
    f = lambda *a: call("qmm_q4_0_q8", *a)
    for shape in ((300, 2048, 1), (300, 2048, 16), (4096, 256, 512), (70, 96, 3)):
        need = call("qmm_q4_0_q8_ws_bytes", *shape)
        assert need == call("qmm_q4_0_q8act_ws_bytes", *shape) > 0
        assert f(FAKE, FAKE, FAKE, FAKE, *shape, FAKE, need - 1, S) == WS
    assert call("qmm_q4_0_q8_ws_bytes", 0, 64, 1) == 0
    good = [FAKE, FAKE, FAKE, FAKE, 64, 256, 2, FAKE, BIG, S]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return f(*a)

    for i in (0, 1, 2, 3, 7):
        assert with_(i, None) == NUL
    assert with_(4, 0) == SHAPE and with_(5, 40) == SHAPE and with_(6, 65536) == SHAPE
    for i, off in ((0, 8), (1, 4), (2, 2), (3, 2), (7, 8)):
        assert with_(i, FAKE + off) == ALIGN


def test_draft_arguments():
    need = call("draft_verify_ws_bytes", 2, 4, 1000)
    assert need > 0
    #        target ld   draft ld   tokens n     u     acc   out   B G V     T    cap  ws    bytes
    good = [FAKE, 1000, FAKE, 1000, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 1000, 1.0, 0.0, FAKE, need, S]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return call("draft_verify", *a)

    for i in (0, 2, 4, 6, 7, 8, 14):
        assert with_(i, None) == NUL
    assert with_(1, 999) == SHAPE and with_(3, 999) == SHAPE and with_(1, 2 ** 61) == SHAPE
    for i, vals in ((9, (0, -1, 65536)), (10, (0, -1, 65)), (11, (0, -5, 2 ** 31))):
        for v in vals:
            assert with_(i, v) == SHAPE
    for v in (0.0, -1.0, float("nan"), float("inf")):
        assert with_(12, v) == ARG
    for v in (-1.0, float("nan"), float("inf")):
        assert with_(13, v) == ARG
    for i in (0, 2, 4, 5, 6, 7, 8):
        assert with_(i, FAKE + 2) == ALIGN
    assert with_(14, FAKE + 8) == ALIGN
    assert with_(15, need - 1) == WS
    assert call("draft_verify_ws_bytes", 0, 4, 1000) == 0
    assert call("draft_verify_ws_bytes", 2, 65, 1000) == 0
    assert call("draft_verify_ws_bytes", 2, 4, 0) == 0


@pytest.mark.parametrize("cap,ok", [(65536.0, True), (65537.0, False), (1e9, False), (3e38, False)])
def test_draft_softcap_has_a_largest_value(cap, ok):
    # the workspace is checked last: a call that gets there has passed the cap
    rc = call("draft_verify", FAKE, 1000, FAKE, 1000, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 1000, 1.0, cap, FAKE, 1, S)
    assert rc == (WS if ok else ARG)


def test_binding_refuses_tensors_of_the_host():
    """An address in host memory would fault the GPU."""
    t = torch.zeros(64)
    c = torch.zeros(2, 1, 16, 64, dtype=torch.int8)
    s = torch.zeros(2, 1, 16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        qmv.rmsnorm_add(t, None, t, None, t, 64, 1, 1e-6, stream=0)
    with pytest.raises(ValueError):
        qmv.KVCache(c, c, s, s)
    with pytest.raises(ValueError):
        qmv.KVBatch(torch.zeros(1, 2, dtype=torch.int32), i, i[:1], 1)


def test_binding_checks_descriptors():
    c = torch.zeros(2, 1, 16, 64, dtype=torch.int8)
    s = torch.zeros(2, 1, 16)
    for args in ((c, c), (c, c, s, None), (c, c, s, s.double()), (c, c, s[:1], s), (c.half(), c.half(), s, s),
                 (c, c.half(), s, s), (c.float(), c.float()), (c[0], c[0], s[0], s[0])):
        with pytest.raises(ValueError, match="int8|float16|scale"):
            qmv.KVCache(*args)
    t = torch.zeros(2, 3, dtype=torch.int32)
    i = torch.zeros(3, dtype=torch.int32)
    for args in ((t.long(), i, i[:2]), (t, i[:2], i[:2]), (t, i, i), (t[0], i, i[:2])):
        with pytest.raises(ValueError, match="int32|entries"):
            qmv.KVBatch(*args, 1)


def test_binding_refuses_descriptors_of_another_gpu(monkeypatch):
    """Made while one GPU was current, used while another is."""
    monkeypatch.setattr(qmv, "_device", lambda: 0)
    objects = []
    for cls, device in ((qmv.KVCache, 0), (qmv.KVCache, 1), (qmv.KVBatch, 0), (qmv.KVBatch, 1)):
        o = cls.__new__(cls)
        o.ref, o.device = FAKE, device
        objects.append(o)
    c0, c1, b0, b1 = objects
    assert qmv._desc(c0, b0) == (FAKE, FAKE)
    for c, b in ((c1, b0), (c0, b1), (c1, b1)):
        with pytest.raises(ValueError, match="another GPU"):
            qmv.kv_write(c, b, FAKE, 64, FAKE, 64, stream=0)
        with pytest.raises(ValueError, match="another GPU"):
            qmv.kv_read(c, b, FAKE, 64, FAKE, 64, stream=0)
        with pytest.raises(ValueError, match="another GPU"):
            qmv.attn_paged(c, b, FAKE, 64, FAKE, 64, 1, 1.0, 0, FAKE, 256, stream=0)
