"""attn_paged over 8-bit keys of small codes: pages filled by other means than
kv_write need not use the codes' range, and a score must not be rounded to a
step that only rows with a code of 127 can afford.  The bound is
step_ref.attention's (its value term needs codes of 64 or more, which the
values here have)."""
import numpy as np
import pytest

from test_gpu_step_attn import Call, both

pytestmark = pytest.mark.gpu


@both
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", ["one code of 1", "codes of -1, 0, 1", "one code of 127", "codes to -128"])
def test_keys_of_small_codes(kind, dim, wide):
    c = Call([300, 40], [2, 1], 4, 2, dim, 16, "q8", seed=dim, scale=1.0, wide=wide)
    rng = np.random.default_rng(dim)
    shape = c.P.k.shape
    if kind == "one code of 1" or kind == "one code of 127":
        k = np.zeros(shape, np.int8)
        at = rng.integers(0, dim, shape[:3])
        np.put_along_axis(k, at[..., None], 1 if kind == "one code of 1" else 127, axis=3)
        spread = 25.0 if kind == "one code of 1" else 25.0 / 127
    elif kind == "codes of -1, 0, 1":
        k, spread = rng.integers(-1, 2, shape).astype(np.int8), 25.0 / dim ** 0.5
    else:
        k, spread = rng.integers(-128, 128, shape).astype(np.int8), 0.3 / dim ** 0.5
    c.P.k[:] = k
    seen = ~np.isnan(c.P.ks)
    c.P.ks[seen] = (rng.random(int(seen.sum())) + 0.5).astype(np.float32) * np.float32(spread)
    c.check(f"{kind}, D {dim}")


@both
def test_large_queries_of_alternating_sign(wide):
    """The digits' sums are as large as they get: every code -128 or 127 against queries near their largest magnitude."""
    c = Call([200], [2], 4, 2, 256, 16, "q8", seed=3, scale=1e-6, wide=wide)
    rng = np.random.default_rng(4)
    c.P.k[:] = np.where(rng.random(c.P.k.shape) < 0.5, -128, 127).astype(np.int8)
    c.q[:] = np.where(rng.random(c.q.shape) < 0.5, -1.0, 1.0).astype(np.float32) * rng.uniform(0.98, 1.0, c.q.shape).astype(np.float32)
    c.P.k[c.P.table[0, 1], :] = 127
    c.P.k[c.P.table[0, 2], :] = -128
    c.q[:, :256] = 1.0
    c.q[:, 256:512] = -1.0
    c.scale = 0.02
    c.check("largest sums")
