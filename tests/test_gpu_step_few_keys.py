"""attn_paged where a row sees one key or a few: nothing averages the rounding of
a weight out."""
import numpy as np
import pytest

import step_ref as R
from gpu_util import assert_within, say
from test_gpu_step_attn import Call, both

pytestmark = pytest.mark.gpu


@both
@pytest.mark.parametrize("fmt", ["q8", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_key(dim, fmt, wide):
    """The weight is the sum of the weights, so the result is the value but for roundings: of p times the value's
    scale (half a step, 1 eps = 2^-24), its two float16 terms (each to 2^-11 of what is left: 2^-22, 4 eps), their
    products' sum (two additions) and the division: 8 eps."""
    c = Call([1] * 20, [1] * 20, 32, 16, dim, 16, fmt, seed=dim, wide=wide)
    say(f"one key {fmt} D {dim}")
    c.upload()
    c.enqueue()
    got = c.result()[:, : c.width].reshape(20, 16, 2, dim)
    v = np.stack([c.P.rows("v", b)[0] for b in range(20)])[:, :, None]
    assert_within(got, np.broadcast_to(v, got.shape), np.broadcast_to(8 * R.EPS32 * np.abs(v) + 1e-30, got.shape), "one key")


@both
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seed", range(2))
@pytest.mark.parametrize("spread", [1.0, 0.003])
def test_few_keys_of_small_values(spread, seed, dim, wide):
    """step_ref.attention's bound over values of 2^-4 down to 2^-33."""
    lens = [2, 3, 4, 5, 9]
    c = Call(lens, lens, 256, 16, dim, 16, "q8", seed=seed, q_scale=0.05, spread=spread, wide=wide)
    rng = np.random.default_rng(seed)
    seen = ~np.isnan(c.P.vs)
    c.P.vs[seen] *= (10.0 ** rng.uniform(-6, 0, int(seen.sum()))).astype(np.float32)
    c.check(f"few keys, D {dim}, values {spread}")
