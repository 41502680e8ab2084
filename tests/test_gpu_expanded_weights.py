"""GPU: the weights that attention over expanded keys multiplies its values with are the ones
that it sums, so that values which are all the same come back as they are."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle.numerics import widen  # noqa: E402
from tests.gpu_parity import gamma  # noqa: E402
from tests.sparse_checks import ROUND, values  # noqa: E402
from tests.test_gpu_expanded import Case, pkv  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heavy", [False, True])
@pytest.mark.parametrize("h,new,keys", [(2, [140, 9], [140, 300]), (3, [400], [400]),
                                        (2, [40], [1300]), (50, [20], [1100])])
def test_equal_values_come_back(pkv, dtype, d, heavy, h, new, keys):  # noqa: F811
    """A weighted mean of equal values is the value: numerator and denominator are sums of the
    same terms, at most n of them, each off by gamma_{2 n + 304} of itself (twice that for
    tensor-core sums that cut).  For bf16 that is far less than half the smaller distance
    between two values (2^-9), so that the output's rounding gives the value itself.
    heavy: key 130 of a sequence, behind the first tile, outweighs the others by up to
    2^7.5, a factor that is no bf16 number and differs from query to query."""
    rng = np.random.default_rng(h + d)
    c = Case(rng, dtype, h, d, new, keys, k_scale=0.1 if heavy else 1.0)
    n = max(keys)
    slack = 2 * 2 * gamma(2 * n + 304)
    assert dtype == "f32" or slack < 2.0 ** -9
    c.kv[:c.ks[-1], :, d:] = values(rng, (h, d), dtype)[None]
    if heavy:
        at = [k for k in c.ks[:-1] + 130 if k < c.ks[-1]]
        c.r[:c.ks[-1], 0] = 0
        c.r[at, 0] = 0x3F80 if dtype == "bf16" else 1.0
        up = (rng.uniform(0, 7.5, c.q.shape[:2]) * np.log(2.0) / c.scale).astype(np.float32)
        c.q[..., d] = (up.view(np.uint32) >> 16).astype(np.uint16) if dtype == "bf16" else up
    want = widen(c.kv[0, :, d:], dtype)
    out, code = c.run(pkv)
    assert code == 0
    got = out[:c.qs[-1]].float().cpu().numpy().astype(np.float64)
    if dtype == "bf16":
        assert (got == want).all(), int((got != want).sum())
    else:
        assert (np.abs(got - want) <= (ROUND[dtype] + slack) * np.abs(want)).all()
