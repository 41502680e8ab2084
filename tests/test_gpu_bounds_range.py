"""GPU: key bounds and scores at the ends of their arithmetic, against the float64
restatement."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import sparse  # noqa: E402
from tests.sparse_checks import i32, to_dev  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib.device_error(clear=True)
    return lib


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("large", [1.0, 300.0, 2.0 ** 40, 2.0 ** 57, 3e38])
def test_tiny_keys_beside_large_ones_are_rounded_outwards(pkv, dtype, d, large):
    """A dimension whose keys are far below the block's unit, down to the least
    subnormal: its upper end is 1 where a key is positive, its lower one -1 where a
    key is negative."""
    tiny = [2.0 ** -149 if dtype == "f32" else 2.0 ** -133, 2.0 ** -126, 2.0 ** -110, 2.0 ** -60]
    k = np.zeros((4, 1, 16, d), dtype=np.float32)
    k[:, 0, 2, 0] = large
    k[1, 0, 9, 0] = -large
    for i, x in enumerate(tiny):
        k[:, 0, i, 1 + i] = x                      # zeros below it
        k[:, 0, i, 11 + i] = -x                    # zeros above it
        k[:, 0, :, 21 + i], k[:, 0, :, 31 + i] = x, -x
        k[:, 0, :8, 41 + i], k[:, 0, 8:, 41 + i] = x, -x
    if dtype == "bf16":
        k = (k.view(np.uint32) >> 16).astype(np.uint16)
    t = np.arange(4, dtype=np.int32)[:, None]
    kd = to_dev(k, dtype)
    bounds, exps = np.zeros((4, 1, 2, d), np.int8), np.zeros((4, 1), np.int8)
    b_d, e_d = to_dev(bounds), to_dev(exps)
    pkv.pkv_block_bounds(b_d, e_d, kd, pkv.cache_desc(kd, 1), i32(t), i32([16] * 4))
    assert pkv.device_error() == 0
    sparse.update_bounds(bounds, exps, k, t, np.arange(5), [16] * 4, dtype)
    assert np.array_equal(e_d.cpu().numpy(), exps)
    assert np.array_equal(b_d.cpu().numpy(), bounds)
    assert (bounds[0, 0, 0, 1:5] == 1).all() and (bounds[0, 0, 1, 11:15] == -1).all()
