"""GPU: softmax weights keep all their bits through the sparse attention's products."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.sparse_checks import EXP2_REL, ROUND, i32, to_dev  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib.device_error(clear=True)
    return lib


def _leading_bits(x):
    """x cut to the eight leading bits that a bf16 value holds."""
    return (x.astype(np.float32).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)


@pytest.mark.parametrize("dtype,hq", [("bf16", 1), ("bf16", 4), ("bf16", 8), ("f32", 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_the_last_bits_of_a_weight_reach_the_output(pkv, dtype, hq, d):
    """Three keys a row: two of weight 1 whose values are minus the weight w's leading
    sixteen bits, one of weight w and value 1.  The output is what is left of w,
    (w - b0 - b1) / (2 + w), below 2^-15 w; sums and products on the way are exact.

    The score s of the third key is exact; the factor log2 e and its product with s
    are rounded, so the exponent x is off by 2^-23 |x| at most, which moves w by ln 2
    times that, exp2 by EXP2_REL: those times w / (2 + w), relative to the
    denominator 2^-23 of the output, and half a step of its type.
    """
    rows = 64
    # scores of 2^-7 .. 2 in steps that bf16 holds, all with the same sign
    s = -np.arange(1, rows * hq + 1).reshape(rows, hq) / 128.0 if hq == 1 else \
        -(1.0 + np.arange(rows * hq).reshape(rows, hq) % 128) / 64.0
    w = np.exp(s)
    b0 = _leading_bits(w)
    b1 = _leading_bits((w - b0).astype(np.float32))
    out = np.zeros((rows, hq, d))
    k = np.zeros((rows, 1, 16, d), np.float32)
    v = np.full((rows, 1, 16, d), np.nan, np.float32)
    k[:, 0, 2, 0] = 1.0
    v[:, 0, :3] = 0.0
    # head g has its value in dimension g alone, and elsewhere those of the others
    for g in range(hq):
        v[:, 0, 0, g], v[:, 0, 1, g], v[:, 0, 2, g] = -b0[:, g], -b1[:, g], 1.0
    q = np.zeros((rows, hq, d), np.float32)
    q[:, :, 0] = s
    if dtype == "bf16":
        for x in (k, v[:, :, :3], q):
            assert np.array_equal(_leading_bits(x), x)
        k, v, q = ((x.view(np.uint32) >> 16).astype(np.uint16) for x in (k, v, q))
    kd, vd, qd = to_dev(k, dtype), to_dev(v, dtype), to_dev(q, dtype)
    table = i32(np.arange(rows)[:, None])
    sel = i32(np.zeros((rows, 1, 1)))
    got = pkv.paged_attention_sparse(torch.empty_like(qd), qd, kd, vd, pkv.cache_desc(kd, hq),
                                     table, i32([3] * rows), sel, scale=1.0)
    assert pkv.device_error() == 0
    got = got.float().cpu().numpy().astype(np.float64)
    for g in range(hq):
        ref = (w[:, g] - b0[:, g].astype(np.float64) - b1[:, g]) / (2.0 + w[:, g])
        x = np.abs(s[:, g]) * np.log2(np.e)
        off = (np.log(2.0) * x * 2.0 ** -23 + EXP2_REL) * w[:, g] / (2.0 + w[:, g])
        bound = off + (2.0 ** -22 + ROUND[dtype]) * (np.abs(ref) + off)
        err = np.abs(got[:, g, g] - ref)
        assert (err <= bound).all(), (err / bound).max()
