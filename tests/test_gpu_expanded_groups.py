"""GPU: attention over expanded keys with so many units that neighbouring ones of a sequence
are planned in groups of four and taken head by head."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import latent  # noqa: E402
from tests.latent_checks import assert_close, expanded_bound  # noqa: E402
from tests.test_gpu_expanded import Case, pkv  # noqa: E402, F401

pytestmark = pytest.mark.gpu


# rows: of a unit.  Sequences of one to eleven units, in and out of fours, some of whose first
# queries (a whole unit of them and a part) see no key
@pytest.mark.parametrize("dtype,d,h,rows,new,keys", [
    ("bf16", 64, 160, 256, [1500, 257, 1, 0, 300, 1100, 600], [1500, 400, 9, 5, 20, 1111, 333]),
    ("bf16", 128, 112, 256, [1281, 513, 40, 1024], [1281, 900, 700, 700]),
    ("bf16", 128, 1250, 256, [255], [300]),       # a unit a head, and no more
    ("f32", 64, 80, 64, [700, 65, 0, 1, 256, 129], [700, 90, 3, 1, 100, 400]),
    ("f32", 128, 80, 64, [300, 449, 1, 193, 64, 63], [333, 449, 30, 100, 64, 80]),
    ("f32", 128, 124, 128, [641, 600], [641, 350]),
])
def test_groups_of_units(pkv, dtype, d, h, rows, new, keys):  # noqa: F811
    c = Case(np.random.default_rng(h), dtype, h, d, new, keys)
    tokens, sms = c.q.shape[0], torch.cuda.get_device_properties(0).multi_processor_count
    assert -(-tokens // rows) * h >= 8 * sms                  # grouped
    if dtype == "f32":                                        # and with this many rows a unit
        assert tokens * h // 64 >= 2 * sms
        assert rows == (128 if d == 128 and -(-tokens // len(new)) >= 512 else 64)
    out, code = c.run(pkv)
    assert code == 0
    assert torch.isfinite(out[:c.qs[-1]]).all() and (out[c.qs[-1]:] == 7.0).all()
    for s, (m, n) in enumerate(zip(new, keys)):
        if m > n:
            assert (out[c.qs[s]:c.qs[s] + m - n] == 0).all()
    # every row of the first, a middle and the last head
    pick = sorted({0, h // 2 + 1, h - 1})
    args = (np.ascontiguousarray(c.q[:, pick]), np.ascontiguousarray(c.kv[:, pick, :d]),
            np.ascontiguousarray(c.kv[:, pick, d:]), c.r, c.qs, c.ks, c.scale, dtype)
    ref = latent.expanded(*args)
    assert_close(out[:, pick], ref, expanded_bound(*args, ref))
    again, _ = c.run(pkv, ws_byte=0x11)
    assert torch.equal(out, again)
