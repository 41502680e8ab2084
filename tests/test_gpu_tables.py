"""GPU: block tables and slots built on the device against the request-by-request model."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import sparse  # noqa: E402
from tests.sparse_checks import i32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib.device_error(clear=True)
    return lib


class Step:
    """Buffers of one step and the call."""

    def __init__(self, n, tokens, width):
        def full(*shape, dtype=torch.int32):
            return torch.full(shape, -77, dtype=dtype, device="cuda")

        self.tables, self.ctx, self.start = full(n, width), full(n), full(n + 1)
        self.slots, self.pos = full(tokens, dtype=torch.int64), full(tokens)

    def call(self, pkv, dt, rows, cached, new, **kw):
        pkv.pkv_tables_step(dt, rows, cached, new, self.tables, self.ctx, self.start, self.slots,
                            self.pos, **kw)
        return self

    def check(self, ctx, start, slots, pos, tables):
        assert np.array_equal(self.ctx.cpu().numpy(), ctx)
        assert np.array_equal(self.start.cpu().numpy(), start)
        assert np.array_equal(self.slots.cpu().numpy(), slots)
        assert np.array_equal(self.pos.cpu().numpy(), pos)
        assert np.array_equal(self.tables.cpu().numpy(), tables)


def _same_state(dt, model):
    assert np.array_equal(dt.block_table.cpu().numpy(), model.table)
    n = int(dt.free_count.item())
    assert dt.free_list[:n].cpu().tolist() == model.free


# in place the step is two launches, with a count of its own one (up to 2048 requests)
IN_PLACE = pytest.mark.parametrize("in_place", [True, False])


def _count(dt, in_place):
    return {} if in_place else dict(free_count_out=torch.full_like(dt.free_count, -3))


def _settle(dt, kw):
    """The caller takes over a count that was written apart."""
    if kw:
        dt.free_count.copy_(kw["free_count_out"])


@IN_PLACE
@pytest.mark.parametrize("bs,rows,width,chunk,seed", [(16, 40, 9, 40, 0), (4, 12, 70, 3, 1),
                                                      (1, 5, 64, 20, 2), (16, 3000, 5, 18, 3),
                                                      (7, 33, 257, 600, 4), (16, 900, 300, 70, 5)])
def test_random_steps_and_releases_match_the_model(pkv, bs, rows, width, chunk, seed, in_place):
    rng = np.random.default_rng(seed)
    nb = rows * max(2, min(width, 2 * chunk // bs + 2))
    order = rng.permutation(nb)
    model = sparse.TablesModel(nb, bs, rows, width, order)
    dt = pkv.DeviceTables.create(nb, bs, rows, width, order)
    lens = np.zeros(rows, dtype=np.int64)
    for it in range(12):
        n = int(rng.integers(1, rows + 1))
        pick = rng.permutation(rows)[:n]
        new = rng.integers(0, chunk + 1, n) if it % 3 else np.ones(n, dtype=np.int64)
        fits = lens[pick] + new <= width * bs
        pick, new = pick[fits], new[fits]
        need = (-(-(lens[pick] + new) // bs) + lens[pick] // -bs).sum()
        if need > len(model.free) or len(pick) == 0:
            live = np.flatnonzero(lens)
            live = rng.permutation(live)[:max(1, len(live) // 2)]
            pkv.pkv_tables_release(dt, i32(live), i32(lens[live]))
            model.release(live, lens[live])
            lens[live] = 0
            _same_state(dt, model)
            continue
        tokens = int(new.sum()) + int(rng.integers(0, 40))
        step = Step(len(pick), tokens, width)
        ref = model.step(pick, lens[pick], new, tokens, width)
        kw = _count(dt, in_place)
        step.call(pkv, dt, i32(pick), i32(lens[pick]), None if it % 3 == 0 else i32(new), **kw)
        _settle(dt, kw)
        step.check(*ref)
        _same_state(dt, model)
        lens[pick] += new
    assert pkv.device_error() == 0


def test_rows_in_order_without_row_list_or_optional_outputs(pkv):
    dt = pkv.DeviceTables.create(20, 16, 4, 5)
    model = sparse.TablesModel(20, 16, 4, 5)
    cached, new = [0, 16, 5], [17, 1, 0]
    model.step([1], [0], [16], 16, 5)
    model.step([2], [0], [5], 5, 5)
    s = Step(1, 16, 5)
    s.call(pkv, dt, i32([1]), i32([0]), i32([16]))
    s = Step(1, 5, 5)
    s.call(pkv, dt, i32([2]), i32([0]), i32([5]))
    s = Step(3, 18, 5)
    pkv.pkv_tables_step(dt, None, i32(cached), i32(new), None, s.ctx, s.start, s.slots)
    ref = model.step(None, cached, new, 18, 5)
    assert s.ctx.tolist() == ref[0].tolist() and s.start.tolist() == ref[1].tolist()
    assert s.slots.tolist() == ref[2].tolist()
    assert (s.pos == -77).all() and (s.tables == -77).all()
    _same_state(dt, model)
    assert pkv.device_error() == 0


def test_a_separate_count_leaves_the_step_repeatable(pkv):
    dt = pkv.DeviceTables.create(30, 4, 3, 8)
    count = torch.empty(1, dtype=torch.int32, device="cuda")
    got = []
    for _ in range(2):
        s = Step(3, 24, 8)
        s.call(pkv, dt, None, i32([0, 0, 0]), i32([5, 9, 1]), free_count_out=count)
        got.append([t.clone() for t in (s.tables, s.ctx, s.start, s.slots, s.pos, count)])
    assert dt.free_count.item() == 30 and count.item() == 30 - (2 + 3 + 1)
    for a, b in zip(*got):
        assert torch.equal(a, b)


@IN_PLACE
def test_requests_that_do_not_fit_wait(pkv, in_place):
    """Blocks, then token rows, run out: the rest of the batch waits and is served
    after a release."""
    model, dt = sparse.TablesModel(6, 4, 5, 4), pkv.DeviceTables.create(6, 4, 5, 4)
    rows, cached, new = [4, 0, 2, 1, 3], [0] * 5, [8, 9, 5, 0, 1]     # 2 + 3 + 2 ... blocks
    ref = model.step(rows, cached, new, 30, 4)
    kw = _count(dt, in_place)
    s = Step(5, 30, 4).call(pkv, dt, i32(rows), i32(cached), i32(new), **kw)
    _settle(dt, kw)
    assert pkv.device_error() == 10                                   # PKV_DEV_NO_FREE_BLOCKS
    s.check(*ref)
    assert ref[0].tolist() == [8, 9, 0, 0, 0]
    _same_state(dt, model)
    pkv.pkv_tables_release(dt, i32([4]), i32([8]))
    model.release([4], [8])
    ref = model.step([2, 3], [0, 0], [5, 1], 5, 4)                    # the last token has no room
    kw = _count(dt, in_place)
    s = Step(2, 5, 4).call(pkv, dt, i32([2, 3]), i32([0, 0]), i32([5, 1]), **kw)
    _settle(dt, kw)
    assert pkv.device_error() == 5                                    # PKV_DEV_BAD_QUERY_LAYOUT
    s.check(*ref)
    assert ref[0].tolist() == [5, 0]
    _same_state(dt, model)


@IN_PLACE
@pytest.mark.parametrize("rows,cached,new,code", [
    ([0, 9, 2], [0, 0, 0], [3, 3, 3], 9), ([0, -1, 2], [0, 0, 0], [3, 3, 3], 9),
    ([2, 0, 2], [0, 0, 0], [3, 3, 3], 9), ([0, 1, 2], [0, -4, 0], [3, 3, 3], 2),
    ([0, 1, 2], [0, 0, 0], [3, -3, 3], 2), ([0, 1, 2], [0, 0, 0], [3, 17, 3], 7),
    ([0, 1, 2], [0, 2**31 - 1, 0], [3, 2**31 - 1, 3], 7),
])
def test_bad_requests_are_skipped_and_flagged(pkv, rows, cached, new, code, in_place):
    model, dt = sparse.TablesModel(12, 4, 4, 4), pkv.DeviceTables.create(12, 4, 4, 4)
    ref = model.step(rows, cached, new, 12, 4)
    kw = _count(dt, in_place)
    s = Step(3, 12, 4).call(pkv, dt, i32(rows), i32(cached), i32(new), **kw)
    _settle(dt, kw)
    assert pkv.device_error() == code
    s.check(*ref)
    _same_state(dt, model)


@IN_PLACE
def test_bad_free_list_and_count(pkv, in_place):
    dt = pkv.DeviceTables.create(4, 4, 2, 4, free_order=[0, 1, 2, 3])
    dt.free_count.fill_(9)
    kw = _count(dt, in_place)
    s = Step(1, 4, 4).call(pkv, dt, i32([0]), i32([0]), i32([4]), **kw)
    _settle(dt, kw)
    assert pkv.device_error() == 1                                    # PKV_DEV_BAD_BLOCK_ID
    assert s.ctx.tolist() == [0] and dt.free_count.item() == 9
    dt.free_count.fill_(4)
    dt.free_list[3] = 55
    s = Step(1, 4, 4).call(pkv, dt, i32([0]), i32([0]), i32([4]), **_count(dt, in_place))
    assert pkv.device_error() == 1
    assert s.slots.tolist() == [-1] * 4                               # appends skip them


def test_release_refuses_rows_it_released(pkv):
    dt = pkv.DeviceTables.create(8, 4, 3, 4)
    Step(2, 10, 4).call(pkv, dt, i32([0, 2]), i32([0, 0]), i32([6, 4]))
    for rows, lens in (([0, 0], [6, 6]), ([5], [4]), ([-1], [4])):
        pkv.pkv_tables_release(dt, i32(rows), i32(lens))
        assert pkv.device_error() == 9
    pkv.pkv_tables_release(dt, i32([2]), i32([-1]))
    assert pkv.device_error() == 2
    pkv.pkv_tables_release(dt, i32([2]), i32([17]))
    assert pkv.device_error() == 7
    pkv.pkv_tables_release(dt, i32([2]), i32([5]))                    # holds one block, not two
    assert pkv.device_error() == 9
    assert dt.free_count.item() == 5
    pkv.pkv_tables_release(dt, i32([2, 0]), i32([4, 6]))
    assert pkv.device_error() == 0 and dt.free_count.item() == 8
    assert (dt.block_table == -1).all()
    pkv.pkv_tables_release(dt, i32([2]), i32([4]))
    assert pkv.device_error() == 9 and dt.free_count.item() == 8


def test_empty_batch_writes_the_padding(pkv):
    dt = pkv.DeviceTables.create(8, 4, 3, 4)
    count = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    s = Step(0, 3, 4)
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    s.call(pkv, dt, None, empty, empty, free_count_out=count)
    assert s.start.tolist() == [0] and count.item() == 8
    assert s.slots.tolist() == [-1] * 3 and s.pos.tolist() == [0] * 3
    assert pkv.device_error() == 0


def test_lengths_in_place_under_a_captured_graph(pkv):
    """A decode loop that never returns to the host: the lengths and the count are
    updated in place by every replay."""
    n, bs, width, steps = 37, 16, 6, 50
    rng = np.random.default_rng(8)
    rows = rng.permutation(50)[:n]
    lens0 = rng.integers(0, 40, n)
    dt = pkv.DeviceTables.create(50 * width, bs, 50, width)
    model = sparse.TablesModel(50 * width, bs, 50, width)
    model.step(rows, [0] * n, lens0, 4000, width)
    Step(n, 4000, width).call(pkv, dt, i32(rows), i32([0] * n), i32(lens0))
    lens, rows_d = i32(lens0), i32(rows)
    s = Step(n, n, width)
    s.ctx = lens
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        s.call(pkv, dt, rows_d, lens, None)
    for i in range(steps):
        g.replay()
    torch.cuda.synchronize()
    for i in range(steps):
        ref = model.step(rows, lens0 + i, None, n, width)
    s.check(*ref)
    _same_state(dt, model)
    assert pkv.device_error() == 0
