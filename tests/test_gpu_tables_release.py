"""GPU: releases of device table rows whose entries are not all blocks of the pool."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.sparse_checks import i32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib.device_error(clear=True)
    return lib


def _serve(pkv, dt, rows, lens):
    """Rows of an empty pool get the blocks of `lens` tokens each."""
    n, width = len(rows), dt.block_table.shape[1]
    out = torch.empty((n, width), dtype=torch.int32, device="cuda")
    ctx, start = i32(np.zeros(n)), i32(np.zeros(n + 1))
    slots = torch.empty(int(sum(lens)), dtype=torch.int64, device="cuda")
    pkv.pkv_tables_step(dt, i32(rows), i32(np.zeros(n)), i32(lens), out, ctx, start, slots)
    return slots


@pytest.mark.parametrize("hole", [-1, -7, 64, 2**31 - 1])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_rows_with_a_hole_keep_their_blocks(pkv, hole, at):
    dt = pkv.DeviceTables.create(64, 4, 5, 6)
    _serve(pkv, dt, [3, 0, 2, 4], [16, 20, 9, 5])
    assert pkv.device_error() == 0
    before = int(dt.free_count.item())
    dt.block_table[0, at] = hole                   # between the first and the last block
    want = dt.block_table.clone()
    free = dt.free_list[:before].clone()
    given = torch.cat([want[3, :4], want[4, :2]])
    pkv.pkv_tables_release(dt, i32([3, 0, 4]), i32([16, 20, 5]))
    assert pkv.device_error() == 1                 # PKV_DEV_BAD_BLOCK_ID
    want[3], want[4] = -1, -1                      # the others of the call are given back
    assert torch.equal(dt.block_table, want)
    count = int(dt.free_count.item())
    assert count == before + 6
    assert torch.equal(dt.free_list[:count], torch.cat([free, given]))
    # what is handed out next are blocks, each of them once
    slots = _serve(pkv, dt, [1], [24])
    assert pkv.device_error() == 0 and (slots >= 0).all() and slots.unique().numel() == 24
    # the row is given back once its entry is right
    ids = set(dt.block_table[2, :3].tolist() + dt.block_table[1].tolist()
              + dt.free_list[:int(dt.free_count.item())].tolist() + dt.block_table[0, :5].tolist())
    dt.block_table[0, at] = (set(range(64)) - ids).pop()
    pkv.pkv_tables_release(dt, i32([0, 1, 2]), i32([20, 24, 9]))
    assert pkv.device_error() == 0 and dt.free_count.item() == 64
    assert sorted(dt.free_list.tolist()) == list(range(64))


@pytest.mark.parametrize("listed", [True, False])
def test_holes_in_many_rows_of_several_passes(pkv, listed):
    """More requests than the kernel takes at once, a tenth of them with a hole."""
    rng = np.random.default_rng(5)
    n, width = 2600, 7
    lens = rng.integers(1, width * 4 + 1, n)
    blocks = -(-lens // 4)
    nb = int(blocks.sum()) + 9
    dt = pkv.DeviceTables.create(nb, 4, n, width, rng.permutation(nb))
    rows = rng.permutation(n) if listed else np.arange(n)
    _serve(pkv, dt, rows, lens)
    assert pkv.device_error() == 0 and dt.free_count.item() == 9
    table = dt.block_table.cpu().numpy()
    holes = (rng.random(n) < 0.1) & (blocks >= 3)
    for i in np.flatnonzero(holes):
        table[rows[i], rng.integers(1, blocks[i] - 1)] = rng.choice([-1, nb])
    dt.block_table.copy_(torch.from_numpy(table))
    want, given = table.copy(), dt.free_list[:9].tolist()
    for i in np.flatnonzero(~holes):
        given += table[rows[i], :blocks[i]].tolist()
        want[rows[i]] = -1
    pkv.pkv_tables_release(dt, i32(rows) if listed else None, i32(lens))
    assert pkv.device_error() == 1
    assert np.array_equal(dt.block_table.cpu().numpy(), want)
    count = int(dt.free_count.item())
    assert dt.free_list[:count].tolist() == given


def test_a_row_with_a_hole_makes_room_for_those_behind_it(pkv):
    """The free list has room for all rows but the one that is skipped."""
    dt = pkv.DeviceTables.create(8, 4, 3, 4)
    _serve(pkv, dt, [0, 1], [16, 16])
    dt.block_table[2, :4] = i32([5, 8, 6, 7])      # a row that no step filled, with an id of 8
    pkv.pkv_tables_release(dt, i32([2, 0, 1]), i32([16, 16, 16]))
    assert pkv.device_error() == 1
    assert dt.free_count.item() == 8 and sorted(dt.free_list.tolist()) == list(range(8))
    assert dt.block_table[2].tolist() == [5, 8, 6, 7]
