"""Device tables of several devices (CPU: stand-ins for tensors of other GPUs)."""

import pytest
import torch

from tests.test_abi_host import _FakeTensor


class _Ints(_FakeTensor):
    def __init__(self, index, shape):
        super().__init__(index, torch.int32, shape)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape[0]


def test_device_tables_lie_on_one_device(lib):
    t = lib.DeviceTables(_Ints(1, (8, 4)), _Ints(1, (32,)), _Ints(1, (1,)), 16)
    assert (t.desc.max_seqs, t.desc.max_blocks, t.desc.num_blocks) == (8, 4, 32)
    with pytest.raises(ValueError, match="free_list is on cuda:0, but block_table is on cuda:1"):
        lib.DeviceTables(_Ints(1, (8, 4)), _Ints(0, (32,)), _Ints(1, (1,)), 16)
    with pytest.raises(ValueError, match="free_count is on cuda:2, but block_table is on cuda:1"):
        lib.DeviceTables(_Ints(1, (8, 4)), _Ints(1, (32,)), _Ints(2, (1,)), 16)
