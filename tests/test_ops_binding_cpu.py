"""What the binding of the operators around the block hands to the library: workspaces, devices, sizes. Needs no GPU."""
import pytest
import torch

from activation_sparse_ffn_03_amd import twell as tw


class _OnGpu:
    """Stands for a contiguous GPU tensor, with an address that is never read."""

    def __init__(self, shape, dtype=torch.float32, index=0, contiguous=True):
        self.shape, self.dtype, self.index, self.contiguous = torch.Size(shape), dtype, index, contiguous
        self.is_cuda, self.device = True, torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self.contiguous

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x100000


def test_workspace_has_to_be_device_memory_in_one_piece():
    """Its size is what the library is told: a host tensor's address, or the bytes that an expanded or strided tensor
    does not hold, would be written by a kernel."""
    x = _OnGpu((4, 64))
    with pytest.raises(ValueError, match="ws must be on the GPU"):
        tw._workspace(torch.empty(4096, dtype=torch.uint8), 1024, x, None)
    with pytest.raises(ValueError, match="ws must be contiguous"):
        tw._workspace(_OnGpu((4096,), torch.uint8, contiguous=False), 1024, x, None)
    with pytest.raises(ValueError, match="ws must be on cuda:0"):
        tw._workspace(_OnGpu((4096,), torch.uint8, index=1), 1024, x, None)
    ws = _OnGpu((4096,), torch.uint8)
    assert tw._workspace(ws, 1024, x, None)[:2] == (0x100000, 4096)
    assert tw._workspace(None, 0, x, None)[:2] == (None, 0)
