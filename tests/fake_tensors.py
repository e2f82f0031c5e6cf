"""Stand-ins for CUDA tensors and for the library, to test the binding without
a GPU: addresses are made up and nothing is read through them."""
import itertools
import math

import torch

_addresses = itertools.count(0x7F0000000000, 1 << 30)


class FakeTensor:
    """What the binding asks a contiguous tensor on a GPU for."""

    def __init__(self, shape, dtype=torch.float32, gpu=0, requires_grad=False):
        self.shape, self.dtype, self.gpu, self.requires_grad = torch.Size(shape), dtype, gpu, requires_grad
        self.device, self.is_cuda, self.address = torch.device("cuda", gpu), True, next(_addresses)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def get_device(self):
        return self.gpu

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.address


class FakeStream:
    def __init__(self, gpu=0, handle=16):
        self.device, self.device_index, self.cuda_stream = torch.device("cuda", gpu), gpu, handle


def fake_empty(*shape, dtype=torch.float32, device=None):
    shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
    return FakeTensor(shape, dtype, torch.device(device).index or 0)
