"""Stand-ins for device tensors and the library, for tests of the Python binding's checks
on a machine without a GPU."""
import torch


class FakeLibrary:
    """Takes every call and launches nothing."""
    def w4a16_status_string(self, status):
        return b"refused"

    def __getattr__(self, name):
        return lambda *args: (1 << 20) if name.endswith("_packed_bytes") else 0


class FakeTensor:
    """What the binding asks of a contiguous tensor on device 0."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, *shape, dtype, recorded=None):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.recorded = [] if recorded is None else recorded   # streams it has to wait for

    def dim(self):
        return len(self.shape)

    def size(self, i):
        return self.shape[i]

    def numel(self):
        return self.shape.numel()

    def stride(self, i):
        return torch.Size(self.shape[i + 1:]).numel()

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x10000

    def record_stream(self, stream):
        self.recorded.append(stream)


def fake(*shape, dtype):
    return FakeTensor(*shape, dtype=dtype)
