"""CPU tests of the cache operators' binding: what it makes of its arguments
before the library is called.  Devices are stand-ins: tensors that say which
one they are on, and a current device that is only a number."""
import pytest
import torch

from diffusion_smooth_group_amd import kv


class T:
    """As much of an int32 tensor on a GPU as the binding looks at."""
    dtype = torch.int32

    def __init__(self, device, *shape):
        self.index, self.shape, self.device = device, shape, f"cuda:{device}" if device >= 0 else "cpu"

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.index

    is_cuda = property(lambda self: self.index >= 0)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096 * (self.index + 2)

    def new_empty(self, n):
        return New(self.index, n)


class New(T):
    def split(self, cuts):
        return [T(self.index, n) for n in cuts]


@pytest.fixture
def devices(monkeypatch):
    """The current device, and the launches with the device that they went to."""
    class Devices:
        now, launches = 0, []

        def __init__(self):
            self.launches = []
    d = Devices()

    class On:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, d.now = d.now, self.index

        def __exit__(self, *_):
            d.now = self.before
    monkeypatch.setattr(kv, "_current_device", lambda: d.now, raising=False)
    monkeypatch.setattr(kv, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(kv, "_call", lambda name, *args: d.launches.append((name, d.now, args[-1])))
    return d


def tables(device, **other):
    t = dict(done=T(device, 3), block_table=T(device, 3, 5), kv_len=T(device, 3), free_pages=T(device, 9), free_count=T(device, 1))
    return t | other


@pytest.mark.parametrize("device", [0, 1, 5])
def test_a_launch_goes_to_the_tensors_device(devices, device):
    kv.release(**tables(device), page_size=16)
    kv.plan(T(device, 3), T(device, 3), T(device, 3, 5), T(device, 9), T(device, 1), 16, 40)
    assert devices.launches == [(n, device, 100 + device) for n in ("svdq_kv_release", "svdq_kv_plan")]
    assert devices.now == 0


@pytest.mark.parametrize("name", ["block_table", "kv_len", "free_pages", "free_count"])
@pytest.mark.parametrize("device", [0, 1, -1])
def test_tensors_of_two_devices_are_refused(devices, name, device):
    args = tables(2)
    args[name] = T(device, *args[name].shape)
    with pytest.raises(ValueError, match=name):
        kv.release(**args, page_size=16)
    assert not devices.launches


def test_tensors_of_the_host_are_refused(devices):
    with pytest.raises(ValueError):
        kv.release(**tables(-1), page_size=16)
    assert not devices.launches
