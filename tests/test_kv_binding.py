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

    def element_size(self):
        return 4

    def stride(self):
        return tuple(range(len(self.shape)))

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


class Rows(T):
    dtype = torch.float16

    def stride(self):
        return self.shape[1] * self.shape[2], self.shape[2], 1


def cache(device):
    c = kv.KVCache.__new__(kv.KVCache)
    c.heads, c.head_dim, c.index, c.device, c.n_pages, c.page_size, c.c = 2, 64, device, f"cuda:{device}", 4, 16, None
    return c


def attention(**change):
    q = Rows(0, 6, 4, 64)
    args = dict(q=q, cache=cache(0), block_table=T(0, 3, 5), q_start=T(0, 4), kv_len=T(0, 3), max_q=2, max_kv=80, out=q, ws=T(0, 1000))
    return kv.attention(**(args | change))


@pytest.mark.parametrize("name", ["max_q", "max_kv", "window"])
@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 8, -(1 << 31) - 1, 1 << 70])
def test_sizes_that_do_not_fit_are_refused(devices, name, value):
    """ctypes would pass their low 32 bits."""
    with pytest.raises(ValueError, match=name):
        attention(**{name: value})
    assert not devices.launches


def test_sizes_that_fit_arrive(devices, monkeypatch):
    seen = []
    monkeypatch.setattr(kv, "_call", lambda name, d, *args: seen.append((d.max_q, d.max_kv, d.window)))
    attention(max_q=(1 << 31) - 1, max_kv=(1 << 31) - 1, window=7)
    assert seen == [((1 << 31) - 1, (1 << 31) - 1, 7)]


@pytest.mark.parametrize("change", [dict(requests=1 << 63), dict(q_heads=(1 << 32) + 4), dict(max_q=(1 << 32) + 1), dict(max_kv=(1 << 32) + 8)])
def test_workspace_sizes_that_do_not_fit_are_refused(change):
    args = dict(requests=2, tokens=2, q_heads=4, cache=cache(0), max_q=1, max_kv=80)
    with pytest.raises(ValueError, match=next(iter(change))):
        kv.attention_workspace_size(**(args | change))


def test_cache_and_page_sizes_that_do_not_fit_are_refused(devices):
    for change in (dict(n_pages=1 << 64), dict(page_size=(1 << 32) + 16), dict(heads=(1 << 32) + 1), dict(head_dim=(1 << 32) + 64)):
        with pytest.raises(ValueError, match=next(iter(change))):
            kv.KVCache(**(dict(n_pages=2, page_size=16, heads=1, head_dim=64, fmt=kv.FMT_MXFP4_G32) | change))
    with pytest.raises(ValueError, match="page_size"):
        kv.release(**tables(0), page_size=(1 << 32) + 16)
    assert not devices.launches


@pytest.mark.parametrize("device", [0, 3])
def test_the_layers_linears_go_to_its_device(devices, monkeypatch, device):
    from diffusion_smooth_group_amd.attention_layer import SVDQAttention

    class X:
        shape, dtype, device = (6, 256), torch.float16, "cpu"

        def get_device(self):
            return device
    net = SVDQAttention.__new__(SVDQAttention)
    net.qkv, net.out, net.q_heads, net.cache, net.how, net.window, net.causal = None, None, 4, cache(device), {}, 0, True
    seen = []

    def linear(self, layer, x):
        seen.append(("linear", devices.now))
        return torch.zeros(6, 8 * 64)
    monkeypatch.setattr(SVDQAttention, "_linear", linear)
    net.cache.append = lambda *a, **k: seen.append(("append", devices.now))
    monkeypatch.setattr(kv, "attention", lambda *a, **k: seen.append(("attention", devices.now)))
    net(X(), kv.Plan(*[None] * 7), 1, 10)
    assert seen == [("linear", device), ("append", device), ("attention", device), ("linear", device)] and devices.now == 0


# ------------------------------------------------------------------------ autograd
@pytest.fixture
def taken(monkeypatch):
    """The gradients that the library would be given, with a forward pass that
    doubles (on the CPU: only the wiring is tested)."""
    seen = []

    def forward(q, k, *_):
        return 2 * q, 2 * k

    def backward(gq, gk, q, k, cos, sin, wq, wk, *_):
        seen.extend((gq, gk))
        return 2 * gq, 2 * gk, torch.ones(q.shape[2]), torch.ones(q.shape[2])
    monkeypatch.setattr(kv, "qk_norm_rope", forward)
    monkeypatch.setattr(kv, "qk_norm_rope_backward", backward)
    return seen


LOSSES = {"sum over heads": lambda y, c: (y.sum(1) * c).sum(), "mean over heads": lambda y, c: (y.mean(1) * c).sum(),
          "sum": lambda y, c: y.sum(), "mean over tokens": lambda y, c: (y.mean(0) * c[0]).sum(), "one head": lambda y, c: (y[:, 1] * c).sum(),
          "columns first": lambda y, c: (y.transpose(1, 2) * c[:, :, None]).sum(), "heads first": lambda y, c: (y.transpose(0, 1) * c).sum(),
          "odd columns": lambda y, c: (y[..., 1::2] * c[:, None, 1::2]).sum()}


@pytest.mark.parametrize("loss", list(LOSSES))
@pytest.mark.parametrize("tokens,heads", [(5, 3), (1, 2), (5, 2)])
def test_every_gradient_arrives_as_rows_that_the_library_takes(taken, loss, tokens, heads):
    q, k, c = torch.randn(tokens, heads, 64), torch.randn(tokens, 2, 64), torch.randn(tokens, 64)
    q.requires_grad_(), k.requires_grad_()
    yq, yk = kv.qk_norm_rope_autograd(q, k, None, None, None, None)
    (LOSSES[loss](yq, c) + LOSSES[loss](yk, c)).backward()
    for g, y in zip(taken, (q, k)):
        t, h, d = g.stride()
        assert d == 1 and t % 8 == 0 and t >= 0 and h % 8 == 0 and (g.shape[1] == 1 or h >= 64) and g.data_ptr() % 16 == 0
        want = torch.autograd.grad(LOSSES[loss](y, c), y)[0]
        assert torch.equal(g, want)


def test_a_second_derivative_is_refused(taken):
    """A penalty on the gradient beside another loss: an error, no wrong sum."""
    q, k = torch.randn(5, 2, 64, requires_grad=True), torch.randn(5, 2, 64, requires_grad=True)
    yq, yk = kv.qk_norm_rope_autograd(q, k, None, None, None, None)
    dq, = torch.autograd.grad((yq ** 2).sum() + yk.sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dq.square().sum() + (yk ** 2).sum()).backward()
