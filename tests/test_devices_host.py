"""Tensors of more than one device, and a device that is not the current one, in
the tensor layers: refused or entered before an address reaches a kernel.  Stand-ins
for tensors and for the library's calls; nothing touches a GPU."""
import contextlib
import types

import pytest
import torch


class Tensor:
    """What the tensor layers ask of a tensor."""

    def __init__(self, shape, dtype=torch.float32, dev=0, contiguous=True):
        self.shape, self.dtype, self.dev, self.contiguous = torch.Size(shape), dtype, dev, contiguous
        self.is_cuda, self.device = dev >= 0, torch.device("cuda", dev) if dev >= 0 else torch.device("cpu")

    def stride(self):
        steps = [1]
        for n in reversed(self.shape[1:]):
            steps.insert(0, steps[0] * n)
        return tuple(steps[:len(self.shape)])

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return self.contiguous

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def lib(monkeypatch):
    """The tensor layer over recorded calls; the current GPU is 0."""
    from dense_convolution_gb300 import build
    build.build()
    from dense_convolution_gb300 import conv, head
    seen = types.SimpleNamespace(calls=[], current=0, head=head, conv=conv, streams=[])

    @contextlib.contextmanager
    def device(dev):
        was, seen.current = seen.current, dev
        yield
        seen.current = was

    @contextlib.contextmanager
    def stream(s):
        with device(s.device.index):
            seen.streams.append(s)
            yield

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for layer in (head, conv):
        monkeypatch.setattr(layer, "_current_device", lambda: seen.current, raising=False)
    monkeypatch.setattr(head, "_raw_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Tensor(
        shape if isinstance(shape, (tuple, torch.Size)) else (shape,), dtype, torch.device(device).index))
    monkeypatch.setattr(torch, "empty_like", lambda t: Tensor(t.shape, t.dtype, t.dev))
    for f in ("layernorm_fwd", "layernorm_bwd", "dropout_fwd", "dropout_bwd", "linear_ce_fwd", "linear_ce_bwd"):
        monkeypatch.setattr(head.head_capi, f, lambda *a, f=f: seen.calls.append((f, seen.current, a[-1])))
    return seen


def _cases(head, other):
    """(call, its tensors' names) for every entry of the head, each tensor on GPU 0
    except the one named, which is on `other`."""
    i64 = torch.int64

    def at(bad, name, *shape, dtype=torch.float32):
        return Tensor(shape, dtype, other if bad == name else 0)

    ln, planes = head.LayerNorm(4, 8), head.LayerNorm(4, 8, pixels=2)
    dr, ce = head.Dropout(4, 8), head.LinearCrossEntropy(4, 8, 16, "f32")
    u8 = torch.uint8
    return [
        (lambda b: ln(at(b, "x", 4, 8), at(b, "gamma", 8), at(b, "beta", 8), y=at(b, "y", 4, 8)), ("x", "gamma", "beta", "y")),
        (lambda b: planes(at(b, "x", 2, 8, 2), at(b, "gamma", 8), y=at(b, "y", 4, 8)), ("x", "gamma", "y")),
        (lambda b: ln.backward(at(b, "dy", 4, 8), at(b, "x", 4, 8), at(b, "gamma", 8), at(b, "mean", 4), at(b, "rstd", 4),
                               workspace=at(b, "workspace", 1 << 20, dtype=u8)),
         ("dy", "x", "gamma", "mean", "rstd", "workspace")),
        (lambda b: dr(at(b, "x", 4, 8), 1, residual=at(b, "residual", 4, 8), y=at(b, "y", 4, 8)), ("x", "residual", "y")),
        (lambda b: dr.backward(at(b, "dy", 4, 8), 1, dx=at(b, "dx", 4, 8)), ("dy", "dx")),
        (lambda b: ce(at(b, "h", 4, 8), at(b, "w", 16, 8), at(b, "target", 4, dtype=i64),
                      workspace=at(b, "workspace", 1 << 20, dtype=u8)), ("h", "w", "target", "workspace")),
        (lambda b: ce.backward(at(b, "h", 4, 8), at(b, "w", 16, 8), at(b, "target", 4, dtype=i64), at(b, "lse", 4),
                               at(b, "dloss"), workspace=at(b, "workspace", 1 << 20, dtype=u8)),
         ("h", "w", "target", "lse", "dloss", "workspace")),
    ]


@pytest.mark.parametrize("other", [1, -1])
def test_a_tensor_of_another_device_is_refused(lib, other):
    for call, names in _cases(lib.head, other):
        call(None)
        done = len(lib.calls)
        for name in names:
            with pytest.raises(ValueError):
                call(name)
        assert len(lib.calls) == done


def test_a_call_runs_on_its_tensors_device(lib):
    t = lambda *shape, dtype=torch.float32: Tensor(shape, dtype, 2)
    lib.head.LayerNorm(4, 8)(t(4, 8), t(8))
    lib.head.Dropout(4, 8).backward(t(4, 8), 1)
    ce = lib.head.LinearCrossEntropy(4, 8, 16, "f32")
    ce(t(4, 8), t(16, 8), t(4, dtype=torch.int64))
    assert [c[1:] for c in lib.calls] == [(2, 102)] * 3 and lib.current == 0


def test_a_stream_of_another_device_is_refused(lib):
    on = lambda dev: types.SimpleNamespace(device=torch.device("cuda", dev))
    dr = lib.head.Dropout(4, 8)
    with pytest.raises(ValueError):
        dr(Tensor((4, 8)), 1, stream=on(1))
    assert not lib.calls
    s = on(1)
    dr(Tensor((4, 8), dev=1), 1, stream=s)
    assert lib.streams == [s] and lib.calls[0][1] == 1


def test_a_workspace_that_repeats_itself_is_refused(lib):
    ce = lib.head.LinearCrossEntropy(4, 8, 16, "f32")
    h, w, target = Tensor((4, 8)), Tensor((16, 8)), Tensor((4,), torch.int64)
    with pytest.raises(ValueError):
        ce(h, w, target, workspace=Tensor((1 << 20,), torch.uint8, contiguous=False))


@pytest.mark.parametrize("other", [1, -1])
def test_convolution_tensors_of_another_device_are_refused(lib, other, monkeypatch):
    capi = lib.conv.capi
    monkeypatch.setattr(capi, "conv2d_fwd", lambda *a: lib.calls.append(("fwd", lib.current, a[-1])))
    monkeypatch.setattr(capi, "conv2d_pack_filter", lambda *a: lib.calls.append(("pack", lib.current, a[-1])))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=100 + d.index))
    op = lib.conv.Conv2d(1, 4, 8, 8, 16, 3, 3)
    shapes = {"x": (1, 4, 8, 8), "w": (16, 4, 3, 3), "bias": (16,), "y": (1, 16, 6, 6), "workspace": (1 << 20,)}

    def call(bad, dev=0):
        t = {k: Tensor(v, torch.uint8 if k == "workspace" else torch.float32, other if k == bad else dev)
             for k, v in shapes.items()}
        return op(t["x"], t["w"], y=t["y"], workspace=t["workspace"], bias=t["bias"])

    call(None)
    call(None, dev=2)
    assert lib.calls == [("fwd", 0, 100), ("fwd", 2, 102)]
    for name in shapes:
        with pytest.raises(ValueError):
            call(name)
    with pytest.raises(ValueError):
        op.pack_filter(Tensor(shapes["w"], dev=-1))
    with pytest.raises(ValueError):
        op(Tensor(shapes["x"]), Tensor(shapes["w"]), y=Tensor((1, 16, 6, 5)))
    assert len(lib.calls) == 2
