"""What the Python calls of linear attention and layer norm refuse before the library is called (CPU: the library is a
stand-in that must not be reached, tensors are known by their shapes alone)."""

import pytest

torch = pytest.importorskip("torch")


class _Library:
    """Answers the size queries; any other entry is a launch."""

    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 4096
        if name == "linattn_num_chunks":
            return lambda L, dtype: (L + 127) // 128
        return lambda *a: self.launched.append(name) or 0


@pytest.fixture
def ops(monkeypatch):
    """The wrappers with the stand-in library; the current device is 0."""
    from mamba_selective_ssm_gb300 import ops
    lib = _Library()
    ops._linattn_plan.cache_clear()
    ops._layernorm_plan.cache_clear()
    monkeypatch.setattr(ops, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    yield ops, lib
    ops._linattn_plan.cache_clear()
    ops._layernorm_plan.cache_clear()


class _On(torch.Tensor):
    """A tensor in host memory that says it is on a GPU."""

    index = 0

    @property
    def device(self):
        return torch.device("cuda", self.index)

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.index


def _as(t, index):
    return t.as_subclass(type("_On", (_On,), {"index": index}))


def _on(index, *shape, dtype=torch.float32):
    return _as(torch.zeros(shape, dtype=dtype), index)


def _calls(ops, index):
    """Each wrapper's call with its tensors on cuda:index."""
    t = lambda *shape: _on(index, *shape)
    q, v, g, h = t(2, 8, 2, 16), t(2, 8, 4, 16), t(2, 8, 4), t(2, 4, 16, 16)
    x, w, r = t(6, 32), t(32), t(6)
    return {
        "linattn_fwd": lambda **k: ops.linattn_fwd(q, q, v, g, **k),
        "linattn_bwd": lambda **k: ops.linattn_bwd(q, q, v, g, t(2, 4, 1, 16, 16), v, **k),
        "layernorm_bwd": lambda **k: ops.layernorm_bwd(x, x, w, r, r, **k),
        "layernorm_fwd": lambda: ops.layernorm_fwd(x, w, w, 1e-5),
        "linattn_step": lambda: ops.linattn_step(t(2, 2, 16), t(2, 2, 16), t(2, 4, 16), t(2, 4), h),
    }


NAMES = ["linattn_fwd", "linattn_bwd", "layernorm_bwd", "layernorm_fwd", "linattn_step"]


@pytest.fixture(autouse=True)
def _outputs(monkeypatch):
    """Outputs and scratch asked for on a GPU are made in host memory."""
    empty, zeros, like = torch.empty, torch.zeros, torch.empty_like
    on = lambda make: lambda *a, device=None, **k: _as(make(*a, **k), device.index) if device is not None else make(*a, **k)
    monkeypatch.setattr(torch, "empty", on(empty))
    monkeypatch.setattr(torch, "zeros", on(zeros))
    monkeypatch.setattr(torch, "empty_like", lambda t: _as(like(t.as_subclass(torch.Tensor)), t.index))


@pytest.mark.parametrize("name", NAMES)
def test_the_current_device_is_the_tensors(ops, name):
    ops, lib = ops
    _calls(ops, 0)[name]()
    assert lib.launched == [name]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_another_device_are_refused(ops, name):
    ops, lib = ops
    with pytest.raises(ValueError, match="on cuda:1, but the current device is cuda:0"):
        _calls(ops, 1)[name]()
    assert lib.launched == []


@pytest.mark.parametrize("name", NAMES[:3])
def test_workspace_is_a_dense_tensor_of_the_device(ops, name):
    ops, lib = ops
    call = _calls(ops, 0)[name]
    with pytest.raises(TypeError, match="workspace must be a torch.Tensor"):
        call(workspace=4096)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        call(workspace=torch.zeros(8192, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        call(workspace=_on(0, 64, 256)[:, :128])
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        call(workspace=_on(1, 8192))
    assert lib.launched == []
    call(workspace=_on(0, 8192))
    assert lib.launched == [name]
