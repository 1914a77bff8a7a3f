"""What the Python calls of the gated delta rule and group norm refuse before the library is called (CPU: the library is a
stand-in that must not be reached, tensors are known by their shapes alone)."""

import pytest

torch = pytest.importorskip("torch")


class _Library:
    """Answers the size queries; any other entry is a launch."""

    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 4096
        return lambda *a: self.launched.append(name) or 0


@pytest.fixture
def ops(monkeypatch):
    """The wrappers with the stand-in library; the current device is 0."""
    from mamba_selective_ssm_gb300 import ops
    lib = _Library()
    for plan in (ops._deltarule_plan, ops._groupnorm_plan):
        plan.cache_clear()
    monkeypatch.setattr(ops, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    empty, empty_like = torch.empty, torch.empty_like
    monkeypatch.setattr(torch, "empty", lambda *s, device=None, dtype=None: _as(empty(*s, dtype=dtype), torch.device(device).index))
    monkeypatch.setattr(torch, "empty_like", lambda t: _as(empty(tuple(t.shape), dtype=t.dtype), t.index))
    yield ops, lib
    for plan in (ops._deltarule_plan, ops._groupnorm_plan):
        plan.cache_clear()


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


def _args(index=0):
    t = lambda *shape: _on(index, *shape)
    return {"q": t(2, 8, 2, 16), "k": t(2, 8, 2, 16), "v": t(2, 8, 4, 16), "g": t(2, 8, 4), "beta": t(2, 8, 4), "ckpt": t(2, 4, 4096),
            "do": t(2, 8, 4, 16), "q1": t(2, 2, 16), "v1": t(2, 4, 16), "g1": t(2, 4), "h": t(2, 4, 16, 16), "x": t(6, 5, 32), "w": t(32),
            "s": t(6, 4)}


def _calls(ops, a):
    return {
        "deltarule_fwd": lambda **k: ops.deltarule_fwd(a["q"], a["k"], a["v"], a["g"], a["beta"], **k),
        "deltarule_bwd": lambda **k: ops.deltarule_bwd(a["q"], a["k"], a["v"], a["g"], a["beta"], a["ckpt"], a["do"], **k),
        "deltarule_step": lambda **k: ops.deltarule_step(a["q1"], a["q1"], a["v1"], a["g1"], a["g1"], a["h"], **k),
        "groupnorm_fwd": lambda **k: ops.groupnorm_fwd(a["x"], a["w"], a["w"], 4, 1e-5, **k),
        "groupnorm_bwd": lambda **k: ops.groupnorm_bwd(a["x"], a["x"], a["w"], None, a["s"], a["s"], 4, **k),
    }


NAMES = ["deltarule_fwd", "deltarule_bwd", "deltarule_step", "groupnorm_fwd", "groupnorm_bwd"]


@pytest.mark.parametrize("name", NAMES)
def test_the_call_itself_is_made(ops, name):
    mod, lib = ops
    _calls(mod, _args())[name]()
    assert lib.launched == [name]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_another_device(ops, name):
    mod, lib = ops
    with pytest.raises(ValueError, match="current device"):
        _calls(mod, _args(1))[name]()
    assert not lib.launched


@pytest.mark.parametrize("name, arg", [("deltarule_fwd", n) for n in ("k", "v", "g", "beta")] + [
    ("deltarule_bwd", n) for n in ("k", "v", "g", "beta", "ckpt", "do")] + [("deltarule_step", n) for n in ("v1", "g1", "h")] + [
    ("groupnorm_fwd", "w"), ("groupnorm_bwd", "w"), ("groupnorm_bwd", "s")])
def test_one_tensor_elsewhere_or_of_another_kind(ops, name, arg):
    mod, lib = ops
    a = _args()
    for other in (_as(a[arg], 1), _on(0, *a[arg].shape, dtype=torch.float64), _on(0, *a[arg].shape, 2), torch.zeros(a[arg].shape)):
        with pytest.raises((ValueError, TypeError)):
            _calls(mod, a | {arg: other})[name]()
    assert not lib.launched


def test_strides(ops):
    mod, lib = ops
    a = _args()
    with pytest.raises(ValueError, match="strides"):
        _calls(mod, a | {"q": _as(torch.zeros(2, 2, 8, 16).transpose(1, 2), 0)})["deltarule_fwd"]()
    with pytest.raises(ValueError, match="contiguous"):
        _calls(mod, a | {"x": _as(torch.zeros(5, 6, 32).transpose(0, 1), 0)})["groupnorm_fwd"]()
    with pytest.raises(ValueError, match="contiguous"):
        _calls(mod, a | {"beta": _as(torch.zeros(2, 4, 8).transpose(1, 2), 0)})["deltarule_bwd"]()
    z = _as(torch.zeros(2, 8, 128), 0)  # columns of one projection
    q, k, v = z[..., :32].unflatten(-1, (2, 16)), z[..., 32:64].unflatten(-1, (2, 16)), z[..., 64:].unflatten(-1, (4, 16))
    q, k, v = (_as(t, 0) for t in (q, k, v))
    _calls(mod, a | {"q": q, "k": k, "v": v})["deltarule_fwd"]()
    assert lib.launched == ["deltarule_fwd"]


@pytest.mark.parametrize("name", ["deltarule_fwd", "deltarule_bwd", "groupnorm_fwd", "groupnorm_bwd"])
def test_workspace_is_a_dense_tensor_there(ops, name):
    mod, lib = ops
    for bad in (_on(1, 8192, dtype=torch.uint8), torch.zeros(8192, dtype=torch.uint8), _as(torch.zeros(64, 128).t(), 0), 5):
        with pytest.raises((ValueError, TypeError)):
            _calls(mod, _args())[name](workspace=bad)
    assert not lib.launched


def test_numbers_of_dimensions(ops):
    mod, lib = ops
    a = _args()
    for other in (a["q"][0], 3):
        with pytest.raises((ValueError, TypeError)):
            _calls(mod, a | {"q": other})["deltarule_fwd"]()
    for other in (a["w"], None):
        with pytest.raises((ValueError, TypeError)):
            _calls(mod, a | {"x": other})["groupnorm_fwd"]()
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        _calls(mod, a | {"x": _on(0, 6, 5, 32, dtype=torch.float16)})["groupnorm_fwd"]()
    assert not lib.launched
