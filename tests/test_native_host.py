"""What the package loads: the views module goes by the Python and the torch it was
built for (no GPU needed)."""
import contextlib
import os
import sysconfig
import types

import pytest
import torch

import speculative_decode_verify_prefix_gb300 as vsk
from speculative_decode_verify_prefix_gb300 import _native, api, cache_ops


@pytest.fixture(scope="module", autouse=True)
def built():
    vsk.build()


@pytest.fixture
def unloaded(monkeypatch, tmp_path):
    """A copy of the built views module, not loaded yet."""
    at = tmp_path / os.path.basename(_native.VIEWS_PATH)
    for end in ("", ".torch"):
        with open(_native.VIEWS_PATH + end, "rb") as f:
            (tmp_path / (at.name + end)).write_bytes(f.read())
    monkeypatch.setattr(_native, "VIEWS_PATH", str(at))
    monkeypatch.setattr(_native, "_views", None)
    return at


def test_views_module_is_named_by_the_python_that_built_it():
    assert os.path.basename(_native.VIEWS_PATH).endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert os.path.exists(_native.VIEWS_PATH)


def test_views_module_of_this_torch_is_loaded(unloaded):
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        _native.views()(("q",), (torch.zeros(1),))


@pytest.mark.parametrize("change", [lambda s: s.replace(torch.__version__, "1.0.0"), lambda s: s.replace("torch", "elsewhere"), lambda s: ""])
def test_views_module_of_another_torch_is_not_loaded(unloaded, change):
    stamp = unloaded.with_name(unloaded.name + ".torch")
    stamp.write_text(change(stamp.read_text()))
    with pytest.raises(RuntimeError, match="built against another torch"):
        _native.views()
    unloaded.unlink()
    with pytest.raises(RuntimeError, match="is missing"):
        _native.views()


def test_build_makes_a_views_module_of_another_torch_anew(unloaded):
    stamp = unloaded.with_name(unloaded.name + ".torch")
    want = stamp.read_text()
    assert torch.__version__ in want and os.path.dirname(torch.__file__) in want
    stamp.write_text("1.0.0")
    before = os.stat(unloaded).st_ino
    _native._build_views(False)
    assert stamp.read_text() == want and os.stat(unloaded).st_ino != before
    before = os.stat(unloaded).st_ino
    _native._build_views(False)
    assert os.stat(unloaded).st_ino == before


def test_without_python_headers_the_library_is_built_and_calls_run(unloaded, monkeypatch):
    """Nothing but the views module needs Python.h: build() warns, and the calls pack their views in Python."""
    paths = sysconfig.get_paths()
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a: {**paths, "include": "/nonexistent"})
    monkeypatch.setattr(_native, "VIEWS_SRC", str(unloaded.with_name("views.cpp")))
    unloaded.with_name("views.cpp").write_text("#error no headers\n")
    with pytest.warns(RuntimeWarning, match="was not built"):
        assert vsk.build() == _native.LIB_PATH
    assert not _native._views_match()  # (the old one is not taken for the new source)
    monkeypatch.setattr(cache_ops, "_views", None)
    with pytest.warns(RuntimeWarning, match="longer on the host"):
        with pytest.raises(ValueError, match="q must be a CUDA tensor"):
            vsk.rope_fwd(*[torch.zeros(1, 1, 64, dtype=torch.bfloat16)] * 4, torch.zeros(1), torch.zeros(32))
    assert cache_ops._views is cache_ops._python_views


@pytest.mark.parametrize("bad", [torch.zeros(1), [0, 1], torch.zeros(2).to_sparse()])
def test_both_packers_refuse_alike(bad):
    errors = []
    for pack in (_native.views(), cache_ops._python_views):
        for tensors in ((bad, None), (None, bad), (None, None)):
            with pytest.raises(ValueError) as e:
                pack(("a", "b"), tensors)
            errors.append(str(e.value))
    assert errors[:3] == errors[3:] and errors[0] == "a must be a CUDA tensor" and errors[1] == "b must be a CUDA tensor"


# ------------------------------------------------------------------ workspaces

@pytest.mark.parametrize("given", [True, False])
def test_workspace_is_zeroed_on_the_stream_that_uses_it(monkeypatch, given):
    current, zeroed = [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def zeros(n, **kw):
        zeroed.append(current[-1] if current else None)
        return torch.empty(n, dtype=torch.uint8)

    one, other = types.SimpleNamespace(cuda_stream=0), types.SimpleNamespace(cuda_stream=7)
    device = torch.device("cuda", 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: one)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device: other if raw == 7 else None)  # (any object with a cuda_stream)
    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(api, "_WS", {})
    monkeypatch.setattr(api, "_WS_SIZE", {(device, b, 8, 2, 64, 64, 4): 1024 * b for b in (1, 2)})
    at = (8, 2, 64, 64, 4, other if given else None)
    small = vsk.get_workspace(device, 1, *at)
    assert vsk.get_workspace(device, 1, *at) is small
    large = vsk.get_workspace(device, 2, *at)
    assert large.numel() == 2048 and vsk.get_workspace(device, 1, *at) is large
    assert zeroed == [other if given else None] * 2
    assert list(api._WS) == [(device, 7 if given else 0)]
