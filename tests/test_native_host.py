"""What the package loads: the views module goes by the Python and the torch it was
built for (no GPU needed)."""
import os
import sysconfig

import pytest
import torch

import speculative_decode_verify_prefix_gb300 as vsk
from speculative_decode_verify_prefix_gb300 import _native


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
