"""The convolution's Python calls without the token-wise operators' compiled module, and its build, without a GPU."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "conv2d_batchnorm_silu_gb300"


@pytest.fixture(scope="module")
def built():
    from conv2d_batchnorm_silu_gb300 import _build
    _build.build()
    return _build


@pytest.mark.parametrize("module", ["missing", "foreign"])
def test_the_library_answers_without_the_compiled_module(built, module, tmp_path):
    package = tmp_path / PACKAGE
    package.mkdir()
    for name in os.listdir(built.PKG_DIR):
        if name.endswith(".py"):
            shutil.copy(os.path.join(built.PKG_DIR, name), package / name)
    shutil.copy(built.LIB_PATH, package / os.path.basename(built.LIB_PATH))
    if module == "foreign":
        (package / "_token_ops.so").write_bytes(b"\x7fELF of another machine")
    code = f"""
import torch
from {PACKAGE} import capi
assert capi.__file__.startswith({str(tmp_path)!r})
assert capi.output_dims(640, 640, 3, 3, 2, 1) == (320, 320)
assert capi.raw_status("conv_bn_silu_layer_norm_backward_workspace", -1, 8) == -1
x = torch.zeros(2, 8)
for call in (lambda: capi.layer_norm(x), lambda: capi.layer_norm_backward(x, x, None, x), lambda: capi.quantize_rows(x),
             lambda: capi.layer_norm_quantize(x), lambda: capi.linear_int8(x, x, x, x)):
    try:
        call()
    except ImportError as e:
        assert "_token_ops.so" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("answered")
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                         env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert run.returncode == 0, run.stderr


def test_the_compiled_module_loads_on_first_use(built):
    code = f"""
import sys
sys.path.insert(0, {ROOT!r})
from {PACKAGE} import capi
import torch
assert "{PACKAGE}._token_ops" not in sys.modules
try:
    capi.layer_norm(torch.zeros(2, 8))
except ValueError as e:
    assert "CUDA" in str(e), e
else:
    raise AssertionError("a tensor of the host was taken")
assert "{PACKAGE}._token_ops" in sys.modules
"""
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr


@pytest.fixture
def small_build(built, monkeypatch, tmp_path):
    """_build over a source of a few lines, in a folder of its own."""
    source = tmp_path / "answer.cu"
    source.write_text('extern "C" int answer() { return 42; }\n')
    monkeypatch.setattr(built, "sources", lambda: [str(source)])
    monkeypatch.setattr(built, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(built, "LIB_PATH", str(tmp_path / "libconvbnsilu.so"))
    monkeypatch.setattr(built, "BINDING_PATH", str(tmp_path / "_token_ops.so"))
    monkeypatch.setattr(built, "PKG_DIR", str(tmp_path))
    return built


def answer(path):
    code = f"import ctypes; assert ctypes.CDLL({path!r}).answer() == 42"
    assert subprocess.run([sys.executable, "-c", code]).returncode == 0


def test_the_library_builds_where_there_is_no_pytorch(small_build, monkeypatch):
    import importlib.util
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))
    assert small_build.build() == small_build.LIB_PATH
    answer(small_build.LIB_PATH)
    assert not os.path.exists(small_build.BINDING_PATH) and small_build.up_to_date()


def test_the_library_is_there_when_the_compiled_module_does_not_build(small_build, monkeypatch, tmp_path):
    broken = tmp_path / "binding.cpp"
    broken.write_text("#error headers of another PyTorch\n")
    monkeypatch.setattr(small_build, "BINDING_SOURCE", str(broken))
    with pytest.raises(RuntimeError, match="headers of another PyTorch"):
        small_build.build()
    answer(small_build.LIB_PATH)
    before = os.path.getmtime(small_build.LIB_PATH)
    with pytest.raises(RuntimeError, match="headers of another PyTorch"):  # and is not built again for it
        small_build.build()
    assert os.path.getmtime(small_build.LIB_PATH) == before


def test_the_compiled_module_is_built_again_for_another_pytorch(built, monkeypatch):
    import importlib.metadata
    assert built.up_to_date()
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.1" if name == "torch" else version(name))
    assert not built.up_to_date()
