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
