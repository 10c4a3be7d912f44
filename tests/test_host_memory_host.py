"""C entries that allocate on the host, where the host has no memory for them: a status, not an end of the process."""
import subprocess
import sys

import pytest

CALL = """
import ctypes, resource
from conv2d_batchnorm_silu_gb300 import capi
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 30),) * 2)
o = capi.AdamWOptions(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, step=1, state_bits=8)
print(capi.raw_status({}))
"""


@pytest.mark.parametrize("call", ['"conv_bn_silu_adamw_step", (capi.AdamWTensor * 1)(), 2 ** 31 - 1, ctypes.byref(o), None',
                                  '"conv_bn_silu_fold_batch", ctypes.byref(capi.FoldLayer()), 2 ** 31 - 1, None'])
def test_a_table_that_does_not_fit(call):
    """The table of so many entries is asked for before the first one is read."""
    from conv2d_batchnorm_silu_gb300 import _build
    _build.build()
    from conv2d_batchnorm_silu_gb300 import capi
    run = subprocess.run([sys.executable, "-c", CALL.format(call)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.split() == [str(capi.CBS_ERR_CUDA)], (run.returncode, run.stderr[-300:])
