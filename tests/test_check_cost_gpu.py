"""conv_bn_silu_check reads the error words of the kernels that a program has launched: one that runs the convolution
alone does not wait for those of the int8 linear layer."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import time
import torch
from conv2d_batchnorm_silu_gb300 import capi

def check_time():  # the median of runs of checks, each of which waits for the device
    torch.cuda.synchronize()
    times = []
    for _ in range(41):
        start = time.perf_counter()
        for _ in range(20):
            capi.check()
        times.append(time.perf_counter() - start)
    return sorted(times)[20] / 20

x = torch.randn(1, 16, 16, 64, device="cuda").bfloat16()
w = torch.randn(64, 3, 3, 64, device="cuda").bfloat16()
capi.forward(x, w, torch.ones(64, device="cuda"), torch.zeros(64, device="cuda"), stride=1, pad=1)
check_time()
alone = check_time()
a = torch.ones(700, 400, dtype=torch.int8, device="cuda")
one = torch.ones(1300, device="cuda")
capi.linear_int8(a, a[:1].expand(1300, 400).contiguous(), one[:700], one)
check_time()
print(alone, check_time())
"""


def test_the_convolution_alone_does_not_wait_for_the_linear_layer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    run = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
    alone, both = (float(v) for v in run.stdout.split())
    # three words to read against five, which take equal times
    assert alone < 0.8 * both, (alone, both)
