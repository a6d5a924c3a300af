"""How the binding finds the current stream and device (CPU: with stand-ins for torch's functions)."""
import subprocess
import sys

import pytest

PROBE = """
import torch
from types import SimpleNamespace
{without}
torch.cuda.current_device = lambda: 5
torch.cuda.current_stream = lambda dev=None: SimpleNamespace(cuda_stream=700 + dev)
import nvfp4_block_scaled_08_b200 as nv
assert nv._stream(SimpleNamespace(cuda_stream=42)) == 42 and nv._stream_of(3, SimpleNamespace(cuda_stream=43)) == 43
{then}
"""
DROP = """
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
"""


@pytest.mark.parametrize("without,then", [
    (DROP, "assert nv._stream() == 705 and nv._stream_of(3) == 703"),
    ("torch._C._cuda_getDevice = lambda: 2\ntorch._C._cuda_getCurrentRawStream = lambda dev: 900 + dev",
     "assert nv._stream() == 902 and nv._stream_of(3) == 903")], ids=["public functions", "own bindings"])
def test_current_stream(without, then):
    r = subprocess.run([sys.executable, "-c", PROBE.format(without=without, then=then)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
