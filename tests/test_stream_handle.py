"""How the layer and latent operators get at the current stream's handle."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_calls_where_torch_has_no_raw_stream():
    """A torch without the private name for a stream's handle: calls take the public one's."""
    code = """
import types
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
from gated_delta_rule_110_amd import layer
torch.cuda.current_stream = lambda dev: types.SimpleNamespace(cuda_stream=70 + dev)
torch.cuda.current_device = lambda: 3
got = []
layer._call(lambda *args: got.append(args) or 0, 3, 1, 2)
assert got == [(1, 2, 73)], got
"""
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)
