"""The binding imports wherever torch does (CPU only)."""

from __future__ import annotations

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A torch whose private bindings differ: only the public interface is there.
PROGRAM = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import mixed_precision_w4a16_repack_amd as w4

class Stream:
    cuda_stream = 4711

torch.cuda.current_stream = lambda device=None: Stream() if device == 3 else None
assert w4._raw_stream(3) == 4711
print("imported")
"""


def test_imports_without_torchs_private_stream_call():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "imported", r.stderr
