"""One HIP runtime in a process, whichever of the library and torch comes first."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIRST = {"library": "mq.library()", "size query": "mq.w4a16_gemm_workspace_bytes(64, 4096, 4096)", "torch": "import torch"}


@pytest.mark.parametrize("first", FIRST)
def test_one_runtime(first):
    code = ("import weight_activation_quantized_amd as mq\n" + FIRST[first] + "\nmq.library()\nimport torch\n"
            "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "1"
