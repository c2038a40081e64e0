"""The example that runs the FFN operators together: its own comparisons with
torch hold (the bounds are in the example)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_ffn_block_example():
    p = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "ffn_block.py"), "--small"],
                       capture_output=True, text=True, timeout=110, cwd=ROOT)
    assert p.returncode == 0, p.stdout + p.stderr
    assert "training" in p.stdout and "one token" in p.stdout
