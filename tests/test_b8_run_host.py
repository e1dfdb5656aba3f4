"""The timing command of the 8-bit block operators: its arguments (no device needed)."""
import subprocess
import sys

import pytest


@pytest.mark.parametrize("args,message", [(["linear", "16", "64"], "a linear needs O"), (["sum", "16", "64"], "invalid choice")])
def test_arguments_are_checked(args, message):
    r = subprocess.run([sys.executable, "-m", "sparsity_sbl_quantize_b200.run_b8", *args], capture_output=True, text=True)
    assert r.returncode == 2 and message in r.stderr
