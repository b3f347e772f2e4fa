"""The fine-tuning operators (include/finetune.h) at the edges of their arguments, as
far as the host answers (no GPU needed)."""
import os
import subprocess
import sys

import pytest

import spectral_corrected_optimizer_gb300 as so
from spectral_corrected_optimizer_gb300 import build as sob

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    sob.build()
    return so.lib()


def test_layernorm_workspace_of_every_narrow_width(lib):
    # in a process of its own: a division by zero would end it
    code = ("import spectral_corrected_optimizer_gb300 as so\n"
            "print([so.lib().layernorm_backward_workspace(rows, dim) for rows in (0, 3, 5000) for dim in range(1, 18)])")
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr
    sizes = eval(run.stdout)
    # at least one partial of both vectors, rows padded to 8 values
    assert all(n >= 2 * 4 * (-(-dim // 8) * 8) for n, dim in zip(sizes, 3 * list(range(1, 18)))), sizes
