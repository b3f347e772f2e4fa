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


def test_tensors_on_another_device_than_the_current_one_are_refused(monkeypatch):
    # the library launches on the current device, whose kernels must not be given another one's memory
    torch = pytest.importorskip("torch")
    from spectral_corrected_optimizer_gb300 import finetune, stage_ends
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    assert finetune._stream is stage_ends._stream and finetune._stream(torch.device("cuda", 0)) == 100
    with pytest.raises(ValueError, match="tensors are on cuda:1, the current device is cuda:0"):
        finetune._stream(torch.device("cuda", 1))
    # every operator of both modules asks for its stream there
    for module in (finetune, stage_ends):
        text = open(module.__file__).read()
        assert text.count("_check(lib()") == text.count("_stream(device))") and text.count("_cuda_getCurrentRawStream") <= 1
