"""The layer operators' binding where no GPU is (CPU)."""
import os
import subprocess
import sys

import pytest

import muon_step_03_amd as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_the_gpu_parts_of_pytorch():
    """A PyTorch built without a GPU backend lacks the stream and device queries:
    the package imports all the same, and refuses a call as it does elsewhere."""
    code = (
        "import torch\n"
        "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
        "    if hasattr(torch._C, name):\n"
        "        delattr(torch._C, name)\n"
        "import muon_step_03_amd as M\n"
        "try:\n"
        "    M.checkpoint_save(torch.zeros(4, 64))\n"
        "except ValueError as e:\n"
        "    assert 'on a GPU' in str(e)\n"
        "    print('REFUSED')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "REFUSED" in r.stdout


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_checkpoints_are_on_a_gpu(device):
    """An unwritten checkpoint elsewhere is refused when it is made, like one of
    given tensors."""
    with pytest.raises(ValueError, match="must be on a GPU"):
        M.ActCheckpoint.empty(4, 64, device=device)
