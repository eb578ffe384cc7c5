"""The package on a torch without GPU support: the host-only functions work, and an operator called with host tensors
says what is wrong."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda")]:
    delattr(torch._C, name)
import qlora_fine_tuning_nf4_amd as q
assert q.qlora_resnorm_workspace_bytes(4, 64) > 0 and q.qlora_embed_workspace_bytes(4, 10, 64) > 0
for call in (lambda: q.qlora_resnorm_fwd(torch.ones(2, 8)),
             lambda: q.qlora_embed_fwd(torch.ones(5, 8), torch.zeros(3, dtype=torch.int64))):
    try:
        call()
    except q.QLoRAError as e:
        assert "current GPU" in str(e)
    else:
        raise AssertionError("host tensors were accepted")
print("imported")
"""


def test_import_without_gpu_support():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
