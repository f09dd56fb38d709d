"""The package is imported, and refuses calls, with a torch that was built
without CUDA (whose C module lacks the stream and device queries)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import chunked_linear_attention_gb300 as cla
q, g = torch.zeros(1, 1, 8, 64), torch.zeros(1, 1, 8)
S = torch.zeros(1, 1, 64, 64)
for call in (lambda: cla.delta_rule_chunked_forward(q, q, q, g, g),
             lambda: cla.delta_rule_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], g[..., 0], g[..., 0], S),
             lambda: cla.block_norm_forward(q[0, 0])):
    try:
        call()
    except ValueError as e:
        assert "CUDA device" in str(e)
    else:
        raise SystemExit("a call with CPU tensors was not refused")
print("refused")
"""


def test_import_and_refusals_without_cuda():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr[-2000:]
