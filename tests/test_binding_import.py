"""The package imports, and its calls that need no GPU work, where torch lacks the private functions the
paged calls use when they are there (a torch built without CUDA)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_maybeExchangeDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import compressed_kv_cache_absorbed_b200 as mla
assert mla.mla_cache_row_elems(mla.make_dims(128, 0, 512, 64, 128, 128, "bf16")) == 576
try:
    mla.mla_append_paged(mla.make_dims(128, 0, 512, 64, 128, 128, "bf16"), *[torch.zeros(1)] * 6)
except ValueError as e:
    assert "not a CUDA device" in str(e), e
else:
    raise SystemExit("a CPU cache was taken")
class FakeCuda:
    now = 3
    current_device = staticmethod(lambda: FakeCuda.now)
    @staticmethod
    def set_device(d):
        FakeCuda.now = d
torch.cuda.current_device, torch.cuda.set_device = FakeCuda.current_device, FakeCuda.set_device
assert mla._swap_device(1) == 3 and FakeCuda.now == 1
print("ok")
"""


def test_import_without_the_private_functions():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
