"""The package's host side needs no CUDA build of torch."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_package_imports_where_torch_has_no_cuda_functions():
    """A CPU-only torch has none of the torch._C._cuda_* names: the import, the
    host checks and the workload generators do not ask for them."""
    code = (
        "import torch\n"
        "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
        "    delattr(torch._C, n)\n"
        "import gated_delta_rule_158_b200 as kda\n"
        "from gated_delta_rule_158_b200 import build, workloads\n"
        "workloads.make_prefill_inputs(1, 4, 1, 32, 32, torch.float32, seed=1, device='cpu')\n"
        "print(kda.KDA_ACT_SILU)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["1"]
