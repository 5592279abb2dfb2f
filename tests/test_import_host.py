"""The binding imports under a torch that was built without CUDA: status names, sizes and refusals need no GPU."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)                    # what such a build does not have
from sparse_selected_cell_gb300 import qsa
assert qsa.decode_status(64 | 8) == ["bad page-table entry", "bad sequence length"]
x = torch.zeros(1)
for call, n in ((qsa.paged_attn, 7), (qsa.rope, 3), (qsa.rope_append, 11), (qsa.cache_gather, 5), (qsa.extend_tables, 4)):
    more = (5, 5) if call is qsa.extend_tables else ()
    try:
        call(*[x] * n, *more)
    except (TypeError, ValueError) as e:
        print(call.__name__, e)
    else:
        raise SystemExit(call.__name__ + " took CPU tensors")
"""


def test_import_without_cuda_in_torch():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert len(r.stdout.splitlines()) == 5 and r.stdout.count("must be a CUDA tensor") == 5
