"""A tree whose library is built and whose tensor reader is not: modules import, the scan needs the library
alone, and the operators that use the reader say what is missing when they are called."""

import subprocess
import sys

import pytest

from conftest import ROOT

PROGRAM = """
import sys
sys.modules["sparse_moe_02_amd._tensors"] = None  # what an import of a file that is not there raises, too
import torch
from sparse_moe_02_amd import attn, gdn, pages

z = torch.zeros
bf = lambda *s: z(s, dtype=torch.bfloat16)
def refused(error, f, *a, **k):
    try:
        f(*a, **k)
    except error as e:
        return str(e)
    raise AssertionError(f"{f} was not refused")

scan = (bf(4, 1, 128), bf(4, 1, 128), bf(4, 2, 128), z(4, 2), z(4, 2))
assert "device tensor" in refused(ValueError, gdn.gdn_scan, *scan, z(2, 128, 128))
step = (*scan, z(3, 2, 128, 128), z(4, dtype=torch.int32))
kv = [bf(3, 16, 1, 64)] * 2
i = lambda *s: z(s, dtype=torch.int32)
calls = [(gdn.gdn_step, step), (attn.paged_attn, (bf(2, 2, 64), *kv, i(1, 2), i(2), i(1), 2, 2)),
         (attn.rope_append, (bf(2, 2, 64), bf(2, 1, 64), bf(2, 1, 64), *kv, i(1, 2), i(2), i(1), None))]
for f, a in calls:
    assert "build()" in refused(ImportError, f, *a)
if BUILT:  # it is found once it is there
    del sys.modules["sparse_moe_02_amd._tensors"]
    for f, a in calls:
        assert "build()" not in refused(ValueError, f, *a)
"""


@pytest.mark.parametrize("later", [False, True])
def test_modules_import_without_the_tensor_reader(later):
    pytest.importorskip("torch")
    r = subprocess.run([sys.executable, "-c", PROGRAM.replace("BUILT", str(later))], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr
