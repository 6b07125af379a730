"""The extension module of the operators' calls on tensors whose accessors throw: the Python checks
speak, the process lives."""
import os
import subprocess
import sys

import pytest
import torch

import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import build as spr_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16

# A copy of the module that takes CPU tensors too, so that the rest of its checks is reached here.
SCRIPT = """
import sys, torch
import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import _binding
_binding.MARSHAL_PATH = sys.argv[1]
BF = torch.bfloat16
q, k = torch.zeros(2, 4, 10, 64, dtype=BF), torch.zeros(2, 2, 30, 64, dtype=BF)
x, w, y = torch.zeros(2, 1, 10, 64, dtype=BF), torch.zeros(64, 64, dtype=BF), torch.zeros(2, 1, 10, 64, dtype=BF)
am, nr, pj = spr.make_masked(q, k, k, q), spr.make_norm_rotate(q, None, q, None, rot=0), spr.make_project(x, w, y)
ws = spr.alloc_workspace(am, device="cpu"), spr.alloc_workspace(pj, device="cpu")
sparse = q.to_sparse()
nested = torch.nested.nested_tensor([q[0], q[1, :, :9]])
calls = {
    "plain": lambda: spr.sparsepr_attend_masked(am, q, k, k, q, ws[0]),
    "vmap": lambda: torch.vmap(lambda t: spr.sparsepr_attend_masked(am, t, k, k, q, ws[0]) or t)(q.expand(3, 2, 4, 10, 64)),
    "vmap_norm": lambda: torch.vmap(lambda t: spr.sparsepr_norm_rotate(nr, t, None, q, None) or t)(q.expand(3, 2, 4, 10, 64)),
    "vmap_project": lambda: torch.vmap(lambda t: spr.sparsepr_project(pj, x, t, y, ws[1]) or t)(w.expand(3, 64, 64)),
    "sparse": lambda: spr.sparsepr_attend_masked(am, sparse, k, k, q, ws[0]),
    "nested": lambda: spr.sparsepr_attend_masked(am, nested, k, k, q, ws[0]),
    "nested_plan": lambda: spr.make_masked(nested, k, k, q),
}
assert _binding.load_marshal().plan(1, 0, 0, 0, (nested,)) is None
for name, call in calls.items():
    try:
        call()
    except (ValueError, RuntimeError) as e:
        print(name, "raised", type(e).__name__)
"""


@pytest.fixture(scope="module")
def cpu_module(tmp_path_factory):
    spr_build.build()
    tmp = tmp_path_factory.mktemp("marshal")
    with open(spr_build.MARSHAL_SRC) as f:
        text = f.read()
    test = "!t.is_cuda() || "
    assert text.count(test) == 1
    src, so = str(tmp / "marshal.cpp"), str(tmp / "_marshal.so")
    with open(src, "w") as f:
        f.write(text.replace(test, ""))
    cmd = spr_build.marshal_command()
    cmd[cmd.index(spr_build.MARSHAL_SRC)] = src
    cmd[cmd.index("-o") + 1] = so
    subprocess.check_call(cmd)
    return so


def test_accessors_that_throw(cpu_module):
    run = subprocess.run([sys.executable, "-c", SCRIPT, cpu_module], cwd=ROOT, text=True,
                         stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=300)
    assert run.returncode == 0, run.stdout
    for name in ("plain", "vmap", "vmap_norm", "vmap_project", "sparse", "nested", "nested_plan"):
        assert f"{name} raised" in run.stdout, run.stdout


@pytest.mark.gpu
def test_tensors_without_storage_on_the_gpu():
    q = torch.zeros(2, 4, 10, 64, device="cuda", dtype=BF)
    k = torch.zeros(2, 2, 30, 64, device="cuda", dtype=BF)
    o = torch.empty_like(q)
    prm = spr.make_masked(q, k, k, o)
    ws = spr.alloc_workspace(prm)
    spr.sparsepr_attend_masked(prm, q, k, k, o, ws)
    for call in (lambda: torch.vmap(lambda t: spr.sparsepr_attend_masked(prm, t, k, k, o, ws) or t)(
                     q.expand(3, *q.shape)),
                 lambda: spr.sparsepr_attend_masked(prm, q.to_sparse(), k, k, o, ws),
                 lambda: spr.sparsepr_attend_masked(prm, torch.nested.nested_tensor([q[0], q[1]]), k,
                                                    k, o, ws)):
        with pytest.raises((ValueError, RuntimeError)):
            call()
    spr.sparsepr_attend_masked(prm, q, k, k, o, ws)
    torch.cuda.synchronize()
    assert (o == 0).all()
