"""The extension module is built for, and loaded by, one Python and one torch."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
if {other}:
    torch.__version__ = "9.8.7+other"
import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import _binding, build
if {other}:
    assert not build.marshal_up_to_date()
    assert "9.8.7_other" in build.marshal_command()[build.marshal_command().index("-o") + 1]
    try:
        _binding.load_marshal()
    except RuntimeError as e:
        assert "not built for this Python and torch" in str(e)
    else:
        raise AssertionError("loaded a module of another torch")
else:
    build.build()
    assert build.marshal_up_to_date() and _binding.load_marshal().call
"""


def test_another_torch_has_another_module():
    """After an update of torch the module of the old one is neither up to date nor loaded."""
    for other in (False, True):
        run = subprocess.run([sys.executable, "-c", SCRIPT.format(other=other)], cwd=ROOT, text=True,
                             stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=600)
        assert run.returncode == 0, run.stdout
