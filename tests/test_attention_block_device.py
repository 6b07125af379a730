"""AttentionBlock around the sparse call, on another device than the current one: on the CPU, with the
operators and the device guard replaced by records."""
import contextlib

import torch

import free_block_sparse_means_b200 as spr
from free_block_sparse_means_b200 import attention_block as ab
from free_block_sparse_means_b200 import build as spr_build

BF = torch.bfloat16


def test_the_sparse_call_runs_on_the_blocks_device(monkeypatch):
    """The call enqueues on the current device's stream, so the block's device has to be current."""
    spr_build.build()
    w, wo = torch.zeros(3 * 128, 128, dtype=BF), torch.zeros(128, 128, dtype=BF)
    block = spr.AttentionBlock((1, 64, 128), 2, 64, w, wo, sparse=dict(Ms=16, p=4, Gk=4, Gq=4))
    current, seen = ["another"], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        yield
        current[0] = before
    monkeypatch.setattr(torch.cuda, "device", device)
    for name in ("sparsepr_project", "sparsepr_norm_rotate"):
        monkeypatch.setattr(ab, name, lambda *a, **k: None)
    for name in ("sparsepr_call", "sparsepr_get_stats"):
        monkeypatch.setattr(ab.spr, name, lambda *a, name=name, **k: seen.append((name, current[0])))
    x = torch.zeros(1, 64, 128, dtype=BF)
    block(x, torch.zeros(64, 32), torch.zeros(64, 32))
    block.check()
    assert seen == [("sparsepr_call", x.device), ("sparsepr_get_stats", x.device)]
    assert current == ["another"]
