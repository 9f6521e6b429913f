"""The plan of large batches in a cluster of 16 blocks and in one of 8, which
moe_permute takes on a device without room for 16."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from bit_expert_ffn_route_b200 import build, moe


@pytest.mark.parametrize("T,k,E,blocks,status", [
    (0, 2, 8, 16, moe.MOE_ERR_INVALID_ARG), (4, 0, 8, 16, moe.MOE_ERR_INVALID_ARG),
    (4, 2, 0, 8, moe.MOE_ERR_INVALID_ARG), (4, 2, 8, 4, moe.MOE_ERR_INVALID_ARG),
    (4, 2, 8, 16, moe.MOE_ERR_INVALID_ARG), (4, 17, 8, 8, moe.MOE_ERR_UNSUPPORTED),
    (4, 2, 1025, 8, moe.MOE_ERR_UNSUPPORTED), (65537, 2, 8, 8, moe.MOE_ERR_UNSUPPORTED)])
def test_refusals(T, k, E, blocks, status):
    build.build()
    assert moe.lib().moe_debug_permute_plan(None, T, k, E, blocks, None, None, None, None) == status


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,kind", [
    (1, 1, 1, "wild"), (33, 2, 1024, "wild"), (2049, 10, 512, "distinct"), (4097, 8, 1023, "wild"),
    # segments of a warp of more than 8 rounds, in 8 blocks alone and in both
    (5000, 7, 60, "one"), (9001, 8, 100, "distinct"), (65536, 16, 1024, "wild"), (65536, 16, 7, "wild")])
def test_both_clusters_sort_alike(T, k, E, kind):
    """Against a stable sort of the pairs by expert, and what moe_permute gives."""
    from tests.test_gpu_permute import buffers, make_ids
    ids = torch.from_numpy(make_ids(T, k, E, kind)).cuda()
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    taken = (flat >= 0) & (flat < E)
    order = np.flatnonzero(taken)[np.argsort(flat[taken], kind="stable")]
    row = np.full(T * k, -1, np.int32)
    row[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[taken], minlength=E))])
    outs = []
    for blocks in (16, 8, None):
        o, pr, rp, _ = buffers(T, k, E)
        if blocks is None:
            moe.moe_permute(ids, E, o, pr, rp)
        else:
            moe.moe_debug_permute_plan(ids, E, blocks, o, pr, rp)
        assert np.array_equal(o.cpu().numpy(), offsets), blocks
        assert np.array_equal(pr.cpu().numpy().reshape(-1), row), blocks
        assert np.array_equal(rp.cpu().numpy()[:len(order)], order) and (rp[len(order):] == -7).all(), blocks
        outs.append((o, pr, rp))
    assert all(torch.equal(a, b) for out in outs[1:] for a, b in zip(outs[0], out))


FIRST_CALL = """
import torch
from bit_expert_ffn_route_b200 import moe
T, k, E, D = 1200, 4, 64, 256
i32 = dict(dtype=torch.int32, device="cuda")
ids, x = torch.arange(T * k, **i32).view(T, k) % E, torch.randn(T, D, device="cuda")
o, pr, rp, rows = torch.empty(E + 1, **i32), torch.empty(T, k, **i32), torch.empty(T * k, **i32), torch.empty(T * k, D, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.moe_permute(ids, E, o, pr, rp, x=x, rows=rows)
graph.replay()
torch.cuda.synchronize()
order = ids.view(-1).sort(stable=True).indices
assert torch.equal(rp.long(), order) and torch.equal(rows, x[order // k])
print("ok")
"""


@pytest.mark.gpu
def test_the_first_call_of_a_process_is_captured():
    """The question whether a cluster of 16 fits is asked inside the capture."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, cwd=build.ROOT, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", (r.stdout, r.stderr)
