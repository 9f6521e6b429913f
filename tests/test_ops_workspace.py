"""Workspaces of moe_ops.h: one that was made for a program's largest batch serves
its smaller ones, and a call writes nothing behind the size it asks for."""
import pytest
import torch

from bit_expert_ffn_route_b200 import build, moe

# D, E, k: pairs joined from few and from many chunks, dense products of both widths, dense from 16 tokens on
SHAPES = [(256, 64, 3), (2304, 64, 10), (2048, 512, 10), (8192, 1024, 16), (8192, 16, 2), (1024, 8, 2), (256, 1, 1),
          (256, 32, 5), (4096, 24, 6)]


@pytest.fixture(scope="module")
def built():
    build.build()


@pytest.mark.parametrize("D,E,k", SHAPES)
def test_sizes_never_fall_as_tokens_are_added(built, D, E, k):
    for sizes in ([moe.route_backward_workspace_size(T, D, E, k) for T in [*range(9000), *range(9000, 65537, 61)]],
                  [moe.block_norm_backward_workspace_size(T, D) for T in range(400)]):
        falls = [T for T in range(1, len(sizes)) if sizes[T] < sizes[T - 1]]
        assert sizes[0] > 0 and not falls, (D, E, k, falls[:4])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 15, 16, 17, 512, 513, 1100])
@pytest.mark.parametrize("D,E,k", [(256, 64, 3), (2304, 64, 10), (1024, 8, 2), (256, 32, 5), (256, 1, 1)])
def test_a_call_stays_inside_its_size(built, T, D, E, k):
    """With a workspace of just its size, marked behind it, and with one of 1,100 tokens: the same bits."""
    from tests.test_gpu_permute import buffers
    from tests.test_gpu_route_grad import make
    ids, gates, dg, x, Wr, _ = make(T, k, E, D, "distinct")
    o, pr, rp, _ = buffers(T, k, E)
    moe.moe_permute(ids, E, o, pr, rp)
    n = moe.route_backward_workspace_size(T, D, E, k)
    room = torch.full((n + 4096,), 171, dtype=torch.uint8, device="cuda")
    most = torch.full((moe.route_backward_workspace_size(1100, D, E, k),), 255, dtype=torch.uint8, device="cuda")
    got = []
    for ws in (room[:n], most):
        out = [torch.full((T, k), 3.0, device="cuda"), torch.full((T, D), 3.0, dtype=torch.bfloat16, device="cuda"),
               torch.full((E, D), 3.0, device="cuda"), torch.full((E,), 3.0, device="cuda")]
        moe.moe_route_backward(dg, gates, ids, x, Wr, o, rp, out[0], ws, dx=out[1], dWr=out[2], dbias=out[3])
        got.append(out)
    assert (room[n:] == 171).all()
    assert all(torch.equal(a, b) for a, b in zip(*got))
