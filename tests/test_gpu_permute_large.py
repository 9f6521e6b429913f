"""Rows that together pass 4 GiB: byte offsets beyond 32 bits, on whole packs and on
rows that start anywhere."""
import pytest
import torch

from bit_expert_ffn_route_b200 import moe
from tests.ops_ref_many import U32, check, stored
from tests.test_gpu_permute import buffers

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,D,dtype", [(65536, 5, 8192, torch.bfloat16), (65536, 5, 8191, torch.float16),
                                         (40001, 4, 8191, torch.float32)])
def test_there_and_back(T, k, D, dtype):
    E, step = 64, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn(T, D, generator=g, device="cuda").to(dtype)
    w = torch.rand(T, k, generator=g, device="cuda")
    o, pr, rp, rows = buffers(T, k, E, D, dtype)
    assert rows.numel() * rows.element_size() > 1 << 32
    moe.moe_permute(ids, E, o, pr, rp, x=x, rows=rows)
    N = int(o[E])
    assert N == int((ids >= 0).sum()) and (rows[N:] == 3).all()
    for i in range(0, N, step):
        s = slice(i, min(i + step, N))
        assert torch.equal(rows[s], x[(rp[s] // k).long()]), i
    out, drows = torch.full_like(x, 9.0), torch.full_like(rows, 5.0)
    moe.moe_unpermute(rows, pr, out, weights=w)
    dw = torch.full((T, k), 7.0, device="cuda")
    moe.moe_unpermute_backward(out, pr, drows, rows=rows, weights=w, dweights=dw)
    held = pr >= 0
    for t in range(0, T, step):
        s = slice(t, t + step)
        x64, w64 = x[s].double(), torch.where(held[s], w[s], 0).double()
        n = w64.sum(1, keepdim=True)            # every row of a token is the token itself
        check(out[s], n * x64, stored(n * x64, (k + 1) * U32 * n * x64.abs(), dtype), ("out", t))
        d64 = out[s].double()
        dot, mag = (d64 * x64).sum(1, keepdim=True), (d64 * x64).abs().sum(1, keepdim=True)
        check(dw[s], torch.where(held[s], dot, 0), torch.where(held[s], 1.01 * (D + 1) * U32 * mag, 0), ("dweights", t))
    assert (drows[N:] == 5).all()
    for i in range(0, N, step):
        s = slice(i, min(i + step, N))
        p = rp[s].long()
        want = w.reshape(-1)[p][:, None].double() * out[p // k].double()
        check(drows[s], want, stored(want, U32 * want.abs(), dtype), ("drows", i))
