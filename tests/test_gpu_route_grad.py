"""The router's gradient against the plain 64-bit form, against differences of
the router's own function, and behind moe_route_topk and moe_permute."""
import numpy as np
import pytest
import torch

from bit_expert_ffn_route_b200 import moe, synth
from tests import ops_ref as ref
from tests.ops_ref import check, f64, stored
from tests.test_gpu_permute import buffers, make_ids

pytestmark = pytest.mark.gpu

BF, FL = torch.bfloat16, torch.float32


def make(T, k, E, D, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")       # noqa: E731
    ids = torch.from_numpy(make_ids(T, k, E, kind, seed)).cuda()
    gates = torch.softmax(rand(T, k), 1)
    return ids, gates, rand(T, k), rand(T, D).to(BF), (rand(E, D) * 0.1).to(BF), rand(T, D).to(BF)


def call(ids, gates, dg, x, Wr, add=None, **none):
    T, k = ids.shape
    E, D = Wr.shape
    o, pr, rp, _ = buffers(T, k, E)
    moe.moe_permute(ids, E, o, pr, rp)
    out = {"dlogits": torch.full((T, k), 3.0, device="cuda"), "dx": torch.full((T, D), 3.0, dtype=BF, device="cuda"),
           "dWr": torch.full((E, D), 3.0, device="cuda"), "dbias": torch.full((E,), 3.0, device="cuda")}
    out |= none
    ws = torch.full((moe.route_backward_workspace_size(T, D, E, k),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_route_backward(dg, gates, ids, x, Wr, o, rp, out["dlogits"], ws, dx=out["dx"], dx_add=add, dWr=out["dWr"],
                           dbias=out["dbias"])
    return out


CASES = [(1, 1, 1, 256, "distinct"), (1, 10, 512, 256, "distinct"), (4, 2, 16, 768, "distinct"),
         (33, 16, 16, 256, "distinct"), (70, 3, 9, 512, "wild"), (200, 2, 5, 256, "one"), (40, 4, 8, 256, "none"),
         (531, 10, 64, 2304, "distinct"), (1300, 2, 3, 256, "wild"), (5, 8, 1024, 8192, "distinct"),
         # few experts and many tokens: whole tiles and not, every width of the experts' tile, more blocks than one wave
         (256, 2, 8, 512, "distinct"), (257, 16, 32, 1024, "wild"), (4100, 4, 17, 256, "one"), (700, 6, 64, 256, "none"),
         (600, 5, 33, 512, "wild"), (9601, 16, 16, 256, "distinct"), (300, 8, 65, 256, "distinct"),
         (4100, 6, 17, 256, "one"), (600, 5, 31, 768, "wild"), (16, 1, 1, 256, "distinct"), (90, 5, 32, 4096, "none")]


@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("T,k,E,D,kind", CASES)
def test_against_the_formula(T, k, E, D, kind, with_add):
    ids, gates, dg, x, Wr, add = make(T, k, E, D, kind)
    add = add if with_add else None
    got = call(ids, gates, dg, x, Wr, add)
    want = ref.route_backward(f64(dg), f64(gates), ids.cpu().numpy(), f64(x), f64(Wr), f64(add))
    for name, (v, e), dt in zip(("dlogits", "dx", "dWr", "dbias"), want, (FL, BF, FL, FL)):
        check(got[name], v, stored(v, e, dt), name)
    again = call(ids, gates, dg, x, Wr, add)
    assert all(torch.equal(got[n], again[n]) for n in got)              # the same bits
    # dx may be the buffer that holds what is added
    if with_add:
        same = call(ids, gates, dg, x, Wr, add, dx=add)
        assert torch.equal(same["dx"], got["dx"])
    only = call(ids, gates, dg, x, Wr, dx=None, dbias=None)
    assert torch.equal(only["dWr"], got["dWr"])
    only = call(ids, gates, dg, x, Wr, dx=None, dWr=None)
    assert torch.equal(only["dbias"], got["dbias"]) and torch.equal(only["dlogits"], got["dlogits"])


@pytest.mark.parametrize("T,E", [(15, 40), (20, 20), (900, 20), (900, 16), (900, 100), (8000, 20), (8000, 8)])
def test_what_is_not_finite_stays_with_its_pairs(T, E):
    """An infinity or NaN in x reaches the gradients of that token's experts alone, one in Wr the tokens of that
    expert, one in dgates that token and its experts."""
    k, D = 6, 512
    ids, gates, dg, x, Wr, _ = make(T, k, E, D, "distinct", seed=3)
    clean = call(ids, gates, dg, x, Wr)
    x[3, 17], x[7, 300], Wr[5, 40], dg[11, 1] = float("inf"), float("nan"), float("nan"), float("inf")
    got = call(ids, gates, dg, x, Wr)
    bad_W, bad_x = torch.zeros(E, D, dtype=torch.bool, device="cuda"), torch.zeros(T, D, dtype=torch.bool, device="cuda")
    bad_W[ids[3].long(), 17] = bad_W[ids[7].long(), 300] = True
    bad_W[ids[11].long()] = True
    bad_x[(ids == 5).any(1), 40] = True
    bad_x[11] = True
    assert torch.equal(~got["dWr"].isfinite(), bad_W) and torch.equal(~got["dx"].isfinite(), bad_x)
    # what they do not reach is right: the same sums in another order, or the same bits
    want = ref.route_backward(f64(dg).clip(-1e30, 1e30) * (f64(dg) < 1e30), f64(gates), ids.cpu().numpy(),
                              np.nan_to_num(f64(x), posinf=0, neginf=0), np.nan_to_num(f64(Wr)))
    assert torch.equal(got["dlogits"][:11], clean["dlogits"][:11])
    for name, bad, (v, e), dt in (("dx", bad_x, want[1], BF), ("dWr", bad_W, want[2], FL)):
        ok = (~bad).cpu().numpy()
        check(got[name][~bad], v[ok], stored(v, e, dt)[ok], name)


def test_no_tokens():
    z = torch.zeros(0, 2, device="cuda")
    i = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    Wr = torch.ones(4, 256, dtype=BF, device="cuda")
    dW, db = torch.ones(4, 256, device="cuda"), torch.ones(4, device="cuda")
    ws = moe.alloc_ws(moe.route_backward_workspace_size(0, 256, 4, 2))
    moe.moe_route_backward(z, z, i, torch.zeros(0, 256, dtype=BF, device="cuda"), Wr, torch.zeros(5, dtype=torch.int32,
                           device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), z, ws, dWr=dW, dbias=db)
    assert (dW == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T", [6, 40])
def test_behind_the_router_against_differences(T):
    """moe_route_topk, then the gradient of <c, gates> against central differences of the 64-bit router with the
    selection held fixed.  With step h the differences are off by h^2 / 6 of the third derivative along the
    direction, which for a softmax over logits that move by m per unit step is at most 6 m^3 |c|."""
    D, E, k = 256, 32, 4
    x, Wr = synth.hidden(T, D, seed=3, device="cuda"), synth.router_weight(E, D, seed=3, layer=0, device="cuda")
    bias = synth.zipf_bias(E, 1.1, 0.5, seed=3).cuda()
    ids, gates = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_route_topk(x, Wr, bias, k, ids, gates, moe.alloc_ws(moe.route_workspace_size(T, D, E, k)))
    c = torch.randn(T, k, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    got = call(ids, gates, c, x, Wr)
    i, x64, W64, b64, c64 = ids.cpu().numpy(), f64(x), f64(Wr), f64(bias), f64(c)

    def loss(xv, Wv, bv):
        l = np.take_along_axis(xv @ Wv.T + bv, i, 1)
        g = np.exp(l - l.max(1, keepdims=True))
        return float((c64 * g / g.sum(1, keepdims=True)).sum())

    rng = np.random.default_rng(5)
    h = 1e-4
    _, (dx, e_dx), (dW, e_dW), (db, e_db) = ref.route_backward(c64, f64(gates), i, x64, W64)
    for n, (w, e) in enumerate(((dx, stored(dx, e_dx, BF)), (dW, stored(dW, e_dW, FL)), (db, stored(db, e_db, FL)))):
        base = (x64, W64, b64)
        v = rng.standard_normal(base[n].shape) / np.sqrt(base[n].size)
        up, down = ([b + s * h * v if j == n else b for j, b in enumerate(base)] for s in (1, -1))
        num = (loss(*up) - loss(*down)) / (2 * h)
        moved = np.abs(up[0] @ up[1].T + up[2] - down[0] @ down[1].T - down[2]).max() / (2 * h)
        trunc = h * h * moved ** 3 * np.abs(c64).sum()
        # moe_route_topk's gates are within 1e-6 of the 64-bit ones (its own tests), and enter twice
        tol = ((e * np.abs(v)).sum() + trunc + 1e-9 + 3e-6 * (np.abs(w) * np.abs(v)).sum()
               + 2e-6 * moved * np.abs(c64).sum())
        g = f64(got[("dx", "dWr", "dbias")[n]])
        assert abs(num - (g * v).sum()) <= tol, (n, num, (g * v).sum(), tol)


@pytest.mark.parametrize("T,E", [(20, 16), (64, 16), (900, 16), (20, 100), (900, 100), (4000, 100)])
def test_captured(T, E):
    k, D = 4, 512
    a, b = make(T, k, E, D, "distinct", 1), make(T, k, E, D, "distinct", 2)
    hold = [t.clone() for t in a[:5]]
    o, pr, rp, _ = buffers(T, k, E)
    out = [torch.empty(T, k, device="cuda"), torch.empty(T, D, dtype=BF, device="cuda"),
           torch.empty(E, D, device="cuda"), torch.empty(E, device="cuda")]
    ws = moe.alloc_ws(moe.route_backward_workspace_size(T, D, E, k))

    def step():
        moe.moe_permute(hold[0], E, o, pr, rp)
        moe.moe_route_backward(hold[2], hold[1], hold[0], hold[3], hold[4], o, rp, out[0], ws, dx=out[1], dWr=out[2],
                               dbias=out[3])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for m in (b, a):
        for h, t in zip(hold, m):
            h.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        want = call(*m[:5])
        assert all(torch.equal(g, want[n]) for g, n in zip(out, ("dlogits", "dx", "dWr", "dbias")))
