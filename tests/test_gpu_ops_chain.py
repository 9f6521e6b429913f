"""The operators of moe_ops.h as they are used together.

Serving: a layer whose experts are partly missing.  moe_expert_forward computes
the resident ones; the missed pairs are sorted by expert, computed by the caller
(here in torch, from the dequantised weights), summed back per token and given to
moe_combine as miss_partial.  The layer's output is then the all-resident layer's,
within the library's own bound; the norms between two such layers follow.

Training: gradients of a block (router, experts' rows scaled per expert, weighted
sum, norms) through the operators' backward calls against torch.autograd in 64
bits on the same selection."""
import numpy as np
import pytest
import torch

from bit_expert_ffn_route_b200 import configs, moe, synth
from tests import ops_ref as ref
from tests.harness import bf16_from_u16, oracle_layer, rel_l2_per_token, u16
from tests.test_gpu_permute import buffers

pytestmark = pytest.mark.gpu

BF, FL = torch.bfloat16, torch.float32
TOL_OUT = 1e-2          # of the expert pass, per token


def dequantised(pool, slot, D, F):
    out = []
    for m, shape in enumerate(((F, D), (F, D), (D, F))):
        w = torch.empty(*shape, device="cuda")
        moe.moe_dequantize(pool, slot, m, w)
        out.append(w)
    return out


def missed_rows(pool, slots, xr, offsets, D, F):
    """The experts' rows in fp32, computed by the caller."""
    y = torch.zeros(xr.shape, device="cuda")
    off = offsets.tolist()
    for e, slot in slots.items():
        a, b = off[e], off[e + 1]
        if a < b:
            wg, wu, wd = dequantised(pool, slot, D, F)
            v = xr[a:b].float()
            h = (torch.nn.functional.silu(v @ wg.t()) * (v @ wu.t())).to(BF).float()
            y[a:b] = h @ wd.t()
    return y


@pytest.mark.parametrize("T", [1, 4, 40])
def test_layer_with_missing_experts(T):
    cfg = configs.CONFIGS["tiny"]
    wl = configs.build(cfg, device="cuda", T=T)
    L, D, F, E, k = wl.layers[0], cfg.D, cfg.F, cfg.E, cfg.k
    x = wl.x
    gone = list(range(0, E, 3))
    slots = {e: int(L.slot_table[e]) for e in gone}
    want = oracle_layer(wl.pool, L, k, u16(x))                      # with every expert
    table = L.slot_table.clone()
    table[gone] = -1
    layer = moe.Layer(wl.pool, L.shared_slot, table, L.Wr, L.bias, k, T)
    layer(x)
    # the missed pairs, sorted by expert
    o, pr, rp, rows = buffers(T, k, E, D, BF)
    moe.moe_permute(layer.ids, E, o, pr, rp, x=x, rows=rows, slot_table=table, n_slots=layer.pool.n_slots)
    n = int(layer.miss_count)
    assert int(o[E]) == n
    named = {tuple(m) for m in layer.miss_list[:n].tolist()}
    assert named == {(p // k, p % k, int(layer.ids.view(-1)[p])) for p in rp[:n].tolist()}
    y = missed_rows(layer.pool, slots, rows, o, D, F)
    partial = torch.full((T, D), 7.0, device="cuda")
    moe.moe_unpermute(y, pr, partial, weights=layer.gates)
    out = torch.empty(T, D, dtype=BF, device="cuda")
    moe.moe_combine(layer.expert_out, layer.gates, T, D, k, out, miss_partial=partial)
    assert np.array_equal(layer.ids.cpu().numpy(), want.ids)
    err = rel_l2_per_token(u16(out), want.out)
    assert err.max() <= TOL_OUT, err
    # to the next layer: the stream and its norm
    w = torch.rand(D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") + 0.5
    stream, normed = x.clone(), torch.empty_like(x)
    moe.moe_block_norm(out, stream, residual=stream, w_post=w, w_next=w, normed=normed)
    v, e, _ = ref.norm(ref.f64(out), ref.f64(x), 1.0, None, None, ref.f64(w), 1e-6)
    ref.check(stream, v, ref.stored(v, e, BF), "stream")
    v, e, _ = ref.next_norm(ref.f64(stream), ref.f64(w), 1e-6)
    ref.check(normed, v, ref.stored(v, e, BF), "normed")
    assert moe.Layer(wl.pool, L.shared_slot, L.slot_table, L.Wr, L.bias, k, T)(normed).shape == (T, D)


@pytest.mark.parametrize("experts", ["factor", "vector"])
@pytest.mark.parametrize("T", [5, 300])
def test_gradients_of_a_block(T, experts):
    """x -> router -> rows in expert order, times a factor or a vector per expert -> weighted sum -> norms.  The
    operators pass bf16 between them: each of those roundings is half a step, 2^-8 of the value, and there are at most
    four in a row (rows, their gradient, dy, dx): the gradients are held to 4 * 2^-8 of their norm over tokens (their
    errors are independent), with the fp32 sums far below that.

    The router's gradients come from dgates = <dy, ys>, a sum of D products whose factors carry 4 and 1 of those
    roundings: it is off by at most 5 * 2^-8 of sum |dy ys|, and the logits' gradient g (dg - sum g dg) by g times that
    of its own pair plus the weighted mean of the token's.  dWr and dbias are sums of the latter (times x).  That is
    all there is for `factor`: there y is a multiple of x whatever the gates, the norm behind it takes the multiple
    away, and the loss does not depend on the gates at all (but for eps): the exact gradient is 1e-4 of its terms.  For
    `vector` the products have random signs: relative to the gradient itself the error is 5 * 2^-8, twice for the
    difference in the logits' gradient."""
    D, E, k = 512, 24, 3
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")          # noqa: E731
    x, Wr, bias = rand(T, D).to(BF), synth.router_weight(E, D, seed=2, layer=0, device="cuda"), rand(E) * 0.1
    scale = (rand(E, 1 if experts == "factor" else D) * 0.3 + 1).to(BF)     # stands for the experts
    res, w_post, w_next, gate = rand(T, D).to(BF), rand(D) * 0.1 + 1, rand(D) * 0.1 + 1, rand(D) * 0.1 + 1
    c1, c2 = rand(T, D).to(BF), rand(T, D).to(BF)                           # the loss's gradients
    ids, gates = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_route_topk(x, Wr, bias, k, ids, gates, moe.alloc_ws(moe.route_workspace_size(T, D, E, k)))
    o, pr, rp, rows = buffers(T, k, E, D, BF)
    moe.moe_permute(ids, E, o, pr, rp, x=x, rows=rows)
    of_row = ids.view(-1)[rp.long()].long()
    ys = (rows.float() * scale[of_row].float()).to(BF)
    y, xo, no = (torch.empty(T, D, dtype=BF, device="cuda") for _ in range(3))
    moe.moe_unpermute(ys, pr, y, weights=gates)
    rp_, rn_ = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_block_norm(y, xo, residual=res, gate=gate, gate_mode="channel", w_post=w_post, w_next=w_next, normed=no,
                       rstd_post=rp_, rstd_next=rn_)
    # backward
    dy, dres = torch.empty_like(y), torch.empty_like(y)
    dgate, dwp, dwn = (torch.empty(D, device="cuda") for _ in range(3))
    moe.moe_block_norm_backward(c1, c2, xo, y, dy, moe.alloc_ws(moe.block_norm_backward_workspace_size(T, D)),
                                dresidual=dres, gate=gate, gate_mode="channel", dgate=dgate, w_post=w_post, dw_post=dwp,
                                rstd_post=rp_, w_next=w_next, dw_next=dwn, rstd_next=rn_)
    dys, dgates = torch.empty_like(ys), torch.empty(T, k, device="cuda")
    moe.moe_unpermute_backward(dy, pr, dys, rows=ys, weights=gates, dweights=dgates)
    drows = (dys.float() * scale[of_row].float()).to(BF)
    dx = torch.empty_like(x)
    moe.moe_permute_backward(drows, pr, dx)
    dl, dW, db = torch.empty(T, k, device="cuda"), torch.empty(E, D, device="cuda"), torch.empty(E, device="cuda")
    moe.moe_route_backward(dgates, gates, ids, x, Wr, o, rp, dl,
                           moe.alloc_ws(moe.route_backward_workspace_size(T, D, E, k)), dx=dx, dx_add=dx, dWr=dW,
                           dbias=db)
    # the same in 64 bits
    leaf = lambda t: t.double().clone().requires_grad_(True)                # noqa: E731
    X, W, B, R, G, WP, WN = (leaf(t) for t in (x, Wr, bias, res, gate, w_post, w_next))
    lg = (X @ W.t() + B).gather(1, ids.long())
    Y = (torch.softmax(lg, 1)[:, :, None] * X[:, None, :] * scale.double()[ids.long()]).sum(1)
    n1 = Y * torch.rsqrt(Y.square().mean(1, keepdim=True) + 1e-6) * WP
    XO = R + G * n1
    NO = XO * torch.rsqrt(XO.square().mean(1, keepdim=True) + 1e-6) * WN
    ((c1.double() * XO).sum() + (c2.double() * NO).sum()).backward()
    for name, got, want in (("dx", dx, X.grad), ("dresidual", dres, R.grad), ("dgate", dgate, G.grad),
                            ("dw_post", dwp, WP.grad), ("dw_next", dwn, WN.grad)):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 4 * 2.0 ** -8, (name, rel)
    u, g64 = 2.0 ** -8, gates.double()
    e_dg = 5 * u * (dy.double().abs()[:, None, :] * ys.double()[pr.long()].abs()).sum(2)
    e_dl = g64 * (e_dg + (g64 * e_dg).sum(1, keepdim=True))
    hot = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, ids.long(), e_dl)
    for name, got, want, bound in (("dWr", dW, W.grad, hot.t() @ x.double().abs()), ("dbias", db, B.grad, hot.sum(0))):
        off = (got.double() - want).abs()
        assert (off <= bound + 1e-12).all(), (name, float((off - bound).max()))
        if experts == "vector":
            assert float(off.norm() / want.norm()) <= 10 * u, (name, float(off.norm() / want.norm()))
