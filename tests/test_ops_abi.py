"""Size queries and argument checks of moe_ops.h (no GPU: every call here returns
before it touches the device), and the binding's checks of its tensors."""
import ctypes

import pytest
import torch

from bit_expert_ffn_route_b200 import build, moe

BAD, UNSUP, WS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_OK


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


def at(n, off=0):
    """A pointer that nothing reads: 16 MB apart, 256-byte aligned but for `off`."""
    return ctypes.c_void_p((n << 24) + off)


def test_permute_refusals(L):
    def call(ids=at(1), T=4, k=2, E=8, table=None, n_slots=0, x=at(2), D=64, dt=0, rows=at(3), off=at(4), pr=at(5),
             rp=at(6)):
        return L.moe_permute(ids, T, k, E, table, n_slots, x, D, dt, rows, off, pr, rp, None)

    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(D=0), dict(dt=3), dict(dt=-1), dict(n_slots=-1),
                dict(ids=None), dict(off=None), dict(pr=None), dict(rp=None), dict(x=None), dict(rows=None),
                dict(rows=at(2)), dict(x=at(2, 1)), dict(rows=at(3, 2), dt=2), dict(ids=at(1, 2)), dict(off=at(4, 1)),
                dict(pr=at(5, 2)), dict(rp=at(6, 2)), dict(table=at(7, 2))):
        assert call(**bad) == BAD, bad
    for bad in (dict(T=65537), dict(k=17), dict(E=1025), dict(D=8193)):
        assert call(**bad) == UNSUP, bad


def test_unpermute_refusals(L):
    def call(rows=at(1), n=8, pr=at(2), w=at(3), T=4, k=2, D=64, dt=0, out=at(4), odt=0):
        return L.moe_unpermute(rows, n, pr, w, T, k, D, dt, out, odt, None)

    for bad in (dict(T=-1), dict(k=0), dict(D=0), dict(n=-1), dict(dt=3), dict(odt=1), dict(dt=2, odt=0), dict(pr=None),
                dict(out=None), dict(rows=None), dict(out=at(1)), dict(rows=at(1, 1)), dict(out=at(4, 2), odt=2),
                dict(w=at(3, 2)), dict(pr=at(2, 1))):
        assert call(**bad) == BAD, bad
    for bad in (dict(T=65537), dict(k=17), dict(D=8193)):
        assert call(**bad) == UNSUP, bad
    assert call(T=0, rows=None, pr=None, out=None) == OK

    def back(drows=at(1), n=8, pr=at(2), T=4, k=2, D=64, dt=0, dx=at(4)):
        return L.moe_permute_backward(drows, n, pr, T, k, D, dt, dx, None)

    for bad in (dict(T=-1), dict(n=-1), dict(dt=5), dict(drows=None), dict(pr=None), dict(dx=None), dict(dx=at(1))):
        assert back(**bad) == BAD, bad
    assert back(D=8193) == UNSUP
    assert back(T=0, drows=None, pr=None, dx=None) == OK


def test_unpermute_backward_refusals(L):
    def call(dout=at(1), odt=0, rows=at(2), n=8, pr=at(3), w=at(4), T=4, k=2, D=64, dt=0, drows=at(5), dw=at(6)):
        return L.moe_unpermute_backward(dout, odt, rows, n, pr, w, T, k, D, dt, drows, dw, None)

    for bad in (dict(T=-1), dict(k=0), dict(D=0), dict(n=-1), dict(dt=3), dict(odt=1), dict(dout=None), dict(pr=None),
                dict(rows=None), dict(drows=None, dw=None), dict(drows=at(2)), dict(drows=at(1)), dict(dw=at(6, 2)),
                dict(drows=at(5, 1)), dict(rows=at(2, 1)), dict(dout=at(1, 1)), dict(w=at(4, 1)), dict(pr=at(3, 1))):
        assert call(**bad) == BAD, bad
    for bad in (dict(T=65537), dict(k=17), dict(D=8193)):
        assert call(**bad) == UNSUP, bad
    assert call(T=0, dout=None) == OK


def test_route_backward_sizes_and_refusals(L):
    assert moe.route_backward_workspace_size(100, 256, 8, 2) > 0
    assert moe.route_backward_workspace_size(100, 128, 8, 2) == 0        # D % 256
    assert moe.route_backward_workspace_size(100, 256, 1, 2) == 0        # E < k
    assert moe.route_backward_workspace_size(65537, 256, 8, 2) == 0
    need = moe.route_backward_workspace_size(4, 256, 8, 2)

    def call(dg=at(1), g=at(2), ids=at(3), x=at(4), Wr=at(5), off=at(6), rp=at(7), T=4, D=256, E=8, k=2, add=None,
             dl=at(8), dx=at(9), dW=at(10), db=at(11), ws=at(12), n=need):
        return L.moe_route_backward(dg, g, ids, x, Wr, off, rp, T, D, E, k, add, dl, dx, dW, db, ws, n, None)

    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(D=0), dict(dg=None), dict(g=None), dict(ids=None), dict(x=None),
                dict(Wr=None), dict(off=None), dict(rp=None), dict(dl=None), dict(ws=None), dict(ws=at(12, 16)),
                dict(x=at(4, 8)), dict(Wr=at(5, 8)), dict(dx=at(9, 8)), dict(add=at(13, 8)), dict(dW=at(10, 8)),
                dict(db=at(11, 2)), dict(dx=None, add=at(13)), dict(dx=at(4)), dict(dx=at(5)), dict(dg=at(1, 2)),
                dict(g=at(2, 2)), dict(ids=at(3, 2)), dict(dl=at(8, 2)), dict(off=at(6, 2)), dict(rp=at(7, 2))):
        assert call(**bad) == BAD, bad
    for bad in (dict(T=65537), dict(k=17, E=32), dict(E=1025), dict(E=1), dict(D=128), dict(D=8448)):
        assert call(**bad) == UNSUP, bad
    assert call(n=need - 1) == WS
    assert call(T=0, dg=None, g=None, ids=None, dW=None, db=None, ws=None, n=0) == OK


def test_block_norm_refusals(L):
    nan, inf = float("nan"), float("inf")

    def call(y=at(1), res=at(2), gate=None, mode=0, alpha=1.0, wp=at(4), wn=at(5), eps=1e-6, T=4, D=64, dt=0, xo=at(6),
             no=at(7), rp=None, rn=None):
        return L.moe_block_norm(y, res, gate, mode, alpha, wp, wn, eps, T, D, dt, xo, no, rp, rn, None)

    for bad in (dict(T=-1), dict(D=0), dict(dt=3), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(alpha=nan),
                dict(alpha=inf), dict(y=None), dict(mode=1), dict(mode=3, gate=at(3)), dict(gate=at(3)),
                dict(no=None), dict(wn=None), dict(wn=None, no=None, xo=None), dict(wp=None, rp=at(8)),
                dict(wn=None, no=None, rn=at(8)), dict(no=at(1)), dict(no=at(2)), dict(no=at(6)), dict(y=at(1, 1)),
                dict(res=at(2, 1)), dict(xo=at(6, 1)), dict(no=at(7, 1)), dict(wp=at(4, 2)), dict(wn=at(5, 2)),
                dict(rp=at(8, 2)), dict(rn=at(8, 2)), dict(gate=at(3, 2), mode=1)):
        assert call(**bad) == BAD, bad
    for bad in (dict(T=65537), dict(D=8193)):
        assert call(**bad) == UNSUP, bad
    assert call(T=0, y=None) == OK


def test_block_norm_backward_refusals(L):
    assert moe.block_norm_backward_workspace_size(4, 8193) == 0
    need = moe.block_norm_backward_workspace_size(4, 64)
    assert need > 0

    def call(dxo=at(1), dn=at(2), xo=at(3), y=at(4), gate=at(5), mode=1, alpha=1.0, wp=at(6), rp=at(7), wn=at(8),
             rn=at(9), T=4, D=64, dt=0, dy=at(10), dr=at(11), dg=at(12), dwp=at(13), dwn=at(14), ws=at(15), n=need):
        return L.moe_block_norm_backward(dxo, dn, xo, y, gate, mode, alpha, wp, rp, wn, rn, T, D, dt, dy, dr, dg, dwp,
                                         dwn, ws, n, None)

    for bad in (dict(T=-1), dict(D=0), dict(dt=3), dict(alpha=float("nan")), dict(dy=None), dict(gate=None),
                dict(mode=0), dict(mode=0, gate=None), dict(dn=None), dict(wn=None), dict(rn=None), dict(rp=None),
                dict(xo=None), dict(y=None), dict(wp=None, rp=None), dict(ws=None), dict(ws=at(15, 16)),
                dict(dxo=None, dn=None, wn=None, dwn=None), dict(dy=at(1)), dict(dy=at(4)), dict(dr=at(2)),
                dict(dr=at(10)), dict(dxo=at(1, 1)), dict(dy=at(10, 1)), dict(dg=at(12, 2)), dict(dwp=at(13, 2)),
                dict(dwn=at(14, 2)), dict(rn=at(9, 2))):
        assert call(**bad) == BAD, bad
    for bad in (dict(T=65537), dict(D=8193)):
        assert call(**bad) == UNSUP, bad
    assert call(n=need - 1) == WS
    assert call(T=0, dg=None, dwp=None, dwn=None, ws=None) == OK


def test_binding_refuses_tensors_it_cannot_pass(L):
    """Wrong types, shapes, strides and devices raise before any call (CPU tensors throughout: nothing runs)."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)     # noqa: E731
    ids, x, rows = i32(4, 2), torch.zeros(4, 8), torch.zeros(8, 8)
    plan = i32(6), i32(4, 2), i32(8)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_permute(ids, 5, *plan, x=x, rows=rows)
    for bad in (dict(ids=ids.long()), dict(x=x.double()), dict(x=x.t().contiguous().t()), dict(rows=rows[:7]),
                dict(rows=rows.half()), dict(x=None), dict(rows=None)):
        a = dict(ids=ids, x=x, rows=rows) | bad
        with pytest.raises(ValueError):
            moe.moe_permute(a["ids"], 5, *plan, x=a["x"], rows=a["rows"])
    with pytest.raises(ValueError, match="x must be a contiguous torch.float32 tensor .* strided"):
        moe.moe_permute(ids, 5, *plan, x=torch.zeros(8, 4).t(), rows=rows)
    with pytest.raises(ValueError, match="rows must be a tensor or None"):
        moe.moe_permute(ids, 5, *plan, x=x, rows=[1.0])
    with pytest.raises(ValueError, match="n_slots"):
        moe.moe_permute(ids, 5, *plan, x=x, rows=rows, slot_table=i32(5))
    with pytest.raises(ValueError, match="offsets"):
        moe.moe_permute(ids, 6, *plan, x=x, rows=rows)
    with pytest.raises(ValueError, match="weights"):
        moe.moe_unpermute(rows, ids, x, weights=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="drows, dweights"):
        moe.moe_unpermute_backward(x, ids)
    with pytest.raises(ValueError, match="gate_mode"):
        moe.moe_block_norm(x, x, gate=torch.zeros(8), gate_mode="row")
    with pytest.raises(ValueError, match="gate "):
        moe.moe_block_norm(x, torch.zeros(4, 8), gate=torch.zeros(8), gate_mode="token")


def test_binding_takes_its_arguments_as_python_does(L):
    """By position and by name; a missing, unknown, doubled or surplus one is a TypeError, a number that does not
    fit a ValueError (CPU tensors again)."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)     # noqa: E731
    ids, plan = i32(4, 2), (i32(6), i32(4, 2), i32(8))
    y, xo = torch.zeros(4, 8), torch.zeros(4, 8)
    for call in (lambda: moe.moe_permute(ids, 5, *plan), lambda: moe.moe_permute(ids, E=5, row_pair=plan[2],
                                                                                pair_row=plan[1], offsets=plan[0]),
                 lambda: moe.moe_block_norm(y, xo, None, 0.5), lambda: moe.moe_block_norm(y, x_out=xo, alpha=1)):
        with pytest.raises(ValueError, match="CUDA"):       # every argument was accepted
            call()
    with pytest.raises(TypeError, match="needs row_pair"):
        moe.moe_permute(ids, 5, *plan[:2])
    with pytest.raises(TypeError, match="no parameter 'rowpair'"):
        moe.moe_permute(ids, 5, *plan[:2], rowpair=plan[2])
    with pytest.raises(TypeError, match="two values for E"):
        moe.moe_permute(ids, 5, *plan, E=5)
    with pytest.raises(TypeError, match="at most 4"):
        moe.moe_permute_backward(y, ids, xo, None, None)
    with pytest.raises(TypeError):
        moe.moe_block_norm(y, xo, alpha="1")
    with pytest.raises(TypeError):
        moe.moe_permute(ids, 5.0, *plan)
    with pytest.raises(ValueError, match="E is out of range"):
        moe.moe_permute(ids, 1 << 40, *plan)
    with pytest.raises(ValueError, match="two dimensions"):
        moe.moe_permute(ids.view(-1), 5, *plan)
    with pytest.raises(ValueError, match="ids must be a tensor"):
        moe.moe_permute([[0]], 5, *plan)
    with pytest.raises(AttributeError):
        moe.moe_unsorted
