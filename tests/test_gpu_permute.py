"""Tokens sorted by expert and back, and their gradients, against the plain
64-bit forms of tests/ops_ref.py: plans and copies bit for bit, sums within the
bounds derived there."""
import numpy as np
import pytest
import torch

from bit_expert_ffn_route_b200 import moe
from tests import ops_ref as ref
from tests.ops_ref import U32, check, f64, stored

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32


def make_ids(T, k, E, kind, seed=0):
    g = np.random.default_rng(seed)
    if kind == "one":                       # every pair to one expert
        return np.full((T, k), E - 1, np.int32)
    if kind == "none":                      # no pair has an expert
        return np.where(g.random((T, k)) < 0.5, -1, E).astype(np.int32)
    if kind == "wild":                      # repeated experts in a token, ids outside [0, E)
        return g.integers(-2, E + 2, (T, k)).astype(np.int32)
    score = -0.8 * np.log(np.arange(1, E + 1)) + g.gumbel(size=(T, E))      # distinct experts, skewed
    return np.argsort(-score, axis=1)[:, :k].astype(np.int32)


def buffers(T, k, E, D=None, dtype=None, off=0):
    """Outputs filled with a mark; `off` shifts the rows by that many elements in memory."""
    o = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    pr = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    rp = torch.full((T * k,), -7, dtype=torch.int32, device="cuda")
    return o, pr, rp, None if D is None else shifted((T * k, D), dtype, off, fill=3.0)


def shifted(shape, dtype, off, fill=None, seed=None):
    n = int(np.prod(shape))
    base = torch.empty(n + 16, dtype=dtype, device="cuda")
    v = base[off:off + n].view(shape)
    if fill is not None:
        v.fill_(fill)
    else:
        g = torch.Generator(device="cuda").manual_seed(seed)
        v.copy_(torch.randn(shape, generator=g, device="cuda"))
    return v


CASES = [
    # T, k, E, D, dtype, ids, resident share (None: no slot table), offset in elements
    (1, 1, 1, 1, BF, "wild", None, 0),
    (1, 10, 512, 256, BF, "distinct", None, 0),
    (4, 10, 512, 3072, BF, "distinct", 0.6, 0),
    (24, 16, 16, 40, HF, "distinct", 0.5, 0),
    (25, 3, 60, 1001, FL, "distinct", None, 0),
    (33, 2, 1024, 7, HF, "wild", 0.5, 0),
    (64, 4, 8, 64, BF, "wild", None, 1),
    (64, 4, 8, 64, FL, "one", None, 1),
    (130, 5, 9, 2055, BF, "none", None, 0),
    (300, 6, 31, 128, FL, "wild", 1.0, 0),
    (700, 10, 512, 72, BF, "distinct", None, 0),
    (2049, 10, 512, 24, BF, "distinct", 0.62, 0),
    (5000, 16, 1000, 8, HF, "wild", 0.3, 0),
    # rows that start anywhere, moved in shifted 16-byte blocks
    (900, 6, 31, 203, BF, "wild", 0.5, 0),
    (1100, 4, 16, 67, FL, "distinct", None, 1),
    (600, 7, 40, 130, HF, "distinct", 0.4, 3),
    (1, 16, 16, 8191, BF, "distinct", None, 1),
    (300, 16, 1024, 130, FL, "distinct", None, 0),
    (7, 9, 12, 8190, FL, "wild", None, 2),
]


def setup(case, seed=0):
    T, k, E, D, dtype, kind, share, off = case
    ids = make_ids(T, k, E, kind, seed)
    table, n_slots = None, 0
    if share is not None:
        g = np.random.default_rng(seed + 1)
        n_slots = 2 * E
        table = np.where(g.random(E) < share, g.permutation(2 * E)[:E], -1).astype(np.int32)
        table[::7] = n_slots + 3            # out of range: not resident
    d_ids = torch.from_numpy(ids).cuda()
    d_table = None if table is None else torch.from_numpy(table).cuda()
    return ids, table, n_slots, d_ids, d_table


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"T{c[0]}k{c[1]}E{c[2]}D{c[3]}{c[5]}")
def test_permute(case):
    T, k, E, D, dtype, kind, share, off = case
    ids, table, n_slots, d_ids, d_table = setup(case)
    x = shifted((T, D), dtype, off, seed=5)
    o, pr, rp, rows = buffers(T, k, E, D, dtype, off)
    moe.moe_permute(d_ids, E, o, pr, rp, x=x, rows=rows, slot_table=d_table, n_slots=n_slots)
    torch.cuda.synchronize()
    offsets, pair_row, order = ref.plan(ids, E, table, n_slots)
    N = len(order)
    assert np.array_equal(o.cpu().numpy(), offsets)
    assert np.array_equal(pr.cpu().numpy(), pair_row)
    assert np.array_equal(rp.cpu().numpy()[:N], order) and (rp[N:] == -7).all()
    assert torch.equal(rows[:N], x[torch.from_numpy(order // k).long().cuda()]) and (rows[N:] == 3).all()
    # the plan alone
    o2, pr2, rp2, _ = buffers(T, k, E)
    moe.moe_permute(d_ids, E, o2, pr2, rp2, slot_table=d_table, n_slots=n_slots)
    assert torch.equal(o, o2) and torch.equal(pr, pr2) and torch.equal(rp, rp2)


def test_plan_of_the_largest_batch():
    T, k, E = 65536, 16, 1024
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    o, pr, rp, _ = buffers(T, k, E)
    moe.moe_permute(ids, E, o, pr, rp)
    flat = ids.reshape(-1).cpu().numpy()
    order = np.argsort(flat, kind="stable")[int((flat < 0).sum()):]
    pair_row = np.full(T * k, -1, np.int32)
    pair_row[order] = np.arange(len(order))
    assert np.array_equal(o.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))]))
    assert np.array_equal(rp.cpu().numpy()[:len(order)], order)
    assert np.array_equal(pr.cpu().numpy().reshape(-1), pair_row)


def test_rows_past_32_bits():
    """Row offsets beyond 2^31 elements."""
    T, k, E, D = 34000, 8, 4, 8192
    ids = torch.arange(T * k, device="cuda", dtype=torch.int32).view(T, k) % E
    x = (torch.arange(T, device="cuda") % 251).to(BF)[:, None].expand(T, D).contiguous()
    o, pr, rp, _ = buffers(T, k, E)
    rows = torch.empty(T * k, D, dtype=BF, device="cuda")
    moe.moe_permute(ids, E, o, pr, rp, x=x, rows=rows)
    want = (rp // k % 251).to(BF)
    for c in (0, 1, 4095, D - 1):
        assert torch.equal(rows[:, c], want)
    dx = torch.empty_like(x)
    moe.moe_permute_backward(rows, pr, dx)
    assert torch.equal(dx[:, 5].float(), (x[:, 5].float() * k).to(BF).float())
    dw = torch.empty(T, k, device="cuda")
    one = torch.ones(T, D, dtype=BF, device="cuda")
    moe.moe_unpermute_backward(one, pr, rows=rows, dweights=dw)
    assert torch.equal(dw, (x[:, :1].float() * D).expand(T, k))     # whole numbers below 2^24: exact


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("wide_out", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"T{c[0]}k{c[1]}E{c[2]}D{c[3]}{c[5]}")
def test_unpermute_and_gradients(case, wide_out, weighted):
    T, k, E, D, dtype, kind, share, off = case
    if T * k * D > 3_000_000:
        pytest.skip("the plain form loops over pairs")
    ids, table, n_slots, d_ids, d_table = setup(case, 2)
    o, pr, rp, _ = buffers(T, k, E)
    moe.moe_permute(d_ids, E, o, pr, rp, slot_table=d_table, n_slots=n_slots)
    pair_row, N = pr.cpu().numpy(), int(o[E])
    rows = shifted((T * k, D), dtype, off, seed=8)
    rows[N:] = float("nan")                                     # rows of no pair are never read
    w = torch.rand(T, k, device="cuda") if weighted else None
    odt = FL if wide_out else dtype
    out = shifted((T, D), odt, off, fill=9.0)
    moe.moe_unpermute(rows, pr, out, weights=w)
    want, mag = ref.unpermute(f64(rows), pair_row, f64(w))
    check(out, want, stored(want, (k + 1) * U32 * mag, odt), "out")

    dout = shifted((T, D), odt, off, seed=4)
    drows, dw = shifted((T * k, D), dtype, off, fill=5.0), torch.full((T, k), 7.0, device="cuda")
    moe.moe_unpermute_backward(dout, pr, drows, rows=rows, weights=w, dweights=dw)
    g, held, wdw, wmag = ref.unpermute_backward(f64(dout), f64(rows), pair_row, f64(w))
    assert (drows[torch.from_numpy(~held).cuda()] == 5).all()
    i = torch.from_numpy(held).cuda()
    check(drows[i], g[held], stored(g[held], U32 * np.abs(g[held]), dtype), "drows")
    check(dw, wdw, 1.01 * (D + 1) * U32 * wmag, "dweights")
    # one output without the other
    d2, w2 = shifted((T * k, D), dtype, off, fill=5.0), torch.full((T, k), 7.0, device="cuda")
    moe.moe_unpermute_backward(dout, pr, d2, weights=w)
    moe.moe_unpermute_backward(dout, pr, rows=rows, weights=w, dweights=w2)
    assert torch.equal(d2, drows) and torch.equal(w2, dw)
    if not weighted and not wide_out:
        dx = shifted((T, D), dtype, off, fill=9.0)
        moe.moe_permute_backward(rows, pr, dx)
        assert torch.equal(dx, out)


def test_gradients_against_differences():
    """The loss <c, unpermute(rows, w)> is linear in the rows and in w: its differences are the gradients."""
    T, k, E, D = 19, 3, 5, 16
    ids = torch.from_numpy(make_ids(T, k, E, "wild", 4)).cuda()
    o, pr, rp, _ = buffers(T, k, E)
    moe.moe_permute(ids, E, o, pr, rp)
    rows, w = shifted((T * k, D), FL, 0, seed=1), torch.rand(T, k, device="cuda")
    c = shifted((T, D), FL, 0, seed=2)
    drows, dw = torch.zeros(T * k, D, device="cuda"), torch.zeros(T, k, device="cuda")
    moe.moe_unpermute_backward(c, pr, drows, rows=rows, weights=w, dweights=dw)
    p, r64, w64, c64 = pr.cpu().numpy(), f64(rows), f64(w), f64(c)
    loss = lambda a, b: float((c64 * ref.unpermute(a, p, b)[0]).sum())      # noqa: E731
    rng = np.random.default_rng(0)
    for _ in range(5):
        da, db = rng.standard_normal(r64.shape), rng.standard_normal(w64.shape)
        num = (loss(r64 + da, w64) - loss(r64 - da, w64)) / 2
        assert abs(num - (f64(drows) * da).sum()) <= 4 * U32 * (np.abs(f64(drows) * da)).sum() + 1e-9
        num = (loss(r64, w64 + db) - loss(r64, w64 - db)) / 2
        mag = sum(np.abs(c64[t] * r64[p[t, q]]).sum() * abs(db[t, q])
                  for t in range(T) for q in range(k) if p[t, q] >= 0)
        assert abs(num - (f64(dw) * db).sum()) <= 1.01 * (D + 1) * U32 * mag + 1e-9


def test_rows_outside_the_buffer_are_no_rows():
    T, k, D = 6, 3, 32
    rows = shifted((4, D), BF, 0, seed=1)
    pr = torch.tensor([[0, 4, -1], [3, 1, 2], [-5, 1 << 30, 4], [-(1 << 31), 2, 0], [5, 6, 7], [3, 3, 3]],
                      dtype=torch.int32, device="cuda")
    w = torch.rand(T, k, device="cuda")
    w[2] = float("nan")                                         # the weights of absent rows are not used
    out = torch.full((T, D), 9.0, dtype=BF, device="cuda")
    moe.moe_unpermute(rows, pr, out, weights=w)
    want, mag = ref.unpermute(f64(rows), pr.cpu().numpy(), f64(w))
    check(out, want, stored(want, 4 * U32 * mag, BF), "out")
    assert (out[2] == 0).all() and (out[4] == 0).all()
    dw = torch.full((T, k), 7.0, device="cuda")
    moe.moe_unpermute_backward(out, pr, rows=rows, weights=w, dweights=dw)
    assert (dw[2] == 0).all() and (dw[4] == 0).all() and dw[0, 1] == 0


def test_buffers_that_start_differently():
    """rows and drows apart by less than 16 bytes: their blocks of 16 do not coincide."""
    T, k, E, D = 90, 3, 7, 333
    ids, _, _, d_ids, _ = setup((T, k, E, D, BF, "distinct", None, 0), 3)
    o, pr, rp, _ = buffers(T, k, E)
    moe.moe_permute(d_ids, E, o, pr, rp)
    rows, dout, w = shifted((T * k, D), BF, 1, seed=1), shifted((T, D), BF, 2, seed=2), torch.rand(T, k, device="cuda")
    got = []
    for off in (1, 3):
        drows, dw = shifted((T * k, D), BF, off, fill=5.0), torch.empty(T, k, device="cuda")
        moe.moe_unpermute_backward(dout, pr, drows, rows=rows, weights=w, dweights=dw)
        g, held, wdw, wmag = ref.unpermute_backward(f64(dout), f64(rows), pr.cpu().numpy(), f64(w))
        check(drows, g, stored(g, U32 * np.abs(g), BF), "drows")
        check(dw, wdw, 1.01 * (D + 1) * U32 * wmag, "dweights")
        got.append(drows)
    assert torch.equal(*got)


def test_no_rows():
    """No row at all (an empty buffer): sums are zero, so are the weights' gradients."""
    pr = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    rows, out = torch.empty(0, 40, device="cuda"), torch.full((5, 40), 3.0, device="cuda")
    moe.moe_unpermute(rows, pr, out)
    assert (out == 0).all()
    dw = torch.full((5, 2), 3.0, device="cuda")
    moe.moe_unpermute_backward(out, pr, rows=rows, dweights=dw)
    assert (dw == 0).all()


def test_no_tokens():
    ids = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    o = torch.full((5,), 3, dtype=torch.int32, device="cuda")
    moe.moe_permute(ids, 4, o, ids, torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert (o == 0).all()
    moe.moe_unpermute(torch.zeros(0, 8, device="cuda"), ids, torch.zeros(0, 8, device="cuda"))


@pytest.mark.parametrize("T", [4, 900])
def test_captured_and_on_two_streams(T):
    """One call captured and replayed with other inputs, beside eager calls on another stream."""
    k, E, D = 10, 64, 256
    made = [setup((T, k, E, D, BF, "distinct", None, 0), s) for s in (1, 2, 3)]
    xs = [shifted((T, D), BF, 0, seed=s) for s in (1, 2, 3)]
    ids, x = made[0][3].clone(), xs[0].clone()
    o, pr, rp, rows = buffers(T, k, E, D, BF)
    out, w = torch.empty(T, D, dtype=BF, device="cuda"), torch.rand(T, k, device="cuda")

    def step(stream=None):
        moe.moe_permute(ids, E, o, pr, rp, x=x, rows=rows, stream=stream)
        moe.moe_unpermute(rows, pr, out, weights=w, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = torch.cuda.Stream()
    for m, v in zip(made, xs):
        ids.copy_(m[3])
        x.copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            o2, pr2, rp2, rows2 = buffers(T, k, E, D, BF)
            out2 = torch.empty_like(out)
            moe.moe_permute(ids, E, o2, pr2, rp2, x=x, rows=rows2, stream=other)
            moe.moe_unpermute(rows2, pr2, out2, weights=w, stream=other)
        torch.cuda.synchronize()
        offsets, pair_row, order = ref.plan(m[0], E)
        assert np.array_equal(pr.cpu().numpy(), pair_row) and np.array_equal(pr2.cpu().numpy(), pair_row)
        assert torch.equal(rows, rows2) and torch.equal(out, out2)
