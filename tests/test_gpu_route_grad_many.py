"""The router's gradient of many tokens against the 64-bit form: every width of the
sliced kernel, joins of few and of many chunks, and dense blocks of many tiles."""
import pytest
import torch

from tests.ops_ref_many import check, route_backward, stored
from tests.test_gpu_route_grad import call, make

pytestmark = pytest.mark.gpu

BF, FL = torch.bfloat16, torch.float32

# T, k, E, D, ids.  dx in slices of Wr: 12,288 pairs or more and enough of them per expert
SLICED = [
    # up to 800 experts, 128 columns to a slice: each number of ranks, odd and even; the last tile of tokens not full
    (12290, 1, 64, 256, "distinct"), (6201, 2, 33, 512, "wild"), (4100, 3, 800, 8192, "distinct"),
    (3101, 4, 64, 2048, "wild"), (2501, 5, 800, 4096, "wild"), (2101, 6, 100, 768, "distinct"),
    (1801, 7, 300, 2304, "wild"), (1601, 8, 65, 512, "distinct"), (1401, 9, 90, 1280, "wild"),
    (1301, 10, 512, 2048, "distinct"), (1201, 11, 64, 256, "distinct"), (1101, 12, 128, 1024, "wild"),
    (1001, 13, 40, 512, "distinct"), (901, 14, 256, 2048, "wild"), (851, 15, 33, 256, "distinct"),
    (769, 16, 800, 4096, "distinct"),
    # beyond 800, 64 columns
    (12289, 1, 801, 2048, "distinct"), (6201, 2, 1024, 4096, "wild"), (2101, 6, 801, 2048, "distinct"),
    (1301, 10, 1024, 2048, "wild"), (801, 16, 900, 4096, "distinct"),
    # few experts with many chunks each: the wide join
    (8301, 4, 20, 1024, "distinct"), (30001, 3, 17, 256, "wild")]
# few experts: blocks of 4 to 14 tiles of 32 tokens, the last block and its last tile ragged
DENSE = [(6001, 2, 8, 2048, "distinct"), (4001, 6, 24, 2048, "wild"), (12001, 3, 16, 4096, "wild"),
         (9001, 5, 32, 1024, "wild"), (20000, 2, 8, 1024, "distinct"), (3001, 16, 31, 8192, "distinct")]


def against_the_formula(T, k, E, D, kind, terms):
    ids, gates, dg, x, Wr, add = make(T, k, E, D, kind, seed=5)
    if k == 1:
        gates = gates / 2                       # a single gate of 1 has no gradient at all; the formula takes any
    for a in (add, None):
        got = call(ids, gates, dg, x, Wr, a)
        want = route_backward(dg, gates, ids, x, Wr, a, terms)
        for name, (v, e), dt in zip(("dlogits", "dx", "dWr", "dbias"), want, (FL, BF, FL, FL)):
            assert v.abs().max() > 0, name
            check(got[name], v, stored(v, e, dt), name)
    again = call(ids, gates, dg, x, Wr)
    assert all(torch.equal(got[n], again[n]) for n in got)              # the same bits
    same = call(ids, gates, dg, x, Wr, add.clone(), dWr=None)
    held = add.clone()                                                  # dx in the buffer that holds what is added
    assert torch.equal(call(ids, gates, dg, x, Wr, held, dx=held, dbias=None)["dx"], same["dx"])
    assert torch.equal(same["dbias"], got["dbias"])
    only = call(ids, gates, dg, x, Wr, dx=None)
    assert all(torch.equal(only[n], got[n]) for n in ("dlogits", "dWr", "dbias"))


@pytest.mark.parametrize("T,k,E,D,kind", SLICED)
def test_slices(T, k, E, D, kind):
    against_the_formula(T, k, E, D, kind, 1)


@pytest.mark.parametrize("T,k,E,D,kind", DENSE)
def test_dense_blocks_of_many_tiles(T, k, E, D, kind):
    against_the_formula(T, k, E, D, kind, 6)


@pytest.mark.parametrize("T,k,E,D", [(8000, 6, 100, 512), (2100, 6, 900, 2048), (6001, 2, 8, 2048), (4001, 6, 24, 2048)])
def test_what_is_not_finite_stays_with_its_pairs(T, k, E, D):
    """In a block's later tiles and its last token too; gradients that no such value reaches are right."""
    ids, gates, dg, x, Wr, _ = make(T, k, E, D, "distinct", seed=3)
    inf, nan = float("inf"), float("nan")
    hit_x = {(100, 17): inf, (127, 300): nan, (T - 1, 1): -inf, (T // 2, 40): nan}
    for (t, c), v in hit_x.items():
        x[t, c] = v
    Wr[5, 40], Wr[E - 1, D - 1] = nan, inf
    dg[70, 1], dg[T - 2, 0] = inf, nan
    got = call(ids, gates, dg, x, Wr)
    bad_W = torch.zeros(E, D, dtype=torch.bool, device="cuda")
    bad_x = torch.zeros(T, D, dtype=torch.bool, device="cuda")
    for t, c in hit_x:
        bad_W[ids[t].long(), c] = True
    for t in (70, T - 2):
        bad_W[ids[t].long()] = True
        bad_x[t] = True
    bad_x[(ids == 5).any(1), 40] = True
    bad_x[(ids == E - 1).any(1), D - 1] = True
    assert torch.equal(~got["dWr"].isfinite(), bad_W) and torch.equal(~got["dx"].isfinite(), bad_x)
    clean = dg.clone()
    clean[70], clean[T - 2] = 0, 0
    want = route_backward(clean, gates, ids, x.nan_to_num(0, 0, 0), Wr.nan_to_num(0, 0, 0), None, 6)
    for name, bad, (v, e), dt in (("dx", bad_x, want[1], BF), ("dWr", bad_W, want[2], FL)):
        check(got[name][~bad], v[~bad], stored(v, e, dt)[~bad], name)


def test_on_a_stream_that_is_not_current():
    from bit_expert_ffn_route_b200 import moe
    from tests.test_gpu_permute import buffers
    T, k, E, D = 1301, 10, 64, 1024
    ids, gates, dg, x, Wr, _ = make(T, k, E, D, "distinct")
    want = call(ids, gates, dg, x, Wr)
    o, pr, rp, _ = buffers(T, k, E)
    out = [torch.empty(T, k, device="cuda"), torch.empty(T, D, dtype=BF, device="cuda"), torch.empty(E, D, device="cuda"),
           torch.empty(E, device="cuda")]
    ws = moe.alloc_ws(moe.route_backward_workspace_size(T, D, E, k))
    side, late = torch.cuda.Stream(), torch.full((T, k), 7.0, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)           # what the calls read is written late on their own stream
        late.copy_(dg)
    moe.moe_permute(ids, E, o, pr, rp, stream=side)
    moe.moe_route_backward(late, gates, ids, x, Wr, o, rp, out[0], ws, dx=out[1], dWr=out[2], dbias=out[3], stream=side)
    side.synchronize()
    assert all(torch.equal(g, want[n]) for g, n in zip(out, ("dlogits", "dx", "dWr", "dbias")))
