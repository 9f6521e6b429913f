"""The norms and their gradients where a group of threads takes many tokens (more
than twice the rows it keeps in flight, so that every place of its ring is used
again), in every layout of the rows and every size of block."""
import pytest
import torch

from bit_expert_ffn_route_b200 import moe
from tests import test_gpu_block_norm as few
from tests.ops_ref import U32
from tests.ops_ref_many import check, next_norm, norm, norm_backward, stored
from tests.test_gpu_permute import shifted

pytestmark = pytest.mark.gpu

BF, HF, FL, EPS = torch.bfloat16, torch.float16, torch.float32, 1e-6

# T, D, dtype, gate mode, w_post, residual, w_next, alpha, offset in elements
CASES = [
    # rows of whole packs, every operand: each size of block
    (3001, 2048, BF, "channel", True, True, True, 1.0, 0),
    (3001, 1024, FL, "channel", True, True, True, 0.5, 0),
    (2001, 4096, HF, "channel", True, True, True, 1.0, 0),
    (2001, 2048, FL, "channel", True, True, True, 1.0, 0),
    (1001, 4096, FL, "channel", True, True, True, 1.0, 0),
    (1001, 8192, BF, "none", True, True, True, 1.414, 0),
    (1001, 8192, FL, "channel", True, True, True, 1.0, 0),
    # whole packs, other operands: the norm before a block, a gate per token, the end of the last block
    (3001, 2048, BF, "none", False, True, True, 1.0, 0),
    (5, 2048, BF, "none", False, True, True, 1.0, 0),
    (3001, 1536, FL, "none", False, True, True, 1.0, 0),
    (3001, 2048, BF, "token", True, True, True, 0.5, 0),
    (3001, 2048, HF, "channel", True, True, False, 1.0, 0),
    (1001, 8192, HF, "token", False, True, True, 1.0, 0),
    (33001, 200, BF, "channel", True, True, True, 1.0, 0),      # a warp per token
    (33001, 100, FL, "token", True, True, True, 1.0, 0),
    # pairs
    (5601, 1026, HF, "channel", True, True, True, 1.0, 0),
    (1001, 6002, HF, "token", True, True, True, 1.0, 0),
    (33001, 202, BF, "channel", True, True, True, 1.0, 2),
    # rows that start anywhere
    (3001, 2055, BF, "channel", True, True, True, 1.0, 3),
    (3001, 1001, FL, "token", True, True, True, 1.0, 0),
    (2001, 3333, BF, "token", False, True, True, 1.0, 0),
    (1001, 3001, FL, "none", True, True, True, 1.0, 1),
    (1001, 8191, HF, "channel", True, True, True, 1.0, 0),
    (1001, 5001, FL, "channel", True, False, True, 1.0, 0),
    (33001, 201, BF, "channel", True, True, True, 1.0, 0),
    (33001, 99, FL, "none", False, True, True, 1.0, 0),
]
NAMES = [f"T{c[0]}D{c[1]}{str(c[2])[6:]}{c[3]}{int(c[4])}{int(c[5])}{int(c[6])}" for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=NAMES)
def test_forward(case):
    few.test_forward(case)
    a = few.make(case)                          # in place of the block's output, while later rows of it are fetched
    o = few.forward(a, case[-1])
    moe.moe_block_norm(**a, x_out=a["y"], normed=o["normed"], eps=EPS)
    assert torch.equal(a["y"], o["x_out"])


@pytest.mark.parametrize("case", CASES, ids=NAMES)
def test_backward(case):
    few.test_backward(case)


@pytest.mark.parametrize("which", ["w_post", "w_next", "gate"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_factors_that_are_not_on_a_pack(which, off):
    """A vector of fp32 factors that starts 4, 8 or 12 bytes into a pack: the same numbers."""
    case = (700, 512, BF, "channel", True, True, True, 1.0, 0)
    a = few.make(case)
    a[which] = shifted((512,), FL, off, fill=0.0).copy_(a[which])
    x, e = norm(a["y"].double(), a["residual"].double(), 1.0, a["gate"].double(), a["w_post"].double(),
                a["w_next"].double(), EPS)
    o = few.forward(a)
    check(o["x_out"], x, stored(x, e, BF), "x_out")
    n, e = next_norm(o["x_out"].double(), a["w_next"].double(), EPS)
    check(o["normed"], n, stored(n, e, BF), "normed")
    dx, dn = shifted((700, 512), BF, 0, seed=20), shifted((700, 512), BF, 0, seed=21)
    g = few.backward(a, o, dx, dn)
    want = norm_backward(dx.double(), dn.double(), o["x_out"].double(), a["y"].double(), 1.0, a["gate"].double(),
                         a["w_post"].double(), a["w_next"].double(), EPS)
    for name, (v, m) in want.items():
        e = (3 * (512 + 24) + 700 + 8) * U32 * m
        check(g[name], v, stored(v, e, BF if name in ("dy", "dresidual") else FL), name)


def test_the_largest_matrices():
    """65,536 tokens of 8,192 fp32: byte offsets up to 2^31.  The bounds are those of tests/ops_ref.py."""
    T, D, step = 65536, 8192, 4096
    g = torch.Generator(device="cuda").manual_seed(9)
    new = lambda: torch.randn(T, D, generator=g, device="cuda")     # noqa: E731
    vec = lambda: 1 + 0.2 * torch.randn(D, generator=g, device="cuda")      # noqa: E731
    y, res, wp, wn, gate = new(), new(), vec(), vec(), vec()
    x, normed = torch.full_like(y, 9.0), torch.full_like(y, 9.0)
    rp, rn = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_block_norm(y, x, residual=res, alpha=0.5, gate=gate, gate_mode="channel", w_post=wp, w_next=wn, normed=normed,
                       rstd_post=rp, rstd_next=rn, eps=EPS)
    f = [v.double() for v in (gate, wp, wn)]
    for t in range(0, T, step):
        s = slice(t, t + step)
        want, e = norm(y[s].double(), res[s].double(), 0.5, *f, EPS)
        check(x[s], want, stored(want, e, FL), ("x_out", t))
        want, e = next_norm(x[s].double(), f[2], EPS)
        check(normed[s], want, stored(want, e, FL), ("normed", t))
    dx, dn = res, normed                        # any values; reused as they are
    dy, dr = torch.full_like(y, 9.0), torch.full_like(y, 9.0)
    sums = {n: torch.empty(D, device="cuda") for n in ("dgate", "dw_post", "dw_next")}
    ws = moe.alloc_ws(moe.block_norm_backward_workspace_size(T, D))
    moe.moe_block_norm_backward(dx, dn, x, y, dy, ws, dresidual=dr, alpha=0.5, gate=gate, gate_mode="channel", w_post=wp,
                                w_next=wn, rstd_post=rp, rstd_next=rn, **sums)
    each = 3 * (D + 24) * U32
    total = {n: [0.0, 0.0] for n in sums}
    for t in range(0, T, step):
        s = slice(t, t + step)
        part = norm_backward(dx[s].double(), dn[s].double(), x[s].double(), y[s].double(), 0.5, *f, EPS)
        for n, got in (("dy", dy), ("dresidual", dr)):
            v, m = part[n]
            check(got[s], v, stored(v, (each + U32) * m, FL), (n, t))
        for n in sums:
            total[n] = [a + b for a, b in zip(total[n], part[n])]
    for n, (v, m) in total.items():
        check(sums[n], v, stored(v, (each + (T + 8) * U32) * m, FL), n)


def test_on_a_stream_that_is_not_current():
    case = (900, 1024, BF, "channel", True, True, True, 1.0, 0)
    a = few.make(case)
    o = few.forward(a)
    dx, dn = shifted((900, 1024), BF, 0, seed=20), shifted((900, 1024), BF, 0, seed=21)
    want = few.backward(a, o, dx, dn)
    side, late = torch.cuda.Stream(), torch.full_like(a["y"], 7.0)
    out = {n: torch.empty_like(v) for n, v in o.items()}
    got = {n: torch.empty_like(v) for n, v in want.items()}
    ws = moe.alloc_ws(moe.block_norm_backward_workspace_size(900, 1024))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)           # y is written late, on the calls' own stream
        late.copy_(a["y"])
    b = dict(a, y=late)
    moe.moe_block_norm(**b, **out, eps=EPS, stream=side)
    moe.moe_block_norm_backward(dx, dn, out["x_out"], late, ws=ws, gate=a["gate"], gate_mode="channel", w_post=a["w_post"],
                                w_next=a["w_next"], rstd_post=out["rstd_post"], rstd_next=out["rstd_next"], stream=side,
                                **got)
    side.synchronize()
    assert all(torch.equal(v, o[n]) for n, v in out.items()) and all(torch.equal(v, want[n]) for n, v in got.items())


def test_two_calls_side_by_side():
    """On two streams, each with a workspace of its own: the bits of one after the other."""
    cases = [(2001, 1024, BF, "channel", True, True, True, 1.0, 0), (901, 1023, HF, "token", True, True, True, 1.0, 0)]
    work = []
    for c in cases:
        a = few.make(c)
        o = few.forward(a)
        d = [shifted(c[:2], c[2], 0, seed=s) for s in (20, 21)]
        work.append((a, o, d, few.backward(a, o, *d), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for a, o, d, _, stream in work:
            with torch.cuda.stream(stream):
                got.append((few.forward(a), few.backward(a, o, *d)))
        torch.cuda.synchronize()
        for (o2, g2), (_, o, _, g, _) in zip(got, work):
            assert all(torch.equal(v, o2[n]) for n, v in o.items()) and all(torch.equal(v, g2[n]) for n, v in g.items())
