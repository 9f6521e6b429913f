"""The norms between two blocks and their gradients against the plain 64-bit
forms and against differences."""
import numpy as np
import pytest
import torch

from bit_expert_ffn_route_b200 import moe
from tests import ops_ref as ref
from tests.ops_ref import U32, check, f64, stored
from tests.test_gpu_permute import shifted

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6

# T, D, dtype, gate mode, w_post, residual, w_next, alpha, offset in elements
CASES = [
    (1, 1, BF, "channel", True, True, True, 1.0, 0),
    (1, 3072, BF, "channel", True, True, True, 1.0, 0),
    (3, 8, HF, "token", True, True, True, 0.5, 0),
    (5, 7, FL, "none", True, True, True, 1.414, 0),
    (4, 8192, BF, "token", True, True, True, 1.0, 0),
    (4, 8192, FL, "channel", True, True, True, -1.0, 0),
    (3, 8191, HF, "channel", True, True, True, 1.0, 0),
    (3, 4097, FL, "token", True, True, True, 1.0, 0),
    (9, 256, BF, "none", False, False, True, 1.0, 0),       # the norm before the first block
    (9, 2055, BF, "none", False, True, True, 1.0, 0),
    (300, 512, BF, "channel", True, True, False, 1.0, 0),   # after the last block
    (700, 320, HF, "token", False, True, True, 0.25, 1),
    (1000, 64, BF, "channel", False, True, True, 1.0, 1),
    (2100, 136, FL, "channel", True, True, True, 1.0, 0),
    (33, 2048, FL, "none", True, False, False, 1.0, 1),
    (701, 322, HF, "token", True, True, True, 0.25, 0),     # rows of pairs
    (301, 1026, BF, "channel", True, True, True, 1.0, 2),
    (150, 2048, BF, "none", True, True, True, 1.0, 2),
    (5, 6002, HF, "channel", True, False, True, 1.414, 0),
    (701, 321, HF, "token", True, True, True, 0.25, 0),     # rows that start in turn on a pair and inside one
    (301, 1023, BF, "channel", True, True, True, 1.0, 3),
    (150, 3071, BF, "none", True, True, True, 1.0, 0),
    (1, 3071, HF, "channel", True, True, True, 1.0, 1),
    (2, 3072, BF, "channel", True, True, True, 1.0, 1),
    (5, 6001, HF, "channel", True, False, True, 1.414, 0),
    (3, 4095, BF, "token", False, True, True, 1.0, 0),
    (4, 8192, BF, "channel", True, True, True, 1.0, 1),
    (7301, 17, BF, "token", True, True, True, 1.0, 0),
    (900, 1, HF, "channel", True, True, True, 1.0, 0),
    (7300, 18, BF, "token", True, True, True, 1.0, 0),      # 24 tokens in a block
    (7300, 24, BF, "channel", True, True, True, 1.0, 0),
]
NAMES = [f"T{c[0]}D{c[1]}{c[3]}{int(c[4])}{int(c[5])}{int(c[6])}" for c in CASES]


def make(case, seed=0):
    T, D, dt, mode, post, res, nxt, alpha, off = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    vec = lambda n, m, s: torch.randn(n, generator=g, device="cuda") * s + m      # noqa: E731
    a = {"y": shifted((T, D), dt, off, seed=seed + 1), "alpha": alpha, "gate_mode": mode,
         "residual": shifted((T, D), dt, off, seed=seed + 2) if res else None,
         "gate": {"none": None, "channel": vec(D, 0.8, 0.3), "token": vec(T, 0.8, 0.3)}[mode],
         "w_post": vec(D, 1.0, 0.2) if post else None, "w_next": vec(D, 1.0, 0.2) if nxt else None}
    a["y"].mul_(0.7)
    return a


def forward(a, off=0, keep=True):
    T, D = a["y"].shape
    dt = a["y"].dtype
    o = {"x_out": shifted((T, D), dt, off, fill=9.0),
         "normed": None if a["w_next"] is None else shifted((T, D), dt, off, fill=9.0),
         "rstd_post": torch.full((T,), 9.0, device="cuda") if keep and a["w_post"] is not None else None,
         "rstd_next": torch.full((T,), 9.0, device="cuda") if keep and a["w_next"] is not None else None}
    moe.moe_block_norm(**a, **o, eps=EPS)
    return o


@pytest.mark.parametrize("case", CASES, ids=NAMES)
def test_forward(case):
    T, D, dt, mode, post, res, nxt, alpha, off = case
    a = make(case)
    o = forward(a, off)
    x, err, rp = ref.norm(f64(a["y"]), f64(a["residual"]), np.float32(alpha).astype(np.float64), f64(a["gate"]), mode,
                          f64(a["w_post"]), EPS)
    check(o["x_out"], x, stored(x, err, dt), "x_out")
    if post:
        check(o["rstd_post"], rp, rp * (D / 2 + 6) * U32, "rstd_post")
    if nxt:                                                 # of x_out as it is stored
        n, e, r = ref.next_norm(f64(o["x_out"]), f64(a["w_next"]), EPS)
        check(o["normed"], n, stored(n, e, dt), "normed")
        check(o["rstd_next"], r, r * (D / 2 + 6) * U32, "rstd_next")
        # without x_out, without the kept factors, or with x_out in place of the residual: the same
        lone = shifted((T, D), dt, off, fill=9.0)
        moe.moe_block_norm(**a, normed=lone, eps=EPS)
        assert torch.equal(lone, o["normed"])
        if res:
            b = dict(a, residual=shifted((T, D), dt, off, fill=0.0).copy_(a["residual"]))   # laid out alike
            moe.moe_block_norm(**b, x_out=b["residual"], normed=lone, eps=EPS)
            assert torch.equal(lone, o["normed"]) and torch.equal(b["residual"], o["x_out"])
        # two calls: the block's end, then the next block's norm
        moe.moe_block_norm(o["x_out"], w_next=a["w_next"], normed=lone, eps=EPS)
        assert torch.equal(lone, o["normed"])


def backward(a, o, dx_out, dnormed, off=0, ws=None, drop=()):
    T, D = a["y"].shape
    dt = a["y"].dtype
    new = lambda v: None if v is None else torch.full_like(v, 9.0)      # noqa: E731
    g = {"dy": shifted((T, D), dt, off, fill=9.0), "dresidual": shifted((T, D), dt, off, fill=9.0),
         "dgate": new(a["gate"]), "dw_post": new(a["w_post"]), "dw_next": new(a["w_next"])}
    g |= {n: None for n in drop}
    if ws is None:                                          # no initialisation asked for
        ws = torch.full((moe.block_norm_backward_workspace_size(T, D),), 255, dtype=torch.uint8, device="cuda")
    moe.moe_block_norm_backward(dx_out, dnormed, o["x_out"], a["y"], ws=ws, alpha=a["alpha"], gate=a["gate"],
                                gate_mode=a["gate_mode"], w_post=a["w_post"], w_next=a["w_next"],
                                rstd_post=o["rstd_post"], rstd_next=o["rstd_next"], **g)
    return g


@pytest.mark.parametrize("case", CASES, ids=NAMES)
def test_backward(case):
    T, D, dt, mode, post, res, nxt, alpha, off = case
    a = make(case, 3)
    o = forward(a, off)
    dn = shifted((T, D), dt, off, seed=21) if nxt else None
    for dx_out in (shifted((T, D), dt, off, seed=20), None) if nxt else (shifted((T, D), dt, off, seed=20),):
        g = backward(a, o, dx_out, dn, off)
        al = np.float32(alpha).astype(np.float64)
        want = ref.norm_backward(f64(dx_out), f64(dn), f64(o["x_out"]), f64(a["y"]), al, f64(a["gate"]), mode,
                                 f64(a["w_post"]), f64(a["w_next"]), EPS)
        for n, (v, e) in want.items():
            check(g[n], v, stored(v, e, dt if n in ("dy", "dresidual") else FL), n)
        again = backward(a, o, dx_out, dn, off)
        assert all(v is None or torch.equal(v, again[n]) for n, v in g.items())
        few = backward(a, o, dx_out, dn, off, drop=("dresidual", "dgate", "dw_post", "dw_next"))
        assert torch.equal(few["dy"], g["dy"])
        if dx_out is not None:                              # dresidual in place of dx_out
            b = dx_out.clone() if off == 0 else dx_out
            moe.moe_block_norm_backward(b, dn, o["x_out"], a["y"], few["dy"], moe.alloc_ws(
                moe.block_norm_backward_workspace_size(T, D)), dresidual=b, alpha=alpha, gate=a["gate"], gate_mode=mode,
                w_post=a["w_post"], w_next=a["w_next"], rstd_post=o["rstd_post"], rstd_next=o["rstd_next"])
            assert torch.equal(b, g["dresidual"]) and torch.equal(few["dy"], g["dy"])


@pytest.mark.parametrize("T,D,dt", [(300, 1000, BF), (5, 6001, HF), (700, 33, BF), (20, 3072, HF)])
def test_matrices_that_start_differently(T, D, dt):
    """Outputs and inputs at different offsets from a 4-byte boundary: single elements."""
    case = (T, D, dt, "channel", True, True, True, 0.5, 1)
    a = make(case, 5)
    o = forward(a, 0)
    x, err, _ = ref.norm(f64(a["y"]), f64(a["residual"]), 0.5, f64(a["gate"]), "channel", f64(a["w_post"]), EPS)
    check(o["x_out"], x, stored(x, err, dt), "x_out")
    n, e, _ = ref.next_norm(f64(o["x_out"]), f64(a["w_next"]), EPS)
    check(o["normed"], n, stored(n, e, dt), "normed")
    dx_out, dn = shifted((T, D), dt, 2, seed=20), shifted((T, D), dt, 3, seed=21)
    g = backward(a, o, dx_out, dn, 0)
    want = ref.norm_backward(f64(dx_out), f64(dn), f64(o["x_out"]), f64(a["y"]), 0.5, f64(a["gate"]), "channel",
                             f64(a["w_post"]), f64(a["w_next"]), EPS)
    for n, (v, e) in want.items():
        check(g[n], v, stored(v, e, dt if n in ("dy", "dresidual") else FL), n)


@pytest.mark.parametrize("mode", ["none", "channel", "token"])
def test_gradients_against_differences(mode):
    """The loss <c, x_out> + <d, normed> in 64 bits, its central differences along random directions.  With h = 1e-4
    and directions of length 1 they are off by about h^2 times the loss's third derivative, here below 1e2."""
    T, D = 5, 24
    a = make((T, D, FL, mode, True, True, True, 0.5, 0), 7)
    o = forward(a)
    c, d = shifted((T, D), FL, 0, seed=1), shifted((T, D), FL, 0, seed=2)
    g = backward(a, o, c, d)
    base = {n: f64(a[n]) for n in ("y", "residual", "gate", "w_post", "w_next") if a[n] is not None}

    def loss(v):
        x, _, _ = ref.norm(v["y"], v["residual"], 0.5, v.get("gate"), mode, v["w_post"], EPS)
        return float((f64(c) * x).sum() + (f64(d) * ref.next_norm(x, v["w_next"], EPS)[0]).sum())

    want = ref.norm_backward(f64(c), f64(d), f64(o["x_out"]), base["y"], 0.5, base.get("gate"), mode, base["w_post"],
                             base["w_next"], EPS)
    rng, h = np.random.default_rng(1), 1e-4
    for n, out in (("y", "dy"), ("residual", "dresidual"), ("gate", "dgate"), ("w_post", "dw_post"),
                   ("w_next", "dw_next")):
        if n not in base:
            continue
        v = rng.standard_normal(base[n].shape)
        v /= np.linalg.norm(v)
        num = (loss(base | {n: base[n] + h * v}) - loss(base | {n: base[n] - h * v})) / (2 * h)
        # x_out is stored in fp32 and read back: u32 of it, through the second derivative (below 1e2)
        tol = (stored(*want[out], FL) * np.abs(v)).sum() + h * h * 1e2 + U32 * 1e2 * np.abs(f64(o["x_out"])).sum()
        assert abs(num - (f64(g[out]) * v).sum()) <= tol, (n, num, (f64(g[out]) * v).sum(), tol)


def test_rows_without_variance_and_extremes():
    """Rows of zeros (the norm is 0 / sqrt(eps)), of the type's largest values in fp16 after the sum, and NaN in one
    token: the other tokens do not see it."""
    T, D = 4, 64
    a = make((T, D, HF, "channel", True, True, True, 1.0, 0), 2)
    a["y"][0] = 0
    a["residual"][0] = 0
    a["y"][2, 5] = float("nan")
    o = forward(a)
    assert (o["x_out"][0] == 0).all() and (o["normed"][0] == 0).all()
    assert torch.isnan(o["normed"][2]).all() and torch.isfinite(o["normed"][[0, 1, 3]]).all()
    g = backward(a, o, shifted((T, D), HF, 0, seed=5) * 1e-3, shifted((T, D), HF, 0, seed=6) * 1e-3)
    assert torch.isfinite(g["dy"][[0, 1, 3]]).all() and torch.isnan(g["dy"][2]).any()


def test_no_tokens():
    z, w = torch.zeros(0, 16, device="cuda"), torch.ones(16, device="cuda")
    moe.moe_block_norm(z, z, w_next=w, normed=z)
    ws = moe.alloc_ws(moe.block_norm_backward_workspace_size(0, 16))
    r, dw = torch.zeros(0, device="cuda"), torch.ones(16, device="cuda")
    moe.moe_block_norm_backward(z, z, z, z, z, ws, w_next=w, rstd_next=r, dw_next=dw)
    assert (dw == 0).all()


def test_captured():
    case = (40, 256, BF, "channel", True, True, True, 1.0, 0)
    a, b = make(case, 1), make(case, 2)
    hold = {n: v.clone() if isinstance(v, torch.Tensor) else v for n, v in a.items()}
    dx, dn = shifted((40, 256), BF, 0, seed=3), shifted((40, 256), BF, 0, seed=4)
    ws = moe.alloc_ws(moe.block_norm_backward_workspace_size(40, 256))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        backward(hold, forward(hold), dx, dn, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = forward(hold)
        g = backward(hold, o, dx, dn, ws=ws)
    for m in (b, a):
        for n, v in m.items():
            if isinstance(v, torch.Tensor):
                hold[n].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        o2 = forward(m)
        g2 = backward(m, o2, dx, dn)
        assert all(torch.equal(v, o2[n]) for n, v in o.items()) and all(torch.equal(v, g2[n]) for n, v in g.items())
