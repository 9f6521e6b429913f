"""64-bit forms for large batches, in torch on the GPU, with the bounds of
tests/ops_ref.py: the router's gradient as products of dense matrices, and the
norms a block of tokens at a time."""
import torch

from tests.ops_ref import TINY, U, U32


def stored(want, err, dtype):
    return 1.01 * err + U[dtype] * (want.abs() + 1.01 * err) + TINY[dtype]


def check(got, want, bound, what):
    assert got.shape == want.shape, what
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist(),
                           bound.expand_as(want)[bad][:4].tolist())


def route_backward(dgates, gates, ids, x, Wr, dx_add=None, terms=1):
    """dlogits, dx, dWr, dbias, each with a bound on its fp32 error.

    terms: additions per pair in the sums of dx and dWr, in steps of u32.  One by one they are 1.  On the tensor cores
    a pair comes as three exact terms, each added with an error of at most two (a sum may be cut off instead of
    rounded): 6."""
    T, k = ids.shape
    E, D = Wr.shape
    inside = (ids >= 0) & (ids < E)
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    g, dg = torch.where(inside, gates.double(), zero), torch.where(inside, dgates.double(), zero)
    dl = g * (dg - (g * dg).sum(1, keepdim=True))
    e_dl = g.abs() * ((k + 3) * U32 * (dg.abs() + (g * dg).abs().sum(1, keepdim=True)))
    at = torch.where(inside, ids.long(), E)

    def spread(v):                              # [T, E]: the token's values at their experts
        return torch.zeros(T, E + 1, dtype=torch.float64, device=x.device).scatter_add_(1, at, v)[:, :E]

    x, Wr = x.double(), Wr.double()
    S, A, B = spread(dl), spread(dl.abs()), spread(e_dl)
    n = torch.bincount(at.reshape(-1), minlength=E + 1)[:E]
    dx, e_dx = S @ Wr, (B + (terms * k + 1) * U32 * A) @ Wr.abs()
    if dx_add is not None:
        dx, e_dx = dx + dx_add.double(), e_dx + (terms * k + 1) * U32 * dx_add.double().abs()
    e_W = B + (terms * n + 1) * U32 * A
    e_b = B + (n + 1) * U32 * A
    return (dl, e_dl), (dx, e_dx), (S.t() @ x, e_W.t() @ x.abs()), (S.sum(0), e_b.sum(0))


def norm(y, residual, alpha, gate, w_post, w_next, eps):
    """x_out with the bound of its fp32 error; a channel gate, every operand given."""
    D = y.shape[1]
    z = y * (1 / ((y * y).mean(1, keepdim=True) + eps).sqrt()) * w_post * gate
    x = alpha * residual + z
    return x, z.abs() * (D / 2 + 11) * U32 + U32 * (x.abs() + (alpha * residual).abs())


def next_norm(x, w_next, eps):
    v = x * (1 / ((x * x).mean(1, keepdim=True) + eps).sqrt()) * w_next
    return v, v.abs() * (x.shape[1] / 2 + 10) * U32


def norm_backward(dx_out, dnormed, x, y, alpha, gate, w_post, w_next, eps):
    """dy, dresidual and this block of tokens' part of dgate, dw_post, dw_next, each with its terms' magnitudes."""
    r = 1 / ((x * x).mean(1, keepdim=True) + eps).sqrt()
    xh, u = x * r, dnormed * w_next
    G = dx_out + r * (u - xh * (xh * u).mean(1, keepdim=True))
    a = dx_out.abs() + r * (u.abs() + xh.abs() * (xh * u).abs().mean(1, keepdim=True))
    ry = 1 / ((y * y).mean(1, keepdim=True) + eps).sqrt()
    yh = y * ry
    v, a_v = gate * G * w_post, gate.abs() * a * w_post.abs()
    dy = ry * (v - yh * (yh * v).mean(1, keepdim=True))
    a_dy = ry * (a_v + yh.abs() * (yh.abs() * a_v).mean(1, keepdim=True))
    return {"dy": (dy, a_dy), "dresidual": (alpha * G, abs(alpha) * a),
            "dgate": ((G * yh * w_post).sum(0), (a * (yh * w_post).abs()).sum(0)),
            "dw_post": ((gate * G * yh).sum(0), (gate.abs() * a * yh.abs()).sum(0)),
            "dw_next": ((dnormed * xh).sum(0), (dnormed * xh).abs().sum(0))}
