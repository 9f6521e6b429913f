"""Plain 64-bit forms of the operators of moe_ops.h, written from their formulas
with numpy loops over tokens and pairs, and the error bounds that their tests use.

Bounds.  u32 = 2^-24 is half a step of fp32 relative to the value, u(t) the same
of the stored type t.  A sum of n products formed in fp32, in any order, is off by
at most n * u32 * sum |terms| (first order; 1.01 covers the higher ones, as n * u32
stays below 1e-3).  Storing adds u(t) * |value|, and half the smallest subnormal
where the value is below the type's normal range."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U32}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def stored(want, err, dtype):
    """Bound on |stored - want| for an fp32 result within err of want, rounded once to dtype."""
    return 1.01 * err + U[dtype] * (np.abs(want) + 1.01 * err) + TINY[dtype]


def check(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4],
                           np.broadcast_to(bound, want.shape)[bad][:4])


# ---------------------------------------------------------------- permutation
def plan(ids, E, slot_table=None, n_slots=0):
    """offsets, pair_row [T][k], and the taken pairs in row order."""
    T, k = ids.shape
    lists = [[] for _ in range(E)]
    for p, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E and (slot_table is None or not 0 <= slot_table[e] < n_slots):
            lists[e].append(p)
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in lists])]).astype(np.int32)
    order = np.array([p for v in lists for p in v], np.int32)
    pair_row = np.full(T * k, -1, np.int32)
    pair_row[order] = np.arange(len(order))
    return offsets, pair_row.reshape(T, k), order


def unpermute(rows, pair_row, weights):
    """The sum, and the sum of the terms' magnitudes."""
    T, k = pair_row.shape
    out = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(out)
    for t in range(T):
        for r in range(k):
            if 0 <= pair_row[t, r] < len(rows):
                v = (1.0 if weights is None else weights[t, r]) * rows[pair_row[t, r]]
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


def unpermute_backward(dout, rows, pair_row, weights):
    """drows, the rows it holds, dweights and the magnitudes of their sums."""
    T, k = pair_row.shape
    drows, held = np.zeros(rows.shape), np.zeros(len(rows), bool)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for r in range(k):
            i = pair_row[t, r]
            if 0 <= i < len(rows):
                drows[i] = (1.0 if weights is None else weights[t, r]) * dout[t]
                held[i] = True
                dw[t, r] = np.sum(dout[t] * rows[i])
                mag[t, r] = np.sum(np.abs(dout[t] * rows[i]))
    return drows, held, dw, mag


# ---------------------------------------------------------------- router
def route_backward(dgates, gates, ids, x, Wr, dx_add=None):
    """dlogits, dx, dWr, dbias, each with a bound on its fp32 error."""
    T, k = ids.shape
    E, D = Wr.shape
    inside = (ids >= 0) & (ids < E)
    g = np.where(inside, gates, 0.0)
    dg = np.where(inside, dgates, 0.0)
    s = (g * dg).sum(1, keepdims=True)
    dl = g * (dg - s)
    e_dl = np.abs(g) * ((k + 3) * U32 * (np.abs(dg) + (np.abs(g * dg)).sum(1, keepdims=True)))
    dx = np.zeros((T, D)) if dx_add is None else dx_add.copy()
    e_dx = (k + 1) * U32 * np.abs(dx)
    dW, e_dW = np.zeros((E, D)), np.zeros((E, D))
    db, e_db = np.zeros(E), np.zeros(E)
    n = np.bincount(ids[inside], minlength=E)
    for t in range(T):
        for r in range(k):
            if not inside[t, r]:
                continue
            e = ids[t, r]
            dx[t] += dl[t, r] * Wr[e]
            e_dx[t] += (e_dl[t, r] + (k + 1) * U32 * np.abs(dl[t, r])) * np.abs(Wr[e])
            dW[e] += dl[t, r] * x[t]
            e_dW[e] += (e_dl[t, r] + (n[e] + 1) * U32 * np.abs(dl[t, r])) * np.abs(x[t])
            db[e] += dl[t, r]
            e_db[e] += e_dl[t, r] + (n[e] + 1) * U32 * np.abs(dl[t, r])
    return (dl, e_dl), (dx, e_dx), (dW, e_dW), (db, e_db)


# ---------------------------------------------------------------- block norm
def norm(y, residual, alpha, gate, gate_mode, w_post, eps):
    """x_out before it is stored, a bound on its fp32 error, and rstd_post."""
    T, D = y.shape
    z, rp = y, None
    e_z = np.zeros_like(y)
    if w_post is not None:
        rp = 1 / np.sqrt((y * y).mean(1) + eps)
        z = y * rp[:, None] * w_post
        # mean of D squares, its square root's half of that, rsqrt (2 steps) and two products
        e_z = np.abs(z) * (D / 2 + 10) * U32
    if gate is not None:
        m = gate[None, :] if gate_mode == "channel" else gate[:, None]
        z, e_z = z * m, e_z * np.abs(m) + np.abs(z * m) * U32
    x = z if residual is None else alpha * residual + z
    # one fused multiply-add; alpha itself is rounded to fp32 once
    err = e_z + U32 * (np.abs(x) + (0 if residual is None else np.abs(alpha * residual)))
    return x, err, rp


def next_norm(x, w_next, eps):
    D = x.shape[1]
    r = 1 / np.sqrt((x * x).mean(1) + eps)
    v = x * r[:, None] * w_next
    return v, np.abs(v) * (D / 2 + 10) * U32, r


def norm_backward(dx_out, dnormed, x, y, alpha, gate, gate_mode, w_post, w_next, eps):
    """Every gradient with a bound on its fp32 error.  The bounds carry the magnitudes of all terms (a) through the
    formula; each fp32 operation and each reduction over D adds (D + 24) u32 of them, and there are three such
    stages one after the other (the first norm's mean, the second's, and the sum over tokens adds T u32)."""
    T, D = x.shape if x is not None else dx_out.shape
    G = np.zeros((T, D)) if dx_out is None else dx_out
    a = np.abs(G)
    dwn = a_dwn = None
    if w_next is not None:
        r = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
        xh, u = x * r, dnormed * w_next
        G = G + r * (u - xh * (xh * u).mean(1, keepdims=True))
        a = a + r * (np.abs(u) + np.abs(xh) * np.abs(xh * u).mean(1, keepdims=True))
        dwn, a_dwn = (dnormed * xh).sum(0), np.abs(dnormed * xh).sum(0)
    yh, z, ry = y, y, 1.0
    if w_post is not None:
        ry = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
        yh = y * ry
        z = yh * w_post
    m, dgate, a_dgate = 1.0, None, None
    if gate is not None:
        m = gate[None, :] if gate_mode == "channel" else gate[:, None]
        ax = 0 if gate_mode == "channel" else 1
        dgate, a_dgate = (G * z).sum(ax), (a * np.abs(z)).sum(ax)
    dz, a_dz = m * G, np.abs(m) * a
    dy, a_dy, dwp, a_dwp = dz, a_dz, None, None
    if w_post is not None:
        v, a_v = dz * w_post, a_dz * np.abs(w_post)
        dy = ry * (v - yh * (yh * v).mean(1, keepdims=True))
        a_dy = ry * (a_v + np.abs(yh) * (np.abs(yh) * a_v).mean(1, keepdims=True))
        dwp, a_dwp = (dz * yh).sum(0), (a_dz * np.abs(yh)).sum(0)
    e = 3 * (D + 24) * U32
    et = e + (T + 8) * U32
    out = {"dy": (dy, e * a_dy), "dresidual": (alpha * G, (e + U32) * np.abs(alpha) * a)}
    if dgate is not None:
        out["dgate"] = (dgate, et * a_dgate)
    if dwp is not None:
        out["dw_post"] = (dwp, et * a_dwp)
    if dwn is not None:
        out["dw_next"] = (dwn, et * a_dwn)
    return out
