"""What the operators around the expert pass are measured on: tokens sorted by
expert and back (with gate weights), their gradients, the router's gradient,
and the norms between two layers' blocks with their gradient.

``run`` computes an operator in plain torch where ``own`` is false, and through
``bit_expert_ffn_route_b200.moe`` where it is true; both return the same
tensors.  ``exact`` computes them in 64 bits, by another route.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    def tokens(name, op, T, E, k, D, dtype, miss=1.0, skew=0.8, out="same"):
        return {"name": name, "op": op, "T": T, "E": E, "k": k, "D": D, "dtype": dtype, "miss": miss, "skew": skew,
                "out": out}

    def norm(name, op, T, D, dtype, gate, post=True, alpha=1.0):
        return {"name": name, "op": op, "T": T, "D": D, "dtype": dtype, "gate": gate, "post": post, "alpha": alpha}

    return [
        # A decode step of 4 tokens (one and three drafts): the pairs whose expert is not resident, gathered for
        # whoever computes them.  Latency.
        tokens("permute_decode_misses", "permute", 4, 512, 10, 3072, "bf16", miss=0.375),
        # A prefill chunk, every pair, as a caller's own experts would take it.
        tokens("permute_chunk", "permute", 4096, 512, 10, 3072, "bf16"),
        # The gradient with respect to the tokens of a long ragged batch: narrow fp32 rows of an odd width, few experts.
        tokens("permute_grad_ragged", "permute_grad", 20011, 60, 3, 1001, "f32", skew=0.0),
        # The decode step's missed pairs back into an fp32 partial sum.
        tokens("unpermute_decode_misses", "unpermute", 24, 512, 10, 3072, "bf16", miss=0.375, out="f32"),
        # The prefill chunk back, weighted.
        tokens("unpermute_chunk", "unpermute", 4096, 512, 10, 3072, "bf16"),
        # Its gradient: the rows' and the weights'.
        tokens("unpermute_grad_chunk", "unpermute_grad", 4096, 512, 10, 3072, "bf16"),
        # An odd width in fp16 over the 256-expert shape, a third of the pairs elsewhere.
        tokens("unpermute_grad_odd", "unpermute_grad", 777, 256, 7, 2055, "f16", miss=0.66),
        # The router's gradient: a small batch over the 256-expert shape, and the prefill chunk.
        tokens("route_grad_small", "route_grad", 100, 256, 10, 3072, "bf16"),
        tokens("route_grad_chunk", "route_grad", 4096, 512, 10, 3072, "bf16"),
        # Between two layers: one token of a decode step, a prefill chunk, and its gradient.
        norm("norm_token", "norm", 1, 3072, "bf16", "channel"),
        norm("norm_chunk", "norm", 4096, 3072, "bf16", "channel"),
        norm("norm_grad_chunk", "norm_grad", 4096, 3072, "bf16", "channel"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "permute_grad", "unpermute", "unpermute_grad", "route_grad", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    T = _spread(rng, 1, 20000)
    if op in ("norm", "norm_grad"):
        D = _spread(rng, 16, 8192)
        T = max(1, min(T, (1 << 26) // (D * BYTES[dtype])))
        return {"op": op, "T": T, "D": D, "dtype": dtype, "gate": rng.choice(["none", "channel", "token"]),
                "post": rng.random() < 0.7, "alpha": rng.choice([1.0, 0.5, 1.414])}
    k = rng.randint(1, 16)
    E = max(k, _spread(rng, 4, 1024))
    D = _spread(rng, 16, 8192)
    if op == "route_grad":                      # the router's own types and widths
        dtype, D = "bf16", 256 * _spread(rng, 1, 32)
    elif rng.random() < 0.5:
        D = max(8, D // 8 * 8)
    T = max(1, min(T, (1 << 27) // (k * D * BYTES[dtype])))
    return {"op": op, "T": T, "E": E, "k": k, "D": D, "dtype": dtype,
            "miss": 1.0 if op == "route_grad" else rng.choice([1.0, 1.0, 0.375, 0.07]), "skew": rng.choice([0.0, 0.8]),
            "out": rng.choice(["same", "f32"]) if op.startswith("unpermute") else "same"}


def work(case):
    T, D, es = case["T"], case["D"], BYTES[case["dtype"]]
    if case["op"] == "norm":                    # y and the residual in, their sum and its norm out
        return {"bytes": 4.0 * T * D * es, "flops": 12.0 * T * D}
    if case["op"] == "norm_grad":               # two gradients, the sum and y in; two gradients out
        return {"bytes": 6.0 * T * D * es + 16.0 * D, "flops": 30.0 * T * D}
    E, k = case["E"], case["k"]
    P = T * k
    N = P * case["miss"]
    eo = 4 if case["out"] == "f32" else es
    tok = T * min(1.0, 1 - (1 - case["miss"]) ** k)     # tokens with a pair among those taken
    if case["op"] == "permute":
        return {"bytes": (tok + N) * D * es + 12.0 * P + 4 * E, "flops": 0.0}
    if case["op"] == "permute_grad":
        return {"bytes": (N + T) * D * es + 4.0 * P, "flops": N * D}
    if case["op"] == "unpermute":
        return {"bytes": N * D * es + T * D * eo + 8.0 * P, "flops": 2.0 * N * D}
    if case["op"] == "unpermute_grad":
        return {"bytes": 2.0 * N * D * es + tok * D * eo + 12.0 * P, "flops": 3.0 * N * D}
    return {"bytes": 4.0 * T * D + 6.0 * E * D + 20.0 * P, "flops": 4.0 * P * D}        # route_grad


# ------------------------------------------------------------------ inputs
def _plan(ids, E, absent):
    """Rows in expert order, pairs in order within an expert.  absent: truth value per expert, or None (all pairs)."""
    P = ids.numel()
    flat = ids.reshape(-1).long()
    key = flat if absent is None else torch.where(absent[flat], flat, E)
    key, order = torch.sort(key, stable=True)
    place = torch.arange(P, device=ids.device)
    taken = key < E
    count = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = count[:E].cumsum(0)
    pair_row = torch.empty(P, dtype=torch.int32, device=ids.device)
    pair_row[order] = torch.where(taken, place, -1).int()
    row_pair = torch.where(taken, order, -1).int()
    return offsets, pair_row.view(ids.shape), row_pair


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, D, dt = case["T"], case["D"], DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    def room(*shape, dtype=dt):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    s = {"case": case}
    if case["op"] in ("norm", "norm_grad"):
        f32 = torch.float32
        s["y"] = normal(T, D, std=0.7)
        s["residual"] = normal(T, D, std=2.0)
        s["w_post"] = normal(D, std=0.1, mean=1.0, dtype=f32) if case["post"] else None
        s["w_next"] = normal(D, std=0.1, mean=1.0, dtype=f32)
        s["gate"] = {"none": None, "channel": normal(D, std=0.2, mean=0.8, dtype=f32),
                     "token": torch.sigmoid(normal(T, dtype=f32))}[case["gate"]]
        if case["op"] == "norm":
            s["x_out"], s["normed"] = room(T, D), room(T, D)
            return s
        # what a training step kept of its forward pass
        s["x_out"], _, s["rstd_post"], s["rstd_next"] = _norm(s)
        s["dx_out"], s["dnormed"] = normal(T, D, std=1e-2), normal(T, D, std=1e-2)
        s["dy"], s["dresidual"] = room(T, D), room(T, D)
        s["dw_post"] = room(D, dtype=f32) if case["post"] else None
        s["dw_next"] = room(D, dtype=f32)
        s["dgate"] = None if s["gate"] is None else torch.zeros_like(s["gate"])
        return s
    E, k, P = case["E"], case["k"], T * case["k"]
    # popularity falls with a power of the rank; tokens draw distinct experts by it
    rank = torch.randperm(E, generator=g, device="cuda").float() + 1
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-12, 1 - 1e-7)
    scores, ids = torch.topk(-case["skew"] * torch.log(rank) - torch.log(-torch.log(u)), k, dim=1)
    s["ids"], s["gates"] = ids.int(), torch.softmax(scores, dim=1)
    s["slot_table"], s["n_slots"] = None, 0
    absent = None
    if case["miss"] < 1:                        # slots for the resident experts, the others missed
        absent = torch.rand(E, generator=g, device="cuda") < case["miss"]
        s["slot_table"] = torch.where(absent, -1, torch.arange(E, device="cuda")).int()
        s["n_slots"] = E
    s["absent"] = absent
    if case["op"] == "permute":
        s["x"] = normal(T, D)
        s["rows"] = room(P, D)
        s["offsets"] = room(E + 1, dtype=torch.int32)
        s["pair_row"] = room(T, k, dtype=torch.int32)
        s["row_pair"] = torch.full((P,), -1, dtype=torch.int32, device="cuda")
        return s
    s["offsets"], s["pair_row"], s["row_pair"] = _plan(s["ids"], E, absent)
    if case["op"] == "permute_grad":
        s["drows"], s["dx"] = normal(P, D), room(T, D)
    elif case["op"] == "unpermute":
        s["rows"], s["out"] = normal(P, D), room(T, D, dtype=torch.float32 if case["out"] == "f32" else dt)
    elif case["op"] == "unpermute_grad":
        s["rows"], s["drows"] = normal(P, D), room(P, D)
        s["dout"] = normal(T, D, dtype=torch.float32 if case["out"] == "f32" else dt)
        s["dweights"] = room(T, k, dtype=torch.float32)
    else:
        s["x"], s["Wr"] = normal(T, D), normal(E, D, std=0.02)
        s["dgates"] = normal(T, k, std=0.1, dtype=torch.float32)
        s["dlogits"], s["dx"] = room(T, k, dtype=torch.float32), room(T, D)
        s["dWr"], s["dbias"] = room(E, D, dtype=torch.float32), room(E, dtype=torch.float32)
    return s


# ------------------------------------------------------------------ plain forms
def _norm(s):
    case, dt = s["case"], s["y"].dtype
    z, rstd_post = s["y"].float(), None
    if s["w_post"] is not None:
        rstd_post = torch.rsqrt(z.square().mean(1) + EPS)
        z = z * rstd_post[:, None] * s["w_post"]
    if s["gate"] is not None:
        z = z * (s["gate"] if case["gate"] == "channel" else s["gate"][:, None])
    x_out = (case["alpha"] * s["residual"].float() + z).to(dt)      # the next block's norm reads what is stored
    xf = x_out.float()
    rstd_next = torch.rsqrt(xf.square().mean(1) + EPS)
    return x_out, (xf * rstd_next[:, None] * s["w_next"]).to(dt), rstd_post, rstd_next


def _norm_grad(s):
    case, dt = s["case"], s["y"].dtype
    xh = s["x_out"].float() * s["rstd_next"][:, None]
    dn = s["dnormed"].float()
    u = dn * s["w_next"]
    G = s["dx_out"].float() + s["rstd_next"][:, None] * (u - xh * (xh * u).mean(1, keepdim=True))
    yf = s["y"].float()
    yh = yf if s["w_post"] is None else yf * s["rstd_post"][:, None]
    z = yh if s["w_post"] is None else yh * s["w_post"]
    dz, dgate = G, None
    if case["gate"] == "channel":
        dz, dgate = G * s["gate"], (G * z).sum(0)
    elif case["gate"] == "token":
        dz, dgate = G * s["gate"][:, None], (G * z).sum(1)
    dy, dw_post = dz, None
    if s["w_post"] is not None:
        v = dz * s["w_post"]
        dy, dw_post = s["rstd_post"][:, None] * (v - yh * (yh * v).mean(1, keepdim=True)), (dz * yh).sum(0)
    return dy.to(dt), (case["alpha"] * G).to(dt), dgate, dw_post, (dn * xh).sum(0)


def _of_pairs(rows, pair_row):
    """[T, k, D] in 32 bits: the row of every pair, zero where it has none."""
    v = rows[pair_row.clamp(min=0).long()].float()
    return torch.where((pair_row >= 0)[:, :, None], v, torch.zeros((), device=v.device))


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        return _norm(s)[:2]
    if op == "norm_grad":
        return _norm_grad(s)
    T, E, k = case["T"], case["E"], case["k"]
    if op == "permute":
        offsets, pair_row, row_pair = _plan(s["ids"], E, s["absent"])
        x = s["x"]
        rows = torch.where((row_pair >= 0)[:, None], x[(row_pair.clamp(min=0) // k).long()],
                           torch.zeros((), dtype=x.dtype, device=x.device))
        return rows, offsets, pair_row, row_pair
    if op == "permute_grad":
        return _of_pairs(s["drows"], s["pair_row"]).sum(1).to(s["drows"].dtype)
    if op == "unpermute":
        return (s["gates"][:, :, None] * _of_pairs(s["rows"], s["pair_row"])).sum(1).to(s["out"].dtype)
    if op == "unpermute_grad":
        dout, held = s["dout"].float(), s["row_pair"] >= 0
        pair = s["row_pair"].clamp(min=0).long()
        drows = torch.where(held[:, None], s["gates"].reshape(-1)[pair][:, None] * dout[pair // k],
                            torch.zeros((), device=dout.device)).to(s["rows"].dtype)
        return drows, (_of_pairs(s["rows"], s["pair_row"]) * dout[:, None, :]).sum(2)
    g, dg = s["gates"], s["dgates"]
    dl = g * (dg - (g * dg).sum(1, keepdim=True))
    dense = torch.zeros(T, E, device=dl.device).scatter_add_(1, s["ids"].long(), dl)
    return dl, (dense @ s["Wr"].float()).to(s["x"].dtype), dense.t() @ s["x"].float(), dense.sum(0)


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    from bit_expert_ffn_route_b200 import moe
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        moe.moe_block_norm(s["y"], s["x_out"], residual=s["residual"], alpha=case["alpha"], gate=s["gate"],
                           gate_mode=case["gate"], w_post=s["w_post"], w_next=s["w_next"], normed=s["normed"],
                           eps=EPS)
        return s["x_out"], s["normed"]
    if op == "norm_grad":
        if "ws" not in s:                       # a program keeps its workspace
            s["ws"] = moe.alloc_ws(moe.block_norm_backward_workspace_size(case["T"], case["D"]))
        moe.moe_block_norm_backward(s["dx_out"], s["dnormed"], s["x_out"], s["y"], s["dy"], s["ws"],
                                    dresidual=s["dresidual"], alpha=case["alpha"], gate=s["gate"],
                                    gate_mode=case["gate"], dgate=s["dgate"], w_post=s["w_post"],
                                    dw_post=s["dw_post"], rstd_post=s["rstd_post"], w_next=s["w_next"],
                                    dw_next=s["dw_next"], rstd_next=s["rstd_next"])
        return s["dy"], s["dresidual"], s["dgate"], s["dw_post"], s["dw_next"]
    if op == "permute":
        moe.moe_permute(s["ids"], case["E"], s["offsets"], s["pair_row"], s["row_pair"], x=s["x"], rows=s["rows"],
                        slot_table=s["slot_table"], n_slots=s["n_slots"])
        return s["rows"], s["offsets"], s["pair_row"], s["row_pair"]
    if op == "permute_grad":
        moe.moe_permute_backward(s["drows"], s["pair_row"], s["dx"])
        return s["dx"]
    if op == "unpermute":
        moe.moe_unpermute(s["rows"], s["pair_row"], s["out"], weights=s["gates"])
        return s["out"]
    if op == "unpermute_grad":
        moe.moe_unpermute_backward(s["dout"], s["pair_row"], s["drows"], rows=s["rows"], weights=s["gates"],
                                   dweights=s["dweights"])
        return s["drows"], s["dweights"]
    if "ws" not in s:
        s["ws"] = moe.alloc_ws(moe.route_backward_workspace_size(case["T"], case["D"], case["E"], case["k"]))
    moe.moe_route_backward(s["dgates"], s["gates"], s["ids"], s["x"], s["Wr"], s["offsets"], s["row_pair"],
                           s["dlogits"], s["ws"], dx=s["dx"], dWr=s["dWr"], dbias=s["dbias"])
    return s["dlogits"], s["dx"], s["dWr"], s["dbias"]


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, T, D = case["op"], case["T"], case["D"]
    d = {n: v.double() for n, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op in ("norm", "norm_grad"):
        one = torch.ones((), dtype=torch.float64, device="cuda")
        gate = {"none": one, "channel": d.get("gate"), "token": d["gate"].view(T, 1) if case["gate"] == "token" else 0}
        gate, wn, wp = gate[case["gate"]], d["w_next"], d.get("w_post")
        y, dt = d["y"], s["y"].dtype
        ry = 1 / ((y * y).sum(1, keepdim=True) / D + EPS).sqrt() if case["post"] else one
        z = y * ry * (wp if case["post"] else one)
        if op == "norm":
            total = gate * z + case["alpha"] * d["residual"]
            x = total.to(dt).double()           # the next block's norm reads what is stored
            return total, x * wn / ((x * x).sum(1, keepdim=True) / D + EPS).sqrt()
        x, rx = d["x_out"], 1 / ((d["x_out"] ** 2).sum(1, keepdim=True) / D + EPS).sqrt()
        # d/dx of n_i = w_i x_i r(x): r w_i dn_i - x_i r^3 / D sum_j w_j dn_j x_j
        G = d["dx_out"] + rx * wn * d["dnormed"] - x * rx ** 3 / D * (wn * d["dnormed"] * x).sum(1, keepdim=True)
        dz = gate * G
        if case["post"]:
            dy = ry * wp * dz - y * ry ** 3 / D * (wp * dz * y).sum(1, keepdim=True)
        else:
            dy = dz
        dgate = {"none": None, "channel": (G * z).sum(0), "token": (G * z).sum(1)}[case["gate"]]
        return (dy, case["alpha"] * G, dgate, (dz * y * ry).sum(0) if case["post"] else None,
                (d["dnormed"] * x * rx).sum(0))
    E, k, P = case["E"], case["k"], T * case["k"]
    pair = torch.arange(P, device="cuda")
    flat = s["ids"].reshape(-1).long()
    taken = torch.ones(P, dtype=torch.bool, device="cuda") if s["absent"] is None else s["absent"][flat]
    at = (flat * P + pair)[taken].sort().values % P         # the taken pairs in row order
    N = at.numel()
    if op == "permute":
        rows = torch.zeros(P, D, dtype=torch.float64, device="cuda")
        rows[:N] = d["x"][at // k]
        return rows, None, None, None
    w = d["gates"].reshape(-1)
    if op in ("permute_grad", "unpermute"):
        rows = d["drows" if op == "permute_grad" else "rows"][:N]
        if op == "unpermute":
            rows = rows * w[at][:, None]
        return torch.zeros(T, D, dtype=torch.float64, device="cuda").index_add_(0, at // k, rows)
    if op == "unpermute_grad":
        drows = torch.zeros(P, D, dtype=torch.float64, device="cuda")
        drows[:N] = d["dout"][at // k] * w[at][:, None]
        dw = torch.zeros(P, dtype=torch.float64, device="cuda")
        dw[at] = (d["dout"][at // k] * d["rows"][:N]).sum(1)
        return drows, dw.view(T, k)
    jac = torch.diag_embed(d["gates"]) - d["gates"][:, :, None] * d["gates"][:, None, :]
    dl = (jac @ d["dgates"][:, :, None])[:, :, 0]
    hot = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    hot[torch.arange(T, device="cuda")[:, None], s["ids"].long()] = dl
    return dl, hot @ d["Wr"], hot.t() @ d["x"], hot.sum(0)
