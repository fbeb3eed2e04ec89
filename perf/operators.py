"""What the grouped operators cost: the row grouping, the expert products over
ragged groups, the per-request adapters and the MoE block of any number of
tokens, each as a user's program calls it and as a plain form in 32 bits.

Shapes: the Qwen3-30B-A3B layer (d = 2048, I = 768, 128 experts, top-8), the
tiny block of the tests (d = 256, I = 128, 8 experts, top-2) and generic ones.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    qwen = {"E": 128, "I": 768, "d": 2048, "top": 8}
    return [
        # the pairs of a 16-token step, grouped by expert
        {"name": "group 128", "op": "group", "n": 128, "G": 128, "none": 0.0},
        # the pairs of a long prompt chunk, one in ten for an expert that another rank holds
        {"name": "group 65536", "op": "group", "n": 65536, "G": 128, "none": 0.1},
        # gate/up of a decode step with few requests: one or two rows per expert
        {"name": "swiglu 5 tokens", "op": "swiglu", "T": 5, "skew": False, **qwen},
        # gate/up of a prompt chunk under skewed routing
        {"name": "swiglu 4096 tokens", "op": "swiglu", "T": 4096, "skew": True, **qwen},
        # down products of a short, odd prompt: about 21 rows per expert
        {"name": "down 333 tokens", "op": "product", "T": 333, "top": 8, "E": 128, "K": 768, "N": 2048, "layout": 1,
         "skew": False},
        # a generic grouped projection, weights stored by output channel, few large ragged groups
        {"name": "product 9001 rows", "op": "product", "T": 9001, "top": 1, "E": 16, "K": 1096, "N": 2016,
         "layout": 0, "skew": True},
        # the whole block, smallest: the tiny block of the tests at a few tokens
        {"name": "block tiny", "op": "block", "T": 7, "E": 8, "I": 128, "d": 256, "top": 2, "skew": False,
         "residual": False},
        # the whole block for a short prompt (more tokens than a decode step may have)
        {"name": "block 300 tokens", "op": "block", "T": 300, "skew": False, "residual": True, **qwen},
        # the whole block for a long prompt chunk under skewed routing: the largest
        {"name": "block 8192 tokens", "op": "block", "T": 8192, "skew": True, "residual": True, **qwen},
        # one decoding request with its adapter beside a shared projection
        {"name": "adapter 1 token", "op": "adapter", "T": 1, "A": 1, "K": 2048, "N": 2048, "r": 16, "w": True,
         "base": False, "runs": False},
        # a decode batch, every request with an adapter of its own choice, added to a block's output
        {"name": "adapter 64 tokens", "op": "adapter", "T": 64, "A": 32, "K": 2048, "N": 2048, "r": 32, "w": False,
         "base": True, "runs": False},
        # prompts of many requests side by side, each a run of tokens with one adapter or none
        {"name": "adapter 4100 tokens", "op": "adapter", "T": 4100, "A": 9, "K": 2048, "N": 4096, "r": 64, "w": True,
         "base": True, "runs": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(lo, min(hi, m * max(1, _log(rng, lo, hi) // m)))


def draw(rng):
    op = rng.choice(["group", "swiglu", "product", "block", "adapter"])
    skew = rng.random() < 0.5
    if op == "group":
        return {"op": op, "n": _log(rng, 1, 65536), "G": _log(rng, 1, 1024), "none": rng.choice([0.0, 0.1, 0.9])}
    if op == "adapter":
        A = _log(rng, 1, 64)
        form = rng.choice([(True, False), (True, True), (False, True)])
        return {"op": op, "T": _log(rng, 1, 4100), "A": A, "K": _mult(rng, 256, 4096, 8), "N": _mult(rng, 256, 4096, 8),
                "r": 8 * rng.randint(1, 16), "w": form[0], "base": form[1], "runs": rng.random() < 0.5}
    E = _log(rng, 4, 128)
    top = rng.randint(1, min(8, E))
    if op == "product":
        return {"op": op, "T": _log(rng, 1, 4096), "top": top, "E": E, "K": _mult(rng, 64, 2048, 8),
                "N": _mult(rng, 64, 2048, 8), "layout": rng.randint(0, 1), "skew": skew}
    d = 2 ** rng.randint(8, 11)
    if op == "swiglu":
        return {"op": op, "T": _log(rng, 1, 4096), "E": E, "I": _mult(rng, 16, 768, 8), "d": d, "top": top, "skew": skew}
    return {"op": op, "T": _log(rng, 1, 6000), "E": E, "I": _mult(rng, 16, 768, 8), "d": d, "top": top, "skew": skew,
            "residual": rng.random() < 0.5}


def _active(groups, rows, top=1):
    """Groups that hold a row, expected for even routing of rows / top tokens to top of the groups each."""
    return groups * (1.0 - (1.0 - top / groups) ** (rows / top))


def work(case):
    c = case
    if c["op"] == "group":
        return {"bytes": 8 * c["n"] + 4 * (c["G"] + 1), "flops": c["n"]}
    if c["op"] == "adapter":
        T, K, N, r = c["T"], c["K"], c["N"], c["r"]
        by = 2 * T * (K + N) + 2 * r * (K + N) * _active(c["A"], T)
        by += (2 * N * K if c["w"] else 0) + (2 * T * N if c["base"] else 0)
        return {"bytes": by, "flops": 2 * T * r * (K + N) + (2 * T * N * K if c["w"] else 0)}
    P, ea = c["T"] * c["top"], _active(c["E"], c["T"] * c["top"], c["top"])
    if c["op"] == "product":
        x = P if c["layout"] else c["T"]
        return {"bytes": 2 * (ea * c["K"] * c["N"] + x * c["K"] + P * c["N"]), "flops": 2 * P * c["K"] * c["N"]}
    T, I, d = c["T"], c["I"], c["d"]
    if c["op"] == "swiglu":
        return {"bytes": 2 * (2 * ea * I * d + T * d + P * I), "flops": 4 * P * I * d}
    return {"bytes": 2 * (3 * ea * I * d + c["E"] * d + (3 if c["residual"] else 2) * T * d),
            "flops": 6 * P * I * d + 2 * T * c["E"] * d}


# ------------------------------------------------------------------ inputs
def _weights(g, *shape, fan):
    """bf16 N(0, 1/fan) with a lognormal scale per row, as the layers of this framework are drawn."""
    w = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = w.view(-1, *shape[-2:])
    for e in range(flat.shape[0]):
        s = torch.exp(torch.randn((shape[-2], 1), generator=g, device=DEV)) / math.sqrt(fan)
        flat[e] = (torch.randn(shape[-2:], generator=g, device=DEV) * s).to(torch.bfloat16)
    return w


def _tokens(g, T, d):
    """RMS-normalised tokens with heavy tails (a normal over the root of a mean of four squares)."""
    z = torch.randn((T, d), generator=g, device=DEV)
    h = torch.randn((T, d, 4), generator=g, device=DEV).square().mean(-1).sqrt()
    t = z / h
    return (t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def _routed(g, T, E, top, skew):
    """[T, top] distinct experts of each token."""
    s = torch.randn((T, E), generator=g, device=DEV)
    if skew:
        s = s + torch.randn((E,), generator=g, device=DEV)
    return s.topk(top, dim=1).indices.to(torch.int32)


def _plan(ids, groups):
    """The grouping of ids: offsets [groups + 1] and rows [n], stable, ids outside [0, groups) behind the last."""
    key = torch.where((ids >= 0) & (ids < groups), ids, torch.full_like(ids, groups)).long()
    counts = torch.bincount(key, minlength=groups + 1)
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts[:groups].cumsum(0)
    return offsets, torch.sort(key, stable=True).indices.to(torch.int32), int(counts[:groups].max())


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "group":
        ids = torch.randint(0, c["G"], (c["n"],), generator=g, device=DEV, dtype=torch.int32)
        drop = torch.rand((c["n"],), generator=g, device=DEV) < c["none"]
        s["ids"] = torch.where(drop, torch.full_like(ids, -1), ids)
        s["offsets"] = torch.zeros(c["G"] + 1, dtype=torch.int32, device=DEV)
        s["rows"] = torch.zeros(c["n"], dtype=torch.int32, device=DEV)
    elif c["op"] == "swiglu":
        E, I, d, T, top = c["E"], c["I"], c["d"], c["T"], c["top"]
        s["x"] = _tokens(g, T, d)
        s["w_gate"], s["w_up"] = _weights(g, E, I, d, fan=d), _weights(g, E, I, d, fan=d)
        s["offsets"], s["rows"], s["most"] = _plan(_routed(g, T, E, top, c["skew"]).flatten(), E)
        s["a"] = torch.zeros((T * top, I), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "product":
        E, K, N, T, top = c["E"], c["K"], c["N"], c["T"], c["top"]
        s["x"] = _tokens(g, T * top if c["layout"] else T, K)
        s["w"] = _weights(g, E, K, N, fan=K) if c["layout"] else _weights(g, E, N, K, fan=K)
        s["offsets"], s["rows"], s["most"] = _plan(_routed(g, T, E, top, c["skew"]).flatten(), E)
        s["y"] = torch.zeros((T * top, N), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "block":
        E, I, d, T = c["E"], c["I"], c["d"], c["T"]
        s["x"] = _tokens(g, T, d)
        s["weights"] = {"w_router": (torch.randn((E, d), generator=g, device=DEV) / math.sqrt(d)).to(torch.bfloat16),
                        "router_bias": torch.randn((E,), generator=g, device=DEV) if c["skew"] else None,
                        "w_gate": _weights(g, E, I, d, fan=d), "w_up": _weights(g, E, I, d, fan=d),
                        "w_down": _weights(g, E, I, d, fan=d)}
        s["residual"] = torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16) if c["residual"] else None
        s["y"] = torch.zeros_like(s["x"])
        s["ids"] = torch.zeros((T, c["top"]), dtype=torch.int32, device=DEV)
        # the most tokens that an expert takes: the room that a padded product needs
        s["most"] = int(torch.bincount(_route(s["x"], s["weights"], c["top"])[0].flatten(), minlength=E).max())
    else:
        T, A, K, N, r = c["T"], c["A"], c["K"], c["N"], c["r"]
        s["x"] = _tokens(g, T, K)
        s["w"] = _weights(g, N, K, fan=K) if c["w"] else None
        s["base"] = torch.randn((T, N), generator=g, device=DEV).to(torch.bfloat16) if c["base"] else None
        s["a"], s["b"] = _weights(g, A, r, K, fan=K), _weights(g, A, N, r, fan=r)
        s["scale"] = 0.25 + torch.rand((A,), generator=g, device=DEV)
        if c["runs"]:  # runs of tokens, each with one adapter (or none: -1)
            cut = (torch.rand((T,), generator=g, device=DEV) < 12.0 / max(T, 12)).cumsum(0)
            of = torch.randint(-1, A, (T + 1,), generator=g, device=DEV, dtype=torch.int32)
            ids = of[cut]
        else:
            ids = torch.randint(0, A, (T,), generator=g, device=DEV, dtype=torch.int32)
        s["offsets"], s["rows"], _ = _plan(ids, A)
        s["y"] = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    if own:
        from calibration_free_channel_b200 import moe_reader as M
        if c["op"] == "group":
            nb = M.moe_reader_group_workspace_bytes(c["n"], c["G"])
        elif c["op"] == "adapter":
            nb = M.moe_reader_adapter_workspace_bytes(c["T"], c["A"], c["K"], c["N"], c["r"])
        elif c["op"] == "block":
            s["layer"] = M.Layer(s["weights"], c["top"])
            nb = M.moe_reader_block_workspace_bytes(c["T"], c["E"], c["top"], c["I"], c["d"])
            s["struct"] = s["layer"].struct()
        else:
            nb = M.moe_reader_grouped_workspace_bytes(c["E"], c["T"] * c["top"])
        s["ws"] = torch.zeros(nb, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------ one pass each
def _route(x, w, top):
    """Chosen experts [T, top] and their softmax weights; logits in 64 bits, ties to the lower id."""
    logits = x.double() @ w["w_router"].double().T
    if w["router_bias"] is not None:
        logits = logits + w["router_bias"].double()
    vals, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    e = torch.exp(vals[:, :top] - vals[:, :1])
    return ids[:, :top], (e / e.sum(1, keepdim=True)).float()


def _padded(offsets, most, last):
    """[groups, most] sorted positions of each group (clamped where a group has fewer), and the group and the
    place in it of each sorted position."""
    at = (offsets[:-1, None].long() + torch.arange(most, device=DEV)).clamp(max=last)
    p = torch.arange(last + 1, device=DEV, dtype=torch.int32)
    group = torch.searchsorted(offsets[1:].contiguous(), p, right=True).clamp(max=offsets.numel() - 2)
    return at, group, p.long() - offsets[group].long()


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def run(s):
    c = s["case"]
    if own:
        return _run_own(s)
    if c["op"] == "group":
        G = c["G"]
        key = torch.where((s["ids"] >= 0) & (s["ids"] < G), s["ids"], torch.full_like(s["ids"], G))
        counts = (key[:, None] == torch.arange(G, device=DEV, dtype=torch.int32)).sum(0)
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0)])
        return offsets.to(torch.int32), torch.sort(key, stable=True).indices.to(torch.int32)
    if c["op"] == "swiglu":
        at, group, place = _padded(s["offsets"], s["most"], s["rows"].numel() - 1)
        x = s["x"].float()[s["rows"][at].long() // c["top"]]
        g = torch.bmm(x, s["w_gate"].float().transpose(1, 2))
        u = torch.bmm(x, s["w_up"].float().transpose(1, 2))
        return (_silu(g) * u)[group, place].to(torch.bfloat16)
    if c["op"] == "product":
        at, group, place = _padded(s["offsets"], s["most"], s["rows"].numel() - 1)
        if c["layout"]:
            y = torch.bmm(s["x"].float()[at], s["w"].float())[group, place]
            return torch.zeros_like(s["y"]).index_copy_(0, s["rows"].long(), y.to(torch.bfloat16))
        x = s["x"].float()[s["rows"][at].long() // c["top"]]
        return torch.bmm(x, s["w"].float().transpose(1, 2))[group, place].to(torch.bfloat16)
    if c["op"] == "block":
        w, top, T = s["weights"], c["top"], c["T"]
        ids, share = _route(s["x"], w, top)
        rows = torch.sort(ids.flatten(), stable=True).indices
        counts = (ids.reshape(-1, 1) == torch.arange(c["E"], device=DEV)).sum(0)
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0)]).to(torch.int32)
        at, group, place = _padded(offsets, s["most"], T * top - 1)
        x = s["x"].float()[rows[at] // top]
        a = _silu(torch.bmm(x, w["w_gate"].float().transpose(1, 2))) * torch.bmm(x, w["w_up"].float().transpose(1, 2))
        out = torch.bmm(a, w["w_down"].float())[group, place] * share.flatten()[rows][:, None]
        y = torch.zeros_like(out).index_copy_(0, rows, out).view(T, top, c["d"]).sum(1)
        if c["residual"]:
            y = y + s["residual"].float()
        return y.to(torch.bfloat16), ids.to(torch.int32)
    T, A, r = c["T"], c["A"], c["r"]
    x, of = s["x"].float(), torch.arange(A, device=DEV).repeat_interleave(r)
    p = torch.arange(T, device=DEV, dtype=torch.int32)
    group = torch.searchsorted(s["offsets"][1:].contiguous(), p, right=True)
    mine = torch.zeros_like(group).index_copy_(0, s["rows"].long(), group)  # the adapter of each token, A for none
    z = (x @ s["a"].float().view(A * r, -1).T) * s["scale"][of] * (mine[:, None] == of)
    y = z @ s["b"].float().transpose(1, 2).reshape(A * r, -1)
    if c["w"]:
        y = y + x @ s["w"].float().T
    if c["base"]:
        y = y + s["base"].float()
    return y.to(torch.bfloat16)


def _run_own(s):
    from calibration_free_channel_b200 import moe_reader as M
    c, ws = s["case"], s["ws"]
    if c["op"] == "group":
        M.moe_reader_group_rows(c["n"], c["G"], s["ids"], s["offsets"], s["rows"], ws, ws.numel())
        return s["offsets"], s["rows"]
    if c["op"] == "swiglu":
        M.moe_reader_grouped_swiglu(c["E"], c["T"] * c["top"], c["T"], c["I"], c["d"], s["x"], s["rows"], c["top"],
                                    s["offsets"], s["w_gate"], s["w_up"], s["a"], ws, ws.numel())
        return s["a"]
    if c["op"] == "product":
        P = c["T"] * c["top"]
        M.moe_reader_grouped_product(c["E"], P, s["x"].shape[0], P, c["N"], c["K"], c["layout"], s["x"],
                                     None if c["layout"] else s["rows"], 1 if c["layout"] else c["top"], s["offsets"],
                                     s["w"], s["y"], s["rows"] if c["layout"] else None, ws, ws.numel())
        return s["y"]
    if c["op"] == "block":
        M.moe_reader_forward_grouped(s["struct"], c["T"], s["x"], s["residual"], s["y"], s["ids"], ws, ws.numel())
        return s["y"], s["ids"]
    M.moe_reader_adapter_product(c["T"], c["A"], c["N"], c["K"], c["r"], s["x"], s["w"], s["base"], s["offsets"],
                                 s["rows"], s["a"], s["b"], s["scale"], s["y"], ws, ws.numel())
    return s["y"]


# ------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    """The operators from their definitions, one group at a time."""
    c, s = case, prepare(case, seed)
    if c["op"] == "group":
        ids, G = s["ids"], c["G"]
        parts = [(ids == e).nonzero().flatten() for e in range(G)] + [((ids < 0) | (ids >= G)).nonzero().flatten()]
        ends = [0]
        for rows in parts[:G]:
            ends.append(ends[-1] + rows.numel())
        return torch.tensor(ends, dtype=torch.int32, device=DEV), torch.cat(parts).to(torch.int32)
    if c["op"] == "adapter":
        y = torch.zeros((c["T"], c["N"]), dtype=torch.float64, device=DEV)
        if c["w"]:
            y += s["x"].double() @ s["w"].double().T
        if c["base"]:
            y += s["base"].double()
        off = s["offsets"].tolist()
        for a in range(c["A"]):
            rows = s["rows"][off[a]:off[a + 1]].long()
            z = s["x"][rows].double() @ s["a"][a].double().T
            y[rows] += s["scale"][a].double() * (z @ s["b"][a].double().T)
        return y
    if c["op"] == "block":
        w, top = s["weights"], c["top"]
        lg = s["x"].double() @ w["w_router"].double().T + (0 if w["router_bias"] is None else w["router_bias"].double())
        best = lg.topk(top, dim=1)
        if 6.0 * c["T"] * top * c["I"] * c["d"] > 4e11:
            return None, best.indices.to(torch.int32)
        share = torch.softmax(best.values, dim=1)
        y = torch.zeros((c["T"], c["d"]), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            t, k = (best.indices == e).nonzero(as_tuple=True)
            xe = s["x"][t].double()
            g = xe @ w["w_gate"][e].double().T
            a = g * torch.sigmoid(g) * (xe @ w["w_up"][e].double().T)
            y[t] += share[t, k][:, None] * (a @ w["w_down"][e].double())
        if c["residual"]:
            y += s["residual"].double()
        return y, best.indices.to(torch.int32)
    off, P = s["offsets"].tolist(), c["T"] * c["top"]
    out = torch.zeros((P, c["I"] if c["op"] == "swiglu" else c["N"]), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        p = torch.arange(off[e], off[e + 1], device=DEV)
        if c["op"] == "swiglu":
            xe = s["x"][s["rows"][p].long() // c["top"]].double()
            g = xe @ s["w_gate"][e].double().T
            out[p] = g * torch.sigmoid(g) * (xe @ s["w_up"][e].double().T)
        elif c["layout"]:
            out[s["rows"][p].long()] = s["x"][p].double() @ s["w"][e].double()
        else:
            out[p] = s["x"][s["rows"][p].long() // c["top"]].double() @ s["w"][e].double().T
    return out
