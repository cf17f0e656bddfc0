"""Measured cases of the int8 products with token and channel scales, dense and grouped by expert, and of the
row quantisation, expert positions and combine that go with them.

A token's activations are int8 codes with one binary32 scale per row, a weight's are int8 codes with one scale per
output channel: y[t, n] = (sum_k Xq[t, k] Wq[n, k]) sx[t] sw[n] + b[n].  With `gated` the outputs come in pairs
(gate channel j, value channel F + j of 2 F) and silu(gate) * value is returned.
"""
import torch

own = False

HALF, BF16, F32 = "float16", "bfloat16", "float32"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token through an up projection: bound by reading the weight once, latency counts
        {"name": "product one token", "op": "product", "T": 1, "N": 11008, "K": 4096, "dtype": HALF, "bias": False,
         "gated": False},
        # a ragged prompt, wide projection with a bias
        {"name": "product 333 tokens", "op": "product", "T": 333, "N": 13824, "K": 5120, "dtype": BF16, "bias": True,
         "gated": False},
        # a full prefill batch of a large model: bound by the tensor cores
        {"name": "product 4096 tokens", "op": "product", "T": 4096, "N": 28672, "K": 8192, "dtype": HALF,
         "bias": False, "gated": False},
        # a decode step of 8 sequences: few rows for each expert, some experts with none
        {"name": "grouped decode", "op": "grouped", "T": 8, "k": 2, "E": 16, "N": 4096, "K": 2048, "dtype": BF16,
         "bias": False, "gated": False},
        # a prompt over many small experts, the gate and up projections in one product
        {"name": "grouped ragged", "op": "grouped", "T": 999, "k": 4, "E": 32, "N": 4096, "K": 2048, "dtype": F32,
         "bias": False, "gated": True},
        # a full prefill batch over few large experts
        {"name": "grouped prefill", "op": "grouped", "T": 4096, "k": 2, "E": 8, "N": 22016, "K": 4096, "dtype": F32,
         "bias": False, "gated": True},
        # the activations of a prompt before a projection
        {"name": "quantize rows", "op": "quantize", "T": 2048, "k": 0, "K": 4096, "dtype": HALF},
        # the same, written to the rows that the experts' product reads
        {"name": "quantize to experts", "op": "quantize", "T": 1021, "k": 4, "K": 5120, "dtype": BF16},
        # the routing of a decode step and of a large batch, padding tokens with no expert among them
        {"name": "positions decode", "op": "positions", "T": 16, "k": 2, "E": 8},
        {"name": "positions batch", "op": "positions", "T": 8192, "k": 8, "E": 128},
        # the experts' outputs of a decode step and of a prompt, summed for each token
        {"name": "combine decode", "op": "combine", "T": 16, "k": 2, "N": 4096, "dtype": HALF},
        {"name": "combine prompt", "op": "combine", "T": 4096, "k": 4, "N": 5120, "dtype": BF16},
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["product", "product", "grouped", "grouped", "quantize", "positions", "combine"])
    dtype = rng.choice([HALF, BF16, F32])
    if op == "product":
        K, N = 16 * _log(rng, 16, 512), _log(rng, 250, 28672)
        gated = rng.random() < 0.3
        N = N // 32 * 32 + 32 if gated else N
        return {"op": op, "T": _log(rng, 1, 4096), "N": min(N, 28672), "K": K, "dtype": dtype,
                "bias": rng.random() < 0.4, "gated": gated}
    if op == "grouped":
        E, K = _log(rng, 4, 128), 16 * _log(rng, 16, 256)
        gated = rng.random() < 0.5
        N = _log(rng, 250, min(22016, 7 * 10 ** 8 // (E * K)))
        N = N // 32 * 32 + 32 if gated else N
        return {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, min(E, 8)), "E": E, "N": min(N, 22016), "K": K,
                "dtype": dtype, "bias": rng.random() < 0.3, "gated": gated}
    if op == "quantize":
        return {"op": op, "T": _log(rng, 1, 8192), "k": rng.choice([0, 1, 2, 4, 8]), "K": 16 * _log(rng, 16, 512),
                "dtype": dtype}
    if op == "positions":
        return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, 8), "E": _log(rng, 8, 256)}
    return {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, 8), "N": 8 * _log(rng, 32, 1024), "dtype": dtype}


# ------------------------------------------------------------------ inputs

def _codes(g, *shape):
    """int8 codes as absmax quantisation of normal values leaves them."""
    return torch.randn(*shape, device="cuda", generator=g).mul_(30.0).round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, mean, *shape):
    return (torch.rand(*shape, device="cuda", generator=g) + 0.5) * mean


def _routing(g, T, k, E):
    """A router's choice: k distinct experts for each token, some of them more popular, and their weights."""
    logits = torch.randn(T, E, device="cuda", generator=g) + 0.4 * torch.randn(E, device="cuda", generator=g)
    top, ids = logits.topk(k, dim=1)
    return ids, torch.softmax(top, dim=1)


def _places(ids, E):
    """For each entry of ids its place in the order by expert (-1 for none), and where each expert's rows begin."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=ids.device, dtype=key.dtype)).to(torch.int32)
    at = torch.arange(flat.numel(), device=ids.device, dtype=torch.int32)
    places = torch.empty_like(at)
    places[order] = torch.where(key < E, at, torch.full_like(at, -1))
    return places.view(ids.shape), offsets


def _activations(g, T, K, dtype):
    """Normal values with a few wide channels, as hidden states have them."""
    X = torch.randn(T, K, device="cuda", generator=g)
    X[:, torch.randperm(K, device="cuda", generator=g)[:4]] *= 12.0
    return X.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case)
    if "dtype" in case:
        s["dtype"] = getattr(torch, case["dtype"])
    if op in ("product", "grouped"):
        rows, groups = case["T"], ()
        if op == "grouped":
            ids, _ = _routing(g, case["T"], case["k"], case["E"])
            _, s["offsets"] = _places(ids, case["E"])
            s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
            rows, groups = case["T"] * case["k"], (case["E"],)
        s["Xq"], s["sx"] = _codes(g, rows, case["K"]), _scales(g, 1 / 30, rows)
        s["Wq"] = _codes(g, *groups, case["N"], case["K"])
        s["sw"] = _scales(g, 1 / 30 / case["K"] ** 0.5, *groups, case["N"])
        s["b"] = torch.randn(*groups, case["N"], device="cuda", generator=g) if case["bias"] else None
    elif op == "quantize":
        s["X"] = _activations(g, case["T"], case["K"], s["dtype"])
        s["places"] = None
        if case["k"]:
            ids, _ = _routing(g, case["T"], case["k"], 2 * case["k"])
            s["places"], _ = _places(ids, 2 * case["k"])
    elif op == "positions":
        ids, _ = _routing(g, case["T"], case["k"], case["E"])
        padding = torch.rand(case["T"], 1, device="cuda", generator=g) < 0.03
        s["ids"] = torch.where(padding, torch.full_like(ids, -1), ids)
    else:
        ids, s["weights"] = _routing(g, case["T"], case["k"], 16)
        padding = torch.rand(case["T"], 1, device="cuda", generator=g) < 0.03
        s["places"], _ = _places(torch.where(padding, torch.full_like(ids, -1), ids), 16)
        s["Y"] = torch.randn(case["T"] * case["k"], case["N"], device="cuda", generator=g).to(s["dtype"])
    return s


# ------------------------------------------------------------------ one pass

def _gate(z):
    """silu of the first half of the last axis times the second half."""
    g, u = z.chunk(2, dim=-1)
    return g / (1 + torch.exp(-g)) * u


def _scaled(acc, sx, sw, b, gated):
    z = acc * sx * sw
    z = z if b is None else z + b
    return _gate(z) if gated else z


def run(s):
    op = s["op"]
    if own:
        import int8_mixed_precision_outlier_b200 as L
        if op == "product":
            return L.llmint8_scaled_matmul(s["Xq"], s["sx"], s["Wq"], s["sw"], bias=s["b"], gated=s["gated"],
                                           dtype=s["dtype"])
        if op == "grouped":
            return L.llmint8_grouped_matmul(s["Xq"], s["sx"], s["offsets"], s["Wq"], s["sw"], bias=s["b"],
                                            gated=s["gated"], dtype=s["dtype"])
        if op == "quantize":
            q, scale = L.llmint8_quantize_rows(s["X"], s["places"])
            return {"values": torch.mul(q, scale[:, None], out=torch.empty_like(q, dtype=s["dtype"])), "scale": scale}
        if op == "positions":
            places, offsets = L.llmint8_expert_positions(s["ids"], s["E"])
            return {"positions": places, "offsets": offsets}
        return L.llmint8_expert_combine(s["Y"], s["places"], s["weights"])
    if op == "product":
        acc = s["Xq"].float() @ s["Wq"].float().T
        return _scaled(acc, s["sx"][:, None], s["sw"], s["b"], s["gated"]).to(s["dtype"])
    if op == "grouped":
        # every expert's rows, padded to the longest: one batched product
        start, end = s["offsets"][:-1, None], s["offsets"][1:, None]
        at = start + torch.arange(s["most"], device="cuda")
        inside = at < end
        at = torch.where(inside, at, torch.zeros_like(at))
        acc = s["Xq"].float()[at] @ s["Wq"].float().transpose(1, 2)
        b = None if s["b"] is None else s["b"][:, None]
        y = _scaled(acc, s["sx"][at][:, :, None], s["sw"][:, None], b, s["gated"])
        return y[inside].to(s["dtype"])
    if op == "quantize":
        x = s["X"].float()
        scale = (x.abs().amax(dim=1).double() / 127).float()
        q = torch.round(x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]).clamp(-127, 127)
        values = (q * scale[:, None]).to(s["dtype"])
        if s["places"] is None:
            return {"values": values, "scale": scale}
        at = s["places"].reshape(-1).long()
        out, out_scale = values.new_empty(at.numel(), values.shape[1]), scale.new_empty(at.numel())
        out[at] = values.repeat_interleave(s["k"], dim=0)
        out_scale[at] = scale.repeat_interleave(s["k"])
        return {"values": out, "scale": out_scale}
    if op == "positions":
        places, offsets = _places(s["ids"], s["E"])
        return {"positions": places, "offsets": offsets}
    there = s["places"] >= 0
    y = s["Y"][torch.where(there, s["places"], torch.zeros_like(s["places"]))].float()
    return (torch.where(there, s["weights"], torch.zeros_like(s["weights"]))[:, :, None] * y).sum(1).to(s["dtype"])


# ------------------------------------------------------------------ work and exact values

def _size(name):
    return 4 if name == F32 else 2


def work(case):
    op, T = case["op"], case["T"]
    if op in ("product", "grouped"):
        N, K = case["N"], case["K"]
        rows, groups = T, 1.0
        if op == "grouped":  # experts that some token chose, were they equally popular
            rows, groups = T * case["k"], case["E"] * (1 - (1 - case["k"] / case["E"]) ** T)
        out = N // 2 if case["gated"] else N
        return {"bytes": rows * (K + 4) + groups * N * (K + 4 + 4 * case["bias"]) + rows * out * _size(case["dtype"]),
                "flops": 2.0 * rows * N * K}
    if op == "quantize":  # the codes are one byte; what this pass returns of them has the type of X
        rows = T * max(1, case["k"])
        return {"bytes": T * case["K"] * _size(case["dtype"]) + rows * (case["K"] * (1 + _size(case["dtype"])) + 4),
                "flops": 2.0 * T * case["K"]}
    if op == "positions":
        return {"bytes": 12 * T * case["k"] + 4 * (case["E"] + 1), "flops": T * case["k"]}
    return {"bytes": T * (case["k"] + 1) * case["N"] * _size(case["dtype"]) + 8 * T * case["k"],
            "flops": 2.0 * T * case["k"] * case["N"]}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "product":
        z = torch.einsum("tk,nk->tn", s["Xq"].double(), s["Wq"].double())
        z *= torch.outer(s["sx"].double(), s["sw"].double())
        if s["b"] is not None:
            z += s["b"].double()
        return z[:, : z.shape[1] // 2] * torch.sigmoid(z[:, : z.shape[1] // 2]) * z[:, z.shape[1] // 2:] \
            if s["gated"] else z
    if op == "grouped":
        bounds, parts = s["offsets"].tolist(), []
        for e in range(s["E"]):
            lo, hi = bounds[e], bounds[e + 1]
            z = s["Xq"][lo:hi].double().mm(s["Wq"][e].double().t())
            z = z * s["sx"][lo:hi, None].double() * s["sw"][e].double()
            if s["b"] is not None:
                z = z + s["b"][e].double()
            half = z.shape[1] // 2
            parts.append(z[:, :half] * torch.sigmoid(z[:, :half]) * z[:, half:] if s["gated"] else z)
        return torch.cat(parts)
    if op == "quantize":
        # the scale and the quotient are binary32 by definition (each rounded once), the value is code * scale
        x = s["X"].double()
        scale = (x.abs().max(dim=1).values / 127).float().double()
        q = torch.where(scale[:, None] > 0, (x / scale[:, None]).float().double(), torch.zeros_like(x)).round()
        values = q * scale[:, None]
        if s["places"] is not None:
            row = torch.argsort(s["places"].reshape(-1).long()) // s["k"]
            values, scale = values[row], scale[row]
        return {"values": values, "scale": scale}
    if op == "positions":
        return None
    out = torch.zeros(case["T"], case["N"], device="cuda", dtype=torch.float64)
    for j in range(case["k"]):
        at = s["places"][:, j].long()
        out += torch.where(at >= 0, s["weights"][:, j].double(), 0.0)[:, None] * s["Y"][at.clamp(min=0)].double()
    return out
