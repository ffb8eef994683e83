"""The layer's operators around frozen quantised weights, as a benchmark: the dense
quantised products (forward and input gradient), the router's balance and z losses,
the router's backward pass and the combine's.

``listed()`` gives fixed cases, ``draw(rng)`` more of the same ranges; ``prepare``
makes one case's inputs on the GPU from a seed, ``run`` makes one pass (in plain torch
operations, or through the library where ``own`` is set), ``exact`` the same outputs in
64 bits, and ``work`` the bytes and operations that a pass cannot do without.
"""
import math
import random

import torch

own = False

_BF16, _F32, _F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------ cases

def _linear(op, T, N, K, bits=4, group=128, f32=False, row_bias=False, residual=False, pad=0):
    return {"op": op, "T": T, "N": N, "K": K, "bits": bits, "group": group, "f32": f32, "row_bias": row_bias,
            "residual": residual, "pad": pad}


def _router(op, T, E, k, renorm=True, padded=False, disabled=0):
    return {"op": op, "T": T, "E": E, "k": k, "renorm": renorm, "padded": padded, "disabled": disabled}


def listed():
    return [
        # one token's output projection of a 2048-wide layer, its residual added: latency counts
        dict(_linear("linear", 1, 2048, 2048, residual=True), name="linear_T1"),
        # a batch of 8 decoded tokens through an output vocabulary of odd size, float32 logits
        dict(_linear("linear", 8, 49999, 4096, f32=True), name="linear_logits_T8"),
        # a prompt of 4096 tokens through an up projection
        dict(_linear("linear", 4096, 8192, 2048), name="linear_prompt_T4096"),
        # the gradient past a 2-bit matrix with a row bias and finer groups, a short ragged batch
        dict(_linear("linear_grad", 37, 5111, 2048, bits=2, group=64, pad=24), name="linear_grad_T37"),
        # the same for a single token through a square projection (online tuning)
        dict(_linear("linear_grad", 1, 4096, 4096), name="linear_grad_T1"),
        # a training batch of 4096 tokens
        dict(_linear("linear_grad", 4096, 8192, 2048), name="linear_grad_T4096"),
        # per-expert counts and losses of a decode batch (256 experts, 8 picks)
        dict(_router("balance", 32, 256, 8), name="balance_T32"),
        # a padded training batch, eight experts switched off
        dict(_router("balance", 8191, 128, 8, padded=True, disabled=8), name="balance_T8191"),
        # the router's gradient of a small batch (64 experts, 2 picks)
        dict(_router("route_backward", 64, 64, 2), name="route_backward_T64"),
        # a large batch over 512 experts, gates from the softmax over all of them
        dict(_router("route_backward", 16384, 512, 4, renorm=False, padded=True), name="route_backward_T16384"),
        # the combine's gradient of a decode batch
        dict(op="combine_backward", T=8, H=5120, k=2, name="combine_backward_T8"),
        # and of a training batch
        dict(op="combine_backward", T=4096, H=2048, k=8, name="combine_backward_T4096"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng: random.Random):
    op = rng.choice(["linear", "linear_grad", "linear", "linear_grad", "balance", "route_backward",
                     "combine_backward"])
    if op in ("linear", "linear_grad"):
        K = 128 * _log_int(rng, 1, 96)
        N = _log_int(rng, 1, min(60000, 49999 * 4096 // K))
        T = _log_int(rng, 1, max(1, min(4096, 4096 * 8192 * 2048 // (N * K))))
        return _linear(op, T, N, K, bits=rng.choice([4, 4, 2]), group=rng.choice([128, 128, 64, 32]),
                       f32=rng.random() < 0.3, row_bias=op == "linear" and rng.random() < 0.4,
                       residual=op == "linear" and rng.random() < 0.4, pad=8 * rng.choice([0, 0, 1, 5, 16]))
    if op == "combine_backward":
        k = rng.randint(1, 10)
        H = 128 * _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(1, min(65536 // k, 4096 * 8 * 2048 // (k * H))))
        return {"op": op, "T": T, "H": H, "k": k}
    E = _log_int(rng, 4, 1024)
    k = rng.randint(1, min(10, E))
    T = _log_int(rng, 1, min(65536 // k, 16384 * 512 // E))
    return _router(op, T, E, k, renorm=rng.random() < 0.7, padded=rng.random() < 0.5,
                   disabled=rng.choice([0, 0, (E - k) // 4]))


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _padded(t, pad):
    """t's rows as the first columns of a wider buffer (a slice of a fused projection)."""
    if not pad:
        return t
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _prepare_linear(c, g):
    T, N, K, bits, G = c["T"], c["N"], c["K"], c["bits"], c["group"]
    s = {"case": c}
    s["q"] = torch.randint(0, 256, (K // 128, N, 16 * bits), generator=g, device="cuda", dtype=torch.uint8)
    s["scale"] = (0.005 + 0.015 * _rand(g, N, K // G)).half()
    zero = torch.randint(0, 1 << bits, (N, K // G), generator=g, device="cuda").float()
    s["bias"] = (-zero * s["scale"].float()).half()
    out_type = _F32 if c["f32"] else _BF16
    if c["op"] == "linear":
        s["x"] = _padded(_randn(g, T, K).to(_BF16), c["pad"])
        s["row_bias"] = 0.1 * _randn(g, N) if c["row_bias"] else None
        s["residual"] = _randn(g, T, N).to(_BF16) if c["residual"] else None
        s["y"] = torch.empty(T, N, dtype=out_type, device="cuda")
    else:
        # gradients: small, of very different sizes from token to token, none where a token has no loss
        size = 1e-3 * torch.exp(2 * _randn(g, T, 1)) * (_rand(g, T, 1) > 0.1)
        s["dy"] = _padded((size * _randn(g, T, N)).to(out_type), c["pad"])
        s["dx"] = torch.empty(T, K, dtype=_BF16, device="cuda")
    return s


def _prepare_router(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    s = {"case": c}
    logits = 1.2 * _randn(g, T, E) - torch.log(1 + torch.arange(E, device="cuda", dtype=_F32))
    if c["disabled"]:
        off = torch.randperm(E, generator=g, device="cuda")[:c["disabled"]]
        logits[:, off] = float("-inf")
    s["valid"] = None
    gate_size = torch.ones(T, 1, device="cuda")
    if c["padded"]:
        # tokens behind the ends of their sequences: not valid, some with no logits at all
        s["valid"] = (torch.arange(T, device="cuda") % 512 < 400).to(torch.uint8)
        none = (torch.arange(T, device="cuda") % 512) >= 480
        logits[none] = float("-inf")
        gate_size = s["valid"].float()[:, None]
    s["logits"] = logits.contiguous()
    top, ids = torch.topk(logits, k, dim=1)
    s["ids"] = ids.to(torch.int32).contiguous()
    den = top.double() if c["renorm"] else logits.double()
    gates = torch.exp(top.double() - top[:, :1].double()) / torch.exp(den - top[:, :1].double()).sum(1, keepdim=True)
    s["gates"] = torch.nan_to_num(gates, nan=0.0).float().contiguous()
    if c["op"] == "route_backward":
        s["dgates"] = (gate_size * _randn(g, T, k)).contiguous()
        s["dlosses"] = torch.tensor([1e-2, 1e-3], device="cuda") * (1 + 0.1 * _rand(g, 2))
        take = torch.isfinite(logits).any(1)
        if s["valid"] is not None:
            take = take & (s["valid"] != 0)
        s["counts"] = torch.zeros(E, dtype=torch.int32, device="cuda").index_add_(
            0, ids[take].reshape(-1), torch.ones(int(take.sum()) * k, dtype=torch.int32, device="cuda"))
        s["n_valid"] = take.sum().to(torch.int32).reshape(1)
        s["dlogits"] = torch.empty(T, E, device="cuda")
    else:
        s["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        s["prob_mean"] = torch.empty(E, device="cuda")
        s["n_valid"] = torch.empty(1, dtype=torch.int32, device="cuda")
        s["losses"] = torch.empty(2, device="cuda")
    return s


def _prepare_combine(c, g):
    T, H, k = c["T"], c["H"], c["k"]
    return {
        "case": c,
        "dout": (1e-3 * _randn(g, T, H)).to(_BF16),
        "y_rows": _randn(g, T * k, H).to(_BF16),
        "pair_to_row": torch.randperm(T * k, generator=g, device="cuda").to(torch.int32),
        "gates": torch.softmax(_randn(g, T, k), 1),
        "dy_rows": torch.empty(T * k, H, dtype=_BF16, device="cuda"),
        "dgates": torch.empty(T, k, device="cuda"),
    }


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("linear", "linear_grad"):
        return _prepare_linear(case, g)
    if case["op"] == "combine_backward":
        return _prepare_combine(case, g)
    return _prepare_router(case, g)


# ------------------------------------------------------------ plain forms

def _dequant(s):
    """The matrix [N][K] in float32 from its group-major codes."""
    c, q = s["case"], s["q"]
    if c["bits"] == 4:
        codes = torch.stack((q & 15, q >> 4), dim=-1)
    else:
        codes = torch.stack((q & 3, (q >> 2) & 3, (q >> 4) & 3, q >> 6), dim=-1)
    codes = codes.reshape(q.shape[0], q.shape[1], 128).permute(1, 0, 2).reshape(c["N"], c["K"] // c["group"], c["group"])
    return (codes.float() * s["scale"].float()[:, :, None] + s["bias"].float()[:, :, None]).reshape(c["N"], c["K"])


def _plain_linear(s):
    y = s["x"].float() @ _dequant(s).t()
    if s["row_bias"] is not None:
        y = y + s["row_bias"]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(s["y"].dtype)}


def _plain_linear_grad(s):
    return {"dx": (s["dy"].float() @ _dequant(s)).to(_BF16)}


def _plain_softmax(s):
    """(p, log-sum-exp, rows that have a logit)"""
    L = s["logits"]
    top = L.max(1, keepdim=True).values
    some = top > float("-inf")
    top = torch.where(some, top, torch.zeros_like(top))
    e = torch.exp(L - top)
    total = e.sum(1, keepdim=True)
    p = torch.where(some, e / total, torch.zeros_like(e))
    lse = torch.where(some, top + torch.log(total), torch.zeros_like(top))
    return p, lse, some


def _takes_part(s, some):
    take = some[:, 0]
    return take if s["valid"] is None else take & (s["valid"] != 0)


def _plain_balance(s):
    c = s["case"]
    p, lse, some = _plain_softmax(s)
    take = _takes_part(s, some)
    n = take.sum()
    counts = torch.zeros(c["E"], dtype=torch.int32, device="cuda").index_add_(
        0, s["ids"].reshape(-1), take.to(torch.int32)[:, None].expand(-1, c["k"]).reshape(-1))
    m = n.clamp(min=1).float()
    prob_mean = (p * take[:, None]).sum(0) / m
    balance = c["E"] * (counts.float() / (m * c["k"]) * prob_mean).sum()
    z = (lse[:, 0].square() * take).sum() / m
    return {"counts": counts, "prob_mean": prob_mean, "n_valid": n.to(torch.int32).reshape(1),
            "losses": torch.stack((balance, z))}


def _plain_route_backward(s):
    c = s["case"]
    p, lse, some = _plain_softmax(s)
    take = _takes_part(s, some).float()[:, None]
    ids, g, dg = s["ids"].long(), s["gates"], s["dgates"]
    m = s["n_valid"].clamp(min=1).float()
    f = s["counts"].float() / (m * c["k"])
    d = take * (s["dlosses"][0] * c["E"] / m * p * (f - (p * f).sum(1, keepdim=True))
                + s["dlosses"][1] * 2 / m * lse * p)
    dot = (g * dg).sum(1, keepdim=True)
    if c["renorm"]:
        return {"dlogits": d.scatter_add(1, ids, g * (dg - dot))}
    return {"dlogits": (d - p * dot).scatter_add(1, ids, g * dg)}


def _plain_combine_backward(s):
    c = s["case"]
    rows = s["pair_to_row"].long()
    dout = s["dout"].float()
    y = s["y_rows"][rows].float().reshape(c["T"], c["k"], c["H"])
    dgates = (y * dout[:, None, :]).sum(2)
    dy = torch.empty_like(s["dy_rows"])
    dy[rows] = (s["gates"][:, :, None] * dout[:, None, :]).reshape(-1, c["H"]).to(_BF16)
    return {"dgates": dgates, "dy_rows": dy}


_PLAIN = {"linear": _plain_linear, "linear_grad": _plain_linear_grad, "balance": _plain_balance,
          "route_backward": _plain_route_backward, "combine_backward": _plain_combine_backward}


# ------------------------------------------------------- the library's calls

def _own_linear(s):
    import quantized_expert_ffn_gemv_amd as moe
    c = s["case"]
    if "w" not in s:
        s["w"] = moe.QMatrix(c["bits"], c["group"], s["q"], s["scale"], s["bias"])
        s["buf"] = moe.LinearBuffers.allocate(s["w"], c["T"], s["y"].dtype)
    moe.linear(s["w"], s["x"], s["y"], s["buf"], row_bias=s["row_bias"], residual=s["residual"])
    return {"y": s["y"]}


def _own_linear_grad(s):
    import quantized_expert_ffn_gemv_amd as moe
    c = s["case"]
    if "w" not in s:
        s["w"] = moe.QMatrix(c["bits"], c["group"], s["q"], s["scale"], s["bias"])
        s["buf"] = moe.LinearBuffers.allocate(s["w"], c["T"], s["dy"].dtype, grad=True)
    moe.linear_grad(s["w"], s["dy"], s["dx"], s["buf"])
    return {"dx": s["dx"]}


def _own_balance(s):
    import quantized_expert_ffn_gemv_amd as moe
    c = s["case"]
    if "buf" not in s:
        s["d"] = moe.dims(c["T"], 128, 128, c["E"], c["k"])
        s["buf"] = moe.BalanceBuffers.allocate(s["d"])
    moe.balance_loss(s["d"], s["logits"], s["ids"], s["counts"], s["prob_mean"], s["n_valid"], s["losses"], s["buf"],
                     valid=s["valid"])
    return {"counts": s["counts"], "prob_mean": s["prob_mean"], "n_valid": s["n_valid"], "losses": s["losses"]}


def _own_route_backward(s):
    import quantized_expert_ffn_gemv_amd as moe
    c = s["case"]
    if "d" not in s:
        s["d"] = moe.dims(c["T"], 128, 128, c["E"], c["k"])
    moe.route_backward(s["d"], s["logits"], s["ids"], s["gates"], c["renorm"], s["dlogits"], topk_w_grad=s["dgates"],
                       losses_grad=s["dlosses"], expert_counts=s["counts"], n_valid=s["n_valid"], valid=s["valid"])
    return {"dlogits": s["dlogits"]}


def _own_combine_backward(s):
    import quantized_expert_ffn_gemv_amd as moe
    c = s["case"]
    if "d" not in s:
        s["d"] = moe.dims(c["T"], c["H"], 128, 1024, c["k"])
    moe.combine_backward(s["d"], s["dout"], s["y_rows"], s["pair_to_row"], s["gates"], s["dgates"], s["dy_rows"])
    return {"dgates": s["dgates"], "dy_rows": s["dy_rows"]}


_OWN = {"linear": _own_linear, "linear_grad": _own_linear_grad, "balance": _own_balance,
        "route_backward": _own_route_backward, "combine_backward": _own_combine_backward}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact

def _exact_matrix(s):
    c, q = s["case"], s["q"].to(torch.int32)
    per = 8 // c["bits"]
    shifts = c["bits"] * torch.arange(per, device="cuda", dtype=torch.int32)
    codes = (q.unsqueeze(-1) >> shifts) & ((1 << c["bits"]) - 1)
    codes = codes.flatten(-2).transpose(0, 1).flatten(1).to(_F64)
    spread = lambda v: v.to(_F64).repeat_interleave(c["group"], dim=1)  # noqa: E731
    return codes * spread(s["scale"]) + spread(s["bias"])


def _exact_router(s):
    """Row by row definitions in float64, only over the rows that have a logit."""
    c, L = s["case"], s["logits"].to(_F64)
    has = torch.isfinite(L).sum(1) > 0
    lse = torch.zeros(c["T"], dtype=_F64, device="cuda")
    lse[has] = torch.logsumexp(L[has], 1)
    p = torch.zeros_like(L)
    p[has] = torch.softmax(L[has], 1)
    part = has.to(_F64) if s["valid"] is None else has.to(_F64) * s["valid"].to(_F64)
    return p, lse, part


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "linear":
        y = torch.matmul(s["x"].to(_F64), _exact_matrix(s).transpose(0, 1).contiguous())
        if s["row_bias"] is not None:
            y += s["row_bias"].to(_F64)[None, :]
        if s["residual"] is not None:
            y += s["residual"].to(_F64)
        return {"y": y}
    if op == "linear_grad":
        return {"dx": torch.matmul(s["dy"].to(_F64).contiguous(), _exact_matrix(s))}
    if op == "combine_backward":
        by_token = s["y_rows"].to(_F64)[s["pair_to_row"].long()].view(c["T"], c["k"], c["H"])
        dgates = torch.matmul(by_token, s["dout"].to(_F64).unsqueeze(-1)).squeeze(-1)
        dy = torch.zeros(c["T"] * c["k"], c["H"], dtype=_F64, device="cuda")
        token = torch.arange(c["T"], device="cuda").repeat_interleave(c["k"])
        dy[s["pair_to_row"].long()] = s["gates"].to(_F64).view(-1, 1) * s["dout"].to(_F64)[token]
        return {"dgates": dgates, "dy_rows": dy}
    p, lse, part = _exact_router(s)
    if op == "balance":
        picks = torch.bincount(s["ids"].long().view(-1), weights=part.repeat_interleave(c["k"]), minlength=c["E"])
        n = float(part.sum())
        m = max(n, 1.0)
        mean = torch.matmul(part, p) / m
        losses = torch.stack((c["E"] * torch.dot(picks, mean) / (m * c["k"]), torch.dot(part, lse * lse) / m))
        return {"counts": None, "prob_mean": mean, "n_valid": None, "losses": losses}
    m = float(max(int(s["n_valid"]), 1))
    f = s["counts"].to(_F64) / (m * c["k"])
    a, z = (float(v) for v in s["dlosses"].to(_F64))
    d = p * ((f[None, :] - torch.mv(p, f)[:, None]) * (a * c["E"] / m) + (lse * (2 * z / m))[:, None]) * part[:, None]
    g, dg = s["gates"].to(_F64), s["dgates"].to(_F64)
    inner = (g * dg).sum(1)
    at = (torch.arange(c["T"], device="cuda").repeat_interleave(c["k"]), s["ids"].long().view(-1))
    if c["renorm"]:
        d.index_put_(at, (g * (dg - inner[:, None])).view(-1), accumulate=True)
    else:
        d -= p * inner[:, None]
        d.index_put_(at, (g * dg).view(-1), accumulate=True)
    return {"dlogits": d}


# -------------------------------------------------------------------- work

def work(case):
    c, T = case, case["T"]
    if c["op"] in ("linear", "linear_grad"):
        N, K = c["N"], c["K"]
        wide = 4 if c["f32"] else 2
        nbytes = N * K * c["bits"] // 8 + 4 * N * (K // c["group"])
        nbytes += T * (2 * K + wide * N)
        nbytes += (4 * N if c["row_bias"] else 0) + (2 * T * N if c["residual"] else 0)
        return {"bytes": nbytes, "flops": 2 * T * N * K}
    if c["op"] == "combine_backward":
        pairs, H = T * c["k"], c["H"]
        return {"bytes": 2 * T * H + 4 * pairs * H + 12 * pairs, "flops": 3 * pairs * H}
    E, k = c["E"], c["k"]
    nbytes = 4 * T * E + 4 * T * k + (T if c["padded"] else 0)
    if c["op"] == "balance":
        return {"bytes": nbytes + 8 * E + 12, "flops": 5 * T * E}
    return {"bytes": nbytes + 4 * T * E + 8 * T * k + 4 * E + 12, "flops": 9 * T * E}
