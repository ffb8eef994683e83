"""Operators for tuning and scoring over the layer's frozen quantised weights, as a
benchmark: low-rank adapters of many requests beside a shared projection (forward and
gradients), log probabilities of given tokens with entropy and top alternatives (and
their gradient), and activation checkpoints in 8 bits with the gradients that read them.

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

def _adapter(op, T, K, N, R, n, ragged=False, mixed=True, none=False, f32=False, saved=False, pad=0):
    """ragged: ranks differ; mixed: adapters in any order (else a run of tokens each); none: some
    tokens use no adapter; f32: y (or dy) float32; saved: x from an 8-bit checkpoint; pad: extra
    columns of the wider buffers that the rows are slices of."""
    return {"op": op, "T": T, "K": K, "N": N, "R": R, "n": n, "ragged": ragged, "mixed": mixed, "none": none, "f32": f32,
            "saved": saved, "pad": pad}


def _logprobs(op, T, V, f32=True, top=0, masked=False, padded=False, entropy=True):
    return {"op": op, "T": T, "V": V, "f32": f32, "top": top, "masked": masked, "padded": padded, "entropy": entropy}


def listed():
    return [
        # a batch of decoded tokens, each with its request's adapter or none, ranks 16, 8 and 4
        dict(_adapter("adapter", 48, 4096, 4096, 16, 32, ragged=True, none=True), name="adapter_T48"),
        # prompts of eight requests through an up projection
        dict(_adapter("adapter", 4096, 2048, 8192, 32, 8, mixed=False), name="adapter_T4096"),
        # gradients of a short ragged batch through a projection of odd size, float32 dy
        dict(_adapter("adapter_grad", 37, 2048, 5111, 8, 3, ragged=True, none=True, f32=True), name="adapter_grad_T37"),
        # a training batch over four adapters, the inputs kept in 8 bits
        dict(_adapter("adapter_grad", 4096, 2048, 8192, 16, 4, saved=True), name="adapter_grad_T4096"),
        # one decoded token's log probability, entropy and 20 alternatives: latency counts
        dict(_logprobs("logprobs", 1, 49999, top=20), name="logprobs_T1"),
        # scoring a padded batch of sequences, bf16 logits with a part of the vocabulary masked
        dict(_logprobs("logprobs", 4096, 49999, f32=False, top=5, masked=True, padded=True), name="logprobs_T4096"),
        # the gradient of a small batch
        dict(_logprobs("logprobs_grad", 8, 49999), name="logprobs_grad_T8"),
        # and of a training batch with its padding
        dict(_logprobs("logprobs_grad", 4096, 49999, f32=False, padded=True), name="logprobs_grad_T4096"),
        # a decode batch's layer input kept and restored
        {"op": "checkpoint", "T": 8, "K": 2048, "pad": 0, "name": "checkpoint_T8"},
        # the expert rows of a training batch (4096 tokens, 8 picks)
        {"op": "checkpoint", "T": 32768, "K": 2048, "pad": 0, "name": "checkpoint_T32768"},
        # the gates' gradient of that batch from the checkpoint of its expert rows
        {"op": "gates_saved", "T": 4096, "H": 2048, "k": 8, "rows_grad": False, "name": "gates_saved_T4096"},
        # the router's weight gradient of a training batch from the checkpoint of its input
        {"op": "router_weight", "T": 8192, "H": 2048, "E": 128, "saved": True, "name": "router_weight_T8192"},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng: random.Random):
    op = rng.choice(["adapter", "adapter", "adapter_grad", "adapter_grad", "logprobs", "logprobs", "logprobs_grad",
                     "checkpoint", "gates_saved", "router_weight"])
    if op in ("adapter", "adapter_grad"):
        K, N = 128 * _log_int(rng, 1, 64), _log_int(rng, 8, 16384)
        R = rng.choice([4, 8, 16, 16, 32, 64, _log_int(rng, 1, 128)])
        n = _log_int(rng, 1, 256)
        T = _log_int(rng, 1, max(1, min(4096, 4096 * 8 * 32 * (2048 + 8192) // (n * R * (K + N)))))
        return _adapter(op, T, K, N, R, n, ragged=rng.random() < 0.4, mixed=rng.random() < 0.6, none=rng.random() < 0.4,
                        f32=rng.random() < 0.3, saved=op == "adapter_grad" and rng.random() < 0.4,
                        pad=8 * rng.choice([0, 0, 1, 5, 16]))
    if op in ("logprobs", "logprobs_grad"):
        V = _log_int(rng, 2, 150000)
        T = _log_int(rng, 1, max(1, min(16384, 4096 * 49999 // V)))
        return _logprobs(op, T, V, f32=rng.random() < 0.5, top=0 if op == "logprobs_grad" else rng.choice([0, 0, 1, 5, 20, 50]),
                         masked=rng.random() < 0.4, padded=rng.random() < 0.4, entropy=rng.random() < 0.7)
    if op == "checkpoint":
        K = 128 * _log_int(rng, 1, 64)
        return {"op": op, "T": _log_int(rng, 1, 32768 * 2048 // K), "K": K, "pad": 8 * rng.choice([0, 0, 1, 5, 16])}
    if op == "gates_saved":
        k, H = rng.randint(1, 10), 128 * _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(1, min(65536 // k, 4096 * 8 * 2048 // (3 * k * H))))
        return {"op": op, "T": T, "H": H, "k": k, "rows_grad": rng.random() < 0.4}
    E, H = _log_int(rng, 4, 1024), 128 * _log_int(rng, 1, 64)
    return {"op": op, "T": _log_int(rng, 1, max(1, min(16384, 8192 * 2048 * 128 // (E * H)))), "H": H, "E": E,
            "saved": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6007 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _rows(t, pad):
    """t's rows as the first columns of a wider buffer."""
    if not pad:
        return t.contiguous()
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _activations(g, T, K):
    """Rows as they come out of a residual stream: a few columns far larger than the rest."""
    big = 1 + 12 * (_rand(g, K) < 0.01)
    return (_randn(g, T, K) * big).to(_BF16)


def _codes(x):
    """8-bit codes and scales of x (bf16 [T, K]), one scale for each 128 columns."""
    v = x.double().reshape(x.shape[0], -1, 128)
    top = v.abs().amax(2, keepdim=True)
    q = torch.round(v * 127 / torch.where(top > 0, top, torch.ones_like(top))).to(torch.int8)
    return q.reshape(x.shape).contiguous(), (top[:, :, 0].float() / 127).contiguous()


def _ranks(c):
    """The rank of the j-th adapter in use."""
    return [max(1, c["R"] >> (j % 3)) if c["ragged"] else c["R"] for j in range(c["n"])]


def _prepare_adapter(c, g):
    T, K, N, R, n = c["T"], c["K"], c["N"], c["R"], c["n"]
    s = {"case": c}
    order = torch.randperm(n, generator=g, device="cuda")
    used = min(n, T)
    # every adapter in use has a token, the rest fall at random places: runs of many lengths
    first = torch.arange(used, device="cuda")
    rest = torch.randint(0, used, (T - used,), generator=g, device="cuda")
    if T > used:
        rest = torch.where(_rand(g, T - used) < 0.3, torch.zeros_like(rest), rest)
    slot = torch.sort(torch.cat((first, rest))).values
    if c["mixed"]:
        slot = slot[torch.randperm(T, generator=g, device="cuda")]
    ids = order[slot]
    if c["none"]:
        ids = torch.where(_rand(g, T) < 0.12, torch.full_like(ids, -1), ids)
    s["ids"] = ids.to(torch.int32).contiguous()
    s["rank"] = None
    if c["ragged"]:
        s["rank"] = torch.empty(n, dtype=torch.int32, device="cuda")
        s["rank"][order] = torch.tensor(_ranks(c), dtype=torch.int32, device="cuda")
    s["a"] = (_randn(g, n, R, K) / math.sqrt(K)).to(_BF16)
    wide = (N + 7) // 8 * 8                       # rows of b start at multiples of 16 bytes
    s["b"] = (0.3 * _randn(g, n, R, wide)).to(_BF16)[:, :, :N]
    s["scale"] = 0.5 + 1.5 * _rand(g, n)
    x = _activations(g, T, K)
    out_type = _F32 if c["f32"] else _BF16
    if c["op"] == "adapter":
        s["x"] = _rows(x, c["pad"])
        s["base"] = _rows(_randn(g, T, N).to(out_type), c["pad"])
        s["y"] = _rows(torch.empty(T, N, dtype=out_type, device="cuda"), c["pad"])
        s["h"] = torch.empty(T, R, device="cuda")
        return s
    if c["saved"]:
        s["q"], s["q_scale"] = _codes(x)
    else:
        s["x"] = _rows(x, c["pad"])
    size = 1e-3 * torch.exp(2 * _randn(g, T, 1)) * (_rand(g, T, 1) > 0.1)
    s["dy"] = _rows((size * _randn(g, T, N)).to(out_type), c["pad"])
    s["h"] = _randn(g, T, R)                      # as the forward pass left it
    s["dx_base"] = _rows((1e-2 * size * _randn(g, T, K)).to(_BF16), c["pad"])
    s["dx"] = _rows(torch.empty(T, K, dtype=_BF16, device="cuda"), c["pad"])
    s["da"] = torch.empty(n, R, K, device="cuda")
    s["db"] = torch.empty(n, R, N, device="cuda")
    return s


def _prepare_logprobs(c, g):
    T, V = c["T"], c["V"]
    kind = _F32 if c["f32"] else _BF16
    s = {"case": c}
    logits = _randn(g, T, V)
    logits *= 1 + 2.5 * _rand(g, T, 1)            # rows between nearly even and confident
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    likely = torch.randint(0, V, (T,), generator=g, device="cuda")
    tokens = torch.where(_rand(g, T) < 0.6, likely, tokens)
    logits[torch.arange(T, device="cuda"), likely] += 14 * _rand(g, T)
    if c["masked"]:
        off = _rand(g, V) < 0.2                   # never drawn, the given tokens excepted
        keep = logits[torch.arange(T, device="cuda"), tokens]
        logits[:, off] = float("-inf")
        logits[torch.arange(T, device="cuda"), tokens] = keep
    none = torch.zeros(T, dtype=torch.bool, device="cuda")
    if c["padded"]:
        # rows behind the ends of their sequences, some of them without any logit
        at = torch.arange(T, device="cuda") % 512
        none = at >= 400
        logits[at >= 480] = float("-inf")
        tokens = torch.where(none, torch.full_like(tokens, -1), tokens)
    s["logits"] = logits.to(kind)
    s["tokens"] = tokens.to(torch.int32)
    if c["op"] == "logprobs":
        s["logp"], s["stats"] = torch.empty(T, device="cuda"), torch.empty(T, 2, device="cuda")
        s["entropy"] = torch.empty(T, device="cuda") if c["entropy"] else None
        s["top_ids"] = torch.empty(T, c["top"], dtype=torch.int32, device="cuda") if c["top"] else None
        s["top_logp"] = torch.empty(T, c["top"], device="cuda") if c["top"] else None
        return s
    # what the forward pass left: (maximum, logarithm of the sum relative to it) and the entropy, by
    # pieces of rows, since in 64 bits
    stats, entropy = [], []
    for piece in s["logits"].split(max(1, (1 << 26) // V)):
        v = piece.double()
        m = v.amax(1, keepdim=True)
        d = (v - torch.where(m > float("-inf"), m, torch.zeros_like(m))).clamp(min=-800.0)
        e = torch.exp(d)
        total = e.sum(1, keepdim=True)
        some = m > float("-inf")
        log_total = torch.where(some, torch.log(total), torch.full_like(total, float("-inf")))
        stats.append(torch.cat((m, log_total), 1).float())
        entropy.append(torch.where(some, torch.log(total) - (e * d).sum(1, keepdim=True) / total, torch.zeros_like(m))[:, 0].float())
    s["stats"], s["entropy"] = torch.cat(stats).contiguous(), torch.cat(entropy).contiguous()
    s["dlogp"] = torch.where(none, torch.zeros(T, device="cuda"), -(0.5 + _rand(g, T)) / T)
    s["dentropy"] = torch.where(none, torch.zeros(T, device="cuda"), 0.01 * _randn(g, T) / T) if c["entropy"] else None
    s["dlogits"] = torch.empty(T, V, dtype=kind, device="cuda")
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] in ("adapter", "adapter_grad"):
        return _prepare_adapter(c, g)
    if c["op"] in ("logprobs", "logprobs_grad"):
        return _prepare_logprobs(c, g)
    if c["op"] == "checkpoint":
        return {"case": c, "x": _rows(_activations(g, c["T"], c["K"]), c["pad"]),
                "q": torch.empty(c["T"], c["K"], dtype=torch.int8, device="cuda"),
                "scale": torch.empty(c["T"], c["K"] // 128, device="cuda"),
                "back": _rows(torch.empty(c["T"], c["K"], dtype=_BF16, device="cuda"), c["pad"])}
    T, H = c["T"], c["H"]
    if c["op"] == "gates_saved":
        k = c["k"]
        q, scale = _codes(_activations(g, T * k, H))
        return {"case": c, "dout": (1e-3 * _randn(g, T, H)).to(_BF16), "q": q, "scale": scale,
                "pair_to_row": torch.randperm(T * k, generator=g, device="cuda").to(torch.int32),
                "gates": torch.softmax(_randn(g, T, k), 1), "dgates": torch.empty(T, k, device="cuda"),
                "dy_rows": torch.empty(T * k, H, dtype=_BF16, device="cuda") if c["rows_grad"] else None}
    s = {"case": c, "dw": torch.empty(c["E"], H, device="cuda"), "dbias": torch.empty(c["E"], device="cuda")}
    x = _activations(g, T, H)
    if c["saved"]:
        s["q"], s["scale"] = _codes(x)
    else:
        s["x"] = x
    # gradients past the softmax: a few experts a token get most of it
    size = 1e-3 * torch.exp(2 * _randn(g, T, 1))
    s["dlogits"] = (size * _randn(g, T, c["E"]) * torch.where(_rand(g, T, c["E"]) < 0.1, 1.0, 0.02)).contiguous()
    return s


# ------------------------------------------------------------ plain forms

def _spread(h, s):
    """h [T, R] in the places [T, n * R] of each token's adapter, scaled; zeros elsewhere and past its rank."""
    c = s["case"]
    n, R = c["n"], c["R"]
    ids = s["ids"].long()
    mine = (ids[:, None] == torch.arange(n, device="cuda")[None, :]).float() * s["scale"][None, :]
    if s["rank"] is None:
        return (mine[:, :, None] * h[:, None, :]).reshape(-1, n * R)
    live = (torch.arange(R, device="cuda")[None, :] < s["rank"][:, None]).float()
    return (mine[:, :, None] * live[None, :, :] * h[:, None, :]).reshape(-1, n * R)


def _shrunk(v, m, s):
    """v [T, C] times each token's own adapter's m [R, C] (of [n, R, C]); zeros past its rank and without one."""
    c = s["case"]
    n, R = c["n"], c["R"]
    every = (v @ m.float().reshape(n * R, -1).t()).reshape(-1, n, R)
    ids = s["ids"].long()
    h = torch.gather(every, 1, ids.clamp(min=0)[:, None, None].expand(-1, 1, R))[:, 0]
    keep = (ids >= 0)[:, None].expand(-1, R)
    if s["rank"] is not None:
        keep = keep & (torch.arange(R, device="cuda")[None, :] < s["rank"][ids.clamp(min=0)][:, None])
    return torch.where(keep, h, torch.zeros_like(h))


def _plain_adapter(s):
    c = s["case"]
    h = _shrunk(s["x"].float(), s["a"], s)
    y = s["base"].float() + _spread(h, s) @ s["b"].float().reshape(c["n"] * c["R"], c["N"])
    return {"y": y.to(s["y"].dtype), "h": h}


def _plain_x(s):
    """x in float32, as it is or from its checkpoint."""
    if "q" not in s:
        return s["x"].float()
    scale = s["q_scale"] if "q_scale" in s else s["scale"]
    return (s["q"].float().reshape(s["q"].shape[0], -1, 128) * scale[:, :, None]).reshape(s["q"].shape)


def _plain_adapter_grad(s):
    c = s["case"]
    n, R = c["n"], c["R"]
    dy = s["dy"].float()
    g = _spread(_shrunk(dy, s["b"], s), s)
    dx = s["dx_base"].float() + g @ s["a"].float().reshape(n * R, c["K"])
    da = g.t() @ _plain_x(s)
    db = _spread(s["h"], s).t() @ dy
    return {"dx": dx.to(_BF16), "da": da.reshape(n, R, c["K"]), "db": db.reshape(n, R, c["N"])}


def _plain_logprobs(s):
    c, L = s["case"], s["logits"].float()
    V, top = c["V"], c["top"]
    m = L.max(1, keepdim=True).values
    some = m > float("-inf")
    d = L - torch.where(some, m, torch.zeros_like(m))
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.where(some, torch.log(total), torch.full_like(total, float("-inf")))
    tokens = s["tokens"].long()
    here = tokens >= 0
    picked = torch.gather(d, 1, tokens.clamp(min=0)[:, None]) - log_total
    out = {"logp": torch.where(here, picked[:, 0], torch.zeros_like(picked[:, 0]))}
    if c["entropy"]:
        mean = (e * torch.where(e > 0, d, torch.zeros_like(d))).sum(1, keepdim=True) / total
        out["entropy"] = torch.where(some, log_total - mean, torch.zeros_like(mean))[:, 0]
    if top:
        # one 64-bit key an element: larger values first, equal ones by the lower index
        bits = (L + 0.0).view(torch.int32)
        ordered = bits ^ ((bits >> 31) & 0x7FFFFFFF)
        key = ordered.long() * (1 << 32) + (V - 1 - torch.arange(V, device="cuda"))[None, :]
        if top > V:
            key = torch.cat((key, torch.full((key.shape[0], top - V), -(1 << 62), device="cuda")), 1)
        best = torch.topk(key, top, dim=1).values
        at = (V - 1 - (best & 0xFFFFFFFF)).clamp(min=0, max=V - 1)
        value = torch.where(best > -(1 << 62), torch.gather(L, 1, at), torch.full_like(at, 0, dtype=_F32) - float("inf"))
        there = value > float("-inf")
        out["top_ids"] = torch.where(there, at, torch.full_like(at, -1)).to(torch.int32)
        low = value - torch.where(some, m, torch.zeros_like(m)) - log_total
        out["top_logp"] = torch.where(there, low, torch.full_like(value, float("-inf")))
    return out


def _plain_logprobs_grad(s):
    c, L = s["case"], s["logits"].float()
    m, log_total = s["stats"][:, :1], s["stats"][:, 1:]
    some = m > float("-inf")
    logp = L - torch.where(some, m, torch.zeros_like(m)) - torch.where(some, log_total, torch.zeros_like(m))
    p = torch.exp(logp)
    tokens = s["tokens"].long()
    w = s["dlogp"][:, None] * (tokens >= 0).float()[:, None]
    d = -w * p
    if c["entropy"]:
        bent = torch.where(p > 0, logp, torch.zeros_like(logp)) + s["entropy"][:, None]
        d = d - s["dentropy"][:, None] * p * bent
    d = d.scatter_add(1, tokens.clamp(min=0)[:, None], w)
    return {"dlogits": d.to(s["dlogits"].dtype)}


def _plain_checkpoint(s):
    # in 64 bits: a quotient half way between two codes has to be seen as one
    q, scale = _codes(s["x"])
    back = q.double().reshape(q.shape[0], -1, 128) * scale.double()[:, :, None]
    return {"scale": scale, "x": back.reshape(q.shape).to(_BF16)}


def _plain_gates_saved(s):
    c = s["case"]
    rows = s["pair_to_row"].long()
    dout = s["dout"].float()
    y = _plain_x(s)[rows].reshape(c["T"], c["k"], c["H"])
    out = {"dgates": (y * dout[:, None, :]).sum(2)}
    if c["rows_grad"]:
        dy = torch.empty_like(s["dy_rows"])
        dy[rows] = (s["gates"][:, :, None] * dout[:, None, :]).reshape(-1, c["H"]).to(_BF16)
        out["dy_rows"] = dy
    return out


def _plain_router_weight(s):
    return {"dw": s["dlogits"].t() @ _plain_x(s), "dbias": s["dlogits"].sum(0)}


_PLAIN = {"adapter": _plain_adapter, "adapter_grad": _plain_adapter_grad, "logprobs": _plain_logprobs,
          "logprobs_grad": _plain_logprobs_grad, "checkpoint": _plain_checkpoint, "gates_saved": _plain_gates_saved,
          "router_weight": _plain_router_weight}


# ------------------------------------------------------- the library's calls

def _own_adapter(s):
    import quantized_expert_ffn_gemv_amd as moe
    c = s["case"]
    if "set" not in s:
        s["set"] = moe.Adapters(s["a"], s["b"], s["scale"], s["rank"])
        s["buf"] = moe.AdapterBuffers.allocate(s["set"], c["T"])
    moe.adapter(s["set"], s["ids"], s["x"], s["y"], s["buf"], base=s["base"], h=s["h"])
    return {"y": s["y"], "h": s["h"]}


def _own_adapter_grad(s):
    import quantized_expert_ffn_gemv_amd as moe
    c = s["case"]
    if "set" not in s:
        s["set"] = moe.Adapters(s["a"], s["b"], s["scale"], s["rank"])
        s["buf"] = moe.AdapterBuffers.allocate(s["set"], c["T"], grad=True)
        s["kept"] = moe.Checkpoint(s["q"], s["q_scale"]) if c["saved"] else s["x"]
    moe.adapter_grad(s["set"], s["ids"], s["dy"], s["kept"], s["h"], s["buf"], dx=s["dx"], dx_base=s["dx_base"],
                     da=s["da"], db=s["db"])
    return {"dx": s["dx"], "da": s["da"], "db": s["db"]}


def _own_logprobs(s):
    import quantized_expert_ffn_gemv_amd as moe
    c = s["case"]
    if "buf" not in s:
        s["buf"] = moe.LogprobBuffers.allocate(c["T"], c["V"], c["top"])
    moe.logprobs(s["logits"], s["tokens"], s["logp"], s["stats"], s["buf"], entropy=s["entropy"], top_ids=s["top_ids"],
                 top_logp=s["top_logp"])
    out = {"logp": s["logp"]}
    if c["entropy"]:
        out["entropy"] = s["entropy"]
    if c["top"]:
        out["top_ids"], out["top_logp"] = s["top_ids"], s["top_logp"]
    return out


def _own_logprobs_grad(s):
    import quantized_expert_ffn_gemv_amd as moe
    moe.logprobs_grad(s["logits"], s["tokens"], s["stats"], s["dlogits"], logp_grad=s["dlogp"], entropy=s["entropy"],
                      entropy_grad=s["dentropy"])
    return {"dlogits": s["dlogits"]}


def _own_checkpoint(s):
    import quantized_expert_ffn_gemv_amd as moe
    if "kept" not in s:
        s["kept"] = moe.Checkpoint(s["q"], s["scale"])
    moe.checkpoint_save(s["x"], s["kept"])
    moe.checkpoint_restore(s["kept"], s["back"])
    return {"scale": s["scale"], "x": s["back"]}


def _own_gates_saved(s):
    import quantized_expert_ffn_gemv_amd as moe
    c = s["case"]
    if "d" not in s:
        s["d"] = moe.dims(c["T"], c["H"], 128, 1024, c["k"])
        s["kept"] = moe.Checkpoint(s["q"], s["scale"])
    moe.combine_backward(s["d"], s["dout"], s["kept"], s["pair_to_row"], s["gates"], s["dgates"], s["dy_rows"])
    return {"dgates": s["dgates"], "dy_rows": s["dy_rows"]} if c["rows_grad"] else {"dgates": s["dgates"]}


def _own_router_weight(s):
    import quantized_expert_ffn_gemv_amd as moe
    c = s["case"]
    if "d" not in s:
        s["d"] = moe.dims(c["T"], c["H"], 128, c["E"], 1)
        s["buf"] = moe.RouterWeightBuffers.allocate(s["d"])
        s["kept"] = moe.Checkpoint(s["q"], s["scale"]) if c["saved"] else s["x"]
    moe.router_weight_grad(s["d"], s["dlogits"], s["kept"], s["dw"], s["buf"], bias_grad=s["dbias"])
    return {"dw": s["dw"], "dbias": s["dbias"]}


_OWN = {"adapter": _own_adapter, "adapter_grad": _own_adapter_grad, "logprobs": _own_logprobs,
        "logprobs_grad": _own_logprobs_grad, "checkpoint": _own_checkpoint, "gates_saved": _own_gates_saved,
        "router_weight": _own_router_weight}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact

def _exact_saved(q, scale):
    return q.to(_F64) * scale.to(_F64).repeat_interleave(128, dim=1)


def _exact_adapter(s):
    """Adapter by adapter: its tokens' rows times its factors, cut to its rank."""
    c = s["case"]
    T, K, N, R, n = c["T"], c["K"], c["N"], c["R"], c["n"]
    ids = s["ids"].tolist()
    ranks = [R] * n if s["rank"] is None else s["rank"].tolist()
    scales = s["scale"].to(_F64).tolist()
    grad = c["op"] == "adapter_grad"
    if grad:
        x = _exact_saved(s["q"], s["q_scale"]) if c["saved"] else s["x"].to(_F64)
        dy, h = s["dy"].to(_F64), s["h"].to(_F64)
        dx = s["dx_base"].to(_F64).clone()
        da, db = torch.zeros(n, R, K, dtype=_F64, device="cuda"), torch.zeros(n, R, N, dtype=_F64, device="cuda")
    else:
        x = s["x"].to(_F64)
        y, h = s["base"].to(_F64).clone(), torch.zeros(T, R, dtype=_F64, device="cuda")
    for i in sorted(set(ids) - {-1}):
        at = torch.tensor([t for t in range(T) if ids[t] == i], device="cuda")
        r = ranks[i]
        A, B = s["a"][i, :r].to(_F64), s["b"][i, :r].to(_F64)
        if not grad:
            part = torch.mm(x[at], A.t().contiguous())
            h[at, :r] = part
            y[at] += scales[i] * torch.mm(part, B)
            continue
        g = scales[i] * torch.mm(dy[at], B.t().contiguous())
        dx[at] += torch.mm(g, A)
        da[i, :r] = torch.mm(g.t().contiguous(), x[at])
        db[i, :r] = scales[i] * torch.mm(h[at, :r].t().contiguous(), dy[at])
    return {"dx": dx, "da": da, "db": db} if grad else {"y": y, "h": h}


def _exact_logprobs(s):
    c = s["case"]
    T, V, top = c["T"], c["V"], c["top"]
    out = {"logp": [], "entropy": [], "top_logp": [], "dlogits": []}
    for t0 in range(0, T, max(1, (1 << 27) // V)):
        rows = slice(t0, min(T, t0 + max(1, (1 << 27) // V)))
        v = s["logits"][rows].to(_F64)
        tok = s["tokens"][rows].long()
        empty = torch.isinf(v).all(1)
        v[empty] = 0.0
        logp = torch.log_softmax(v, 1)
        finite = torch.isfinite(logp)
        p = torch.exp(logp)
        H = -torch.where(finite, p * logp, torch.zeros_like(p)).sum(1)
        H[empty] = 0.0
        p[empty] = 0.0
        row = torch.arange(v.shape[0], device="cuda")
        if c["op"] == "logprobs":
            got = logp[row, tok.clamp(min=0)]
            got[empty] = float("-inf")
            got[tok < 0] = 0.0
            out["logp"].append(got)
            out["entropy"].append(H)
            if top:
                logp[empty] = float("-inf")
                best = torch.full((v.shape[0], top), float("-inf"), dtype=_F64, device="cuda")
                best[:, :min(top, V)] = torch.sort(torch.topk(logp, min(top, V), dim=1).values, 1, descending=True).values
                out["top_logp"].append(best)
        else:
            w = s["dlogp"][rows].to(_F64) * (tok >= 0)
            d = -w[:, None] * p
            if c["entropy"]:
                d -= s["dentropy"][rows].to(_F64)[:, None] * p * (torch.where(finite, logp, torch.zeros_like(logp)) + H[:, None])
            d[row[tok >= 0], tok[tok >= 0]] += w[tok >= 0]
            out["dlogits"].append(d)
    if c["op"] == "logprobs_grad":
        return {"dlogits": torch.cat(out["dlogits"])}
    full = {"logp": torch.cat(out["logp"])}
    if c["entropy"]:
        full["entropy"] = torch.cat(out["entropy"])
    if top:
        full["top_ids"], full["top_logp"] = None, torch.cat(out["top_logp"])
    return full


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op in ("adapter", "adapter_grad"):
        return _exact_adapter(s)
    if op in ("logprobs", "logprobs_grad"):
        return _exact_logprobs(s)
    if op == "checkpoint":
        v = s["x"].to(_F64).contiguous().view(c["T"], c["K"] // 128, 128)
        step = torch.linalg.vector_norm(v, ord=float("inf"), dim=2) / 127
        back = torch.where(step[..., None] > 0, torch.round(v / step[..., None]), torch.zeros_like(v)) * step[..., None]
        # the division by a rounded step may turn a tie: those are taken as they are defined, to even
        twice = v * 254
        tie = torch.remainder(twice, 127 * step[..., None]) == 0
        half = torch.where(tie, twice / torch.where(step > 0, 127 * step, torch.ones_like(step))[..., None], torch.zeros_like(v))
        odd = tie & (torch.remainder(torch.round(half), 2) == 1)
        low = torch.floor(torch.round(half) / 2)
        even = low + (torch.remainder(low, 2) == 1).to(_F64)
        return {"scale": step, "x": torch.where(odd, even * step[..., None], back).view(c["T"], c["K"])}
    if op == "gates_saved":
        by_token = _exact_saved(s["q"], s["scale"])[s["pair_to_row"].long()].view(c["T"], c["k"], c["H"])
        out = {"dgates": torch.matmul(by_token, s["dout"].to(_F64).unsqueeze(-1)).squeeze(-1)}
        if c["rows_grad"]:
            dy = torch.zeros(c["T"] * c["k"], c["H"], dtype=_F64, device="cuda")
            token = torch.arange(c["T"], device="cuda").repeat_interleave(c["k"])
            dy[s["pair_to_row"].long()] = s["gates"].to(_F64).view(-1, 1) * s["dout"].to(_F64)[token]
            out["dy_rows"] = dy
        return out
    x = _exact_saved(s["q"], s["scale"]) if c["saved"] else s["x"].to(_F64)
    d = s["dlogits"].to(_F64)
    return {"dw": torch.matmul(d.t().contiguous(), x), "dbias": d.sum(0)}


# -------------------------------------------------------------------- work

def work(case):
    c, T = case, case["T"]
    if c["op"] in ("adapter", "adapter_grad"):
        K, N, R, n = c["K"], c["N"], c["R"], c["n"]
        used = min(n, T)
        ranks = sum(_ranks(c)[:used])
        weights = 2 * ranks * (K + N)             # the rows within their ranks of the adapters in use
        wide = 4 if c["f32"] else 2
        mean = ranks / used
        if c["op"] == "adapter":
            return {"bytes": weights + T * (2 * K + 2 * wide * N + 4 * R + 4), "flops": int(2 * T * mean * (K + N))}
        x = T * (K + 4 * (K // 128)) if c["saved"] else 2 * T * K
        return {"bytes": weights + x + T * (wide * N + 4 * K + 4 * R + 4) + 4 * n * R * (K + N),
                "flops": int(4 * T * mean * (K + N))}
    if c["op"] in ("logprobs", "logprobs_grad"):
        V, wide = c["V"], 4 if c["f32"] else 2
        live = T
        if c["padded"] and c["op"] == "logprobs_grad":
            live = sum(1 for t in range(T) if t % 512 < 400)     # a row without a gradient is not read
        if c["op"] == "logprobs":
            return {"bytes": T * (wide * V + 8 + 8 * c["top"] + (4 if c["entropy"] else 0)), "flops": 5 * T * V}
        return {"bytes": wide * V * (T + live) + 20 * T, "flops": 6 * live * V}
    if c["op"] == "checkpoint":
        return {"bytes": T * c["K"] * 6 + 8 * T * (c["K"] // 128), "flops": 6 * T * c["K"]}
    H = c["H"]
    if c["op"] == "gates_saved":
        P = T * c["k"]
        return {"bytes": 2 * T * H + P * H + 4 * P * (H // 128) + 8 * P + (2 * P * H + 4 * P if c["rows_grad"] else 0),
                "flops": (3 if c["rows_grad"] else 2) * P * H}
    E = c["E"]
    x = T * (H + 4 * (H // 128)) if c["saved"] else 2 * T * H
    return {"bytes": 4 * T * E + x + 4 * E * H + 4 * E, "flops": 2 * T * E * H}
