"""Cases, plain forms and 64-bit forms of the mixture-of-experts and adapter operators.

Four operators over token rows grouped by an index that is known only on the device:

  route     softmax top-k choice of experts, the rows sorted by expert, and the gradient of the logits
  experts   matrix products grouped by expert with ragged sizes: up (gathered rows, activation), down,
            and the backward pass of a down projection (input gradient through the activation, weight gradient)
  combine   the weighted sum of each token's expert rows, and its backward pass
  lora      low-rank adapters of many requests at once beside a shared column-parallel projection

`own` selects the framework's entry points; otherwise every operator is computed from elementary torch
operations in 32 bits and rounded once at the end.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # Serving, one request decoding one token: latency is all.
        dict(name="route one token", op="route", N=1, E=64, k=8, gate="topk", dtype="f32", masked=0, grad=False),
        # Training step: a packed batch with padding tokens (every expert masked), gradient included.
        dict(name="route training batch", op="route", N=16384, E=128, k=8, gate="softmax", dtype="f32", masked=300,
             grad=True),
        # One token through 2 of 8 experts of the width of the Llama-3-8B MLP: pure weight streaming.
        dict(name="experts up one token", op="up", N=1, E=8, k=2, h=4096, F=14336, act="swiglu", grad=False),
        # The same layer's down projection: a long contraction and few output tiles.
        dict(name="experts down 16 tokens", op="down", N=16, E=8, k=2, h=4096, F=14336, act="none", grad=False),
        # A decode batch over many small experts: a handful of rows for each.
        dict(name="experts up 61 tokens fine", op="up", N=61, E=64, k=6, h=2048, F=1024, act="swiglu", grad=False),
        # A prompt: the largest product, bound by the tensor cores.
        dict(name="experts up prompt", op="up", N=4096, E=8, k=2, h=4096, F=14336, act="swiglu", grad=False),
        # Training step of many small experts: input and weight gradients of the down projection.
        dict(name="experts backward fine", op="bwd", N=4093, E=64, k=6, h=2048, F=1024, act="swiglu", grad=True),
        # The expert rows of a prompt come back to their tokens.
        dict(name="combine prompt", op="combine", N=4096, E=8, k=2, h=4096, grad=False),
        # The same in training, many experts for each token; padding tokens have none.
        dict(name="combine gradient", op="combine", N=8191, E=64, k=6, h=2048, grad=True),
        # One request with an adapter decodes one token: QKV-sized projection over 8 shards.
        dict(name="lora one token", op="lora", N=1, k=4096, n=6144, t=8, L=8, rank=16),
        # 64 requests, each with one of 32 adapters, decode together.
        dict(name="lora 64 requests", op="lora", N=64, k=4096, n=6144, t=8, L=32, rank=16),
        # Several prompts of uneven lengths, each with its adapter, in one batch.
        dict(name="lora prompts", op="lora", N=4000, k=4096, n=6144, t=8, L=8, rank=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    return max(lo, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["route", "up", "down", "bwd", "combine", "lora"])
    E = _log(rng, 2, 64)
    k = rng.randint(1, min(8, E))
    if op == "route":
        N = _log(rng, 1, 16384)
        E = _log(rng, 2, 256)
        return dict(op=op, N=N, E=E, k=rng.randint(1, min(8, E)), gate=rng.choice(["softmax", "topk"]),
                    dtype=rng.choice(["f32", "bf16"]), masked=rng.randint(0, N // 8), grad=rng.random() < 0.5)
    if op == "combine":
        return dict(op=op, N=_log(rng, 1, 8192), E=E, k=k, h=_eights(rng, 256, 4096), grad=rng.random() < 0.5)
    if op == "lora":
        t = rng.choice([1, 2, 4, 8])
        return dict(op=op, N=_log(rng, 1, 4096), k=_eights(rng, 256, 4096), n=t * _eights(rng, 256, 6144 // t), t=t,
                    L=_log(rng, 1, 32), rank=8 * rng.randint(1, 8))
    while True:
        N, h, F = _log(rng, 1, 4096), _eights(rng, 256, 4096), _eights(rng, 128, 14336)
        if E * h * F <= 8 * 4096 * 14336 and N * k * h * F <= 8192 * 4096 * 14336 / (3 if op == "bwd" else 1):
            act = "none" if op == "down" else rng.choice(["swiglu", "gelu", "gelu_tanh", "none"])
            return dict(op=op, N=N, E=E, k=k, h=h, F=F, act=act, grad=op == "bwd")


# ---------------------------------------------------------------------------------------------- inputs
def _normal(gen, shape, std=1.0, dtype=BF16):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    return x if std == 1.0 else x.mul_(std)


def _plan(gen, N, E, k, idle=0):
    """Expert choices of N tokens with uneven popularity, and the rows sorted by expert; the last `idle` tokens
    have no expert."""
    score = torch.randn((N, E), generator=gen, device="cuda") + 0.5 * torch.randn((1, E), generator=gen, device="cuda")
    expert = score.topk(k, dim=1).indices.to(torch.int32)
    if idle:
        expert[N - idle:] = -1
    flat = expert.reshape(-1).to(torch.int64)
    flat = torch.where(flat < 0, E, flat)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    rows = int(offsets[-1])
    slot = torch.empty_like(order)
    slot[order] = torch.arange(N * k, device="cuda")
    slot = torch.where(flat < E, slot, -1).reshape(N, k)
    token = (order // k).to(torch.int32)
    return dict(expert=expert, offsets=offsets.to(torch.int32), row_token=token, slot=slot.to(torch.int32), rows=rows,
                cap=max(1, int(counts.max())))


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"c": c}
    op, N = c["op"], c["N"]
    if op == "route":
        E, k = c["E"], c["k"]
        dt = F32 if c["dtype"] == "f32" else BF16
        logits = torch.randn((N, E), generator=gen, device="cuda") + 0.5 * torch.randn((1, E), generator=gen, device="cuda")
        if c["masked"]:
            logits[N - c["masked"]:] = -math.inf           # padding tokens
        s["logits"] = logits.to(dt)
        s["dweight"] = torch.randn((N, k), generator=gen, device="cuda")
        s["expert"] = torch.full((N, k), -7, dtype=torch.int32, device="cuda")
        s["weight"] = torch.zeros((N, k), device="cuda")
        s["slot"] = torch.full((N, k), -7, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["row_token"] = torch.full((N * k,), -7, dtype=torch.int32, device="cuda")
        s["dlogits"] = torch.zeros((N, E), dtype=dt, device="cuda")
        return s
    if op == "lora":
        k, n, t, L, r = c["k"], c["n"], c["t"], c["L"], c["rank"]
        s["x"] = _normal(gen, (N, k))
        s["w"] = _normal(gen, (t, k, n // t), 0.02)
        s["a"] = _normal(gen, (L, k, r), 1.0 / math.sqrt(k))
        s["b"] = _normal(gen, (t, L, r, n // t), 0.5)
        s["scale"] = 0.5 + torch.rand(L, generator=gen, device="cuda")
        # requests: every token of a decode batch is one; prompts are stretches of uneven length
        if N <= 256:
            ids = torch.randint(-1 if N > 1 else 0, L, (N,), generator=gen, device="cuda")
        else:
            cuts = torch.sort(torch.randint(0, N, (2 * L,), generator=gen, device="cuda")).values
            ids = torch.bucketize(torch.arange(N, device="cuda"), cuts) * 7 % (L + 1) - 1
        key = torch.where(ids < 0, L, ids)
        order = torch.sort(key, stable=True).indices
        offsets = torch.zeros(L + 1, dtype=torch.int64, device="cuda")
        offsets[1:] = torch.bincount(key, minlength=L + 1)[:L].cumsum(0)
        s["id"], s["offsets"], s["row_token"] = ids.to(torch.int32), offsets.to(torch.int32), order.to(torch.int32)
        s["y"] = torch.zeros((t, N, n // t), dtype=BF16, device="cuda")
        return s
    E, k, h = c["E"], c["k"], c["h"]
    p = _plan(gen, N, E, k, idle=N // 16 if op == "combine" else 0)
    s.update(p)
    R = N * k
    if op == "combine":
        s["u"] = _normal(gen, (R, h))
        w = torch.rand((N, k), generator=gen, device="cuda")
        s["weight"] = w / w.sum(1, keepdim=True)
        if c["grad"]:
            s["dy"] = _normal(gen, (N, h))
            s["du"] = torch.zeros((R, h), dtype=BF16, device="cuda")
            s["dweight"] = torch.zeros((N, k), device="cuda")
        else:
            s["y"] = torch.zeros((N, h), dtype=BF16, device="cuda")
        return s
    F, wide = c["F"], 2 if c["act"] == "swiglu" else 1
    if op == "up":
        s["x"] = _normal(gen, (N, h))
        s["w"] = _normal(gen, (E, h, wide * F), 0.02)
        s["y"] = torch.zeros((R, F), dtype=BF16, device="cuda")
    elif op == "down":
        s["x"] = _normal(gen, (R, F))
        s["w"] = _normal(gen, (E, F, h), 0.02)
        s["y"] = torch.zeros((R, h), dtype=BF16, device="cuda")
    else:
        s["h_pre"] = _normal(gen, (R, wide * F))
        s["z"] = _normal(gen, (R, F))
        s["du"] = _normal(gen, (R, h))
        s["w"] = _normal(gen, (E, F, h), 0.02)
        s["dh"] = torch.zeros((R, wide * F), dtype=BF16, device="cuda")
        s["dw"] = torch.zeros((E, F, h), device="cuda")
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _act(v, act):
    if act == "swiglu":
        g, u = v.chunk(2, dim=-1)
        return g / (1 + torch.exp(-g)) * u
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _act_back(dz, h, act):
    if act == "swiglu":
        g, u = h.chunk(2, dim=-1)
        s = 1 / (1 + torch.exp(-g))
        return torch.cat([dz * u * s * (1 + g * (1 - s)), dz * g * s], dim=-1)
    if act == "gelu":
        return dz * (0.5 * (1 + torch.erf(h * math.sqrt(0.5))) + h * torch.exp(-0.5 * h * h) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (h + 0.044715 * h * h * h))
        return dz * (0.5 * (1 + th) + 0.5 * h * (1 - th * th) * c * (1 + 3 * 0.044715 * h * h))
    return dz


def _plain_route(s):
    c = s["c"]
    N, E, k = c["N"], c["E"], c["k"]
    v = s["logits"].float()
    top, expert = torch.sort(v, dim=1, descending=True, stable=True)
    top, expert = top[:, :k], expert[:, :k]
    live = top > -math.inf
    m = torch.where(live[:, :1], top[:, :1], 0.0)
    p = torch.exp(v - m)
    chosen = torch.exp(top - m)
    total = (p if c["gate"] == "softmax" else chosen).sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    weight = chosen / total
    flat = torch.where(live, expert, E).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = (flat[:, None] == torch.arange(E, device="cuda")).sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(N * k, device="cuda")
    row = torch.arange(N * k, device="cuda")
    out = {"expert": torch.where(live, expert, -1).to(torch.int32), "weight": weight,
           "slot": torch.where(live, slot.reshape(N, k), -1).to(torch.int32), "offsets": offsets,
           "row_token": torch.where(row < offsets[E], order // k, s["row_token"]).to(torch.int32)}
    if c["grad"]:
        dw = torch.where(live, s["dweight"], 0.0)
        inner = (dw * weight).sum(1, keepdim=True)
        if c["gate"] == "softmax":
            d = torch.zeros_like(v).scatter_(1, expert, dw) - inner
            d = d * (p / total)
        else:
            d = torch.zeros_like(v).scatter_(1, expert, weight * (dw - inner))
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _padded(x, s, index=None):
    """Rows sorted by expert -> [E, cap, width] with zeros behind each expert's last, and where each row lies."""
    rows, E, cap = s["rows"], s["c"]["E"], s["cap"]
    i = torch.arange(rows, device="cuda")
    off = s["offsets"].long()
    e = torch.searchsorted(off[1:], i, right=True)
    j = i - off[e]
    out = torch.zeros((E, cap, x.shape[1]), device="cuda")
    out[e, j] = (x[:rows] if index is None else x[index[:rows].long()]).float()
    return out, e, j


def _plain_linear(s, x, index):
    xp, e, j = _padded(x, s, index)
    y = _act(torch.bmm(xp, s["w"].float())[e, j], s["c"]["act"])
    out = s["y"].clone()
    out[: s["rows"]] = y.to(BF16)
    return out


def _plain_backward(s):
    rows = s["rows"]
    dup, e, j = _padded(s["du"], s)
    zp = _padded(s["z"], s)[0]
    dz = torch.bmm(dup, s["w"].float().transpose(1, 2))[e, j]
    dh = s["dh"].clone()
    dh[:rows] = _act_back(dz, s["h_pre"][:rows].float(), s["c"]["act"]).to(BF16)
    return {"dh": dh, "dw": torch.bmm(zp.transpose(1, 2), dup)}


def _plain_combine(s):
    live = s["slot"] >= 0
    at = torch.where(live, s["slot"], 0).long()
    w = torch.where(live, s["weight"], 0.0)
    if not s["c"]["grad"]:
        return (s["u"][at].float() * w[..., None]).sum(1).to(BF16)
    dy = s["dy"].float()
    dweight = torch.where(live, (s["u"][at].float() * dy[:, None]).sum(2), 0.0)
    du = s["du"].clone()
    du[at[live]] = (w[..., None] * dy[:, None])[live].to(BF16)
    return {"du": du, "dweight": dweight}


def _plain_lora(s):
    c = s["c"]
    N, L, r = c["N"], c["L"], c["rank"]
    x = s["x"].float()
    v = x @ s["a"].float().permute(1, 0, 2).reshape(c["k"], L * r)
    mine = (s["id"][:, None] == torch.arange(L, device="cuda")).float() * s["scale"]
    v = (v.reshape(N, L, r) * mine[..., None]).reshape(N, L * r)
    return (x @ s["w"].float() + v @ s["b"].float().reshape(c["t"], L * r, -1)).to(BF16)


# ---------------------------------------------------------------------------------------------- the framework's
def _own(s):
    import tensor_sharded_matmul_b200 as tp
    c = s["c"]
    op, N = c["op"], c["N"]
    act = {"none": tp.TP_ACT_NONE, "gelu": tp.TP_ACT_GELU, "gelu_tanh": tp.TP_ACT_GELU_TANH,
           "swiglu": tp.TP_ACT_SWIGLU}[c.get("act", "none")]
    if op == "route":
        E, k = c["E"], c["k"]
        gate = tp.TP_GATE_SOFTMAX if c["gate"] == "softmax" else tp.TP_GATE_TOPK
        dt = tp.TP_F32 if c["dtype"] == "f32" else tp.TP_BF16
        if "ws" not in s:
            s["ws_bytes"] = tp.tp_moe_route_ws_bytes(N, E, k)
            s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
        tp.tp_moe_route(s["logits"], dt, N, E, k, gate, s["expert"], s["weight"], s["slot"], s["offsets"], s["row_token"],
                        s["ws"], s["ws_bytes"])
        out = {n: s[n] for n in ("expert", "weight", "slot", "offsets", "row_token")}
        if c["grad"]:
            tp.tp_moe_route_bwd(s["logits"], dt, N, E, k, gate, s["expert"], s["dweight"], s["dlogits"])
            out["dlogits"] = s["dlogits"]
        return out
    if op == "lora":
        if "ws" not in s:
            s["ws_bytes"] = tp.tp_lora_ws_bytes(N, c["rank"])
            s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
        tp.tp_lora_linear(s["x"], N, c["k"], c["n"], c["t"], s["w"], c["L"], c["rank"], s["a"], s["b"], s["scale"],
                          s["offsets"], s["row_token"], s["y"], s["ws"], s["ws_bytes"])
        return s["y"]
    E, R = c["E"], N * c["k"]
    if op == "up":
        tp.tp_ragged_linear(s["x"], N, s["row_token"], s["offsets"], R, E, c["h"], c["F"], act, s["w"], s["y"], tp.TP_BF16,
                            None)
        return s["y"]
    if op == "down":
        tp.tp_ragged_linear(s["x"], R, None, s["offsets"], R, E, c["F"], c["h"], act, s["w"], s["y"], tp.TP_BF16, None)
        return s["y"]
    if op == "bwd":
        tp.tp_ragged_linear_dx(s["du"], s["offsets"], R, E, c["F"], c["h"], s["w"], act,
                               None if act == tp.TP_ACT_NONE else s["h_pre"], s["dh"])
        tp.tp_ragged_linear_dw(s["z"], R, None, s["du"], s["offsets"], R, E, c["F"], c["h"], s["dw"], tp.TP_F32)
        return {"dh": s["dh"], "dw": s["dw"]}
    if not c["grad"]:
        tp.tp_moe_combine(s["u"], tp.TP_BF16, R, s["weight"], s["slot"], N, c["h"], c["k"], s["y"], tp.TP_BF16)
        return s["y"]
    tp.tp_moe_combine_bwd(s["dy"], tp.TP_BF16, s["u"], tp.TP_BF16, R, s["weight"], s["slot"], N, c["h"], c["k"], s["du"],
                          s["dweight"])
    return {"du": s["du"], "dweight": s["dweight"]}


def run(s):
    if own:
        return _own(s)
    c = s["c"]
    op = c["op"]
    if op == "route":
        return _plain_route(s)
    if op == "lora":
        return _plain_lora(s)
    if op == "combine":
        return _plain_combine(s)
    if op == "bwd":
        return _plain_backward(s)
    return _plain_linear(s, s["x"], s["row_token"] if op == "up" else None)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    c = dict(case)
    op, N = c["op"], c["N"]
    if op == "route":
        size = 4 if c["dtype"] == "f32" else 2
        E, k = c["E"], c["k"]
        b = N * E * size + N * k * 16 + (E + 1) * 4
        if c["grad"]:
            b += N * k * 4 + N * E * size
        return {"bytes": b, "flops": N * E * (6 if c["grad"] else 3)}
    if op == "combine":
        live = (N - N // 16) * c["k"]
        b = live * c["h"] * 2 * (2 if c["grad"] else 1) + N * c["h"] * 2 + N * c["k"] * (12 if c["grad"] else 8)
        return {"bytes": b, "flops": live * c["h"] * (3 if c["grad"] else 2)}
    if op == "lora":
        k, n, L, r = c["k"], c["n"], c["L"], c["rank"]
        used = L * (1 - (1 - 1 / L) ** N) if L > 1 else 1
        return {"bytes": 2 * (N * k + k * n + N * n + used * r * (k + n)) + 8 * N,
                "flops": 2.0 * N * (k * n + r * (k + n))}
    E, k, h, F = c["E"], c["k"], c["h"], c["F"]
    R, wide = N * k, 2 if c["act"] == "swiglu" else 1
    active = E * (1 - (1 - k / E) ** N)
    if op == "up":
        return {"bytes": 2 * (N * h + active * h * wide * F + R * F) + 4 * R, "flops": 2.0 * R * h * wide * F}
    if op == "down":
        return {"bytes": 2 * (R * F + active * h * F + R * h), "flops": 2.0 * R * h * F}
    hp = 0 if c["act"] == "none" else wide
    return {"bytes": 2 * (R * h + active * h * F + R * F * hp + R * F * wide + R * F) + 4 * E * F * h,
            "flops": 4.0 * R * h * F}


# ---------------------------------------------------------------------------------------------- 64 bits
def _act64(v, act):
    """The activations from their definitions by other functions than the plain form's (and differentiable)."""
    if act == "swiglu":
        n = v.shape[-1] // 2
        return v[..., :n] * torch.sigmoid(v[..., :n]) * v[..., n:]
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    op, N = c["op"], c["N"]
    D = torch.float64
    if op == "route":
        k = c["k"]
        v = s["logits"].to(D)
        open_ = v > -math.inf
        rank = ((v[:, :, None] < v[:, None, :]) if c["E"] * c["E"] * N <= 1 << 28 else None)
        if rank is not None:       # an expert's place: how many come before it, by value and then by index
            i = torch.arange(c["E"], device="cuda")
            place = rank.sum(2) + ((v[:, :, None] == v[:, None, :]) & (i[None, None, :] < i[None, :, None])).sum(2)
        else:
            place = torch.argsort(torch.argsort(-v, dim=1, stable=True), dim=1)
        order = torch.argsort(place, dim=1)[:, :k]
        taken = (place < k) & open_
        e = torch.where(open_, torch.exp(v - v.clamp(min=-1e300).amax(1, keepdim=True)), 0.0)
        base = e if c["gate"] == "softmax" else torch.where(taken, e, 0.0)
        q = base / base.sum(1, keepdim=True).clamp(min=1e-300)
        out = {"expert": None, "weight": q.gather(1, order), "slot": None, "offsets": None, "row_token": None}
        if c["grad"]:
            dw = torch.zeros_like(v).scatter_(1, order, s["dweight"].to(D)) * taken
            out["dlogits"] = q * (dw - (q * dw).sum(1, keepdim=True))
        return out
    if op == "lora":
        x, off, tok = s["x"].to(D), s["offsets"].tolist(), s["row_token"].long()
        y = torch.stack([x @ s["w"][r].to(D) for r in range(c["t"])])
        for l in range(c["L"]):
            at = tok[off[l]:off[l + 1]]
            if len(at):
                v = float(s["scale"][l]) * (x[at] @ s["a"][l].to(D))
                for r in range(c["t"]):
                    y[r, at] += v @ s["b"][r, l].to(D)
        return y
    if op == "combine":
        slot, w = s["slot"].long(), s["weight"].to(D)
        if not c["grad"]:
            y = torch.zeros((N, c["h"]), dtype=D, device="cuda")
            for j in range(c["k"]):
                m = slot[:, j] >= 0
                y[m] += w[m, j, None] * s["u"][slot[m, j]].to(D)
            return y
        dy = s["dy"].to(D)
        du = s["du"].to(D)
        dwt = torch.zeros((N, c["k"]), dtype=D, device="cuda")
        for j in range(c["k"]):
            m = slot[:, j] >= 0
            du[slot[m, j]] = w[m, j, None] * dy[m]
            dwt[m, j] = (dy[m] * s["u"][slot[m, j]].to(D)).sum(1)
        return {"du": du, "dweight": dwt}
    off = s["offsets"].tolist()
    if op == "bwd":
        dh, dw = s["dh"].to(D), torch.zeros(s["dw"].shape, dtype=D, device="cuda")
        for e in range(c["E"]):
            a, b = off[e], off[e + 1]
            du = s["du"][a:b].to(D)
            h = s["h_pre"][a:b].to(D).requires_grad_(True)
            dh[a:b] = torch.autograd.grad(_act64(h, c["act"]), h, du @ s["w"][e].to(D).t())[0] if b > a else h
            dw[e] = s["z"][a:b].to(D).t() @ du
        return {"dh": dh, "dw": dw}
    y = s["y"].to(D)
    for e in range(c["E"]):
        a, b = off[e], off[e + 1]
        x = s["x"][s["row_token"][a:b].long()] if op == "up" else s["x"][a:b]
        y[a:b] = _act64(x.to(D) @ s["w"][e].to(D), c["act"])
    return y
