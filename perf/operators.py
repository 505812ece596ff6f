"""The operators of a mixture-of-experts layer as measured cases: routing, grouping by expert, the experts' FP8
products, the gated activation with its quantization, and the weighted sum back to tokens.

Sizes: T tokens, k experts per token, E experts, P = T k assignments; an expert's first product is [rows, K] x [N, K]
with N = 2 F (gate and up), its second [rows, F] x [hidden, F].
"""
import torch

own = False

F8 = torch.float8_e4m3fn


def listed():
    return [
        # A decode step of eight sequences: the router is pure latency.
        dict(name="route_decode", op="route", T=8, E=128, k=8, score="softmax", dtype="bf16", bias=False, groups=1,
             top_groups=1, group_score="max", renorm=True, scale=1.0),
        # A prefill chunk with a balance bias and group-limited choice.
        dict(name="route_prefill", op="route", T=8192, E=256, k=8, score="sigmoid", dtype="f32", bias=True, groups=8,
             top_groups=4, group_score="top2", renorm=True, scale=2.5),
        # Grouping one decode batch's assignments.
        dict(name="plan_decode", op="plan", T=24, k=6, E=160, dropped=0.0),
        # Grouping a prefill chunk on a rank that holds three quarters of the experts.
        dict(name="plan_prefill", op="plan", T=8192, k=8, E=256, dropped=0.25),
        # One token: eight experts' weights stream past a single row each.
        dict(name="experts_one_token", op="experts", scheme="fp8_block128", T=1, k=8, E=128, N=2048, K=4096,
             gather=True),
        # A decode batch: nearly every expert is hit by a few rows, per-channel scales.
        dict(name="experts_batch", op="experts", scheme="fp8_row", T=37, k=6, E=64, N=2816, K=2048, gather=True),
        # A short prompt's second product: rows already in expert order, ragged groups.
        dict(name="experts_chunk", op="experts", scheme="fp8_block128", T=1000, k=8, E=60, N=5120, K=1536,
             gather=False),
        # A prefill chunk's first product, bound by the matrix cores.
        dict(name="experts_prefill", op="experts", scheme="fp8_block128", T=8192, k=8, E=64, N=4096, K=2048,
             gather=True),
        # Between the two products of the decode batch.
        dict(name="swiglu_batch", op="swiglu", scheme="fp8_row", M=222, F=1408),
        # Between the two products of the prefill chunk.
        dict(name="swiglu_prefill", op="swiglu", scheme="fp8_block128", M=65536, F=2048),
        # Back to tokens after a decode step, onto the shared expert's output.
        dict(name="combine_decode", op="combine", T=3, k=8, N=4096, add=True, dropped=0.0),
        # Back to tokens after the prefill chunk, some assignments on other ranks.
        dict(name="combine_prefill", op="combine", T=8192, k=8, N=4096, add=False, dropped=0.25),
    ]


def _between(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(lo * (hi / lo) ** rng.random() + rng.random())))


def draw(rng):
    op = rng.choice(["route", "plan", "experts", "experts", "experts", "swiglu", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _between(rng, 4, 256 // groups)
        top = rng.randint(1, groups)
        return dict(op=op, T=_between(rng, 1, 8192), E=E, k=rng.randint(1, min(16, E // groups * top)),
                    score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["bf16", "f16", "f32"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top, group_score=rng.choice(["max", "top2"]),
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    if op == "plan":
        k = rng.randint(1, 8)
        return dict(op=op, T=_between(rng, 1, 8192), k=k, E=_between(rng, k, 512), dropped=rng.choice([0.0, 0.5]))
    if op == "experts":
        while True:
            k = rng.randint(1, 8)
            T, E = _between(rng, 1, 8192), _between(rng, max(4, k), 160)
            N, K = 128 * _between(rng, 2, 40), 128 * _between(rng, 4, 40)
            if T * k * N * K <= 65536 * 4096 * 2048 and E * N * K <= 64 * 4096 * 2048:
                return dict(op=op, scheme=rng.choice(["fp8_block128", "fp8_row"]), T=T, k=k, E=E, N=N, K=K,
                            gather=rng.random() < 0.6)
    if op == "swiglu":
        M = _between(rng, 1, 65536)
        return dict(op=op, scheme=rng.choice(["fp8_block128", "fp8_row"]), M=M,
                    F=128 * _between(rng, 1, min(64, 65536 * 16 // M)))
    k = rng.randint(1, 8)
    T = _between(rng, 1, 8192)
    N = _between(rng, 64, min(8192, 8192 * 8 * 4096 // (T * k)))
    return dict(op=op, T=T, k=k, N=N if rng.random() < 0.25 else N - N % 8, add=rng.random() < 0.5,
                dropped=rng.choice([0.0, 0.5]))


# ------------------------------------------------------------------------------------------------ inputs
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _popular_logits(gen, T, E, dev):
    """Router logits with some experts more popular than others."""
    return torch.randn(T, E, generator=gen, device=dev) + 0.5 * torch.randn(E, generator=gen, device=dev)


def _chosen(gen, T, k, E, dropped, dev):
    """ids i32 [T, k] of distinct experts per token; a `dropped` share of the experts lives elsewhere (id -1)."""
    x = _popular_logits(gen, T, E, dev)
    ids = x.topk(k, dim=1).indices.int()
    return torch.where(ids < E - int(E * dropped), ids, -1)


def _grouped(ids, E):
    """(offsets, order, slots) of the assignments grouped by expert."""
    flat = ids.reshape(-1).long()
    P = flat.numel()
    key = torch.where(flat >= 0, flat, E)
    sorted_key, order = torch.sort(key, stable=True)
    kept = sorted_key < E
    places = torch.arange(P, device=ids.device)
    slots = torch.empty(P, dtype=torch.int64, device=ids.device)
    slots[order] = torch.where(kept, places, -1)
    edges = torch.arange(E + 1, device=ids.device)
    offsets = torch.searchsorted(sorted_key, edges)
    return offsets.int(), torch.where(kept, order, -1).int(), slots.int()


def _f8_scale(amax):
    s = amax / 448.0
    return torch.where(s > 0, s, torch.ones_like(s))


def _quantized_rows(x, scheme):
    """Activation codes (e4m3) and scales of fp32 rows."""
    if scheme == "fp8_row":
        s = _f8_scale(x.abs().amax(1))
        return (x / s[:, None]).to(F8), s
    g = x.view(x.shape[0], -1, 128)
    s = _f8_scale(g.abs().amax(2))
    return (g / s[:, :, None]).view_as(x).to(F8), s


def _quantized_weight(w, scheme):
    """Weight codes (e4m3) [R, K] and scales of stacked fp32 rows."""
    if scheme == "fp8_row":
        return _quantized_rows(w, scheme)
    R, K = w.shape
    b = w.view(R // 128, 128, K // 128, 128)
    s = _f8_scale(b.abs().amax((1, 3)))
    return (b / s[:, None, :, None]).view(R, K).to(F8), s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    c, st = case, {"case": case}
    if c["op"] == "route":
        st["logits"] = _popular_logits(gen, c["T"], c["E"], dev).to(_DTYPES[c["dtype"]])
        st["bias"] = 0.05 * torch.randn(c["E"], generator=gen, device=dev) if c["bias"] else None
    elif c["op"] == "plan":
        st["ids"] = _chosen(gen, c["T"], c["k"], c["E"], c["dropped"], dev)
    elif c["op"] == "experts":
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        ids = _chosen(gen, T, k, E, 0.0, dev)
        st["offsets"], st["order"], st["slots"] = _grouped(ids, E)
        st["most"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())   # rows of the fullest expert
        rows = T if c["gather"] else T * k
        x = torch.randn(rows, K, generator=gen, device=dev).bfloat16().float()
        x[:, torch.randperm(K, generator=gen, device=dev)[: K // 100]] *= 20.0   # outlier channels
        st["a"], st["a_scales"] = _quantized_rows(x, c["scheme"])
        w = (0.02 * torch.randn(E * N, K, generator=gen, device=dev)).bfloat16().float()
        st["w"], st["w_scales"] = _quantized_weight(w, c["scheme"])
    elif c["op"] == "swiglu":
        st["x"] = (1.5 * torch.randn(c["M"], 2 * c["F"], generator=gen, device=dev)).bfloat16()
    else:
        T, k, N = c["T"], c["k"], c["N"]
        ids = _chosen(gen, T, k, 64, c["dropped"], dev)
        st["offsets"], st["order"], st["slots"] = _grouped(ids, 64)
        st["y"] = torch.randn(T * k, N, generator=gen, device=dev).bfloat16()
        st["weights"] = torch.softmax(torch.randn(T, k, generator=gen, device=dev), 1)
        st["add"] = torch.randn(T, N, generator=gen, device=dev).bfloat16() if c["add"] else None
    return st


# ------------------------------------------------------------------------------------------------ plain forms
def _route(st):
    """Scores and choices in 64 bits: the order of near ties is part of the answer."""
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    x = st["logits"].double()
    broken = ((x != x) | (x == float("inf"))).any(1, keepdim=True)
    x = torch.where(broken, float("-inf"), x)
    if c["score"] == "softmax":
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(top > float("-inf"), top, 0.0))
        s = e / e.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    free = x > float("-inf")
    choice = s if st["bias"] is None else s + st["bias"].double()
    key = x if st["bias"] is None else choice
    free = free & (key > float("-inf"))
    key = torch.where(free, key, float("-inf"))
    if G > 1:
        if c["group_score"] == "top2":
            best = torch.where(free, choice, float("-inf")).view(T, G, E // G).sort(2, descending=True).values[:, :, :2]
            rest = torch.where(best[:, :, 1:] > float("-inf"), best[:, :, 1:], 0.0).sum(2)
            score = best[:, :, 0] + rest
        else:
            score = key.view(T, G, E // G).amax(2)
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        key = torch.where(mask[:, :, None], key.view(T, G, E // G), float("-inf")).view(T, E)
    best = torch.sort(key, dim=1, descending=True, stable=True)
    found = best.values[:, :k] > float("-inf")
    ids = best.indices[:, :k]
    w = torch.where(found, s.gather(1, ids), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    w = torch.where(broken, float("nan"), w * c["scale"])
    return torch.where(found, ids, -1).int(), w.float()


def _dequantized(codes, scales, scheme, weight):
    x = codes.float()
    if scheme == "fp8_row":
        return x * scales[:, None]
    if weight:
        R, K = x.shape
        return (x.view(R // 128, 128, K // 128, 128) * scales[:, None, :, None]).view(R, K)
    return (x.view(x.shape[0], -1, 128) * scales[:, :, None]).view_as(x)


def _experts(st):
    """Every expert's rows padded to the fullest one's, and one batched product in 32 bits."""
    c = st["case"]
    E, N, K = c["E"], c["N"], c["K"]
    a = _dequantized(st["a"], st["a_scales"], c["scheme"], False)
    w = _dequantized(st["w"], st["w_scales"], c["scheme"], True).view(E, N, K)
    off = st["offsets"].long()
    place = torch.arange(c["T"] * c["k"], device=a.device)
    rows = st["order"].long() // c["k"] if c["gather"] else place
    expert = torch.searchsorted(off[1:], place, right=True)
    at = (off[:-1, None] + torch.arange(st["most"], device=a.device)).clamp(max=place.numel() - 1)
    y = torch.bmm(a[rows[at]], w.transpose(1, 2))
    return y[expert, place - off[expert]].bfloat16()


def _swiglu(st):
    c, x = st["case"], st["x"].float()
    g, u = x[:, : c["F"]], x[:, c["F"]:]
    codes, scales = _quantized_rows(g / (1.0 + torch.exp(-g)) * u, c["scheme"])
    return codes, scales


def _combine(st):
    c = st["case"]
    slots = st["slots"].long()
    y = torch.where((slots >= 0)[:, None], st["y"][slots.clamp(min=0)].float(), 0.0)
    out = (y.view(c["T"], c["k"], c["N"]) * st["weights"][:, :, None]).sum(1)
    return (out if st["add"] is None else out + st["add"].float()).bfloat16()


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return _own(state)
    return {"route": _route, "plan": lambda s: _grouped(s["ids"], c["E"]), "experts": _experts, "swiglu": _swiglu,
            "combine": _combine}[c["op"]](state)


def _own(st):
    import precision_quantized_linear_amd as pql

    c = st["case"]
    if c["op"] == "route":
        return pql.moe_route(st["logits"], c["k"], score=c["score"], bias=st["bias"], n_groups=c["groups"],
                             top_groups=c["top_groups"], group_score=c["group_score"], renormalize=c["renorm"],
                             scale=c["scale"])
    if c["op"] == "plan":
        plan = pql.moe_plan(st["ids"], c["E"])
        return plan.offsets, plan.order, plan.slots
    if c["op"] == "swiglu":
        q = pql.swiglu_quantize(st["x"], c["scheme"])
        return q.codes.view(F8), q.scales
    E = 64 if c["op"] == "combine" else c["E"]
    plan = pql.MoePlan(c["T"], c["k"], E, st["offsets"], st["order"], st["slots"])
    if c["op"] == "experts":
        a, w = st["a"], st["w"]
        aq = pql.QTensor(c["scheme"], "activation", a.shape[0], c["K"], a.view(torch.uint8), st["a_scales"])
        wq = pql.QTensor(c["scheme"], "weight", w.shape[0], c["K"], w.view(torch.uint8), st["w_scales"])
        return pql.moe_qgemm(aq, wq, plan, gather=c["gather"])
    return pql.moe_combine(st["y"], plan, st["weights"], add=st["add"])


# ------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["T"] * (c["E"] * size + 8 * c["k"]) + (4 * c["E"] if c["bias"] else 0),
                "flops": 8 * c["T"] * c["E"]}
    if c["op"] == "plan":
        return {"bytes": 12 * c["T"] * c["k"] + 4 * (c["E"] + 1), "flops": 0}
    if c["op"] == "experts":
        P, E, N, K = c["T"] * c["k"], c["E"], c["N"], c["K"]
        hit = E * (1.0 - (1.0 - c["k"] / E) ** c["T"])   # experts with at least one row, evenly routed
        rows = c["T"] if c["gather"] else P
        per_row, per_weight = (4, 4 * N) if c["scheme"] == "fp8_row" else (K // 32, N * K // 4096)
        return {"bytes": hit * (N * K + per_weight) + rows * (K + per_row) + 2 * P * N + 4 * (P + E),
                "flops": 2 * P * N * K}
    if c["op"] == "swiglu":
        M, F = c["M"], c["F"]
        return {"bytes": 5 * M * F + 4 * M * (F // 128 if c["scheme"] == "fp8_block128" else 1), "flops": 8 * M * F}
    T, k, N = c["T"], c["k"], c["N"]
    kept = T * k * (1.0 - c["dropped"])
    return {"bytes": 2 * kept * N + (4 if c["add"] else 2) * T * N + 8 * T * k, "flops": 2 * kept * N}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """From the definitions, in 64 bits; codes come as the numbers before their rounding to e4m3."""
    st, c = prepare(case, seed), case
    if c["op"] == "route":
        return _exact_route(st)
    if c["op"] == "plan":
        flat = st["ids"].reshape(-1).cpu()
        P = flat.numel()
        order, slots, offsets = torch.full((P,), -1), torch.full((P,), -1), [0]
        for e in range(c["E"]):
            mine = (flat == e).nonzero().reshape(-1)
            order[offsets[-1]: offsets[-1] + len(mine)] = mine
            slots[mine] = torch.arange(offsets[-1], offsets[-1] + len(mine))
            offsets.append(offsets[-1] + len(mine))
        return torch.tensor(offsets).int(), order.int(), slots.int()
    if c["op"] == "experts":
        off, order = st["offsets"].tolist(), st["order"].long()
        out = torch.empty(c["T"] * c["k"], c["N"], dtype=torch.float64, device=order.device)
        wide = 1 if c["scheme"] == "fp8_row" else 128
        blocks = (lambda s, n: s.double().repeat_interleave(n, 1)[:, : c["K"]]) if wide > 1 else None
        for e in range(c["E"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            at = order[lo:hi].div(c["k"], rounding_mode="floor") if c["gather"] else slice(lo, hi)
            mine = slice(e * c["N"], (e + 1) * c["N"])
            a, w = st["a"][at].double(), st["w"][mine].double()
            if wide > 1:
                a = a * blocks(st["a_scales"][at], 128)
                sw = st["w_scales"][e * (c["N"] // 128): (e + 1) * (c["N"] // 128)]
                w = w * blocks(sw, 128).repeat_interleave(128, 0)
            else:
                a, w = a * st["a_scales"][at].double()[:, None], w * st["w_scales"][mine].double()[:, None]
            out[lo:hi] = torch.mm(a, w.t())
        return out
    if c["op"] == "swiglu":
        x = st["x"].double()
        h = x[:, : c["F"]] * torch.sigmoid(x[:, : c["F"]]) * x[:, c["F"]:]
        group = c["F"] if c["scheme"] == "fp8_row" else 128
        s = h.abs().unflatten(1, (-1, group)).amax(2) / 448.0
        s[s == 0] = 1.0
        codes = h / s.repeat_interleave(group, 1)
        return codes, s.reshape(-1) if c["scheme"] == "fp8_row" else s
    out = torch.zeros(c["T"], c["N"], dtype=torch.float64, device=st["y"].device)
    if st["add"] is not None:
        out += st["add"]
    slots = st["slots"].view(c["T"], c["k"]).long()
    for j in range(c["k"]):
        t = (slots[:, j] >= 0).nonzero().reshape(-1)
        out[t] += st["weights"][t, j].double()[:, None] * st["y"][slots[t, j]].double()
    return out


def _exact_route(st):
    import numpy as np

    c = st["case"]
    x = st["logits"].double().cpu().numpy()
    b = None if st["bias"] is None else st["bias"].double().cpu().numpy()
    ids, weights = np.zeros((c["T"], c["k"]), np.int32), np.zeros((c["T"], c["k"]), np.float64)
    per = c["E"] // c["groups"]
    for t in range(c["T"]):
        if c["score"] == "softmax":
            e = np.exp(x[t] - x[t].max())
            s = e / e.sum()
        else:
            s = 1.0 / (1.0 + np.exp(-x[t]))
        choice, key = (s, x[t]) if b is None else (s + b, s + b)
        allowed = np.arange(c["E"])
        if c["groups"] > 1:
            if c["group_score"] == "top2":
                score = np.sort(choice.reshape(-1, per), axis=1)[:, -2:].sum(1)
            else:
                score = key.reshape(-1, per).max(1)
            kept = np.sort(np.argsort(-score, kind="stable")[: c["top_groups"]])
            allowed = (kept[:, None] * per + np.arange(per)).reshape(-1)
        pick = allowed[np.argsort(-key[allowed], kind="stable")[: c["k"]]]
        w = s[pick]
        ids[t], weights[t] = pick, c["scale"] * (w / w.sum() if c["renorm"] else w)
    return ids, weights
