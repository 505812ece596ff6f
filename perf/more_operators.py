"""The operators of a paged, quantized cache of keys and values as measured cases: slots and positions of a batch's new
tokens, rotary positions, quantizing keys and values into the cache, reading them back, and the attention over it.

Sizes: B sequences, T new tokens in all, L tokens of a sequence in the cache (its new ones included), H query heads, Hk
key / value heads, D the head's size, ps tokens to a page.  A cache is [pages, Hk, ps, D]: bf16, or e4m3 codes with one
scale for all (fp8_tensor) or one per token and head (fp8_row, [pages, Hk, ps]).
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn


def listed():
    return [
        # A decode step of 24 sequences: where its new tokens go, pure latency.
        dict(name="slots_decode", op="slots", B=24, new=1, ctx=9000, ps=16),
        # Prompts of 150 requests at once, some a single token.
        dict(name="slots_prompts", op="slots", B=150, new=200, ctx=9000, ps=64),
        # Query heads of a decode step of seven sequences, far into their contexts.
        dict(name="rope_decode", op="rope", T=7, H=32, D=128, dim=128, layout="half", far=130000, scale=1.0),
        # Query and key heads of a prompt in one pass, half of each head turned, stretched positions.
        dict(name="rope_prompt", op="rope", T=8192, H=40, D=128, dim=64, layout="interleaved", far=900000, scale=1.2),
        # Keys (turned on the way) and values of a decode step.
        dict(name="append_decode", op="append", scheme="fp8_row", T=24, Hk=8, D=128, ps=16, dim=128, layout="half",
             dropped=0.0),
        # A prompt's keys and values, an eighth of the rows padding.
        dict(name="append_prompt", op="append", scheme="fp8_row", T=16384, Hk=8, D=128, ps=64, dim=0, layout="half",
             dropped=0.125),
        # A short prefix back in bf16, one scale for all.
        dict(name="read_prefix", op="read", scheme="fp8_tensor", n=333, Hk=8, D=128, ps=16),
        # A long context back in bf16.
        dict(name="read_context", op="read", scheme="fp8_row", n=60001, Hk=8, D=128, ps=64),
        # One sequence's next token: few rows, the context split over the card.
        dict(name="attend_one", op="attend", scheme="fp8_tensor", B=1, new=1, ctx=6007, H=32, Hk=8, D=128, ps=16,
             causal=True, window=0, lse=False),
        # A decode step of 64 sequences of very different lengths: the cache streams past.
        dict(name="attend_decode", op="attend", scheme="fp8_row", B=64, new=1, ctx=16384, H=32, Hk=4, D=128, ps=64,
             causal=True, window=0, lse=False),
        # Chunks of five prompts over an unquantized cache, each token sees the last 4096.
        dict(name="attend_chunks", op="attend", scheme="bf16", B=5, new=300, ctx=12000, H=16, Hk=2, D=128, ps=32,
             causal=True, window=4096, lse=True),
        # A long prompt's last chunk, bound by the matrix cores.
        dict(name="attend_prompt", op="attend", scheme="fp8_row", B=1, new=8192, ctx=32768, H=32, Hk=8, D=128, ps=64,
             causal=True, window=0, lse=False),
    ]


def _between(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(lo * (hi / lo) ** rng.random() + rng.random())))


def draw(rng):
    op = rng.choice(["slots", "rope", "append", "read", "attend", "attend", "attend", "attend"])
    ps = rng.choice([16, 32, 64, 128])
    if op == "slots":
        return dict(op=op, B=_between(rng, 1, 200), new=_between(rng, 1, 200), ctx=_between(rng, 200, 20000), ps=ps)
    D = rng.choice([64, 128, 128, 192, 256])
    dim = rng.choice([D, D, D // 2, 16 * rng.randint(1, D // 16)])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        H = _between(rng, 1, 64)
        return dict(op=op, T=_between(rng, 1, 8192 * 40 * 128 // (H * D)), H=H, D=D, dim=dim, layout=layout,
                    far=_between(rng, 10, 1000000), scale=rng.choice([1.0, 1.1]))
    scheme = rng.choice(["bf16", "fp8_tensor", "fp8_row", "fp8_row"])
    Hk = _between(rng, 1, 16)
    if op == "append":
        return dict(op=op, scheme=scheme, T=_between(rng, 1, 16384 * 8 * 128 // (Hk * D)), Hk=Hk, D=D, ps=ps,
                    dim=rng.choice([0, dim]), layout=layout, dropped=rng.choice([0.0, 0.3]))
    if op == "read":
        return dict(op=op, scheme=scheme, n=_between(rng, 1, 60001 * 8 * 128 // (Hk * D)), Hk=Hk, D=D, ps=ps)
    while True:
        G = rng.choice([1, 2, 4, 5, 7, 8, 16])
        B = _between(rng, 1, 64)
        new = rng.choice([1, 1, _between(rng, 2, 8), _between(rng, 9, 2048)])
        ctx = _between(rng, max(16, new), 32768)
        if Hk * G <= 64 and B * new * Hk * G * D * ctx <= 2 ** 39 and B * ctx * Hk * D <= 2 ** 29 \
                and B * new * Hk * G <= 2 ** 18:
            return dict(op=op, scheme=scheme, B=B, new=new, ctx=ctx, H=Hk * G, Hk=Hk, D=D, ps=ps,
                        causal=rng.random() < 0.85, window=rng.choice([0, 0, 0, _between(rng, 1, ctx)]),
                        lse=rng.random() < 0.3)


# ------------------------------------------------------------------------------------------------ inputs
def _batch(c):
    """(new tokens, tokens in the cache) of every sequence, lists: the first has `new` and `ctx` in full, the others
    spread from nearly none to all of them.  One new token each where new = 1."""
    new, ctx = [], []
    for b in range(c["B"]):
        share = 1.0 - (b * 0.6180339887) % 1.0
        n = max(1, int(c["new"] * (1.0 - (b * 0.7548776662) % 1.0)))
        new.append(n)
        ctx.append(max(n, int(c["ctx"] * share)))
    return new, ctx


def _freqs(dim, far, dev):
    """Radians per position of each pair (64 bits), the slow ones stretched where positions go far."""
    i = torch.arange(dim // 2, dtype=torch.float64, device=dev)
    f = 10000.0 ** (-2.0 * i / dim)
    return torch.where(f * far < 2 * math.pi * 4, f / 8.0, f)


def _dtype(c):
    return torch.bfloat16 if c["scheme"] == "bf16" else F8


def _scale_of(amax):
    s = amax / 448.0
    return torch.where(s > 0, s, torch.ones_like(s))


def _filled(gen, c, pages, dev):
    """A cache with values in every slot, also behind the sequences' ends."""
    shape = (pages, c["Hk"], c["ps"], c["D"])
    out = {}
    for x, sharp in (("k", 1.5), ("v", 1.0)):
        t = torch.randn(shape, generator=gen, device=dev)
        t *= sharp * (0.5 + torch.rand(shape[:3], generator=gen, device=dev))[..., None]
        if c["scheme"] == "bf16":
            out[x], out[x + "s"] = t.bfloat16(), None
        else:
            s = _scale_of(t.abs().amax() if c["scheme"] == "fp8_tensor" else t.abs().amax(-1))
            t /= s if s.dim() == 0 else s[..., None]
            out[x], out[x + "s"] = t.clamp_(-448, 448).to(F8), s.reshape(1) if s.dim() == 0 else s
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    c, st = case, {"case": case}

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def some(n, of):
        return torch.randperm(of, generator=gen, device=dev)[:n].int()

    if c["op"] in ("slots", "attend"):
        new, ctx = _batch(c)
        st["new"], st["ctx"] = new, ctx
        st["starts"] = i32([0] + torch.tensor(new).cumsum(0).tolist())
        st["lens"] = i32(ctx)
        need = [-(-n // c["ps"]) for n in ctx]
        wide = max(need) + 1
        st["n_pages"] = sum(need) + 3
        ids = some(sum(need), st["n_pages"]).split(need)
        st["pages"] = torch.stack([torch.nn.functional.pad(p, (0, wide - p.numel()), value=-1) for p in ids])
        if c["op"] == "attend":
            st.update(_filled(gen, c, st["n_pages"], dev))
            st["q"] = rand(sum(new), c["H"], c["D"]).bfloat16()
    elif c["op"] == "rope":
        st["x"] = rand(c["T"], c["H"], c["D"]).bfloat16()
        st["positions"] = (torch.rand(c["T"], generator=gen, device=dev) * c["far"]).int()
        st["freqs"] = _freqs(c["dim"], c["far"], dev)
    elif c["op"] == "append":
        T = c["T"]
        st["keys"], st["values"] = rand(T, c["Hk"], c["D"]).bfloat16(), rand(T, c["Hk"], c["D"]).bfloat16()
        st["n_pages"] = -(-T // c["ps"]) + 5
        cache = _filled(gen, c, st["n_pages"], dev)
        if c["scheme"] == "fp8_tensor":
            cache["ks"], cache["vs"] = torch.tensor([0.0117], device=dev), torch.tensor([0.0113], device=dev)
        st.update(cache)
        padding = torch.rand(T, generator=gen, device=dev) < c["dropped"]
        st["slots"] = torch.where(padding, -1, some(T, st["n_pages"] * c["ps"])).int()
        st["live"] = (~padding).nonzero().reshape(-1)
        if c["dim"]:
            st["positions"] = (torch.rand(T, generator=gen, device=dev) * 100000).int()
            st["freqs"] = _freqs(c["dim"], 100000, dev)
    else:
        st["n_pages"] = -(-c["n"] // c["ps"]) + 5
        st.update(_filled(gen, c, st["n_pages"], dev))
        st["slots"] = some(c["n"], st["n_pages"] * c["ps"])
    return st


# ------------------------------------------------------------------------------------------------ plain forms
def _slots(st):
    c = st["case"]
    starts, lens = st["starts"].long(), st["lens"].long()
    t = torch.arange(sum(st["new"]), device=starts.device)
    b = torch.searchsorted(starts, t, right=True) - 1
    pos = lens[b] - (starts[b + 1] - t)
    slot = st["pages"][b, pos // c["ps"]].long() * c["ps"] + pos % c["ps"]
    return slot.int(), pos.int()


def _turned(x, positions, freqs, layout, scale):
    """The first 2 len(freqs) values of every head turned, fp32; angles in 64 bits."""
    a = positions.double()[:, None] * freqs
    cos, sin = (torch.cos(a) * scale).float()[:, None], (torch.sin(a) * scale).float()[:, None]
    d, x = 2 * freqs.numel(), x.float()
    y = x.clone()
    one, two = (slice(0, d // 2), slice(d // 2, d)) if layout == "half" else (slice(0, d, 2), slice(1, d, 2))
    y[..., one] = x[..., one] * cos - x[..., two] * sin
    y[..., two] = x[..., two] * cos + x[..., one] * sin
    return y


def _rope(st):
    c = st["case"]
    return _turned(st["x"], st["positions"], st["freqs"], c["layout"], c["scale"]).bfloat16()


def _at(c, slots):
    slots = slots.long()
    return slots // c["ps"], slots % c["ps"]


def _append(st):
    c, live = st["case"], st["live"]
    k, v = st["keys"].float(), st["values"].float()
    if c["dim"]:
        k = _turned(st["keys"], st["positions"], st["freqs"], c["layout"], 1.0)
    page, off = _at(c, st["slots"][live])
    for x, name in ((k[live], "k"), (v[live], "v")):
        if c["scheme"] == "bf16":
            st[name][page, :, off] = x.bfloat16()
            continue
        s = st[name + "s"]
        if c["scheme"] == "fp8_row":
            s = _scale_of(x.abs().amax(-1))
            st[name + "s"][page, :, off] = s
            s = s[..., None]
        codes = (x / s).clamp(-448, 448).to(F8)
        st[name].view(torch.uint8)[page, :, off] = codes.view(torch.uint8)
    return _stored(st)


def _stored(st):
    out = [st["k"], st["v"]]
    return out + [st["ks"], st["vs"]] if st["case"]["scheme"] == "fp8_row" else out


def _values(st, name, codes, page=None, off=None):
    x = codes.float()
    s = st[name + "s"]
    if s is None:
        return x
    return x * s if s.numel() == 1 and st["case"]["scheme"] == "fp8_tensor" else x * s[page, :, off][..., None]


def _read(st):
    page, off = _at(st["case"], st["slots"])

    def rows(name):
        codes = st[name] if st["ks"] is None else st[name].view(torch.uint8)
        codes = codes[page, :, off]
        return _values(st, name, codes if st["ks"] is None else codes.view(F8), page, off).bfloat16()

    return rows("k"), rows("v")


def _context(st, name, b):
    """Keys or values of sequence b, fp32 [Hk, L, D]."""
    c, n = st["case"], st["ctx"][b]
    page = st["pages"][b, : -(-n // c["ps"])].long()
    x = st[name] if st["ks"] is None else st[name].view(torch.uint8)
    x = x[page]
    x = (x if st["ks"] is None else x.view(F8)).float()
    if c["scheme"] == "fp8_row":
        x *= st[name + "s"][page][..., None]
    elif c["scheme"] == "fp8_tensor":
        x *= st[name + "s"]
    return x.transpose(0, 1).reshape(c["Hk"], -1, c["D"])[:, :n]


def _hidden(c, n, L, dev):
    """[n, L]: key j is hidden from the i-th of the sequence's n new tokens."""
    at = torch.arange(L - n, L, device=dev)[:, None]
    j = torch.arange(L, device=dev)
    hidden = torch.zeros(n, L, dtype=torch.bool, device=dev)
    if c["causal"]:
        hidden |= j > at
    if c["window"]:
        hidden |= j <= at - c["window"]
    return hidden


def _attend(st):
    c = st["case"]
    G, D, dev = c["H"] // c["Hk"], c["D"], st["q"].device
    out = torch.empty_like(st["q"])
    lse = torch.empty(out.shape[:2], dtype=torch.float32, device=dev)
    t = 0
    for b, (n, L) in enumerate(zip(st["new"], st["ctx"])):
        k, v = _context(st, "k", b), _context(st, "v", b)
        hidden = _hidden(c, n, L, dev)
        q = st["q"][t: t + n].float().view(n, c["Hk"], G, D) * D ** -0.5
        for h in range(c["Hk"]):
            s = (q[:, h].reshape(n * G, D) @ k[h].t()).view(n, G, L)
            s.masked_fill_(hidden[:, None], float("-inf"))
            top = s.amax(-1, keepdim=True)
            p = s.sub_(top).exp_()
            total = p.sum(-1)
            o = (p.view(n * G, L) @ v[h]).view(n, G, D) / total[..., None]
            out[t: t + n, h * G: (h + 1) * G] = o.bfloat16()
            lse[t: t + n, h * G: (h + 1) * G] = top[..., 0] + total.log()
        t += n
    return (out, lse) if c["lse"] else out


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _own(state)
    return {"slots": _slots, "rope": _rope, "append": _append, "read": _read,
            "attend": _attend}[state["case"]["op"]](state)


def _own(st):
    import precision_quantized_linear_amd as pql

    c = st["case"]
    if c["op"] == "slots":
        return pql.kv_slots(st["starts"], st["lens"], st["pages"], c["ps"], sum(st["new"]))
    turn = pql.Rope(st["freqs"], c.get("scale", 1.0), c["layout"]) if "freqs" in st else None
    if c["op"] == "rope":
        return pql.rope(st["x"], st["positions"], turn)
    cache = pql.KVCache(c["scheme"], st["n_pages"], c["ps"], c["Hk"], c["D"],
                        *((st[x] if c["scheme"] == "bf16" else st[x].view(torch.uint8)) for x in "kv"), st["ks"], st["vs"])
    if c["op"] == "append":
        pql.kv_append(st["keys"], st["values"], cache, st["slots"], turn, st.get("positions"))
        return _stored(st)
    if c["op"] == "read":
        return pql.kv_read(cache, st["slots"])
    return pql.kv_attention(st["q"], cache, st["starts"], st["lens"], st["pages"], causal=c["causal"],
                            window=c["window"], return_lse=c["lse"])


# ------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "slots":
        new, _ = _batch(c)
        return {"bytes": 8 * c["B"] + 12 * sum(new), "flops": 0}
    if c["op"] == "rope":
        n = c["T"] * c["H"]
        return {"bytes": 4 * n * c["D"] + 4 * c["T"] + 4 * c["dim"], "flops": 3 * n * c["dim"]}
    size, scales = (2, 0) if c["scheme"] == "bf16" else (1, 4 if c["scheme"] == "fp8_row" else 0)
    row = 2 * c["Hk"] * (size * c["D"] + scales)          # one token's keys and values in the cache
    if c["op"] == "append":
        n = c["T"] * (1.0 - c["dropped"])
        return {"bytes": n * (4 * c["Hk"] * c["D"] + row) + 4 * c["T"], "flops": n * c["Hk"] * (3 * c["dim"] + 4 * c["D"])}
    if c["op"] == "read":
        return {"bytes": c["n"] * (4 * c["Hk"] * c["D"] + row + 4), "flops": 2 * c["n"] * c["Hk"] * c["D"]}
    new, ctx = _batch(c)
    pairs, seen = 0, 0
    for n, L in zip(new, ctx):
        first = L - n + 1                                  # keys up to the first new token's own
        w = c["window"] or L
        if c["causal"]:
            short = min(n, max(0, w - first + 1))          # tokens that see less than a whole window
            pairs += short * (2 * first + short - 1) // 2 + (n - short) * min(w, L)
        else:
            pairs += sum(min(L, n - 1 - i + w) for i in range(n))
        seen += min(L, w + n - 1)
    return {"bytes": 4 * sum(new) * c["H"] * c["D"] + seen * row, "flops": 4 * pairs * c["H"] * c["D"]}


# ------------------------------------------------------------------------------------------------ 64 bits
def _rotation(x, positions, freqs, layout, scale):
    """Pairs as complex numbers times scale e^(i position frequency)."""
    d = 2 * freqs.numel()
    x = x.double()
    pairs = x[..., :d].unflatten(-1, (2, -1)).transpose(-1, -2) if layout == "half" else x[..., :d].unflatten(-1, (-1, 2))
    z = torch.view_as_complex(pairs.contiguous())
    turn = torch.polar(torch.full((1,), scale, dtype=torch.float64, device=x.device), torch.outer(positions.double(), freqs))
    y = torch.view_as_real(z * turn[:, None])
    y = y.transpose(-1, -2).flatten(-2) if layout == "half" else y.flatten(-2)
    return torch.cat((y, x[..., d:]), -1)


def exact(case, seed):
    """From the definitions, in 64 bits; codes come as the numbers before their rounding to e4m3."""
    c, st = case, prepare(case, seed)
    if c["op"] == "slots":
        table = st["pages"].tolist()
        pos = [p for n, L in zip(st["new"], st["ctx"]) for p in range(L - n, L)]
        seq = [b for b, n in enumerate(st["new"]) for _ in range(n)]
        slots = [table[b][p // c["ps"]] * c["ps"] + p % c["ps"] for b, p in zip(seq, pos)]
        return torch.tensor(slots).int(), torch.tensor(pos).int()
    if c["op"] == "rope":
        return _rotation(st["x"], st["positions"], st["freqs"], c["layout"], c["scale"])
    if c["op"] == "append":
        k = _rotation(st["keys"], st["positions"], st["freqs"], c["layout"], 1.0) if c["dim"] else st["keys"].double()
        out, scales = [], []
        for name, x in (("k", k), ("v", st["values"].double())):
            held = st[name].double().transpose(1, 2).flatten(0, 1)           # [slots, Hk, D]
            to, x = st["slots"][st["live"]].long(), x[st["live"]]
            if c["scheme"] == "fp8_row":
                s = x.abs().amax(-1) / 448.0
                s[s == 0] = 1.0
                held_s = st[name + "s"].double().transpose(1, 2).flatten(0, 1)
                held_s[to] = s
                scales.append(held_s.unflatten(0, (-1, c["ps"])).transpose(1, 2))
                x = x / s[..., None]
            elif c["scheme"] == "fp8_tensor":
                x = (x / st[name + "s"].double()).clamp(-448.0, 448.0)
            held[to] = x
            out.append(held.unflatten(0, (-1, c["ps"])).transpose(1, 2))
        return out + scales
    if c["op"] == "read":
        out = []
        for name in "kv":
            x = st[name].double().transpose(1, 2).flatten(0, 1)[st["slots"].long()]
            if c["scheme"] == "fp8_row":
                x = x * st[name + "s"].double().transpose(1, 2).flatten(0, 1)[st["slots"].long()][..., None]
            elif c["scheme"] == "fp8_tensor":
                x = x * st[name + "s"].double()
            out.append(x)
        return tuple(out)
    return _exact_attend(st)


def _exact_attend(st):
    """Query blocks of at most 512 tokens, softmax by its logarithm."""
    c = st["case"]
    G, D, dev = c["H"] // c["Hk"], c["D"], st["q"].device
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device=dev)
    t = 0
    for b, (n, L) in enumerate(zip(st["new"], st["ctx"])):
        every = torch.arange(L, device=dev)
        slots = st["pages"][b].long()[every // c["ps"]] * c["ps"] + every % c["ps"]
        for h in range(c["Hk"]):
            kv = []
            for name in "kv":
                x = st[name][:, h].flatten(0, 1) if st["ks"] is None else st[name][:, h].contiguous().view(torch.uint8).flatten(0, 1)
                x = (x[slots] if st["ks"] is None else x[slots].view(F8)).double()
                s = st[name + "s"]
                if s is not None:
                    x = x * (s.double() if c["scheme"] == "fp8_tensor" else s[:, h].flatten()[slots].double()[:, None])
                kv.append(x)
            for i in range(0, n, 512):
                m = min(512, n - i)
                q = st["q"][t + i: t + i + m, h * G: (h + 1) * G].double()
                score = torch.mm(q.flatten(0, 1), kv[0].t()).view(m, G, L) / math.sqrt(D)
                ago = torch.arange(L - n + i, L - n + i + m, device=dev)[:, None] - every
                seen = torch.ones_like(ago, dtype=torch.bool)
                if c["causal"]:
                    seen &= ago >= 0
                if c["window"]:
                    seen &= ago < c["window"]
                score = torch.where(seen[:, None], score, -math.inf)
                z = torch.logsumexp(score, -1)
                lse[t + i: t + i + m, h * G: (h + 1) * G] = z
                p = torch.exp(score - z[..., None])
                out[t + i: t + i + m, h * G: (h + 1) * G] = torch.mm(p.flatten(0, 1), kv[1]).view(m, G, D)
        t += n
    return (out, lse) if c["lse"] else out
