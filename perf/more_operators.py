"""Operators between the projections of a decoder layer: the RMS norm and the
SwiGLU gate whose outputs are a projection's INT8 rows, rotary positions with
the append to a cache held in 4 bits, and causal attention over that cache
for single tokens and for packed prompts.

`run` computes them in elementary torch operations, or, where `own` is set,
by the framework's entry points.  Widths and head layouts are those of the
framework's own workloads (2560, 4096, 5120; 32 or 40 query heads over 8 of
128 features) or generic ones.

The cache.  codes [pages, 2, heads, tokens, D/2] (uint8; 0: keys, 1: values):
byte b of a token's row holds features 2b (low nibble) and 2b + 1.  words
[pages, 2, heads, tokens] (int32): bits of an FP32 scale s whose low four bits
hold the zero point z.  A feature stands for s * (code - z).  Token t of a
sequence is token t % tokens of page block_table[sequence, t // tokens].
"""

import random

import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a chat being decoded: the norm in front of qkv
        dict(name="norm_1", kind="norm", M=1, H=4096, type="f32"),
        # a ragged batch whose residual stream is kept in 16 bits
        dict(name="norm_333_bf16", kind="norm", M=333, H=2560, type="bf16"),
        # a prefill chunk
        dict(name="norm_8192", kind="norm", M=8192, H=5120, type="f32"),
        # the gate of a handful of requests, in front of a wide down projection
        dict(name="swiglu_5", kind="swiglu", M=5, I=14336),
        # a prompt's gate
        dict(name="swiglu_2048", kind="swiglu", M=2048, I=9728),
        # three requests far into long contexts, one position each
        dict(name="rope_3", kind="rope", M=3, Hq=32, Hkv=8, D=128, sections="64", far=1000000, P=64, interleaved=False),
        # a video prompt: time, height and width
        dict(name="rope_video_5000", kind="rope", M=5000, Hq=40, Hkv=8, D=128, sections="16,24,24", far=20000, P=16, interleaved=False),
        # one request, a chat of some length
        dict(name="attn_1", kind="attn", B=1, tokens=1, longest=1500, Hq=32, Hkv=8, D=128, P=64),
        # a serving batch, contexts of every length, small pages
        dict(name="attn_48", kind="attn", B=48, tokens=48, longest=6000, Hq=40, Hkv=8, D=128, P=16),
        # a few requests over whole books
        dict(name="attn_3_long", kind="attn", B=3, tokens=3, longest=120000, Hq=32, Hkv=8, D=128, P=64),
        # ragged prompts side by side, some after a cached prefix; an odd number of heads to a group
        dict(name="prompt_ragged", kind="attn", B=9, tokens=1700, longest=1100, Hq=14, Hkv=2, D=64, P=32),
        # one long prompt
        dict(name="prompt_6000", kind="attn", B=1, tokens=6000, longest=6000, Hq=32, Hkv=8, D=128, P=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    kind = rng.choice(["norm", "swiglu", "rope", "attn", "attn", "prompt", "prompt"])
    while True:
        if kind == "norm":
            c = dict(kind=kind, M=_log(rng, 1, 8192), H=64 * rng.randint(8, 160), type=rng.choice(["f32", "bf16", "f16"]))
            if c["M"] * c["H"] <= 8192 * 5120:
                return c
        elif kind == "swiglu":
            c = dict(kind=kind, M=_log(rng, 1, 4096), I=64 * rng.randint(8, 272))
            if c["M"] * c["I"] <= 2048 * 9728:
                return c
        elif kind == "rope":
            D, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
            a, b = sorted((rng.randint(1, D // 2 - 2), rng.randint(1, D // 2 - 2)))
            s = rng.choice([str(D // 2), "%d,%d,%d" % (a, b - a + 1, D // 2 - b - 1), "%d,%d" % (a, D // 4)]) if a <= D // 4 else str(D // 2)
            c = dict(kind=kind, M=_log(rng, 1, 5000), Hq=hkv * rng.randint(1, 8), Hkv=hkv, D=D, sections=s,
                     far=_log(rng, 1000, 1000000), P=rng.choice([16, 32, 64, 128]), interleaved=rng.random() < 0.4)
            if c["M"] * c["Hq"] * D <= 5000 * 40 * 128:
                return c
        else:
            D, hkv, B = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), _log(rng, 1, 64)
            c = dict(kind="attn", B=B, tokens=B if kind == "attn" else B + _log(rng, 8, 6000), longest=_log(rng, 16, 131072),
                     Hq=hkv * rng.randint(1, 8), Hkv=hkv, D=D, P=rng.choice([16, 32, 64, 128]))
            new, old = _lengths(c)
            keys = sum(n + o for n, o in zip(new, old))
            w = work(c)
            padded = B * c["Hq"] * max(new) * max(n + o for n, o in zip(new, old))
            apart = B * max(n + o for n, o in zip(new, old))               # as the plain form pads them
            if (keys * hkv * D <= 3 * 120000 * 8 * 128 and apart * hkv * D <= 12 * 120000 * 8 * 128
                    and w["flops"] <= 4 * 128 * 32 * 6000 * 3000 and padded <= 32 * 6000 * 6000):
                return c


def _lengths(case):
    """(tokens of each sequence in this call, tokens it has cached before
    them): ragged, and the longest context of exactly `longest` tokens."""
    rng = random.Random("%(B)d %(tokens)d %(longest)d" % case)
    B, tokens, longest = case["B"], case["tokens"], case["longest"]
    cuts = sorted(rng.sample(range(1, tokens), B - 1)) if B > 1 else []
    new = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
    if tokens == B:                # single tokens: contexts spread over their logarithm
        old = [_log(rng, 1, longest) - 1 for _ in range(B)]
        old[rng.randrange(B)] = longest - 1
    else:                          # prompts: every other one after a cached prefix
        old = [0 if rng.random() < 0.5 else rng.randint(0, max(0, longest - n)) for n in new]
    return new, old


_TYPES = dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)


# ---------------------------------------------------------------- inputs

def _acts(M, K, g):
    """Activations: N(0, 1) with 1% of channels x 30."""
    X = torch.randn((M, K), generator=g, device="cuda")
    X[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 30.0
    return X


def _pages(lens, P, g):
    """A block table of scattered pages for sequences of these lengths, -1
    behind the last page, and the number of pages in all."""
    need = [-(-n // P) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    if c["kind"] == "norm":
        t = _TYPES[c["type"]]
        c["X"], c["R"] = _acts(c["M"], c["H"], g).to(t), _acts(c["M"], c["H"], g).mul_(3.0).to(t)
        c["W"] = (torch.rand(c["H"], generator=g, device="cuda") + 0.5).to(t)
    elif c["kind"] == "swiglu":
        c["GU"] = torch.randn((c["M"], 2 * c["I"]), generator=g, device="cuda").mul_(2.0)
    elif c["kind"] == "rope":
        M, D, heads = c["M"], c["D"], c["Hq"] + 2 * c["Hkv"]
        c["parts"] = [int(s) for s in c["sections"].split(",")]
        c["qkv"] = _acts(M, heads * D, g)
        half = sum(c["parts"])
        c["freq"] = (1.0 / 1000000.0 ** (torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        c["pos"] = torch.randint(0, c["far"], (len(c["parts"]), M), generator=g, device="cuda").int()
        pages = -(-M // c["P"]) + 5
        c["slots"] = torch.randperm(pages * c["P"], generator=g, device="cuda")[:M]
        if own:
            import mixed_precision_int_amd as aq
            c["cache"] = aq.aq_kv4_cache(pages, c["P"], c["Hkv"], D)
            c["rope"] = aq.aq_rope_axes(c["freq"], c["parts"], D, interleaved=c["interleaved"])
    else:
        new, old = _lengths(c)
        lens = [a + b for a, b in zip(new, old)]
        P, H, D = c["P"], c["Hkv"], c["D"]
        c["table"], pages = _pages(lens, P, g)
        c["codes"] = torch.randint(0, 256, (pages, 2, H, P, D // 2), generator=g, device="cuda", dtype=torch.uint8)
        # steps as of keys of some units and values of N(0, 1), zero points about the middle
        s = (torch.rand((pages, 2, H, P), generator=g, device="cuda") + 0.5) * 0.3
        z = torch.randint(5, 11, s.shape, generator=g, device="cuda", dtype=torch.int32)
        c["words"] = (s.view(torch.int32) & ~15) | z
        c["q"] = torch.randn((c["tokens"], c["Hq"], D), generator=g, device="cuda")
        c["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0] + new).cumsum(0)
        c["cu"] = None if c["tokens"] == c["B"] else cu.int().cuda()
        c["most"] = (max(new), max(lens))
        if own:
            import mixed_precision_int_amd as aq
            c["cache"] = aq.aq_kv4_cache_of(c["codes"], c["words"])
    return c


# ---------------------------------------------------------------- the operators in plain form

def _codes8(Y):
    """The values that per-row INT8 codes of FP32 rows stand for."""
    s = (Y.abs().amax(-1, keepdim=True).double() / 127).clamp_min(1e-12)
    return (Y.double() / s).round().clamp(-128, 127).float() * s.float()


def _norm(c):
    h = c["X"] + c["R"]
    x = h.double()
    y = x * (1 / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()) * c["W"].double()
    return {"x": _codes8(y.float()), "h": h}


def _swiglu(c):
    g, u = c["GU"].double().chunk(2, dim=1)
    return _codes8((g / (1 + torch.exp(-g)) * u).float())


def _rotate(x, c):
    """The first 2 * half features of each head of FP32 x [M, heads, D]
    rotated, in 64 bits: far positions times small frequencies."""
    half = c["freq"].numel()
    axis = torch.repeat_interleave(torch.arange(len(c["parts"]), device=x.device), torch.tensor(c["parts"], device=x.device))
    angle = c["pos"].double()[axis].T * c["freq"].double()                 # [M, half]
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    x = x.double()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1).float()


def _kv4(x):
    """The values that the 4-bit codes of FP32 vectors stand for."""
    top, low = x.amax(-1, keepdim=True).clamp_min(0).double(), x.amin(-1, keepdim=True).clamp_max(0).double()
    want = ((top - low) / 15).clamp_min(1e-12)
    s = want.float()
    s = torch.where(s.double() < want, torch.nextafter(s, torch.full_like(s, float("inf"))), s)
    s = ((s.view(torch.int32) + 15) & ~15).view(torch.float32).double()
    z = (-low / s).round()
    return (s * (((x.double() / s).round() + z).clamp(0, 15) - z)).float()


def _rope(c):
    M, D, hq, hkv = c["M"], c["D"], c["Hq"], c["Hkv"]
    x = c["qkv"].view(M, hq + 2 * hkv, D)
    r = _rotate(x[:, :hq + hkv], c)
    return {"q": r[:, :hq], "k": _kv4(r[:, hq:]), "v": _kv4(x[:, hq + hkv:])}


def _attention(c):
    """Sequences padded to the longest: scores, softmax and sums in 32 bits."""
    B, H, D, G, dev = c["B"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], c["q"].device
    Q, L = c["most"]
    at = torch.arange(L, device=dev)
    page = c["table"].long()[:, at // c["P"]].clamp_min(0)                 # [B, L]
    codes = c["codes"][page, :, :, (at % c["P"])[None]].permute(2, 0, 3, 1, 4)    # [2, B, H, L, D/2]
    word = c["words"][page, :, :, (at % c["P"])[None]].permute(2, 0, 3, 1)
    s, z = (word & ~15).view(torch.float32), (word & 15).float()
    k, v = ((torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - z[..., None]) * s[..., None]).view(2, B * H, L, D)
    cu = c["cu"] if c["cu"] is not None else torch.arange(B + 1, device=dev, dtype=torch.int32)
    new = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=dev)
    row = (cu[:-1, None] + i).clamp_max(c["tokens"] - 1).long()            # [B, Q]
    q = c["q"][row].view(B, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B * H, G * Q, D)
    S = torch.bmm(q, k.transpose(1, 2).contiguous()).mul_(D ** -0.5).view(B, H, G, Q, L)
    seen = at[None, None, :] <= (c["kv_len"] - new)[:, None, None] + i[None, :, None]
    S.masked_fill_(~seen[:, None, None], -float("inf"))
    S = torch.exp_(S.sub_(S.amax(-1, keepdim=True)))
    S.div_(S.sum(-1, keepdim=True))
    o = torch.bmm(S.view(B * H, G * Q, L), v.contiguous()).view(B, H, G, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, H * G * D)
    return o[i[None] < new[:, None]]


def run(state):
    c = state
    if own:
        import mixed_precision_int_amd as aq
        if c["kind"] == "norm":
            qx, sx, h = aq.aq_norm_quant(c["X"], c["W"], residual=c["R"])
            return {"x": torch.mul(qx, sx[:, None]), "h": h}
        if c["kind"] == "swiglu":
            qx, sx = aq.aq_swiglu_quant(c["GU"])
            return torch.mul(qx, sx[:, None])
        if c["kind"] == "rope":
            q = aq.aq_rope_kv4(c["qkv"], c["rope"], c["pos"], c["cache"], c["slots"])
            k, v = aq.aq_kv4_read(c["cache"], c["slots"])
            return {"q": q, "k": k, "v": v}
        return aq.aq_attn_kv4(c["q"], c["cache"], c["table"], c["kv_len"], cu_q=c["cu"])
    return {"norm": _norm, "swiglu": _swiglu, "rope": _rope, "attn": _attention}[c["kind"]](c)


# ---------------------------------------------------------------- work and 64-bit values

def work(case):
    c = case
    if c["kind"] == "norm":
        b = 4 if c["type"] == "f32" else 2
        return dict(bytes=c["M"] * (c["H"] * (3 * b + 1) + 4) + b * c["H"], flops=8 * c["M"] * c["H"])
    if c["kind"] == "swiglu":
        return dict(bytes=c["M"] * (9 * c["I"] + 4), flops=10 * c["M"] * c["I"])
    if c["kind"] == "rope":
        M, D, hq, hkv = c["M"], c["D"], c["Hq"], c["Hkv"]
        # the rows read, q written, the cache's bytes written, its values as they are read back
        return dict(bytes=M * (4 * (2 * hq + 2 * hkv) * D + 2 * 2 * hkv * (D // 2 + 4) + 2 * hkv * D * 4), flops=M * D * (6 * (hq + hkv) + 8 * hkv))
    new, old = _lengths(c)
    keys = sum(n + o for n, o in zip(new, old))
    pairs = sum(n * o + n * (n + 1) // 2 for n, o in zip(new, old))
    return dict(bytes=8 * c["tokens"] * c["Hq"] * c["D"] + keys * 2 * c["Hkv"] * (c["D"] // 2 + 4), flops=4 * c["D"] * c["Hq"] * pairs)


def exact(case, seed):
    """The definitions in 64 bits, head by head."""
    c = prepare(case, seed)
    if c["kind"] in ("norm", "swiglu"):
        if c["kind"] == "norm":
            h = c["X"].double() + c["R"].double()
            rows = h.to(_TYPES[c["type"]]).double()
            y = torch.nn.functional.rms_norm(rows, (c["H"],), c["W"].double(), 1e-6).float().double()
        else:
            y = (torch.nn.functional.silu(c["GU"][:, :c["I"]].double()) * c["GU"][:, c["I"]:].double()).float().double()
        s = torch.clamp(y.abs().max(1, keepdim=True).values / 127, min=1e-12)
        x = torch.clamp(torch.round(y / s), -128, 127) * s.float().double()
        return {"x": x, "h": h} if c["kind"] == "norm" else x
    if c["kind"] == "rope":
        M, D, hq, hkv = c["M"], c["D"], c["Hq"], c["Hkv"]
        x = c["qkv"].view(M, hq + 2 * hkv, D).double().clone()
        i = 0
        for axis, part in enumerate(c["parts"]):
            for _ in range(part):
                turn = torch.polar(torch.ones(M, dtype=torch.float64, device=x.device), c["pos"][axis].double() * c["freq"][i].double())[:, None]
                at = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + sum(c["parts"]))
                y = torch.complex(x[:, :hq + hkv, at[0]], x[:, :hq + hkv, at[1]]) * turn
                x[:, :hq + hkv, at[0]], x[:, :hq + hkv, at[1]] = y.real, y.imag
                i += 1

        def held(y):
            y = y.float().double()
            top, low = torch.clamp(y.max(-1, keepdim=True).values, min=0), torch.clamp(y.min(-1, keepdim=True).values, max=0)
            want = torch.clamp((top - low) / 15, min=1e-12)
            # the 20-bit significands: steps of 2^-19 of the power of two below
            unit = torch.exp2(torch.floor(torch.log2(want)) - 19)
            s = torch.ceil(want / unit) * unit
            z = torch.round(-low / s)
            return s * (torch.clamp(torch.round(y / s) + z, 0, 15) - z)
        return {"q": x[:, :hq], "k": held(x[:, hq:hq + hkv]), "v": held(x[:, hq + hkv:])}
    new, old = _lengths(c)
    G, D, out, first = c["Hq"] // c["Hkv"], c["D"], torch.zeros((c["tokens"], c["Hq"], c["D"]), dtype=torch.float64, device="cuda"), 0
    for b, (n, o) in enumerate(zip(new, old)):
        pages = c["table"][b, :-(-(n + o) // c["P"])].long()
        for h in range(c["Hkv"]):
            x = c["codes"][pages][:, :, h].transpose(0, 1).reshape(2, -1, D // 2)[:, :n + o].int()
            w = c["words"][pages][:, :, h].transpose(0, 1).reshape(2, -1)[:, :n + o]
            kv = torch.empty((2, n + o, D), dtype=torch.float64, device="cuda")
            kv[..., 0::2], kv[..., 1::2] = x % 16, x // 16
            kv = (kv - (w % 16)[..., None]) * (w - w % 16).view(torch.float32).double()[..., None]
            for j in range(h * G, h * G + G):
                S = c["q"][first:first + n, j].double() @ kv[0].T / D ** 0.5
                S = S + torch.full((n, n + o), -float("inf"), dtype=torch.float64, device="cuda").triu(o + 1)
                out[first:first + n, j] = torch.softmax(S, 1) @ kv[1]
        first += n
    return out.view(c["tokens"], -1)
