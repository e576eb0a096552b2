"""Cases and plain forms of a prompt's way into the cache and of eviction by accumulated attention weight.

  rotary    query and key rows turned by their positions: pairs in halves or interleaved, part of the head,
            frequencies scaled for long contexts
  prompt    causal attention over whole prompts of different lengths, grouped heads, packed or padded, with the
            logarithm of each row's sum
  weigh     attention weight that the newest tokens' queries give each token of the 8-bit paged cache, added to
            what the token has gathered so far
  heaviest  the slots an eviction keeps: the first and the last tokens and the heaviest of the others, per head

Shapes: the 28-layer Qwen-7B-shaped, the Llama-8B-shaped and the long-context workloads of this repository.
"""
import math

import torch

own = False

TOP = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one layer of a decode step of the Llama-shaped batch, positions far into a long context
        dict(name="rotary_step", op="rotary", B=64, H=8, G=4, d=128, dim=128, n=1, lo=1, at=131072, interleaved=False,
             scaling="bands", base=500000.0, factor=8.0),
        # one layer of eight prompts of the Qwen-shaped heads
        dict(name="rotary_prompt", op="rotary", B=8, H=4, G=7, d=128, dim=128, n=4096, lo=4096, at=0,
             interleaved=False, scaling="none", base=1000000.0, factor=1.0),
        # one layer of a ragged chunk, half of small heads turned, interleaved pairs, positions interpolated
        dict(name="rotary_part", op="rotary", B=32, H=8, G=4, d=64, dim=32, n=128, lo=40, at=5000, interleaved=True,
             scaling="linear", base=10000.0, factor=4.0),
        # one short prompt, one head: the smallest call, where only latency counts
        dict(name="prompt_tiny", op="prompt", B=1, H=1, G=1, d=64, lo=64, hi=64, packed=True),
        # one layer of a batch of ragged Llama-shaped prompts, packed
        dict(name="prompt_ragged", op="prompt", B=16, H=8, G=4, d=128, lo=612, hi=1112, packed=True),
        # one layer of a long prompt of the Qwen-shaped heads
        dict(name="prompt_long", op="prompt", B=1, H=4, G=7, d=128, lo=16384, hi=16384, packed=False),
        # one layer of a decode step of the Llama-shaped ragged batch
        dict(name="weigh_step", op="weigh", B=64, H=8, G=4, d=128, bs=16, fmt="e4m3", lo=612, hi=1112, n=1, decay=1.0),
        # one layer of a decode step over the long-context caches
        dict(name="weigh_long", op="weigh", B=4, H=4, G=7, d=128, bs=64, fmt="int8", lo=32768, hi=32768, n=1,
             decay=0.99),
        # one layer of whole prompts of the Qwen-shaped batch
        dict(name="weigh_prompt", op="weigh", B=8, H=4, G=7, d=128, bs=16, fmt="e4m3", lo=1536, hi=1536, n=1536,
             decay=0.0),
        # one layer of the Llama-shaped ragged batch, 1112 -> 512 slots
        dict(name="heaviest_ragged", op="heaviest", L=1, B=64, H=8, lo=612, hi=1112, budget=512),
        # every layer of the Qwen-shaped batch, 1536 -> 1024 slots
        dict(name="heaviest_event", op="heaviest", L=28, B=8, H=4, lo=1536, hi=1536, budget=1024),
        # every layer of the long-context caches, 32768 -> 4096 slots
        dict(name="heaviest_long", op="heaviest", L=28, B=4, H=4, lo=32768, hi=32768, budget=4096),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["rotary", "prompt", "prompt", "weigh", "weigh", "heaviest"])
    c = dict(op=op, H=rng.choice([1, 2, 4, 8]), G=rng.randint(1, 8), d=rng.choice([64, 128]))
    if op == "rotary":
        c["B"] = log(1, 64)
        c["n"] = rng.choice([1, log(2, max(3, min(4096, 32768 // c["B"])))])
        c["lo"] = max(1, int(c["n"] * rng.choice([1.0, 0.3])))
        c["at"] = rng.choice([0, log(1, 1000000)])
        c["dim"] = c["d"] // rng.choice([1, 1, 2, 4])
        c["interleaved"] = rng.random() < 0.5
        c["scaling"] = rng.choice(["none", "linear", "ntk", "bands"])
        c["base"] = rng.choice([10000.0, 500000.0, 1000000.0])
        c["factor"] = 1.0 if c["scaling"] == "none" else rng.choice([2.0, 4.0, 8.0])
    elif op == "prompt":
        c["B"] = log(1, 16)
        c["hi"] = log(1, max(2, min(16384, int((7.0e9 / (c["B"] * c["H"] * c["G"])) ** 0.5))))
        c["lo"] = max(1, int(c["hi"] * rng.choice([1.0, 0.6, 0.1])))
        c["packed"] = rng.random() < 0.5
    elif op == "weigh":
        c["B"] = log(1, 64)
        many = int((2.5e9 / (c["B"] * c["H"] * c["G"])) ** 0.5)
        c["n"] = rng.choice([1, 1, rng.randint(2, 4), log(5, min(1536, many))])
        most = min(32768, 1048576 // (c["B"] * c["H"]), 3_000_000_000 // (c["B"] * c["H"] * c["G"] * c["n"]))
        c["hi"] = log(c["n"] + 8, max(c["n"] + 9, most))
        c["lo"] = max(1, int(c["hi"] * rng.choice([1.0, 0.7, 0.3])))
        c["bs"] = rng.choice([8, 16, 16, 24, 32, 64, 128])
        c["fmt"] = rng.choice(["e4m3", "int8"])
        c["decay"] = rng.choice([1.0, 1.0, 0.9, 0.0])
    else:
        c["L"] = rng.choice([1, 1, 4, 28])
        c["B"] = log(1, 64)
        c["hi"] = log(16, min(32768, 14_000_000 // (c["L"] * c["B"] * c["H"])))
        c["lo"] = max(1, int(c["hi"] * rng.choice([1.0, 0.5])))
        c["budget"] = max(8, c["hi"] // rng.choice([2, 3, 8]))
        del c["G"], c["d"]
    return c


def _lens(c):
    """The sequences' lengths: spread over [lo, hi] in a scattered order, the same for every seed."""
    B, lo, hi = c["B"], c["lo"], c.get("hi", c.get("n"))
    return [hi if B == 1 else lo + (hi - lo) * ((i * 37 + 11) % B) // (B - 1) for i in range(B)]


def _queries(c, length):
    """Queries of a sequence in a weighing: the newest n tokens."""
    return min(c["n"], length)


def work(c):
    """Bytes: bf16 rows (2), codes (1), scales, weights, sums, positions and indices (4).  Flops: the products."""
    lens, B, H = _lens(c), c["B"], c["H"]
    if c["op"] == "rotary":
        rows = sum(lens) * H * (c["G"] + 1)
        return {"bytes": rows * c["d"] * 4 + sum(lens) * 4, "flops": rows * c["dim"] * 3.0}
    if c["op"] == "prompt":
        rows, pairs = sum(lens) * H, sum(m * (m + 1) / 2 for m in lens)
        return {"bytes": rows * (4 * c["d"] * (c["G"] + 1) + 4 * c["G"]), "flops": 4.0 * H * c["G"] * c["d"] * pairs}
    if c["op"] == "weigh":
        nq = [_queries(c, m) for m in lens]
        seen = sum(n * m - n * (n - 1) / 2 for n, m in zip(nq, lens))
        blocks = sum(-(-m // c["bs"]) for m in lens)
        cache = H * (sum(lens) * c["d"] + blocks * 4) + blocks * 4
        gathered = H * sum(lens) * (8 if c["decay"] else 4)
        return {"bytes": cache + gathered + sum(nq) * H * c["G"] * (2 * c["d"] + 4),
                "flops": 2.0 * H * c["G"] * c["d"] * seen}
    units = c["L"] * H
    return {"bytes": units * (sum(lens) * 4 + B * (max(lens) * 4 + c["budget"] * 4 + 4)), "flops": 0}


# ----------------------------------------------------------------- inputs ----

def _bf16(shape, g, spread=0.0):
    """N(0, 1) rows in bf16; with `spread`, a factor 2^(spread * N(0, 1)) for each row."""
    x = torch.randn(shape, generator=g, device="cuda")
    if spread:
        x *= torch.exp2(spread * torch.randn((*shape[:-1], 1), generator=g, device="cuda"))
    return x.to(torch.bfloat16)


def _as_codes(x, fmt):
    """Codes of [N, H, bs, d] rows and one power-of-two scale for each block and head."""
    amax = x.abs().amax((-1, -2)).clamp(min=2.0 ** -60)
    scale = torch.exp2(torch.ceil(torch.log2(amax / TOP[fmt])))
    y = (x / scale[..., None, None]).clamp(-TOP[fmt], TOP[fmt])
    return (y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)), scale


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, B, H = c["op"], c["B"], c["H"]
    lens = _lens(c)
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s = dict(c=c, length=length)
    if op == "rotary":
        G, d, n = c["G"], c["d"], c["n"]
        # one projection's output: queries, keys and values side by side, token-major
        qkv = _bf16((1, B, n, H * G + 2 * H, d), g, 0.4)
        s["q"] = qkv[..., :H * G, :].permute(0, 1, 3, 2, 4)
        s["k"] = qkv[..., H * G:H * G + H, :].permute(0, 1, 3, 2, 4)
        s["q_out"], s["k_out"] = (torch.zeros((1, B, n, x, d), dtype=torch.bfloat16, device="cuda").permute(0, 1, 3, 2, 4)
                                  for x in (H * G, H))
        start = (torch.rand(B, generator=g, device="cuda") * (c["at"] + 1)).int()
        s["pos"] = start[:, None] + torch.arange(n, dtype=torch.int32, device="cuda")
    elif op == "prompt":
        G, d, hi = c["G"], c["d"], c["hi"]
        # packed: the sequences one after another, each begins at a multiple of 8 rows; padded: hi rows for each
        firsts = [0]
        for m in lens:
            firsts.append(firsts[-1] + -(-m // 8) * 8)
        N = firsts[-1] if c["packed"] else hi
        lead = () if c["packed"] else (B,)
        rows = dict(zip("qkv", (_bf16((*lead, N, x, d), g, 0.4) for x in (H * G, H, H))))
        rows["q"] *= 1.5
        at = torch.arange(N, device="cuda")
        if c["packed"]:
            s["first"] = torch.tensor(firsts[:-1], dtype=torch.int32, device="cuda")
            inside = ((at >= s["first"][:, None]) & (at < (s["first"] + length)[:, None])).any(0)
        else:
            s["first"], inside = None, at < length[:, None]
        for k, x in rows.items():  # what lies between and behind the sequences is whatever was there last
            x.masked_fill_(~inside[..., None, None], float("nan"))
            s[k] = x.transpose(-3, -2)
        s["out"] = torch.zeros((*lead, N, H * G, d), dtype=torch.bfloat16, device="cuda").transpose(-3, -2)
        s["lse"] = torch.zeros((*lead, H * G, N), device="cuda")
    elif op == "weigh":
        G, d, n, bs, fmt = c["G"], c["d"], c["n"], c["bs"], c["fmt"]
        M = -(-c["hi"] // bs) + 1
        nb = (length + bs - 1) // bs
        N = sum(-(-m // bs) for m in lens) + 5
        perm = torch.randperm(N, generator=g, device="cuda").int()
        cols = torch.arange(M, device="cuda")
        at = (nb.cumsum(0) - nb)[:, None] + cols
        table = torch.where(cols < nb[:, None], perm[at.clamp(max=N - 1)], -1).int().contiguous()
        ref = torch.ones(N, dtype=torch.int32, device="cuda")
        kp, ks = _as_codes(_bf16((N, H, bs, d), g, 0.4).float(), fmt)
        vp, vs = torch.zeros_like(kp), torch.ones_like(ks)
        s.update(kp=kp[None], ks=ks[None], vp=vp[None], vs=vs[None], table=table, ref=ref,
                 free=perm.flip(0).contiguous(), top=torch.tensor([5], dtype=torch.int32, device="cuda"))
        s["q"] = (1.5 * _bf16((1, B, n, H * G, d), g, 0.4)).permute(0, 1, 3, 2, 4)
        s["n_q"] = length.clamp(max=n).int()
        s["lse"] = torch.logsumexp(_scores(s), -1).reshape(1, B, H * G, n)  # as the attention left it
        older = torch.arange(c["hi"], device="cuda") < (length - s["n_q"])[:, None]
        old = torch.rand((1, B, H, c["hi"]), generator=g, device="cuda").log().neg() * 4  # new tokens have none
        s["w"] = torch.where(older[:, None], old, 0)
    else:
        L, hi = c["L"], c["hi"]
        # gathered attention weight: few tokens have most of it
        w = torch.rand((L, B, H, hi), generator=g, device="cuda").log().neg().square() * 3
        s["w"] = torch.where(torch.arange(hi, device="cuda") < length[:, None, None], w, 0)
        s["kept"] = torch.zeros((L, B, H, c["budget"]), dtype=torch.int32, device="cuda")
        s["n_kept"] = torch.zeros((L, B, H), dtype=torch.int32, device="cuda")
        s["w_out"] = torch.zeros_like(s["w"])
    if own:
        import eviction_gb300 as kvc
        s["h"] = kvc.Handle(kvc.Config(c.get("L", 1), B, H, c.get("G", 1), c.get("d", 64), max(c.get("hi", 1), 1),
                                       c.get("budget", 1), window=1, n_sink=SINKS, n_recent=RECENT))
        if op == "rotary":
            s["rope"] = kvc.Rope(c["dim"], base=c["base"], interleaved=c["interleaved"], scaling=c["scaling"],
                                 factor=c["factor"], low=LOW, high=HIGH, original=ORIGINAL)
        if op == "weigh":
            s["cache"] = kvc.Cache8(s["kp"], s["vp"], s["ks"], s["vs"], s["table"], length, s["free"], s["top"], s["ref"])
    return s


LOW, HIGH, ORIGINAL = 1.0, 4.0, 8192  # turns over ORIGINAL tokens between which frequencies go from scaled to unscaled
SINKS, RECENT = 4, 64


# ------------------------------------------------------------------- runs ----

def run(s):
    return _own(s) if own else PLAIN[s["c"]["op"]](s)


def _own(s):
    h, op = s["h"], s["c"]["op"]
    if op == "rotary":
        h.rotary(s["rope"], s["pos"], s["q"], s["k"], s["q_out"], s["k_out"], n_tok=s["length"])
        return s["q_out"], s["k_out"]
    if op == "prompt":
        h.prompt_attend(s["q"], s["k"], s["v"], s["out"], lse=s["lse"], first=s["first"], n_tok=s["length"])
        return s["out"], s["lse"]
    if op == "weigh":
        h.cache8_weigh(s["cache"], s["q"], s["lse"], s["w"], n_q=s["n_q"], decay=s["c"]["decay"])
        return s["w"]
    h.keep_heaviest(s["w"], s["length"], s["kept"], s["n_kept"], s["w_out"])
    return s["kept"], s["n_kept"], s["w_out"]


# ------------------------------------------------------------ plain forms ----

def _plain_rotary(s):
    c = s["c"]
    dim, half = c["dim"], c["dim"] // 2
    i = torch.arange(half, dtype=torch.float64, device="cuda")
    base = c["base"] * (c["factor"] ** (dim / (dim - 2)) if c["scaling"] == "ntk" else 1.0)
    f = base ** (-2 * i / dim)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "bands":
        mix = ((ORIGINAL * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = (1 - mix) * f / c["factor"] + mix * f
    angle = (s["pos"].double()[..., None] * f)[None, :, None]  # far positions: in 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    there = (torch.arange(c["n"], device="cuda") < s["length"][:, None])[None, :, None, :, None]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        x = x.float()
        turn, rest = x[..., :dim], x[..., dim:]
        if c["interleaved"]:
            a, b = turn[..., 0::2], turn[..., 1::2]
            y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = turn[..., :half], turn[..., half:]
            y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        out.copy_(torch.where(there, torch.cat((y, rest), -1), out.float()))
    return s["q_out"], s["k_out"]


def _padded(s, x, T):
    """Rows [heads, N, d] of packed sequences, or [B, heads, N, d], as [B, heads, T, d] in 32 bits, zeros behind."""
    there = (torch.arange(T, device="cuda") < s["length"][:, None])[:, None, :, None]
    if s["first"] is not None:
        at = (s["first"].long()[:, None] + torch.arange(T, device="cuda")).clamp(max=x.shape[1] - 1)
        x = x[:, at].transpose(0, 1)
    return torch.where(there, x.float(), 0)


def _plain_prompt(s):
    c = s["c"]
    B, H, G, d, T = c["B"], c["H"], c["G"], c["d"], c["hi"]
    q, k, v = (_padded(s, s[x], T) for x in "qkv")
    z = (q * d ** -0.5).reshape(B, H, G * T, d) @ k.transpose(-1, -2)
    z = z.reshape(B, H, G, T, T)
    t = torch.arange(T, device="cuda")
    z.masked_fill_(t > t[:, None], -torch.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = ((p.reshape(B, H, G * T, T) @ v).reshape(B, H, G, T, d) / total).reshape(B, H * G, T, d)
    lse = (top + total.log()).reshape(B, H * G, T)
    there = t < s["length"][:, None]  # [B, T]
    if s["first"] is None:
        s["out"].copy_(torch.where(there[:, None, :, None], out, s["out"].float()))
        s["lse"].copy_(torch.where(there[:, None], lse, s["lse"]))
    else:
        at = (s["first"].long()[:, None] + t)[there]
        s["out"][:, at] = out.transpose(1, 2)[there].transpose(0, 1).to(torch.bfloat16)
        s["lse"][:, at] = lse.transpose(1, 2)[there].transpose(0, 1)
    return s["out"], s["lse"]


def _scores(s):
    """[B, H, G, n, T] scaled products of the queries with the cache's keys, -inf where a query does not see."""
    c = s["c"]
    B, H, G, d, n, bs, T = c["B"], c["H"], c["G"], c["d"], c["n"], c["bs"], c["hi"]
    t = torch.arange(T, device="cuda")
    blk = s["table"].long()[:, t // bs].clamp(min=0)  # [B, T]
    k = s["kp"][0].view(torch.uint8)[blk, :, t % bs].view(s["kp"].dtype).float() * s["ks"][0][blk][..., None]
    z = (s["q"][0].float() * d ** -0.5).reshape(B, H, G * n, d) @ k.permute(0, 2, 3, 1)
    last = (s["length"] - s["n_q"])[:, None] + torch.arange(n, device="cuda")  # the last token that a query sees
    return z.reshape(B, H, G, n, T).masked_fill_((t > last[..., None])[:, None, None], -torch.inf)


def _plain_weigh(s):
    c = s["c"]
    p = (_scores(s) - s["lse"].reshape(*s["lse"].shape[1:2], c["H"], c["G"], c["n"], 1)).exp()
    there = (torch.arange(c["n"], device="cuda") < s["n_q"][:, None])[:, None, None, :, None]
    new = torch.where(there, p, 0).sum((2, 3))
    held = (torch.arange(c["hi"], device="cuda") < s["length"][:, None])[:, None]
    s["w"][0] = torch.where(held, s["w"][0] * c["decay"] + new, s["w"][0])
    return s["w"]


def _plain_heaviest(s):
    c = s["c"]
    T, K = c["hi"], c["budget"]
    t = torch.arange(T, device="cuda")
    length = s["length"][:, None, None]
    recent = min(RECENT, K)
    must = (t >= length - recent) | (t < min(SINKS, K - recent))
    w = s["w"].masked_fill(must, torch.inf).masked_fill(t >= length, -torch.inf)
    order = w.argsort(dim=-1, descending=True, stable=True)  # equal weights: the lowest slot first
    n = length.clamp(max=K)
    order = torch.nn.functional.pad(order[..., :K], (0, max(0, K - T)), value=T)
    slots = torch.where(torch.arange(K, device="cuda") < n, order, T).sort(-1).values
    s["kept"].copy_(torch.where(slots < T, slots, -1))
    s["n_kept"].copy_(n[None, :, :, 0].expand_as(s["n_kept"]))
    got = torch.where(slots < T, s["w"].gather(-1, slots.clamp(max=T - 1)), 0)
    s["w_out"].copy_(torch.nn.functional.pad(got[..., :T], (0, max(0, T - K))))
    return s["kept"], s["n_kept"], s["w_out"]


PLAIN = {"rotary": _plain_rotary, "prompt": _plain_prompt, "weigh": _plain_weigh, "heaviest": _plain_heaviest}


# ------------------------------------------------------------------ exact ----

def exact(c, seed):
    """From the definitions, in 64 bits, on the state that prepare() makes."""
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    return {"rotary": _exact_rotary, "prompt": _exact_prompt, "weigh": _exact_weigh, "heaviest": _exact_heaviest}[c["op"]](s)


def _exact_frequency(c, i):
    """Radians a token of pair i."""
    f = math.pow(c["base"], -2.0 * i / c["dim"])
    if c["scaling"] == "linear":
        return f / c["factor"]
    if c["scaling"] == "ntk":
        return math.pow(c["base"] * math.pow(c["factor"], c["dim"] / (c["dim"] - 2.0)), -2.0 * i / c["dim"])
    if c["scaling"] == "bands":
        turns = ORIGINAL * f / (2.0 * math.pi)
        if turns >= HIGH:
            return f
        if turns <= LOW:
            return f / c["factor"]
        part = (turns - LOW) / (HIGH - LOW)
        return part * f + (1.0 - part) * f / c["factor"]
    return f


def _exact_rotary(s):
    c, got = s["c"], []
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = out.double().contiguous()
        for b, m in enumerate(_lens(c)):
            z = x[0, b, :, :m].double()
            f = torch.tensor([_exact_frequency(c, i) for i in range(c["dim"] // 2)], dtype=torch.float64, device="cuda")
            e = torch.polar(torch.ones((m, len(f)), dtype=torch.float64, device="cuda"), s["pos"][b, :m].double()[:, None] * f)
            pair = torch.arange(c["dim"] // 2, device="cuda")
            i, j = (2 * pair, 2 * pair + 1) if c["interleaved"] else (pair, pair + c["dim"] // 2)
            r = torch.complex(z[..., i], z[..., j]) * e
            z[..., i], z[..., j] = r.real, r.imag
            y[0, b, :, :m] = z
        got.append(y)
    return tuple(got)


def _exact_prompt(s):
    c = s["c"]
    G, d = c["G"], c["d"]
    out, lse = s["out"].double().contiguous(), s["lse"].double()
    for b, m in enumerate(_lens(c)):
        lo = 0 if s["first"] is None else int(s["first"][b])
        q, k, v = (x[:, lo:lo + m] for x in ((s["q"], s["k"], s["v"]) if s["first"] is not None else (s["q"][b], s["k"][b], s["v"][b])))
        o, a = (out, lse) if s["first"] is not None else (out[b], lse[b])
        for h in range(c["H"]):
            kh, vh = k[h].double(), v[h].double()
            for r0 in range(0, m, 4096):
                r1 = min(m, r0 + 4096)
                sees = torch.arange(r1, device="cuda") <= torch.arange(r0, r1, device="cuda")[:, None]
                for g in range(G):
                    z = q[h * G + g, r0:r1].double() @ kh[:r1].T / math.sqrt(d)
                    z = torch.where(sees, z, -torch.inf)
                    norm = torch.logsumexp(z, -1)
                    a[h * G + g, lo + r0:lo + r1] = norm
                    o[h * G + g, lo + r0:lo + r1] = torch.exp(z - norm[:, None]) @ vh[:r1]
    return out, lse


def _exact_weigh(s):
    c = s["c"]
    G, bs = c["G"], c["bs"]
    w = s["w"].double()
    for b, m in enumerate(_lens(c)):
        n = _queries(c, m)
        blocks = s["table"][b, : -(-m // bs)].long()
        k = s["kp"][0].view(torch.uint8)[blocks].view(s["kp"].dtype).to(torch.float64) * s["ks"][0][blocks].double()[:, :, None, None]
        for h in range(c["H"]):
            key = k[:, h].reshape(-1, c["d"])[:m]
            total = torch.zeros(m, dtype=torch.float64, device="cuda")
            for g in range(G):
                z = s["q"][0, b, h * G + g, :n].double() @ key.T / math.sqrt(c["d"]) - s["lse"][0, b, h * G + g, :n].double()[:, None]
                total += torch.exp(z).tril(m - n).sum(0)
            w[0, b, h, :m] = c["decay"] * w[0, b, h, :m] + total
    return w


def _exact_heaviest(s):
    """The kept slots are whole numbers, which the plain form gives too; the weights that go with them are copies."""
    c = s["c"]
    T, K = c["hi"], c["budget"]
    w = s["w"].double()
    t, n = torch.arange(T, device="cuda"), s["length"].long()[:, None, None]
    tail = min(RECENT, K)
    must = ((t >= n - tail) | (t < min(SINKS, K - tail))) & (t < n)
    other = ((t < n) & ~must).expand(w.shape)
    want = (n.clamp(max=K) - must.sum(-1, keepdim=True)).expand(w.shape[:-1] + (1,))  # of the others
    least = torch.where(other, w, -1).sort(-1, descending=True).values.gather(-1, (want - 1).clamp(min=0))
    more, equal = other & (w > least), other & (w == least)
    keep = must | ((more | (equal & (equal.cumsum(-1) <= want - more.sum(-1, keepdim=True)))) & (want > 0))
    w_out = torch.zeros_like(w)
    unit, slot = keep.reshape(-1, T).nonzero(as_tuple=True)
    place = keep.reshape(-1, T).cumsum(-1)[unit, slot] - 1
    w_out.reshape(-1, T)[unit, place] = w.reshape(-1, T)[unit, slot]
    return None, None, w_out
