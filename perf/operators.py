"""Cases and plain forms of the 8-bit paged cache operators.

A cache holds keys and values as 8-bit codes in pages ("blocks") of `bs` tokens, with one power-of-two scale
for each block and head: pools [L, n_blocks, H, bs, d], scales [L, n_blocks, H], one block table per sequence
shared by all layers.  A code stands for code * scale; codes are e4m3 floats or signed 8-bit integers, and the
scale of a block is the smallest power of two (2^-64 at least, 2^64 at most) under which the largest finite
magnitude of its rows is at most 448 (e4m3) or 127 (int8).  Five operators:

  append   quantise the newest tokens' keys and values into their blocks
  attend   softmax attention of the newest tokens' queries over the cache
  gather   the cache as dense, left-padded bf16 rows (what the compression event reads)
  compact  the rows that an event kept, per head, requantised into new blocks
  pages    block tables: free sequences, grow them, fork them (full blocks shared, a started one copied)

Shapes: the 28-layer Qwen-7B-shaped, the Llama-8B-shaped and the long-context workloads of this repository.
"""
import torch

own = False

E_MIN, E_MAX = -64, 64
TOP = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one sequence, one head: the smallest decode step, where only latency counts
        dict(name="attend_tiny", op="attend", L=1, B=1, H=1, G=1, d=64, bs=16, fmt="e4m3", lo=768, hi=768, n=1),
        # one layer of a decode step of the Llama-shaped ragged batch
        dict(name="attend_ragged", op="attend", L=1, B=64, H=8, G=4, d=128, bs=16, fmt="e4m3", lo=612, hi=1112, n=1),
        # one layer of a decode step over the long-context caches (few units, a long axis)
        dict(name="attend_long", op="attend", L=1, B=4, H=4, G=7, d=128, bs=64, fmt="int8", lo=32768, hi=32768, n=1),
        # one layer of a chunk of 128 new tokens (prompt in pieces) over Qwen-shaped caches
        dict(name="attend_chunk", op="attend", L=1, B=32, H=4, G=7, d=128, bs=16, fmt="e4m3", lo=1024, hi=1536, n=128),
        # one layer of a decode step: one new token for each of 32 sequences
        dict(name="append_step", op="append", L=1, B=32, H=4, G=7, d=128, bs=16, fmt="int8", lo=1024, hi=1535, n=1),
        # one layer of a long prompt's pieces: 4000 new tokens a sequence, starting inside a block
        dict(name="append_prompt", op="append", L=1, B=8, H=8, G=4, d=128, bs=16, fmt="e4m3", lo=4100, hi=4611, n=4000),
        # one layer of the ragged batch made dense for an event
        dict(name="gather_ragged", op="gather", L=1, B=64, H=8, G=4, d=128, bs=16, fmt="int8", lo=612, hi=1112),
        # every layer of a Qwen-shaped batch made dense for an event
        dict(name="gather_event", op="gather", L=28, B=8, H=4, G=7, d=128, bs=16, fmt="e4m3", lo=1536, hi=1536),
        # the ragged batch's event, one layer, 1112 -> 512 slots
        dict(name="compact_ragged", op="compact", L=1, B=64, H=8, G=4, d=128, bs=16, fmt="e4m3", lo=612, hi=1112,
             budget=512),
        # the Qwen-shaped event over all layers, 1536 -> 1024 slots
        dict(name="compact_event", op="compact", L=28, B=8, H=4, G=7, d=128, bs=16, fmt="e4m3", lo=1536, hi=1536,
             budget=1024),
        # a batch of sequences ends and the next one is admitted
        dict(name="pages_admit", op="admit", L=1, B=64, H=1, G=4, d=64, bs=16, fmt="int8", lo=100, hi=1112),
        # eight samples of each of eight prompts end and eight new ones start from the prompts' caches
        dict(name="pages_fork", op="fork", L=28, B=72, H=4, G=7, d=128, bs=64, fmt="e4m3", lo=900, hi=1500,
             parents=8),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["attend", "attend", "chunk", "append", "gather", "compact", "admit", "fork"])
    c = dict(op="attend" if op == "chunk" else op, L=1, H=rng.choice([1, 2, 4, 8]), G=rng.randint(1, 8),
             d=rng.choice([64, 128]), bs=rng.choice([8, 16, 16, 24, 32, 64, 128]), fmt=rng.choice(["e4m3", "int8"]))
    if op == "attend":
        c["B"] = log(1, 64)
        c["hi"] = log(64, min(32768, 524288 // (c["B"] * c["H"])))
        c["n"] = rng.choice([1, 1, 1, 2, 3, 4])
        c["lo"] = max(c["n"], int(c["hi"] * rng.choice([1.0, 0.7, 0.2])))
    elif op == "chunk":
        c["B"] = log(1, 16)
        c["n"] = log(5, 128)
        c["hi"] = log(c["n"] + 8, max(c["n"] + 9, min(4096, 140_000_000 // (c["B"] * c["H"] * c["G"] * c["n"]))))
        c["lo"] = max(c["n"], int(c["hi"] * rng.choice([1.0, 0.6])))
    elif op == "append":
        c["B"] = log(1, 32)
        c["n"] = rng.choice([1, 1, log(2, min(4000, 250_000 // (c["B"] * c["H"])))])
        c["lo"] = c["n"] + rng.randint(0, 500)
        c["hi"] = c["lo"] + rng.randint(0, 300)
    elif op in ("gather", "compact"):
        c["L"] = rng.choice([1, 1, 2, 4])
        c["B"] = log(1, 32)
        c["hi"] = log(64, min(4096, 1_300_000 // (c["L"] * c["B"] * c["H"])))
        c["lo"] = max(1, int(c["hi"] * rng.choice([1.0, 0.5])))
        if op == "compact":
            c["budget"] = max(8, c["hi"] // rng.choice([2, 3, 8]))
    elif op == "admit":
        c["H"], c["d"] = 1, 64
        c["B"] = log(2, 128)
        c["hi"] = log(32, 2048)
        c["lo"] = max(1, c["hi"] // 5)
    else:
        c["L"], c["H"], c["bs"] = rng.choice([1, 4, 8]), min(4, c["H"]), min(64, c["bs"])
        c["parents"] = rng.randint(1, 8)
        c["B"] = c["parents"] * (1 + rng.randint(1, 8))
        c["hi"] = log(32, 1500)
        c["lo"] = max(1, c["hi"] // 2)
    return c


def _lens(c):
    """The sequences' lengths: spread over [lo, hi] in a scattered order, the same for every seed."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    n = c.get("parents", B)
    got = [hi if n == 1 else lo + (hi - lo) * ((i * 37 + 11) % n) // (n - 1) for i in range(n)]
    if "parents" in c:  # the children: as many for each parent, one after another
        k = B // n - 1
        got += [got[i // k] for i in range(n * k)]
    return got


def work(c):
    """Bytes: codes (1 each), scales (4), bf16 rows (2), tables and indices (4).  Flops: the products."""
    L, B, H, G, d, bs = c["L"], c["B"], c["H"], c["G"], c["d"], c["bs"]
    lens = _lens(c)
    blocks = sum(-(-n // bs) for n in lens)
    tokens = sum(lens)
    if c["op"] == "attend":
        n = c["n"]
        seen = sum(n * m - n * (n - 1) // 2 for m in lens)
        cache = 2 * L * H * (tokens * d + blocks * 4) + blocks * 4
        return {"bytes": cache + L * B * H * G * n * (4 * d + 4), "flops": 4.0 * L * H * G * d * seen}
    if c["op"] == "append":
        n = c["n"]
        touched = sum(-(-m // bs) - (m - n) // bs for m in lens)
        return {"bytes": 2 * L * H * (B * n * d * 3 + touched * 4) + touched * 4, "flops": 0}
    if c["op"] == "gather":
        T = max(lens)
        return {"bytes": 2 * L * H * (tokens * d + blocks * 4 + B * T * d * 2) + blocks * 4, "flops": 0}
    if c["op"] == "compact":
        kept = sum(min(m, c["budget"]) for m in lens)
        new = sum(-(-min(m, c["budget"]) // bs) for m in lens)
        rows = kept * (2 * 2 * d + 4 + 8)  # codes read and written, the index, the credit read and written
        return {"bytes": L * H * (rows + 2 * (blocks + new) * 4) + (blocks + new) * 4, "flops": 0}
    if c["op"] == "admit":  # table entries read and written, stack and counts too
        return {"bytes": blocks * 4 * 8, "flops": 0}
    kids = lens[c["parents"]:]
    return {"bytes": 2 * L * H * sum(2 * (m % bs) * d + (8 if m % bs else 0) for m in kids)
            + sum(-(-m // bs) for m in kids) * 4 * 8, "flops": 0}


# ----------------------------------------------------------------- inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(shape, g, spread=0.0):
    """N(0, 1) rows in bf16; with `spread`, a factor 2^(spread * N(0, 1)) for each row."""
    x = torch.randn(shape, generator=g, device="cuda")
    if spread:
        x *= torch.exp2(spread * torch.randn((*shape[:-1], 1), generator=g, device="cuda"))
    return x.to(torch.bfloat16)


def _pool(L, N, H, bs, d, fmt, g):
    """A pool whose every row holds codes of N(0, 1) rows, and its scales."""
    codes = torch.empty((L, N, H, bs, d), dtype=torch.uint8, device="cuda")
    scale = torch.empty((L, N, H), device="cuda")
    for i in range(L):
        x = _bf16((N, H, bs, d), g, 0.4).float()
        s = _scale(x.abs().amax((-1, -2)), fmt)
        scale[i] = s
        codes[i] = _codes(x / s[..., None, None], fmt).view(torch.uint8)
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8), scale


def prepare(c, seed):
    g = _gen(seed)
    L, B, H, G, d, bs, fmt, op = (c[k] for k in ("L", "B", "H", "G", "d", "bs", "fmt", "op"))
    lens = _lens(c)
    dev = dict(dtype=torch.int32, device="cuda")
    P = c.get("parents", B)
    held = [-(-m // bs) for m in lens]
    M = max(held) + 1
    kept = [min(m, c["budget"]) for m in lens] if op == "compact" else []
    length = torch.tensor(lens, **dev)
    cols = torch.arange(M, **dev)
    nb = (length + bs - 1) // bs
    seq = torch.arange(B, device="cuda")
    shares = torch.where(seq < P, 0, length // bs)  # a child has its parent's full blocks
    used = sum(held[:P]) + sum(m % bs > 0 for m in lens[P:])
    N = used + sum(-(-m // bs) for m in kept) + 5
    perm = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    alone = nb - shares
    at = (alone.cumsum(0) - alone)[:, None] + cols - shares[:, None]
    table = torch.where(cols < nb[:, None], perm[at.clamp(0, N - 1).long()], -1)
    mother = torch.where(seq < P, seq, (seq - P) // max(1, B // P - 1))
    table = torch.where(cols < shares[:, None], table[mother], table)
    ref = torch.zeros(N, **dev)
    _count(ref, table, 1)
    free = torch.where(torch.arange(N, device="cuda") < N - used, perm.flip(0), 0).to(torch.int32)
    top = torch.tensor(N - used, **dev)
    kp, ks = _pool(L, N, H, bs, d, fmt, g)
    vp, vs = _pool(L, N, H, bs, d, fmt, g)
    s = dict(c=c, kp=kp, vp=vp, ks=ks, vs=vs, table=table.to(torch.int32).contiguous(), length=length, free=free,
             top=top.to(torch.int32).reshape(1), ref=ref)
    if op == "attend":
        n = c["n"]
        # queries as a projection leaves them, token-major; each leans on a few of its cache's keys
        q = _bf16((L, B, n, H * G, d), g).float()
        at = (torch.rand((B, 3), generator=g, device="cuda") * length[:, None]).long()
        keys = _values(kp.view(torch.uint8)[:, table.long().gather(1, at // bs), :, at % bs], fmt)  # [B,3,L,H,d]
        lean = keys.sum(1).permute(1, 0, 2, 3).repeat_interleave(G, 2)  # codes: their direction is what counts
        lean = lean / lean.square().mean(-1, keepdim=True).sqrt().clamp(min=1e-6)
        q += 0.4 * torch.randn((L, B, n, H * G, 1), generator=g, device="cuda").abs() * lean[:, :, None]
        s["q"] = q.to(torch.bfloat16).permute(0, 1, 3, 2, 4)
        s["out"] = torch.zeros((L, B, n, H * G, d), dtype=torch.bfloat16, device="cuda").permute(0, 1, 3, 2, 4)
        s["lse"] = torch.zeros((L, B, H * G, n), device="cuda")
        # what lies behind a sequence's end is no one's: whatever was there last, NaN codes among it
        last = (length - 1) // bs
        behind = table.gather(1, last.long()[:, None])[:, 0].long()
        stale = (torch.arange(bs, device="cuda") > ((length - 1) % bs)[:, None])[None, :, None, :, None]
        for p in (kp, vp):
            u = p.view(torch.uint8)
            u[:, behind] = torch.where(stale, 255, u[:, behind])
    elif op == "append":
        s["k"], s["v"] = (_bf16((L, B, c["n"], H, d), g, 0.5).permute(0, 1, 3, 2, 4) for _ in "kv")
        s["n_new"] = torch.full((B,), c["n"], **dev)
    elif op == "gather":
        T = max(lens)
        s["pad"] = torch.zeros(B, **dev)
        s["out"] = tuple(torch.zeros((L, B, H, T, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    elif op == "compact":
        T, K = max(lens), c["budget"]
        s["pad"] = T - length
        keep = torch.minimum(length, torch.tensor(K, **dev))
        score = torch.rand((L, B, H, T), generator=g, device="cuda")
        score = score.masked_fill(torch.arange(T, device="cuda") < s["pad"][:, None, None], -1)
        idx = score.topk(min(K, T), -1).indices
        held_k = torch.arange(idx.shape[-1], device="cuda") < keep[:, None, None]
        idx = torch.where(held_k, idx, T).sort(-1).values
        s["kept"] = torch.full((L, B, H, K), -1, **dev)
        s["kept"][..., : idx.shape[-1]] = torch.where(idx < T, idx, -1).to(torch.int32)
        s["n_kept"] = keep[None, :, None].expand(L, B, H).contiguous()
        s["credit"] = torch.rand((L, B, H, T), generator=g, device="cuda")
        s["credit_out"] = torch.zeros((L, B, H, K), device="cuda")
        s["new_table"], s["new_length"] = torch.full((B, M), -1, **dev), torch.zeros(B, **dev)
        _grow(s["new_table"], s["new_length"], s["free"], s["top"], s["ref"], keep, bs)
    elif op == "admit":
        s["n_new"], s["all"] = length.clone(), torch.arange(B, **dev)
    else:
        s["kids"] = torch.arange(P, B, **dev)
        s["mothers"] = (torch.arange(B - P, **dev) // (B // P - 1)).to(torch.int32)
    if own:
        import eviction_gb300 as kvc
        s["h"] = kvc.Handle(kvc.Config(L, B, H, G, d, max(lens), c.get("budget", 1), window=max(1, c.get("n", 1)) if
                                       op == "attend" else 1, n_recent=0))
        s["cache"] = kvc.Cache8(kp, vp, ks, vs, s["table"], length, free, s["top"], ref)
        if op == "compact":
            s["new"] = kvc.Cache8(kp, vp, ks, vs, s["new_table"], s["new_length"], free, s["top"], ref)
    return s


# ------------------------------------------------------------------- runs ----

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    h, cache, op = s["h"], s["cache"], s["c"]["op"]
    if op == "attend":
        h.cache8_attend(cache, s["q"], s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "append":
        h.cache8_append(cache, s["k"], s["v"], s["n_new"])
        return s["kp"], s["vp"], s["ks"], s["vs"]
    if op == "gather":
        h.cache8_gather(cache, s["out"][0].shape[3], s["pad"], s["out"][0], s["out"][1])
        return s["out"], s["pad"]
    if op == "compact":
        h.cache8_compact(cache, s["new"], s["credit"].shape[3], s["pad"], s["kept"], s["n_kept"],
                         credit_post=s["credit"], credit_out=s["credit_out"])
        return s["kp"], s["vp"], s["ks"], s["vs"], s["credit_out"]
    if op == "admit":
        h.cache8_free(cache, s["all"])
        h.cache8_grow(cache, s["n_new"])
    else:
        h.cache8_free(cache, s["kids"])
        h.cache8_fork(cache, s["mothers"], s["kids"])
    return _pages(s)


def _pages(s):
    got = [s["table"], s["length"], s["free"], s["top"], s["ref"]]
    return got + ([s["kp"], s["vp"], s["ks"], s["vs"]] if s["c"]["op"] == "fork" else [])


# ------------------------------------------------------------ plain forms ----

def _values(codes, fmt):
    """fp32 values of uint8-held codes (without the scale)."""
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).to(torch.float32)


def _codes(x, fmt):
    """Codes of x (already divided by the scale), nearest, ties to even."""
    if fmt == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn)
    return x.round().clamp(-127, 127).to(torch.int8)


def _scale(amax, fmt):
    """The smallest power of two in [2^E_MIN, 2^E_MAX] with amax / scale <= TOP."""
    m, x = torch.frexp(amax)  # amax = m 2^x, m in [0.5, 1)
    edge, base = (0.875, 9) if fmt == "e4m3" else (0.9921875, 7)  # TOP = edge 2^base
    e = (x - base + (m > edge)).clamp(E_MIN, E_MAX)
    e = torch.where(amax == 0, torch.full_like(e, E_MIN), e)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _rows(pool, scale, blk, r, fmt):
    """fp32 rows [B, T, L, H, d] at blocks blk [B, T], rows r [B, T]."""
    return _values(pool.view(torch.uint8)[:, blk, :, r], fmt) * scale[:, blk].permute(1, 2, 0, 3)[..., None]


def _blocks_at(s, pos):
    bs = s["c"]["bs"]
    return s["table"].long().gather(1, (pos // bs).clamp(0, s["table"].shape[1] - 1)).clamp(min=0), pos % bs


def _plain(s):
    c = s["c"]
    op = c["op"]
    if op == "attend":
        return _plain_attend(s)
    if op == "append":
        return _plain_append(s)
    if op == "gather":
        return _plain_gather(s)
    if op == "compact":
        return _plain_compact(s)
    if op == "admit":
        _free(s["table"], s["length"], s["free"], s["top"], s["ref"], s["all"])
        _grow(s["table"], s["length"], s["free"], s["top"], s["ref"], s["n_new"], c["bs"])
    else:
        _free(s["table"], s["length"], s["free"], s["top"], s["ref"], s["kids"])
        _fork(s)
    return _pages(s)


def _plain_attend(s):
    c = s["c"]
    L, B, H, G, d, n = (c[k] for k in ("L", "B", "H", "G", "d", "n"))
    T = c["hi"]
    t = torch.arange(T, device="cuda").expand(B, T)
    blk, r = _blocks_at(s, t)
    there = (t < s["length"][:, None])[:, :, None, None, None]
    k = torch.where(there, _rows(s["kp"], s["ks"], blk, r, c["fmt"]), 0).permute(2, 0, 3, 1, 4)  # [L,B,H,T,d]
    v = torch.where(there, _rows(s["vp"], s["vs"], blk, r, c["fmt"]), 0).permute(2, 0, 3, 1, 4)
    q = s["q"].float().reshape(L, B, H, G * n, d) * d ** -0.5
    z = (q @ k.transpose(-1, -2)).reshape(L, B, H, G, n, T)
    last = s["length"][:, None] - n + torch.arange(n, device="cuda")  # the last position that query j sees
    sees = (t[:, None] <= last[:, :, None])[None, :, None, None]
    z = z.masked_fill(~sees, -torch.inf)
    top = z.amax(-1, keepdim=True)
    p = (z - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p.reshape(L, B, H, G * n, T) @ v).reshape(L, B, H, G, n, d) / total
    return (out.reshape(L, B, H * G, n, d).to(torch.bfloat16),
            (top + total.log()).reshape(L, B, H * G, n))


def _plain_append(s):
    c = s["c"]
    bs, n, fmt, B = c["bs"], c["n"], c["fmt"], c["B"]
    start = s["length"].long() - n
    first = start // bs
    nb = (n + bs - 2) // bs + 1  # blocks that n tokens can touch
    w = torch.arange(nb * bs, device="cuda")
    pos = (first[:, None] * bs + w).clamp(max=s["length"][:, None].long() - 1)  # past the end: the last row again
    w = pos - first[:, None] * bs
    blk, r = _blocks_at(s, pos)
    new = pos >= start[:, None]
    from_new = (pos - start[:, None]).clamp(min=0)
    seen = w // bs  # block of the row, among the touched ones
    head = (first * bs < start)[:, None] & (torch.arange(nb, device="cuda") == 0)  # blocks with older rows
    blk0 = _blocks_at(s, (first[:, None] + torch.arange(nb, device="cuda")) * bs)[0]
    last = (s["length"].long() - 1) // bs - first  # the last block touched
    held = torch.arange(nb, device="cuda") <= last[:, None]
    blk0 = torch.where(held, blk0, blk0.gather(1, last[:, None]))
    for pool, scale, x in ((s["kp"], s["ks"], s["k"]), (s["vp"], s["vs"], s["v"])):
        x = x.permute(1, 3, 0, 2, 4).float()  # [B, n, L, H, d]
        x = x[torch.arange(B, device="cuda")[:, None], from_new]
        x = torch.where(new[..., None, None, None], x, _rows(pool, scale, blk, r, fmt))
        # largest new magnitude of each touched block (an old row counts through the old scale)
        a = torch.where(new[..., None, None], x.abs().amax(-1), 0)  # [B, W, L, H]
        a = torch.zeros((B, nb, *a.shape[2:]), device="cuda").scatter_reduce(
            1, seen[..., None, None].expand(a.shape), a, "amax")
        sc = _scale(a, fmt)
        old = torch.where(head[..., None, None], scale[:, blk0].permute(1, 2, 0, 3), 0)
        sc = torch.maximum(sc, old)
        sc = torch.where(held[..., None, None], sc, sc.gather(1, last[:, None, None, None].expand(B, 1, *sc.shape[2:])))
        x = x / sc.gather(1, seen[..., None, None].expand(*seen.shape, *sc.shape[2:]))[..., None]
        pool.view(torch.uint8)[:, blk, :, r] = _codes(x, fmt).view(torch.uint8)
        scale[:, blk0] = sc.permute(2, 0, 1, 3)
    return s["kp"], s["vp"], s["ks"], s["vs"]


def _plain_gather(s):
    c = s["c"]
    B, T = c["B"], s["out"][0].shape[3]
    pad = T - s["length"]
    pos = torch.arange(T, device="cuda") - pad[:, None].long()
    blk, r = _blocks_at(s, pos.clamp(min=0))
    there = (pos >= 0)[..., None, None, None]
    got = tuple(torch.where(there, _rows(p, sc, blk, r, c["fmt"]), 0).to(torch.bfloat16).permute(2, 0, 3, 1, 4)
                for p, sc in ((s["kp"], s["ks"]), (s["vp"], s["vs"])))
    return got, pad.to(torch.int32)


def _plain_compact(s):
    c = s["c"]
    L, B, H, d, bs, K, fmt = (c[k] for k in ("L", "B", "H", "d", "bs", "budget", "fmt"))
    nb = -(-K // bs)
    keep = s["new_length"].long()
    j = torch.arange(nb * bs, device="cuda").expand(B, -1)
    j = torch.minimum(j, keep[:, None] - 1)  # past the end: the last row again
    row = j[None, :, None].expand(L, B, H, -1)
    slot = s["kept"].long().gather(3, row)
    pos = slot - s["pad"].long()[:, None, None]
    li = torch.arange(L, device="cuda")[:, None, None, None]
    bi = torch.arange(B, device="cuda")[:, None, None]
    hi = torch.arange(H, device="cuda")[:, None]
    src = s["table"].long()[bi, pos // bs]
    dst = s["new_table"].long()[bi, row // bs]
    for pool, scale in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
        u = pool.view(torch.uint8)
        x = _values(u[li, src, hi, pos % bs], fmt) * scale[li, src, hi][..., None]
        a = torch.zeros((L, B, H, nb), device="cuda").scatter_reduce(3, row // bs, x.abs().amax(-1), "amax")
        sc = _scale(a, fmt).gather(3, row // bs)
        u[li, dst, hi, row % bs] = _codes(x / sc[..., None], fmt).view(torch.uint8)
        scale[li, dst, hi] = sc
    at = torch.arange(K, device="cuda")
    credit = s["credit"].gather(3, s["kept"].clamp(min=0).long())
    return s["kp"], s["vp"], s["ks"], s["vs"], torch.where(at < s["n_kept"][..., None], credit, 0)


def _count(ref, table, by):
    """ref[block] += by for every entry of `table` that is a block."""
    e = table.reshape(-1)
    ref.scatter_add_(0, e.clamp(min=0).long(), torch.where(e >= 0, by, 0).to(ref.dtype))


def _grow(table, length, free, top, ref, n_new, bs):
    B, M = table.shape
    cols = torch.arange(M, device="cuda")
    have, want = (length + bs - 1) // bs, (length + n_new + bs - 1) // bs
    need = want - have
    base = top - need.sum()
    at = base + (need.cumsum(0) - need)[:, None] + cols - have[:, None]
    new = (cols >= have[:, None]) & (cols < want[:, None])
    table.copy_(torch.where(new, free[at.clamp(0, free.numel() - 1).long()], table))
    _count(ref, torch.where(new, table, -1), 1)
    top.copy_(base)
    length += n_new


def _free(table, length, free, top, ref, seqs):
    """Entries in list order; a block is pushed where its last holder among them stands."""
    e = table[seqs.long()].reshape(-1)
    is_block = e >= 0
    _count(ref, e, -1)
    at = torch.arange(e.numel(), device="cuda")
    lastly = torch.full_like(ref, -1, dtype=torch.int64).scatter_reduce(
        0, e.clamp(min=0).long(), torch.where(is_block, at, -1), "amax")
    push = is_block & (ref[e.clamp(min=0).long()] == 0) & (lastly[e.clamp(min=0).long()] == at)
    to = torch.where(push, top + push.cumsum(0) - 1, free.numel()).long()
    more = torch.cat([free, free[:1]])
    more.scatter_(0, to, e)
    free.copy_(more[:-1])
    top += push.sum()
    table[seqs.long()] = -1
    length[seqs.long()] = 0


def _fork(s):
    bs, free, top, ref, table, length = s["c"]["bs"], s["free"], s["top"], s["ref"], s["table"], s["length"]
    src, dst = s["mothers"].long(), s["kids"].long()
    n = length[src]
    full, part = n // bs, n % bs
    started = (part > 0).to(torch.int32)
    base = top - started.sum()
    block = free[(base + started.cumsum(0) - started).clamp(0, free.numel() - 1).long()]
    cols = torch.arange(table.shape[1], device="cuda")
    shared = torch.where(cols < full[:, None], table[src], -1)
    _count(ref, shared, 1)
    rows = torch.where((cols == full[:, None]) & (part > 0)[:, None], block[:, None], shared)
    _count(ref, torch.where(part > 0, block, -1), 1)
    old = table[src].gather(1, ((n - 1) // bs).clamp(min=0).long()[:, None])[:, 0].clamp(min=0).long()
    to = torch.where(part > 0, block.long(), old)  # nothing started: the block onto itself
    here = (torch.arange(bs, device="cuda") < part[:, None])[None, :, None, :, None]
    for pool, scale in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
        u = pool.view(torch.uint8)
        u[:, to] = torch.where(here, u[:, old], u[:, to])
        scale[:, to] = scale[:, old]
    table[dst] = rows
    length[dst] = n
    top.copy_(base)


# ------------------------------------------------------------------ exact ----

def exact(c, seed):
    """From the definitions, in 64 bits, on the state that prepare() makes."""
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    return {"attend": _exact_attend, "append": _exact_append, "gather": _exact_gather,
            "compact": _exact_compact}.get(c["op"], lambda s: None)(s)


def _exact_page(s, which, l, b, upto):
    """Rows [upto, H, d] of one sequence's cache in 64 bits."""
    bs = s["c"]["bs"]
    blocks = s["table"][b, : -(-upto // bs)].long()
    codes = s[which + "p"][l].view(torch.uint8)[blocks]  # [nb, H, bs, d]
    codes = codes.view(s[which + "p"].dtype).to(torch.float64) * s[which + "s"][l][blocks].double()[:, :, None, None]
    return codes.transpose(1, 2).reshape(-1, s["c"]["H"], s["c"]["d"])[:upto]


def _exact_attend(s):
    c = s["c"]
    G, n = c["G"], c["n"]
    out, lse = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda"), torch.zeros_like(s["lse"]).double()
    for l in range(c["L"]):
        for b, m in enumerate(s["length"].tolist()):
            k, v = _exact_page(s, "k", l, b, m), _exact_page(s, "v", l, b, m)
            for h in range(c["H"]):
                q = s["q"][l, b, h * G:(h + 1) * G].double().reshape(G * n, -1)
                z = (q @ k[:, h].T / c["d"] ** 0.5).reshape(G, n, m)
                z = z + torch.full((n, m), -torch.inf, dtype=torch.float64, device="cuda").triu(m - n + 1)
                a = torch.logsumexp(z, -1)
                lse[l, b, h * G:(h + 1) * G] = a
                out[l, b, h * G:(h + 1) * G] = torch.exp(z - a[..., None]) @ v[:, h]
    return out, lse


def _exact_code(x, fmt):
    """The nearest code of each x (64 bits, in units of the scale), ties to even, as the value it stands for."""
    if fmt == "int8":
        return x.round().clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)  # spacing of e4m3 around x
    return ((x / step).round() * step).clamp(-448, 448)


def _exact_scale(a, fmt):
    """Powers of two in turn until the largest magnitude fits."""
    s = torch.full_like(a, 2.0 ** E_MIN)
    for e in range(E_MIN, E_MAX):
        s = torch.where(a > TOP[fmt] * s, 2.0 ** (e + 1), s)
    return s


def _exact_out(s, pools, scales):
    """int8 codes are whole numbers, which the plain form gives too: only e4m3 pools have values here."""
    return (*(pools if s["c"]["fmt"] == "e4m3" else (None, None)), *scales)


def _exact_append(s):
    c = s["c"]
    bs, n, fmt = c["bs"], c["n"], c["fmt"]
    if c["L"] * c["B"] * (n // bs + 2) > 6000:
        return None
    pools, scales = [], []
    for w in "kv":
        pool, scale = s[w + "p"].to(torch.float64), s[w + "s"].double()
        for l in range(c["L"]):
            for b, m in enumerate(s["length"].tolist()):
                for i in range((m - n) // bs, -(-m // bs)):
                    lo, hi, at = max(i * bs, m - n), min(m, i * bs + bs), int(s["table"][b, i])
                    x = s[w][l, b, :, lo - (m - n):hi - (m - n)].double()
                    new = _exact_scale(x.abs().amax((1, 2)), fmt)
                    r = lo - i * bs
                    if r:
                        new = torch.maximum(new, scale[l, at])
                        pool[l, at, :, :r] = _exact_code(pool[l, at, :, :r] * (scale[l, at] / new)[:, None, None], fmt)
                    pool[l, at, :, r:hi - i * bs] = _exact_code(x / new[:, None, None], fmt)
                    scale[l, at] = new
        pools.append(pool)
        scales.append(scale)
    return _exact_out(s, pools, scales)


def _exact_gather(s):
    c = s["c"]
    lens, T = s["length"].tolist(), s["out"][0].shape[3]
    got = [torch.zeros((c["L"], c["B"], c["H"], T, c["d"]), dtype=torch.float64, device="cuda") for _ in "kv"]
    for l in range(c["L"]):
        for b, m in enumerate(lens):
            for g, w in zip(got, "kv"):
                g[l, b, :, T - m:] = _exact_page(s, w, l, b, m).transpose(0, 1)
    return tuple(got), None


def _exact_compact(s):
    c = s["c"]
    bs, fmt = c["bs"], c["fmt"]
    if c["L"] * c["B"] * c["H"] > 600:
        return None
    pools, scales = [], []
    credit = torch.zeros(s["credit_out"].shape, dtype=torch.float64, device="cuda")
    for w in "kv":
        pool, scale = s[w + "p"].to(torch.float64), s[w + "s"].double()
        for l in range(c["L"]):
            for b, m in enumerate(s["length"].tolist()):
                k, row = int(s["n_kept"][l, b, 0]), _exact_page(s, w, l, b, m)
                to = s["new_table"][b, : -(-k // bs)].long()
                for h in range(c["H"]):
                    slot = s["kept"][l, b, h, :k].long()
                    credit[l, b, h, :k] = s["credit"][l, b, h][slot].double()
                    x = torch.zeros((len(to) * bs, c["d"]), dtype=torch.float64, device="cuda")
                    x[:k] = row[slot - s["pad"][b], h]
                    x = x.reshape(len(to), bs, -1)
                    scale[l, to, h] = _exact_scale(x.abs().amax((1, 2)), fmt)
                    x = _exact_code(x / scale[l, to, h][:, None, None], fmt)
                    left = pool[l, to[-1], h, (k - 1) % bs + 1:].clone()
                    pool[l, to, h] = x
                    pool[l, to[-1], h, (k - 1) % bs + 1:] = left
        pools.append(pool)
        scales.append(scale)
    return (*_exact_out(s, pools, scales), credit)
