"""Gathered attention weight of the 8-bit cache and the choice of the heaviest tokens on the GPU,
against plain forms in 64 bits; and a prompt's and an eviction's calls together as a decode loop
makes them."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import prompt_ref as pr
from tests.cache8_bounds import _rows
from tests.test_gpu_cache8 import Pair, _ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def _bf(rng, shape, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(torch.bfloat16).cuda()


class Weigh(Pair):
    """Queries of the newest tokens of a cache, their lse, and what was gathered before."""

    def prepare(self, n, n_q=None, packed=False, q_scale=1.0, cap=None, order="token", exact_lse=True):
        r, G, d = self.ref, self.cfg.group, self.ref.d
        lens = [int(x) for x in r.len]
        self.n, self.n_q, self.packed = n, n_q, packed
        counts = [n if n_q is None else int(n_q[b]) for b in range(r.B)]
        if packed:
            self.first = list(np.cumsum([2] + [c + 3 for c in counts[:-1]]))
            self.n = N = int(self.first[-1]) + counts[-1] + 2
            lead = (r.L,)
        else:
            self.first, N, lead = [0] * r.B, n, (r.L, r.B)
        x = _bf(self.rng, (*lead, N, r.H * G, d), q_scale).transpose(-3, -2)
        self.q = x if order == "token" else x.contiguous()
        self.lse = torch.full((*lead, r.H * G, N), math.nan, device="cuda")
        inside = torch.zeros((*(() if packed else (r.B,)), N), dtype=torch.bool, device="cuda")
        for b in range(r.B):
            (inside if packed else inside[b])[self.first[b]:self.first[b] + counts[b]] = True
        self.q.masked_fill_(~inside[..., None, :, None], math.nan)
        self.cap = cap or max(max(lens), 1) + 3
        self.old = torch.rand((r.L, r.B, r.H, self.cap), device="cuda", dtype=torch.float32,
                              generator=torch.Generator(device="cuda").manual_seed(1)) * 3
        self.counts = counts
        for l in range(r.L):
            for b in range(r.B):
                for h in range(r.H):
                    if counts[b] == 0 or counts[b] > lens[b]:
                        continue
                    q, k = self.queries(l, b, h).double(), self.keys(l, b, h)
                    z = q @ k.T * self.scale
                    sees = torch.arange(lens[b], device="cuda") <= (lens[b] - counts[b]) + torch.arange(
                        counts[b], device="cuda")[:, None]
                    self.lse_of(l, b, h).copy_(torch.logsumexp(z.masked_fill(~sees, -math.inf), -1) +
                                               (0 if exact_lse else 1.5))

    def keys(self, l, b, h):
        m = int(self.ref.len[b])
        return torch.from_numpy(_rows(self.ref, l, b, h, np.arange(m))[0]).cuda()

    def queries(self, l, b, h):
        G = self.cfg.group
        q = self.q[l] if self.packed else self.q[l, b]
        return q[h * G:(h + 1) * G, self.first[b]:self.first[b] + self.counts[b]]

    def lse_of(self, l, b, h):
        G = self.cfg.group
        x = self.lse[l] if self.packed else self.lse[l, b]
        return x[h * G:(h + 1) * G, self.first[b]:self.first[b] + self.counts[b]]

    def run(self, decay=1.0):
        self.w = self.old.clone()
        self.h.cache8_weigh(self.c, self.q, self.lse, self.w, decay=decay,
                            n_q=_ints(self.counts) if self.packed or self.n_q is not None else None,
                            first=_ints(self.first) if self.packed else None)
        return self.w

    def check(self, decay=1.0, status=0, skipped=(), absent=None):
        assert self.h.device_status() == status
        r = self.ref
        for l in range(r.L):
            for b in range(r.B):
                m = 0 if b in skipped else int(r.len[b])
                assert torch.equal(self.w[l, b, :, m:], self.old[l, b, :, m:]), "entries past the end were written"
                for h in range(r.H) if m else ():
                    k = self.keys(l, b, h)
                    want, tol = pr.weigh(self.queries(l, b, h), k, self.lse_of(l, b, h), self.old[l, b, h, :m], decay,
                                         self.scale)
                    if absent is not None:
                        gone = torch.from_numpy(absent[b, :m]).cuda()
                        want = torch.where(gone, decay * self.old[l, b, h, :m].double(), want)
                    off = (self.w[l, b, h, :m].double() - want).abs() - tol
                    assert (off <= 0).all(), (l, b, h, float(off.max()), torch.nonzero(~(off <= 0))[:4].tolist())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,n,H,G,bs", [
    ([1], 1, 1, 1, 16), ([17, 1, 40], 1, 2, 2, 8), ([300, 33, 129], 1, 1, 7, 16), ([31, 32, 33, 65], 2, 2, 4, 24),
    ([100, 50], 4, 1, 8, 64), ([260, 70], 20, 2, 1, 16), ([130, 128, 127], 60, 1, 3, 32), ([400, 150], 128, 1, 7, 16),
    ([300], 300, 2, 2, 16), ([520], 500, 1, 4, 128), ([40], 5, 1, 71, 8), ([30], 3, 1, 300, 8)])
def test_weigh(lens, n, H, G, bs, d, fmt):
    blocks = -(-max(lens) // bs)
    p = Weigh(1, len(lens), H, d, bs, blocks, fmt, G=G, seed=len(lens) * n + G, max_T=64, window=1)
    p.fill(lens)
    n_q = None if min(lens) >= n else [min(m, n) for m in lens]
    for decay in (1.0, 0.9, 0.0):
        p.prepare(n, n_q, order="token" if decay else "dense")
        p.run(decay)
        p.check(decay)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_weigh_packed_prompts_and_layers(fmt):
    lens = [70, 0, 1, 200, 33]
    p = Weigh(2, 5, 2, 128, 16, 13, fmt, G=3, max_T=64, window=1)
    p.fill(lens)
    for n_q in (lens, [1, 0, 1, 1, 1], [10, 0, 0, 150, 33]):
        p.prepare(max(n_q), n_q, packed=True)
        p.run(0.5)
        p.check(0.5)
        p.prepare(max(n_q), n_q)
        p.run(0.5)
        p.check(0.5)


def test_weigh_overwrites_without_reading():
    p = Weigh(1, 2, 1, 64, 16, 8, "e4m3", G=2, max_T=64, window=1)
    p.fill([100, 50])
    for n in (1, 40):
        p.prepare(n)
        p.old[..., :] = math.nan
        p.run(0.0)
        for b, m in ((0, 100), (1, 50)):
            assert torch.isfinite(p.w[0, b, :, :m]).all() and torch.isnan(p.w[0, b, :, m:]).all()


def test_weigh_queries_that_saw_nothing():
    p = Weigh(1, 1, 1, 64, 16, 8, "int8", G=2, max_T=64, window=1)
    p.fill([100])
    for n in (2, 60):
        p.prepare(n)
        p.lse[..., 0, 0] = -math.inf
        p.lse[..., 1, 1] = math.inf
        p.run()
        p.check()


@pytest.mark.parametrize("n", [1, 50])
def test_weigh_spreads(n):
    """Scales far apart and large queries: a token's weight is as good as its own logit."""
    for q_scale in (1e-3, 8.0):
        p = Weigh(1, 2, 1, 128, 8, 30, "int8", G=4, max_T=64, window=1)
        p.grow([240, 100])
        p.append([240, 100], spread=4.0)
        p.prepare(n, q_scale=q_scale)
        p.run()
        p.check()


@pytest.mark.parametrize("n", [1, 70])
def test_weigh_bad_pages_and_lengths(n):
    p = Weigh(1, 4, 1, 64, 16, 8, "e4m3", G=2, max_T=64, window=1)
    p.fill([120, 90, 100, 80])
    p.prepare(n)
    p.c.table[0, 2] = 10 ** 6
    p.c.table[2, 1] = -1
    absent = np.zeros((4, 128), bool)
    absent[0, 32:48] = True
    absent[2, 16:32] = True
    p.run()
    p.check(status=2, absent=absent)
    p = Weigh(1, 4, 1, 64, 16, 8, "e4m3", G=2, max_T=64, window=1)
    p.fill([120, 90, 100, 80])
    p.prepare(n, [n] * 4, cap=110)  # the first sequence is longer
    p.run()
    assert p.h.device_status() == 2
    assert torch.equal(p.w[:, 0], p.old[:, 0]) and not torch.equal(p.w[:, 1], p.old[:, 1])
    p.prepare(n, [n] * 4)
    p.w = p.old.clone()
    p.h.cache8_weigh(p.c, p.q, p.lse, p.w, n_q=_ints([n, 91 if n > 1 else 2, -1, n]))
    assert p.h.device_status() == 2
    assert torch.equal(p.w[:, 1:3], p.old[:, 1:3])
    p.check(skipped=(1, 2))


def test_weigh_same_bits_twice_and_replayed():
    p = Weigh(1, 3, 2, 128, 16, 30, "e4m3", G=4, max_T=64, window=1)
    p.fill([400, 130, 477])
    for n in (1, 100):
        p.prepare(n)
        a = p.run().clone()
        assert torch.equal(a, p.run())
        graph = torch.cuda.CUDAGraph()
        w = p.old.clone()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            p.h.cache8_weigh(p.c, p.q, p.lse, w)
        graph.replay()
        assert torch.equal(w, a)
        w.copy_(p.old)
        graph.replay()
        assert torch.equal(w, a)


@pytest.mark.parametrize("n", [1, 40])
def test_weigh_many_sequences(n):
    """More sequences than are sorted by their lengths: groups of several."""
    B = 270
    lens = [(37 * b) % 71 for b in range(B)]
    lens[200] = 300
    p = Weigh(1, B, 1, 64, 16, 19, "e4m3", n_blocks=1300, G=1, max_T=64, window=1)
    p.fill(lens)
    for packed in (False, True):
        p.prepare(n, [min(n, m) for m in lens], packed=packed)
        p.run(0.5)
        p.check(0.5)


@pytest.mark.parametrize("d,fmt", [(64, "int8"), (128, "e4m3")])
def test_weigh_long_pieces_of_few_heads(d, fmt):
    """Few pairs of tiles and many queries: their queries are cut into parts, which are added up."""
    lens = [520, 0, 300, 257]
    p = Weigh(2, 4, 1, d, 16, 33, fmt, G=16, max_T=64, window=1)
    p.fill(lens)
    for n_q, packed, decay in ((lens, True, 0.5), (lens, False, 1.0), ([400, 0, 7, 256], False, 0.0),
                               ([200, 0, 0, 1], True, 1.0)):
        p.prepare(max(n_q), n_q, packed=packed)
        p.run(decay)
        p.check(decay)
    p.prepare(520, lens)
    p.c.table[0, 3] = 10 ** 6
    p.c.table[3, 16] = -1
    absent = np.zeros((4, 528), bool)
    absent[0, 48:64] = True
    absent[3, 256:] = True
    p.run(0.5)
    p.check(0.5, status=2, absent=absent)


def test_weigh_parts_of_two_captured_calls():
    """Two graphs whose parts lie in the same workspace, replayed in turn and in the other order."""
    p = Weigh(1, 2, 1, 128, 16, 20, "int8", G=16, max_T=64, window=1)
    p.fill([300, 280])
    calls = []
    for n in (280, 200):
        p.prepare(n)
        want = p.run().clone()
        w, graph, stream = p.old.clone(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
            p.h.cache8_weigh(p.c, p.q, p.lse, w)
        calls.append((graph, w, p.old.clone(), want, p.q, p.lse))
    for order in ((0, 1), (1, 0, 0)):
        for i in order:
            calls[i][1].copy_(calls[i][2])
            calls[i][0].replay()
        torch.cuda.synchronize()
        for i in order:
            assert torch.equal(calls[i][1], calls[i][3])
    assert p.h.device_status() == 0


def test_weigh_refuses():
    import eviction_gb300 as kvc
    p = Weigh(1, 2, 2, 64, 16, 8, "e4m3", G=2, max_T=64, window=1)
    p.fill([100, 50])
    p.prepare(2)
    ok = dict(cache=p.c, q=p.q, lse=p.lse, weights=p.old)
    for change, kind in ((dict(cache=None), TypeError), (dict(q=p.q.float()), TypeError), (dict(q=p.q[:, :1]), ValueError),
                         (dict(lse=p.lse[..., :1]), ValueError), (dict(lse=p.lse.double()), TypeError),
                         (dict(lse=p.lse.transpose(-1, -2).contiguous().transpose(-1, -2)), ValueError),
                         (dict(weights=p.old[0]), ValueError), (dict(weights=p.old[:, :, :1]), ValueError),
                         (dict(weights=p.old.cpu()), ValueError), (dict(n_q=_ints([1])), ValueError),
                         (dict(first=_ints([0, 0])), ValueError)):
        with pytest.raises(kind):
            p.h.cache8_weigh(**dict(ok, **change))
    for decay in (-0.1, 1.1, math.nan):
        with pytest.raises(kvc.KvcError, match="decay"):
            p.h.cache8_weigh(**ok, decay=decay)
    with pytest.raises(kvc.KvcError, match="need n_q"):
        p.h.cache8_weigh(p.c, p.q[:, 0], p.lse[:, 0], p.old, first=_ints([0, 1]))
    lib, z = kvc.load_library(), ctypes.c_void_p(0)
    q = p.h._strided(p.q, "q", tuple(p.q.shape), 1)
    l, w = ctypes.c_void_p(p.lse.data_ptr()), ctypes.c_void_p(p.old.data_ptr())
    call = lambda n=2, lse=l, wt=w, cap=p.cap, c=p.c._ref: lib.kvc_cache8_weigh(  # noqa: E731
        p.h._h, c, q, n, z, z, lse, 1.0, wt, cap, z)
    assert call(n=0) == -2 and call(cap=0) == -2 and call(lse=z) == -1 and call(wt=z) == -1
    assert call(wt=ctypes.c_void_p(p.old.data_ptr() + 2)) == -3 and call(cap=2 ** 30) == -2 and call(c=None) == -1
    assert p.h.device_status() == 0


# ---- the choice of the heaviest ----

def _choose(w, lens, budget, n_sink=4, n_recent=64, max_T=None, in_place=False):
    import eviction_gb300 as kvc
    L, B, H, cap = w.shape
    h = kvc.Handle(kvc.Config(L, B, H, 1, 64, max_T or cap, budget, window=1, n_sink=n_sink, n_recent=n_recent))
    kept = torch.full((L, B, H, budget), 7, dtype=torch.int32, device="cuda")
    n_kept = torch.full((L, B, H), 7, dtype=torch.int32, device="cuda")
    src = w.clone()
    out = src if in_place else torch.full_like(w, 7)
    h.keep_heaviest(src, _ints(lens), kept, n_kept, out)
    return kept, n_kept, out, h.device_status()


@pytest.mark.parametrize("d,fmt,bs", [(64, "e4m3", 16), (128, "int8", 8), (128, "e4m3", 128)])
def test_packed_rows_are_appended_as_padded_ones(d, fmt, bs):
    """Packed and padded appends leave the same bytes; rows of no sequence are not read."""
    B, H, M = 4, 3, -(-210 // bs)
    pair = [Weigh(2, B, H, d, bs, M, fmt, seed=7, max_T=64, window=1) for _ in range(2)]
    rng = np.random.default_rng(3)
    for counts in ([37, 0, 1, 100], [1, 1, 1, 1], [90, 64, 0, 9]):
        first = list(np.cumsum([1] + [m + 2 for m in counts[:-1]]))
        n = int(first[-1]) + counts[-1] + 3
        rows = [_bf(rng, (2, n, 2 * H, d), 3.0)[:, :, w * H:(w + 1) * H].transpose(1, 2) for w in (0, 1)]
        inside = torch.zeros(n, dtype=torch.bool, device="cuda")
        padded = [torch.full((2, B, H, max(counts), d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in rows]
        for b, m in enumerate(counts):
            inside[first[b]:first[b] + m] = True
            for x, y in zip(rows, padded):
                y[:, b, :, :m] = x[:, :, first[b]:first[b] + m]
        for x in rows:
            x.masked_fill_(~inside[None, None, :, None], math.nan)
        for p in pair:
            p.h.cache8_grow(p.c, _ints(counts))
        pair[0].h.cache8_append(pair[0].c, *rows, _ints(counts), first=_ints(first))
        pair[1].h.cache8_append(pair[1].c, *padded, _ints(counts))
        for name in ("k_pool", "v_pool", "k_scale", "v_scale"):
            a, b = (getattr(p.c, name).view(torch.uint8) for p in pair)
            assert torch.equal(a, b), name
        assert [p.h.device_status() for p in pair] == [0, 0]


def test_packed_rows_out_of_range_are_skipped_and_refused():
    import eviction_gb300 as kvc
    p = Weigh(1, 4, 1, 64, 16, 4, "e4m3", max_T=64, window=1)
    counts = _ints([5, 5, 5, 5])
    p.h.cache8_grow(p.c, counts)
    x = _bf(np.random.default_rng(1), (1, 1, 30, 64))
    old = p.c.k_pool.view(torch.uint8).clone()
    p.h.cache8_append(p.c, x, x, counts, first=_ints([26, -1, 2 ** 31 - 1, 25]))
    assert p.h.device_status() == 2
    blocks = p.c.table[:, 0].long()
    now = p.c.k_pool.view(torch.uint8)
    for b in range(3):
        assert torch.equal(now[0, blocks[b]], old[0, blocks[b]])
    want = p.c.k_pool.float()[0, blocks[3], 0, :5] * p.c.k_scale[0, blocks[3], 0]
    assert ((want - x[0, 0, 25:].float()).abs() <= 2.0 ** -4 * x[0, 0, 25:].float().abs() + 2.0 ** -10).all()
    now = now.clone()
    with pytest.raises(ValueError):
        p.h.cache8_append(p.c, x[None], x[None], counts, first=_ints([0, 5, 10, 15]))
    with pytest.raises(ValueError):
        p.h.cache8_append(p.c, x, x, counts, first=_ints([0, 5, 10]))
    with pytest.raises(TypeError):
        p.h.cache8_append(p.c, x, x, counts, first=counts.long())
    with pytest.raises(kvc.KvcError):
        p.h.cache8_append(p.c, x[..., :0, :], x[..., :0, :], counts, first=_ints([0, 0, 0, 0]))
    assert torch.equal(p.c.k_pool.view(torch.uint8), now) and p.h.device_status() == 0


def _check_choice(w, lens, budget, n_sink=4, n_recent=64, **kw):
    for in_place in (False, True):
        kept, n_kept, out, status = _choose(w, lens, budget, n_sink, n_recent, in_place=in_place, **kw)
        assert status == 0
        x = w.cpu().numpy()
        for (l, b, h) in np.ndindex(*w.shape[:3]):
            want = pr.heaviest(x[l, b, h].tolist(), lens[b], budget, n_sink, n_recent)
            assert int(n_kept[l, b, h]) == len(want)
            assert kept[l, b, h].tolist() == want + [-1] * (budget - len(want)), (l, b, h)
            got = out[l, b, h].cpu().numpy()
            assert np.array_equal(got[:len(want)], x[l, b, h, want], equal_nan=True) and not got[len(want):].any()


@pytest.mark.parametrize("cap,lens,budget,sink,recent", [
    (1, [1, 0], 1, 0, 0), (5, [5, 3, 0], 2, 1, 1), (70, [70, 69, 64, 1], 66, 4, 64), (100, [100, 99, 31, 33], 32, 4, 16),
    (100, [100, 64], 10, 4, 64), (257, [257, 256, 255], 100, 0, 0), (1000, [1000, 513], 512, 4, 64),
    (1025, [1025, 1024, 1023], 700, 4, 64), (2050, [2050, 1111], 512, 4, 64), (4097, [4097, 4096], 1024, 4, 64),
    (8200, [8200, 3001], 4000, 10, 200), (33000, [33000, 32768, 20000], 4096, 4, 64), (65536, [65536, 40001], 4096, 4, 64),
    (60, [60, 50], 100, 4, 64)])
def test_heaviest(cap, lens, budget, sink, recent):
    g = torch.Generator(device="cuda").manual_seed(cap)
    w = torch.rand((1, len(lens), 2, cap), generator=g, device="cuda").log().neg().square()
    _check_choice(w, lens, budget, sink, recent)


@pytest.mark.parametrize("cap", [300, 1500, 5000, 40000])
def test_heaviest_ties_and_odd_values(cap):
    g = torch.Generator(device="cuda").manual_seed(cap)
    w = torch.randint(0, 4, (2, 2, 2, cap), generator=g, device="cuda").float()
    w[1] *= -1
    w[0, 0, 0] = 0
    w[0, 0, 1, ::2] = -0.0
    w[0, 1, 0, ::3] = math.nan
    w[0, 1, 0, 1::7] = math.inf
    w[0, 1, 1, ::5] = -math.inf
    w[1, 0, 0] = math.nan
    w[1, 0, 1] = 1e-42  # subnormal
    w[1, 0, 1, 100:200] = 2e-42
    _check_choice(w, [cap, cap - 7], cap // 3, 4, 64)
    _check_choice(w, [cap, cap - 7], cap - 5, 0, 0)


def test_heaviest_skips_bad_lengths():
    w = torch.rand((1, 3, 2, 50), device="cuda")
    kept, n_kept, out, status = _choose(w, [50, 51, -1], 20, 1, 1)
    assert status == 2
    assert (kept[:, 1:] == 7).all() and (n_kept[:, 1:] == 7).all() and (out[:, 1:] == 7).all()
    assert (n_kept[:, 0] == 20).all()


def test_heaviest_refuses():
    import eviction_gb300 as kvc
    h = kvc.Handle(kvc.Config(1, 2, 2, 1, 64, 50, 20, window=1))
    w = torch.zeros((1, 2, 2, 50), device="cuda")
    kept, n_kept, lens = _ints(np.zeros((1, 2, 2, 20))), _ints(np.zeros((1, 2, 2))), _ints([50, 40])
    for a, kind in (((w[0], lens, kept, n_kept, w[0]), ValueError), ((w, lens, kept, n_kept, w[..., :40]), ValueError),
                    ((w.double(), lens, kept, n_kept, w.double()), TypeError), ((w, lens[:1], kept, n_kept, w), ValueError),
                    ((w, lens, kept[..., :3], n_kept, w), ValueError), ((w, lens, kept, n_kept.long(), w), TypeError),
                    ((w.cpu(), lens, kept, n_kept, w.cpu()), ValueError)):
        with pytest.raises(kind):
            h.keep_heaviest(*a)
    big = torch.zeros((1, 2, 2, 51), device="cuda")
    with pytest.raises(kvc.KvcError, match="cap"):
        h.keep_heaviest(big, lens, kept, n_kept, big)
    lib, z, p = kvc.load_library(), ctypes.c_void_p(0), ctypes.c_void_p(w.data_ptr())
    i = ctypes.c_void_p(lens.data_ptr())
    assert lib.kvc_keep_heaviest(h._h, p, 0, 50, i, i, i, p, z) == -2
    assert lib.kvc_keep_heaviest(h._h, z, 1, 50, i, i, i, p, z) == -1
    assert lib.kvc_keep_heaviest(h._h, p, 1, 50, ctypes.c_void_p(lens.data_ptr() + 2), i, i, p, z) == -3
    assert h.device_status() == 0


# ---- all of them together ----

def _turn(x, pos, d):
    """fp64 rotation of [..., n, d] rows, rounded to bf16 as the kernel does (a test input)."""
    return pr.rotary(x, pos, pr.frequencies(d), False)[0]


@pytest.mark.parametrize("packed", [False, True])
def test_prompt_to_eviction(packed):
    """Prompts turned, attended, cached, weighed, evicted and decoded further; each step against 64 bits
    on what the step before it left."""
    import eviction_gb300 as kvc
    L, B, H, G, d, bs, budget, steps = 1, 3, 2, 2, 64, 16, 64, 3
    lens = [150, 40, 97]
    cap, M = 192, 12
    cfg = kvc.Config(L, B, H, G, d, cap, budget, window=8, n_sink=2, n_recent=16)
    h = kvc.Handle(cfg)
    rng = np.random.default_rng(5)
    rope = kvc.Rope(d)
    cache = kvc.Cache8.allocate(cfg, 80, bs, M)
    n = max(lens)
    n_tok = _ints(lens)
    # the projections' rows, token-major; positions of each sequence from 0
    qkv = _bf(rng, (B, n, H * G + 2 * H, d))
    raw = qkv.clone()
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, n).contiguous()
    q, k, v = (qkv[:, :, a:b].transpose(1, 2) for a, b in ((0, H * G), (H * G, H * G + H), (H * G + H, H * G + 2 * H)))
    h.rotary(rope, pos, q[None], k[None], n_tok=n_tok)
    want = _turn(raw[:, :, :H * G].transpose(1, 2), pos[:, None], d)
    for b, m in enumerate(lens):
        assert ((q[b, :, :m].double() - want[b, :, :m]).abs() <= 2.0 ** -8 * want[b, :, :m].abs() + 1e-5).all()
    scale = d ** -0.5
    if packed:
        first = _ints(np.cumsum([0] + lens[:-1]))
        flat = lambda x: torch.cat([x[b, :, :m] for b, m in enumerate(lens)], 1)  # noqa: E731
        pq, pk, pv = flat(q), flat(k), flat(v)
        out, lse = torch.empty_like(pq), torch.empty(pq.shape[:-1], device="cuda")
        h.prompt_attend(pq, pk, pv, out, lse=lse, first=first, n_tok=n_tok)
    else:
        first, out, lse = None, torch.empty_like(q), torch.zeros((B, H * G, n), device="cuda")
        h.prompt_attend(q, k, v, out, lse=lse, n_tok=n_tok)
    for b, m in enumerate(lens):
        for g in range(H * G):
            o, l, tol, ltol = pr.attention(q[b, g, :m], k[b, g // G, :m], v[b, g // G, :m], scale)
            at = sum(lens[:b])
            got, gl = (out[g, at:at + m], lse[g, at:at + m]) if packed else (out[b, g, :m], lse[b, g, :m])
            assert ((got.double() - o).abs() <= tol).all() and ((gl.double() - l).abs() <= ltol).all()
    h.cache8_grow(cache, n_tok)
    if packed:
        h.cache8_append(cache, pk[None], pv[None], n_tok, first=first)
    else:
        h.cache8_append(cache, k[None], v[None], n_tok)
    weights = torch.zeros((L, B, H, cap), device="cuda")
    if packed:
        h.cache8_weigh(cache, pq[None], lse[None], weights, n_q=n_tok, first=first)
    else:
        h.cache8_weigh(cache, q[None], lse[None], weights, n_q=n_tok)
    assert h.device_status() == 0

    def held():  # the cache's keys as they are held, [B] of [H, m, d]
        T = int(cache.seq_len.max())
        ko, pad = torch.empty((L, B, H, T, d), dtype=torch.bfloat16, device="cuda"), _ints([0] * B)
        h.cache8_gather(cache, T, pad, ko)
        return [ko[0, b, :, T - int(m):] for b, m in enumerate(cache.seq_len.tolist())]

    for b, key in enumerate(held()):
        for x in range(H):
            at = sum(lens[:b])
            own = (lse[x * G:(x + 1) * G, at:at + lens[b]] if packed else lse[b, x * G:(x + 1) * G, :lens[b]])
            w, tol = pr.weigh(q[b, x * G:(x + 1) * G, :lens[b]], key[x], own, torch.zeros(lens[b], device="cuda"), 1.0, scale)
            assert ((weights[0, b, x, :lens[b]].double() - w).abs() <= tol).all()
    # eviction: the choice, new blocks, the rows, the old blocks back
    kept, n_kept = _ints(np.zeros((L, B, H, budget))), _ints(np.zeros((L, B, H)))
    before, old = weights.cpu().numpy(), held()
    h.keep_heaviest(weights, cache.seq_len, kept, n_kept, weights)
    new = cache.with_sequences(torch.full((B, M), -1, dtype=torch.int32, device="cuda"), _ints([0] * B))
    h.cache8_grow(new, n_kept[0, :, 0].contiguous())
    h.cache8_compact(cache, new, cap, _ints([0] * B), kept, n_kept)
    h.cache8_free(cache, torch.arange(B, dtype=torch.int32, device="cuda"))
    assert h.device_status() == 0
    cache, choice = new, kept.cpu()
    now = [min(m, budget) for m in lens]
    assert cache.seq_len.tolist() == now
    for b, key in enumerate(held()):
        for x in range(H):
            want = pr.heaviest(before[0, b, x].tolist(), lens[b], budget, 2, 16)
            assert choice[0, b, x, :now[b]].tolist() == want
            assert np.array_equal(weights[0, b, x, :now[b]].cpu().numpy(), before[0, b, x, want])
            assert not weights[0, b, x, now[b]:].any()
            # requantised once more: a step of e4m3 at most
            assert ((key[x].double() - old[b][x, want].double()).abs() <= 2.0 ** -3 * old[b][x, want].double().abs() + 2.0 ** -8).all()
    # decoding goes on at the next positions of the text
    one = _ints([1] * B)
    for step in range(steps):
        row = _bf(rng, (1, B, 1, H * G + 2 * H, d))
        q, k, v = (row[..., a:b, :].transpose(2, 3) for a, b in ((0, H * G), (H * G, H * G + H), (H * G + H, H * G + 2 * H)))
        h.rotary(rope, _ints([[m + step] for m in lens]), q, k)
        h.cache8_grow(cache, one)
        h.cache8_append(cache, k, v, one)
        out, lse = torch.empty_like(q), torch.empty((1, B, H * G, 1), device="cuda")
        gathered = weights.clone()
        h.cache8_attend(cache, q, out, lse=lse)
        h.cache8_weigh(cache, q, lse, weights, decay=0.95)
        assert h.device_status() == 0
        for b, key in enumerate(held()):
            m = now[b] + step + 1
            for x in range(H):
                w, tol = pr.weigh(q[0, b, x * G:(x + 1) * G], key[x], lse[0, b, x * G:(x + 1) * G], gathered[0, b, x, :m], 0.95, scale)
                assert ((weights[0, b, x, :m].double() - w).abs() <= tol).all()
                grown = weights[0, b, x, :m].double() - 0.95 * gathered[0, b, x, :m].double()
                assert abs(float(grown.sum()) - G) < 1e-4  # a query's weights sum to 1
