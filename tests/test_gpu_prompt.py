"""Rotary positions and prompt attention on the GPU against plain forms in 64 bits: layouts, lengths
from nothing on, strides, what lies outside the sequences, streams, graphs and refusals."""
import ctypes

import numpy as np
import pytest
import torch

from tests import prompt_ref as pr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def _handle(H=2, G=2, d=64, max_T=64, **kw):
    import eviction_gb300 as kvc
    return kvc.Handle(kvc.Config(kw.pop("L", 1), kw.pop("B", 1), H, G, d, max_T, kw.pop("budget", 16), window=1, **kw))


def _ints(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def _rand(shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


# ---- rotary ----

ROPES = [dict(), dict(interleaved=True), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0, interleaved=True),
         dict(scaling="bands", base=500000.0, factor=8.0, original=8192.0, magnitude=1.2)]


def _check_rotary(x, y, pos, kw, dim, n_tok=None, before=None):
    """x, y [L, S, heads, n, d]; rows past n_tok are what they were before."""
    kw = dict(kw)
    inter, mag = kw.pop("interleaved", False), kw.pop("magnitude", 1.0)
    want, tol = pr.rotary(x, pos[None, :, None], pr.frequencies(dim, **kw), inter, float(np.float32(mag)))
    n = x.shape[3]
    for b in range(x.shape[1]):
        m = n if n_tok is None else n_tok[b]
        assert ((y[:, b, :, :m].double() - want[:, b, :, :m]).abs() <= tol[:, b, :, :m]).all()
        if before is not None:
            assert torch.equal(y[:, b, :, m:], before[:, b, :, m:])


@pytest.mark.parametrize("kw", ROPES)
@pytest.mark.parametrize("d,dim", [(128, 128), (128, 64), (64, 64), (64, 16), (128, 112)])
def test_rotary(kw, d, dim):
    import eviction_gb300 as kvc
    for L, S, n, H, G, n_tok in ((1, 3, 5, 2, 3, None), (2, 2, 1, 1, 1, [1, 0]), (1, 4, 33, 4, 7, [33, 0, 7, 32])):
        h = _handle(H, G, d)
        rope = kvc.Rope(dim, **kw)
        g = torch.Generator().manual_seed(n)
        pos = torch.randint(-3, 200000, (S, n), generator=g, dtype=torch.int32).cuda()
        pos[0, 0] = 0
        q, k = _rand((L, S, H * G, n, d), 1), _rand((L, S, H, n, d), 2)
        qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
        h.rotary(rope, pos, q, k, qo, ko, n_tok=None if n_tok is None else _ints(n_tok))
        assert h.device_status() == 0
        _check_rotary(q, qo, pos, kw, dim, n_tok, torch.full_like(q, 7))
        _check_rotary(k, ko, pos, kw, dim, n_tok, torch.full_like(k, 7))
        # in place: the same bits
        a, b = q.clone(), k.clone()
        h.rotary(rope, pos, a, b, n_tok=None if n_tok is None else _ints(n_tok))
        for got, want, x in ((a, qo, q), (b, ko, k)):
            for s in range(S):
                m = n if n_tok is None else n_tok[s]
                assert torch.equal(got[:, s, :, :m], want[:, s, :, :m])
                assert torch.equal(got[:, s, :, m:], x[:, s, :, m:])
        # only queries, only keys
        a, b = q.clone(), torch.zeros_like(k)
        h.rotary(rope, pos, q=a)
        h.rotary(rope, pos, k=k, k_out=b)
        _check_rotary(q, a, pos, kw, dim)
        _check_rotary(k, b, pos, kw, dim)


def test_rotary_of_a_projection():
    """Queries and keys as slices of one projection, token-major, in place: the values beside them stay."""
    import eviction_gb300 as kvc
    S, n, H, G, d = 3, 50, 2, 4, 64
    h = _handle(H, G, d)
    x = _rand((1, S, n, H * G + 2 * H, d))
    y = x.clone()
    pos = torch.arange(S * n, dtype=torch.int32, device="cuda").reshape(S, n)
    q, k = (y[..., a:b, :].permute(0, 1, 3, 2, 4) for a, b in ((0, H * G), (H * G, H * G + H)))
    h.rotary(kvc.Rope(d), pos, q, k)
    assert torch.equal(y[..., H * G + H:, :], x[..., H * G + H:, :])
    _check_rotary(x[..., :H * G, :].permute(0, 1, 3, 2, 4), q, pos, {}, d)
    _check_rotary(x[..., H * G:H * G + H, :].permute(0, 1, 3, 2, 4), k, pos, {}, d)


def test_rotary_far_positions_and_back():
    import eviction_gb300 as kvc
    h = _handle(1, 1, 128)
    rope = kvc.Rope(128)
    x = _rand((1, 1, 1, 6, 128))
    pos = _ints([[1000000, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1, -2 ** 31, 0]])
    y = torch.empty_like(x)
    h.rotary(rope, pos, q=x, q_out=y)
    _check_rotary(x, y, pos, {}, 128)
    z = torch.empty_like(x)
    back = pos.clone()
    back[0, 4] = 0  # (-2^31 has no opposite)
    h.rotary(rope, -back, q=y, q_out=z)
    assert ((z - x).double().abs()[..., [0, 1, 2, 3, 5], :] <= 2 ** -6 * x.double().norm(dim=-1, keepdim=True)[..., [0, 1, 2, 3, 5], :]).all()


def test_rotary_skips_bad_counts():
    import eviction_gb300 as kvc
    h = _handle(1, 2, 64)
    x = _rand((2, 4, 2, 9, 64))
    y = torch.full_like(x, 7)
    pos = torch.arange(36, dtype=torch.int32, device="cuda").reshape(4, 9)
    h.rotary(kvc.Rope(64), pos, q=x, q_out=y, n_tok=_ints([9, 10, -1, 4]))
    assert h.device_status() == 2
    _check_rotary(x, y, pos, {}, 64, [9, 0, 0, 4], torch.full_like(x, 7))


def test_rotary_refuses():
    import eviction_gb300 as kvc
    h = _handle(2, 2, 64)
    q, pos, rope = _rand((1, 2, 4, 3, 64)), _ints(np.zeros((2, 3))), kvc.Rope(64)
    with pytest.raises(kvc.KvcError, match="larger than head_dim"):
        h.rotary(kvc.Rope(128), pos, q=q)
    for bad, kind in ((dict(q=q.float()), TypeError), (dict(q=q[0]), ValueError), (dict(q=q[..., :32]), ValueError),
                      (dict(q=q.transpose(-1, -2)), ValueError), (dict(q=q.cpu()), ValueError), (dict(), ValueError),
                      (dict(q=q, k=q), ValueError), (dict(q=q, k_out=q), ValueError), (dict(q=q, q_out=q[:, :1]), ValueError),
                      (dict(q=q, n_tok=_ints([1])), ValueError)):
        with pytest.raises(kind):
            h.rotary(rope, pos, **bad)
    for p in (pos[:1], pos.long(), pos.cpu()):
        with pytest.raises((TypeError, ValueError)):
            h.rotary(rope, p, q=q)
    with pytest.raises(TypeError):
        h.rotary(None, pos, q=q)
    with pytest.raises(kvc.KvcError, match="rows overlap"):
        h.rotary(rope, pos, q=q, q_out=q[:, :1].expand(1, 2, 4, 3, 64))
    odd = torch.zeros(1 * 2 * 4 * 3 * 68 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kvc.KvcError, match="multiples of 8"):
        h.rotary(rope, pos, q=odd[:2 * 4 * 3 * 68].reshape(1, 2, 4, 3, 68)[..., :64])
    with pytest.raises(kvc.KvcError, match="16-byte aligned"):
        h.rotary(rope, pos, q=odd[1:1 + q.numel()].reshape(q.shape))
    lib, n = kvc.load_library(), ctypes.c_void_p(0)
    r = h._strided(q, "q", q.shape, 1)
    p = ctypes.c_void_p(pos.data_ptr())
    assert lib.kvc_rotary(h._h, None, r, n, r, n, 1, 2, 3, p, n, n) == -1
    assert lib.kvc_rotary(h._h, rope._ref, n, n, n, n, 1, 2, 3, p, n, n) == -1
    assert lib.kvc_rotary(h._h, rope._ref, r, n, n, n, 1, 2, 3, p, n, n) == -1
    for sizes in ((0, 2, 3), (1, 0, 3), (1, 2, 0)):
        assert lib.kvc_rotary(h._h, rope._ref, r, n, r, n, *sizes, p, n, n) == -2
    assert lib.kvc_rotary(h._h, rope._ref, r, n, r, n, 1, 2 ** 20, 2 ** 11, p, n, n) == -8
    assert lib.kvc_rotary(h._h, rope._ref, r, n, r, n, 1, 2, 3, n, n, n) == -1
    assert lib.kvc_rotary(h._h, rope._ref, r, n, r, n, 1, 2, 3, ctypes.c_void_p(pos.data_ptr() + 2), n, n) == -3
    assert h.device_status() == 0


# ---- prompt attention ----

class Prompts:
    """Ragged prompts, packed (with gaps) or padded; what no sequence has is NaN."""

    def __init__(self, lens, H, G, d, packed, seed=0, q_scale=1.5, v_scale=1.0, gap=3, order="token", n=None):
        self.lens, self.H, self.G, self.d, self.packed = lens, H, G, d, packed
        S = len(lens)
        starts = np.cumsum([gap] + [m + gap for m in lens])
        self.n = n or max(1, int(starts[-1]) if packed else max(lens) + gap)
        lead = () if packed else (S,)
        self.first = [int(s) for s in starts[:-1]] if packed else [0] * S
        inside = torch.zeros((*lead, self.n), dtype=torch.bool, device="cuda")
        for b, m in enumerate(lens):
            (inside if packed else inside[b])[self.first[b]:self.first[b] + m] = True

        def rows(heads, s, scale):
            if order == "token":  # as a projection leaves them
                x = _rand((*lead, self.n, heads, d), s, scale).transpose(-3, -2)
            elif order == "wide":  # a slice of rows that are wider
                x = _rand((*lead, heads, self.n, d + 64), s, scale)[..., 64:]
            else:
                x = _rand((*lead, heads, self.n, d), s, scale)
            return torch.where(inside[..., None, :, None], x, float("nan")) if order == "dense" else \
                x.masked_fill_(~inside[..., None, :, None], float("nan"))

        self.q, self.k, self.v = rows(H * G, seed + 1, q_scale), rows(H, seed + 2, 1.0), rows(H, seed + 3, v_scale)
        self.inside = inside
        self.h = _handle(H, G, d)

    def run(self, lse=True, **kw):
        self.out = torch.full_like(self.q, 7)
        self.lse = torch.full(self.q.shape[:-1], 7.0, device="cuda") if lse else None
        first = _ints(self.first) if self.packed else None
        self.h.prompt_attend(self.q, self.k, self.v, self.out, lse=self.lse, first=first, n_tok=_ints(self.lens), **kw)
        return self.out, self.lse

    def rows(self, b, t, heads=slice(None)):
        t = t if self.packed else t[b]
        return t[heads, self.first[b]:self.first[b] + self.lens[b]]

    def check(self, skipped=()):
        assert self.h.device_status() == (2 if skipped else 0)
        out, lse = self.out, self.lse
        rest = ~self.inside
        for b in skipped:
            (rest if self.packed else rest[b])[self.first[b]:self.first[b] + self.lens[b]] = True
        assert (out[rest[..., None, :, None].expand(out.shape)] == 7).all(), "rows of no sequence were written"
        if lse is not None:
            assert (lse[rest[..., None, :].expand(lse.shape)] == 7).all()
        for b, m in enumerate(self.lens):
            if b in skipped or m <= 0:
                continue
            for hq in range(self.H * self.G):
                w, l, tol, ltol = pr.attention(self.rows(b, self.q, hq), self.rows(b, self.k, hq // self.G),
                                               self.rows(b, self.v, hq // self.G), self.d ** -0.5)
                off = (self.rows(b, out, hq).double() - w).abs() - tol
                assert (off <= 0).all(), (b, hq, float(off.max()), torch.nonzero(~(off <= 0))[:4].tolist())
                if lse is not None:
                    off = (self.rows(b, lse[..., None], hq)[..., 0].double() - l).abs() - ltol
                    assert (off <= 0).all(), (b, hq, float(off.max()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("lens,H,G", [
    ([1], 1, 1), ([0], 1, 1), ([0, 3, 0, 1, 0], 2, 2), ([15, 16, 17], 1, 4), ([63, 64, 65], 2, 1),
    ([127, 128, 129], 1, 1), ([127, 128, 129, 5], 1, 7), ([255, 256, 257], 1, 1), ([300, 17, 511, 513], 2, 3),
    ([130, 1, 260], 1, 8), ([200, 100], 1, 5), ([90, 33], 2, 6), ([140, 31], 1, 16), ([70, 40], 1, 24),
    ([20, 9], 1, 71), ([9, 3], 1, 130)])
def test_prompt(lens, H, G, packed, d):
    p = Prompts(lens, H, G, d, packed, seed=len(lens) + H * G)
    p.run()
    p.check()


@pytest.mark.parametrize("G,d,T", [(1, 128, 1500), (7, 128, 1100), (4, 64, 2050), (2, 128, 4100)])
def test_prompt_long(G, d, T):
    p = Prompts([T, T // 3], 1, G, d, True)
    p.run()
    p.check()


def test_prompt_many_sequences():
    """More sequences than threads of a block, most of them short or empty."""
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 40, 1500)]
    lens[700] = 900
    p = Prompts(lens, 2, 2, 64, True, gap=1)
    p.run()
    p.check()


@pytest.mark.parametrize("order", ["token", "wide", "dense"])
@pytest.mark.parametrize("packed", [True, False])
def test_prompt_strides(order, packed):
    p = Prompts([140, 3, 77], 2, 3, 128, packed, order=order)
    p.run(lse=False)
    p.check()


def test_prompt_one_key_head_for_all():
    """Keys and values that all heads share through a stride of 0, and a sequence axis of stride 0."""
    p = Prompts([150, 90], 2, 2, 64, False)
    p.k = p.k[:, :1].expand_as(p.k)
    p.v = p.v[:1, :, :].expand_as(p.v)
    p.v = torch.where(torch.isnan(p.v), 1.0, p.v)[:1].expand_as(p.v)
    p.run()
    p.check()


@pytest.mark.parametrize("q_scale", [1e-4, 40.0, 3e4])
def test_prompt_logits(q_scale):
    """From all weights alike to one weight that is all: references move, nothing overflows."""
    p = Prompts([400, 129], 1, 2, 128, True, q_scale=q_scale)
    p.run()
    p.check()


def test_prompt_growing_logits():
    """Each key a larger logit than the ones before it, over all of fp32's exponent of exp2: references
    move in every tile."""
    p = Prompts([700], 1, 2, 64, False)
    p.q = torch.ones_like(p.q)
    t = torch.arange(p.n, device="cuda", dtype=torch.float32)
    for slope in (0.01, 0.25, 8.0):
        p.k = (t[:, None] * slope).expand(1, 1, p.n, 64).to(torch.bfloat16).contiguous()
        p.run()
        p.check()
        p.k = p.k.flip(2).contiguous()
        p.run()
        p.check()


def test_prompt_large_values():
    p = Prompts([200], 1, 1, 64, True, v_scale=1e30)
    p.run()
    p.check()


def test_prompt_skips_bad_sequences():
    p = Prompts([40, 50, 60, 70], 1, 2, 64, True)
    keep = list(p.first), list(p.lens)
    for first, lens in ((( -1, None, None, None), None), ((None, 10 ** 9, None, None), None),
                        ((None, None, None, None), (40, -1, 60, 70)), ((None,) * 4, (40, 50, 60, 2 ** 31 - 1))):
        p.out, p.lse = torch.full_like(p.q, 7), torch.full(p.q.shape[:-1], 7.0, device="cuda")
        f = [x if y is None else y for x, y in zip(keep[0], first)]
        n = keep[1] if lens is None else lens
        p.h.prompt_attend(p.q, p.k, p.v, p.out, lse=p.lse, first=_ints(f), n_tok=_ints(n))
        bad = [b for b in range(4) if f[b] != keep[0][b] or n[b] != keep[1][b]]
        p.check(skipped=bad)
    p = Prompts([40, 50], 1, 2, 64, False)
    p.out, p.lse = torch.full_like(p.q, 7), torch.full(p.q.shape[:-1], 7.0, device="cuda")
    p.h.prompt_attend(p.q, p.k, p.v, p.out, lse=p.lse, n_tok=_ints([40, p.n + 1]))
    p.check(skipped=[1])


def test_prompt_whole_rows_without_counts():
    p = Prompts([33, 33, 33], 2, 2, 64, False, gap=0)
    p.out, p.lse = torch.full_like(p.q, 7), torch.full(p.q.shape[:-1], 7.0, device="cuda")
    p.h.prompt_attend(p.q, p.k, p.v, p.out, lse=p.lse)
    p.check()


def test_prompt_same_bits_twice_and_in_any_company():
    """A sequence's result does not depend on the others, and a second run gives the same bits."""
    p = Prompts([260, 100, 513], 2, 4, 128, True)
    a, l = (x.clone() for x in p.run())
    b, m = p.run()
    assert torch.equal(a, b) and torch.equal(l, m)
    lens, first = p.lens, p.first
    for i in range(3):
        p.lens, p.first = [lens[i]], [first[i]]
        p.run()
        assert torch.equal(p.rows(0, p.out), a[:, first[i]:first[i] + lens[i]])
        assert torch.equal(p.rows(0, p.lse[..., None])[..., 0], l[:, first[i]:first[i] + lens[i]])


def test_prompt_on_two_streams_with_one_handle_each():
    ps = [Prompts([300, 200], 2, 2, 128, True, seed=10 * i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(5):
        for p, s in zip(ps, streams):
            with torch.cuda.stream(s):
                p.run()
    torch.cuda.synchronize()
    for p in ps:
        p.check()


def test_prompt_captured_and_replayed():
    """A captured call reads lengths, places and inputs anew at each replay."""
    p = Prompts([200, 120], 2, 2, 64, True)
    n_tok, first = _ints(p.lens), _ints(p.first)
    p.out, p.lse = torch.full_like(p.q, 7), torch.full(p.q.shape[:-1], 7.0, device="cuda")
    call = lambda: p.h.prompt_attend(p.q, p.k, p.v, p.out, lse=p.lse, first=first, n_tok=n_tok)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([200, 120], [17, 3], [1, 119]):
        p.out.fill_(7)
        p.lse.fill_(7)
        p.lens = lens
        n_tok.copy_(_ints(lens))
        p.inside = torch.zeros_like(p.inside)
        for b, m in enumerate(lens):
            p.inside[p.first[b]:p.first[b] + m] = True
        graph.replay()
        p.check()


def test_prompt_refuses():
    import eviction_gb300 as kvc
    p = Prompts([20, 10], 2, 2, 64, False)
    n_tok = _ints([20, 10])
    ok = dict(q=p.q, k=p.k, v=p.v, out=torch.empty_like(p.q))
    for change, kind in ((dict(q=p.q.float()), TypeError), (dict(k=p.k.cpu()), ValueError), (dict(v=p.v[:1]), ValueError),
                         (dict(k=p.q), ValueError), (dict(out=p.k), ValueError), (dict(lse=torch.empty(4, device="cuda")), ValueError),
                         (dict(first=_ints([0])), ValueError), (dict(n_tok=_ints([1])), ValueError),
                         (dict(lse=torch.empty(p.q.shape[:-1], device="cuda", dtype=torch.float64)), TypeError)):
        a = dict(ok, n_tok=n_tok)
        a.update(change)
        with pytest.raises(kind):
            p.h.prompt_attend(**a)
    with pytest.raises(kvc.KvcError, match="need n_tok"):
        x = Prompts([20, 10], 2, 2, 64, True)
        x.h.prompt_attend(x.q, x.k, x.v, torch.empty_like(x.q), first=_ints(x.first))
    with pytest.raises(kvc.KvcError, match="rows overlap"):
        p.h.prompt_attend(**dict(ok, out=p.q[:, :1].expand_as(p.q)), n_tok=n_tok)
    lib, z = kvc.load_library(), ctypes.c_void_p(0)
    r = {k: p.h._strided(t, k, tuple(t.shape), 0, None) for k, t in ok.items()}
    c = ctypes.c_void_p(n_tok.data_ptr())
    call = lambda S, n, q=r["q"], f=z, t=c: lib.kvc_prompt_attend(  # noqa: E731
        p.h._h, q, r["k"], r["v"], S, n, f, t, r["out"], z, z)
    assert call(0, 23) == -2 and call(2, 0) == -2 and call(2 ** 10, 2 ** 21) == -8
    assert call(2, 23, q=None) == -1 and call(2, 23, t=ctypes.c_void_p(n_tok.data_ptr() + 1)) == -3
    assert call(2, 23, f=ctypes.c_void_p(n_tok.data_ptr() + 2)) == -3
    assert p.h.device_status() == 0
