"""GPU parity of the 8-bit paged cache with the 64-bit model of tests/cache8_ref.py: codes, scales,
tables and counts bit for bit, attention within the arithmetic's error; what is refused changes
nothing; and the calls together as a decode loop makes them."""
import ctypes

import numpy as np
import pytest
import torch

from tests import cache8_ref as cr

pytestmark = pytest.mark.gpu

DT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


# Room in the table beyond what a test's sequences need: which of the attention kernels a call goes
# to depends on the table's capacity, and with this much room calls of more than 32 query rows go to
# the one for many.
ROOM = [1, 64]


def _both_kernels(cases):
    """Each case (the last two values: heads of a group, queries) without room and, if it has more
    than 32 query rows, with room."""
    return [(*c, room) for c in cases for room in ROOM if room == 1 or c[-2] * c[-1] > 32]


def _ints(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


class Pair:
    """A model cache and the same one on the GPU."""

    def __init__(self, L, B, H, d, bs, max_blocks, fmt, n_blocks=None, seed=0, G=1, window=8,
                 budget=32, max_T=512, room=1, **cfg):
        import eviction_gb300 as kvc
        n_blocks = n_blocks or B * max_blocks + 3
        max_blocks *= room
        self.rng = np.random.default_rng(seed)
        self.ref = cr.RefCache(L, B, H, d, n_blocks, bs, max_blocks, fmt)
        self.ref.free_list[:] = self.rng.permutation(n_blocks)
        for p in self.ref.pool:  # what no one wrote may be anything, NaN codes among it
            p[:] = self.rng.integers(0, 256, p.shape, dtype=np.uint8)
        self.cfg = kvc.Config(L, B, H, G, d, max_T, budget, window=window, n_recent=0, **cfg)
        self.h = kvc.Handle(self.cfg)
        r = self.ref
        self.c = kvc.Cache8(*[torch.from_numpy(p.copy()).cuda().view(DT[fmt]) for p in r.pool],
                            *[torch.from_numpy(s.copy()).cuda() for s in r.scale], _ints(r.table),
                            _ints(r.len), _ints(r.free_list), _ints([r.top]), _ints(r.ref))
        self.scale = d ** -0.5

    def same(self, ref=None, c=None):
        ref, c = ref or self.ref, c or self.c
        assert np.array_equal(c.table.cpu().numpy(), ref.table)
        assert np.array_equal(c.seq_len.cpu().numpy(), ref.len)
        assert int(c.free_top.item()) == ref.top
        assert np.array_equal(c.free_list.cpu().numpy(), ref.free_list)
        assert np.array_equal(c.ref_count.cpu().numpy(), ref.ref)
        for t, p in zip((c.k_pool, c.v_pool), ref.pool):
            assert np.array_equal(t.view(torch.uint8).cpu().numpy(), p)
        for t, s in zip((c.k_scale, c.v_scale), ref.scale):
            assert np.array_equal(t.cpu().numpy(), s)

    def sync_up(self):
        """Copy the model's state over (after the model was prepared by hand)."""
        r, c = self.ref, self.c
        for t, p in zip((c.k_pool, c.v_pool), r.pool):
            t.view(torch.uint8).copy_(torch.from_numpy(p))
        for t, s in zip((c.k_scale, c.v_scale), r.scale):
            t.copy_(torch.from_numpy(s))
        for t, a in ((c.table, r.table), (c.seq_len, r.len), (c.free_list, r.free_list),
                     (c.ref_count, r.ref)):
            t.copy_(torch.from_numpy(np.ascontiguousarray(a)))
        c.free_top.fill_(r.top)

    def grow(self, n):
        want = self.ref.grow(n)
        self.h.cache8_grow(self.c, _ints(n))
        assert self.h.device_status() == want
        return want

    def new_rows(self, n, spread=1.0, token_major=False):
        r = self.ref
        x = self.rng.standard_normal((r.L, r.B, n, r.H, r.d))
        x *= 2.0 ** (spread * self.rng.standard_normal((r.L, r.B, n, r.H, 1)))
        t = torch.from_numpy(x).to(torch.bfloat16).cuda().permute(0, 1, 3, 2, 4)
        return t if token_major else t.contiguous()

    def append(self, n_new, n=None, spread=1.0, token_major=False, rows=None):
        n = n or max(1, max(n_new))
        k, v = rows or (self.new_rows(n, spread, token_major), self.new_rows(n, spread, token_major))
        want = self.ref.append(k.double().cpu().numpy(), v.double().cpu().numpy(), n_new)
        self.h.cache8_append(self.c, k, v, _ints(n_new))
        assert self.h.device_status() == want

    def fill(self, lens, spread=0.7):
        assert self.grow(lens) == 0
        if max(lens):
            self.append(lens, spread=spread)

    def attend(self, n, n_q=None, token_major=False, lse=True, q_scale=1.0):
        r, G = self.ref, self.cfg.group
        shape = (r.L, r.B, n, r.H * G, r.d) if token_major else (r.L, r.B, r.H * G, n, r.d)
        q = (torch.from_numpy(self.rng.standard_normal(shape)) * q_scale).to(torch.bfloat16).cuda()
        out = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
        if token_major:
            q, out = q.permute(0, 1, 3, 2, 4), out.permute(0, 1, 3, 2, 4)
        ls = torch.full((r.L, r.B, r.H * G, n), 7.0, device="cuda") if lse else None
        self.h.cache8_attend(self.c, q, out, lse=ls, n_q=None if n_q is None else _ints(n_q))
        assert self.h.device_status() == 0
        self.check_attend(q, out, ls, n_q)
        return q, out, ls

    def check_attend(self, q, out, ls, n_q=None):
        want, lse, tol, ltol = self.ref.attend(q.double().cpu().numpy(), self.scale, n_q)
        got = out.double().cpu().numpy()
        n = q.shape[3]
        for b in range(self.ref.B):
            nq = n if n_q is None else int(n_q[b])
            assert (got[:, b, :, nq:] == 7.0).all(), "rows past n_q were written"
            off = np.abs(got - want)[:, b, :, :nq] - tol[:, b, :, :nq]
            assert (off <= 0).all(), (b, off.max())
            if ls is not None:
                g, w = ls.double().cpu().numpy()[:, b], lse[:, b]
                assert (g[:, :, nq:] == 7.0).all()
                g, w, t = g[:, :, :nq], w[:, :, :nq], ltol[:, b, :, :nq]
                empty = np.isneginf(w)
                assert np.array_equal(np.isneginf(g), empty)
                assert (np.abs(g[~empty] - w[~empty]) <= t[~empty]).all()


# ---- append ----

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 16), (128, 5), (64, 1), (128, 64), (64, 24), (128, 130)])
def test_append_matches_model(fmt, d, bs):
    """Several calls in a row: block starts and ends inside a call, counts of zero, growing scales."""
    p = Pair(2, 4, 3, d, bs, -(-220 // bs), fmt, seed=bs)
    p.same()
    for i, n_new in enumerate([[0, 1, 17, 40], [1, 0, 33, 1], [1, 1, 1, 1], [70, 64, 3, 16], [1, 2, 0, 5]]):
        assert p.grow(n_new) == 0
        p.append(n_new, spread=2.0, token_major=bool(i % 2))
        p.same()


def test_append_again_changes_nothing():
    p = Pair(1, 2, 2, 64, 16, 8, "e4m3")
    p.fill([20, 37])
    p.grow([9, 30])
    rows = p.new_rows(30, 3.0), p.new_rows(30, 3.0)
    p.append([9, 30], rows=rows)
    p.same()
    before = [t.view(torch.uint8).clone() for t in (p.c.k_pool, p.c.v_pool)]
    p.h.cache8_append(p.c, *rows, _ints([9, 30]))
    assert all(torch.equal(a, t.view(torch.uint8)) for a, t in zip(before, (p.c.k_pool, p.c.v_pool)))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_extremes(fmt):
    """Zero rows, the smallest and largest bf16 values, infinities and NaN."""
    p = Pair(1, 1, 6, 64, 16, 4, fmt)
    p.grow([20])
    k, v = p.new_rows(20), p.new_rows(20)
    k[0, 0, 0] = 0
    k[0, 0, 1] *= 1e-38
    k[0, 0, 2] *= 2.0 ** 120
    v[0, 0, 3, 4, 7] = float("nan")
    v[0, 0, 4, 18, 0] = float("-inf")
    k[0, 0, 5, :, ::2] = float("inf")
    p.append([20], rows=(k, v))  # the model and the library both report NONFINITE
    p.same()
    p.grow([3])
    p.append([3])
    p.same()


def test_append_skips_what_it_cannot_write():
    p = Pair(1, 4, 2, 64, 16, 8, "int8")
    p.fill([20, 20, 20, 20])
    p.ref.table[2, 1] = 10 ** 6
    p.ref.table[3, 0] = -5
    p.sync_up()
    p.append([21, -1, 8, 18], n=25)  # too many, negative, bad blocks
    p.same()
    p.append([26, 1, 1, 1], n=25)
    p.same()


def test_shared_blocks_are_not_written():
    """Counting more tokens as new than there are reaches blocks that a fork shares: they stay."""
    p = Pair(1, 3, 2, 64, 16, 8, "e4m3")
    p.fill([40, 0, 20])
    assert p.ref.fork([0], [1]) == 0
    p.h.cache8_fork(p.c, _ints([0]), _ints([1]))
    p.append([0, 30, 20])
    p.same()


# ---- attend ----

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,H,bs,G,n,room", _both_kernels([
    (64, 1, 16, 1, 1), (128, 2, 16, 7, 1), (128, 1, 5, 4, 1), (64, 2, 64, 3, 2), (128, 2, 24, 8, 3),
    (64, 1, 8, 5, 8), (128, 1, 16, 13, 1), (64, 1, 1, 2, 5), (128, 1, 16, 7, 37), (64, 2, 16, 4, 64),
    (128, 1, 130, 3, 128)]))
def test_attend_matches_model(fmt, d, H, bs, G, n, room):
    lens = [0, 1, n, 130, 131 + n, 64, 16, 95]
    p = Pair(2, len(lens), H, d, bs, -(-300 // bs), fmt, G=G, window=128, seed=n + bs, room=room)
    p.fill(lens)
    p.attend(n, token_major=bool(bs % 2))


@pytest.mark.parametrize("n,n_q", [(5, [0, 1, 5, 3, 2]), (40, [40, 0, 17, 1, 33])])
@pytest.mark.parametrize("room", ROOM)
def test_attend_ragged_queries(n, n_q, room):
    p = Pair(1, 5, 2, 128, 16, 8, "e4m3", G=3, window=64, room=room)
    p.fill([100, 50, 17, 1, 16])
    p.attend(n, n_q=n_q)
    p.attend(n, n_q=n_q, token_major=True, lse=False)


@pytest.mark.parametrize("G,room", [(2, 1), (8, 1), (8, 1024)])
def test_attend_queries_before_the_first_token(G, room):
    """More queries than tokens: the first ones see nothing and get zeros."""
    p = Pair(1, 3, 1, 64, 16, 4, "int8", G=G, window=16, room=room)
    p.fill([3, 0, 9])
    q, out, lse = p.attend(9)
    assert (out[0, 0, :, :6] == 0).all() and (out[0, 1] == 0).all()
    assert torch.isneginf(lse[0, 0, :, :6]).all() and torch.isneginf(lse[0, 1]).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("H,bs,lens,G,n,room", _both_kernels([
    (1, 16, [3000], 1, 1), (2, 64, [2500, 7, 1777], 7, 1), (1, 7, [1999, 1024, 1025], 4, 2),
    (1, 16, [2048], 8, 20), (2, 16, [3000, 1, 2047], 7, 20)]))
def test_attend_long(fmt, H, bs, lens, G, n, room):
    p = Pair(1, len(lens), H, 128, bs, -(-max(lens) // bs), fmt, G=G, window=32, room=room)
    p.fill(lens)
    p.attend(n)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("B,H,longest,n", [(100, 2, 300, 1), (70, 1, 900, 2), (33, 1, 60, 20), (3, 1, 6000, 1)])
@pytest.mark.parametrize("G", [1, 2])
def test_attend_many_and_uneven_sequences(fmt, B, H, longest, n, G):
    """Heads cut anywhere: lengths from nothing to the longest, some sequences without queries."""
    p = Pair(1, B, H, 64, 16, -(-longest // 16), fmt, window=32, seed=B, G=G, room=1 if G == 1 else 64)
    lens = p.rng.integers(0, longest + 1, B) * (p.rng.random(B) < 0.8)
    lens[0], lens[-1] = longest, 1
    p.fill(lens.tolist())
    p.attend(n)
    n_q = p.rng.integers(0, n + 1, B)
    n_q[:3] = 0
    p.attend(n, n_q=n_q)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n,room", [(1, 1), (40, 1), (40, 64)])
def test_attend_scales_far_apart(fmt, n, room):
    """Blocks whose value scales lie 2^60 apart, and sharp softmaxes."""
    p = Pair(1, 2, 1, 64, 8, 30, fmt, G=2, window=64, room=room)
    p.fill([200, 123])
    for w, lo, hi in ((0, -3, 1), (1, -50, 10)):
        p.ref.scale[w] *= 2.0 ** p.rng.integers(lo, hi, p.ref.scale[w].shape)
    p.sync_up()
    p.attend(n)
    p.attend(n, q_scale=30.0)
    p.attend(n, q_scale=1e-4)


@pytest.mark.parametrize("n,room", [(1, 1), (5, 1), (40, 1), (40, 64)])
def test_attend_reads_nothing_behind_a_sequence(n, room):
    """NaN codes past the end and in free blocks change nothing; -1 past the table's blocks is fine."""
    p = Pair(1, 3, 2, 128, 16, 12, "e4m3", G=4, window=64, seed=3, room=room)
    p.fill([n + 3, 100, 33])
    for w in (0, 1):
        used = np.zeros(p.ref.pool[w].shape[1:4:2], bool)  # [n_blocks, bs]
        for b, m in enumerate(p.ref.len):
            for t in range(m):
                used[p.ref.table[b, t // 16], t % 16] = True
        p.ref.pool[w][:] = np.where(used[None, :, None, :, None], p.ref.pool[w], 0x7F)
    p.sync_up()
    p.attend(n)


@pytest.mark.parametrize("G,room", [(2, 1), (10, 1), (10, 1024)])
def test_attend_infinite_and_nan_queries(G, room):
    """A query row that is not finite spoils its own output only."""
    p = Pair(1, 1, 1, 64, 16, 8, "e4m3", G=G, window=8, room=room)
    p.fill([70])
    q, out, _ = p.attend(4)
    q2 = q.clone()
    q2[0, 0, 1, 2, 5] = float("nan")
    q2[0, 0, 0, 3, 5] = float("inf")
    out2 = torch.zeros_like(out)
    p.h.cache8_attend(p.c, q2, out2)
    spoilt = torch.zeros(G, 4, dtype=torch.bool, device="cuda")
    spoilt[1, 2] = spoilt[0, 3] = True
    assert torch.isnan(out2[0, 0, 1, 2]).all()
    assert torch.equal(out2[0, 0][~spoilt], out[0, 0][~spoilt])


@pytest.mark.parametrize("n,room", [(1, 1), (40, 1), (40, 256)])
def test_attend_bad_pages_are_absent(n, room):
    """Tokens in a block out of range do not count; bad lengths and counts are skipped."""
    p = Pair(1, 4, 1, 64, 16, 8, "int8", G=2, window=64, room=room)
    p.fill([60, 60, 60, 60])
    good = p.ref.table.copy()
    p.ref.table[0, 3] = 10 ** 7   # the last block: 12 tokens
    p.ref.table[1, 3] = -1
    p.ref.len[2] = 16 * 8 * room + 1  # above max_blocks * block_size
    p.ref.len[3] = -7
    p.sync_up()
    q = torch.from_numpy(p.rng.standard_normal((1, 4, 2, n, 64))).to(torch.bfloat16).cuda()
    out = torch.full_like(q, 7.0)
    p.h.cache8_attend(p.c, q, out)
    assert p.h.device_status() == cr.BAD_INDEX
    assert (out[:, 2:] == 7.0).all()
    p.ref.table[:] = good
    p.ref.len[:] = 48             # as if the last block were not there
    q0 = q.double().cpu().numpy()
    if n == 1:
        want, _, tol, _ = p.ref.attend(q0, p.scale)
        assert (np.abs(out.double().cpu().numpy() - want)[:, :2] <= tol[:, :2]).all()
    else:
        assert torch.isfinite(out[:, :2]).all()
    out.fill_(7.0)
    p.ref.len[:] = 60
    p.sync_up()
    p.h.cache8_attend(p.c, q, out, n_q=_ints([n + 1, -1, 0, 0]))
    assert p.h.device_status() == cr.BAD_INDEX and (out == 7.0).all()


@pytest.mark.parametrize("room", ROOM)
def test_attend_is_repeatable(room):
    p = Pair(1, 3, 2, 128, 16, 130, "e4m3", G=7, window=64, room=room)
    p.fill([2000, 500, 1])
    for n in (1, 3, 50):
        q, out, lse = p.attend(n) if n == 1 else (torch.randn((1, 3, 14, n, 128), device="cuda").to(
            torch.bfloat16), *(torch.empty((1, 3, 14, n, 128), dtype=torch.bfloat16, device="cuda"),
                               torch.empty((1, 3, 14, n), device="cuda")))
        p.h.cache8_attend(p.c, q, out, lse=lse)
        for _ in range(3):
            o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
            p.h.cache8_attend(p.c, q, o2, lse=l2)
            assert torch.equal(out, o2) and torch.equal(lse, l2)


# ---- gather and compact ----

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,bs,lens,T", [(64, 16, [0, 1, 100, 64], 100), (128, 5, [33, 7], 61),
                                         (128, 64, [130, 64, 1], 131), (64, 1, [9], 9)])
def test_gather_matches_model(fmt, d, bs, lens, T):
    p = Pair(2, len(lens), 3, d, bs, -(-140 // bs), fmt)
    p.fill(lens, spread=3.0)
    k, v, pad, _ = p.ref.gather(T)
    ko = torch.full((2, len(lens), 3, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vo, po = torch.full_like(ko, 7.0), torch.full((len(lens),), -1, dtype=torch.int32, device="cuda")
    p.h.cache8_gather(p.c, T, po, ko, vo)
    assert p.h.device_status() == 0
    assert np.array_equal(po.cpu().numpy(), pad)
    assert np.array_equal(ko.double().cpu().numpy(), k) and np.array_equal(vo.double().cpu().numpy(), v)
    k2 = torch.zeros_like(ko)
    p.h.cache8_gather(p.c, T, po, k2)
    assert torch.equal(k2, ko)


def test_gather_too_long_or_bad():
    p = Pair(1, 3, 1, 64, 16, 8, "int8")
    p.fill([50, 20, 40])
    k, _, pad, _ = p.ref.gather(40)
    p.ref.table[2, 1] = 999
    p.sync_up()
    ko = torch.full((1, 3, 1, 40, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    po = torch.zeros(3, dtype=torch.int32, device="cuda")
    p.h.cache8_gather(p.c, 40, po, ko)
    assert p.h.device_status() == cr.BAD_INDEX
    assert po.tolist() == [40, 20, 0] == pad.tolist()
    k[0, 2, 0, 16:32] = 0
    assert np.array_equal(ko.double().cpu().numpy(), k)


def _kept(p, budget, T, lens):
    L, B, H = p.ref.L, p.ref.B, p.ref.H
    kept, nk = np.full((L, B, H, budget), -1, np.int32), np.zeros((L, B, H), np.int32)
    for b, n in enumerate(lens):
        m = min(budget, n)
        nk[:, b] = m
        for l in range(L):
            for h in range(H):
                kept[l, b, h, :m] = np.sort(p.rng.permutation(n)[:m]) + T - n
    return kept, nk


@pytest.mark.parametrize("fmt,to,bs,to_bs", [("e4m3", "e4m3", 16, 16), ("int8", "int8", 16, 16),
                                             ("e4m3", "int8", 5, 64), ("int8", "e4m3", 64, 7),
                                             ("int8", "int8", 130, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_compact_matches_model(fmt, to, bs, to_bs, d):
    import eviction_gb300 as kvc
    lens, budget, T = [90, 0, 45, 200, 44], 45, 200
    p = Pair(2, 5, 2, d, bs, -(-200 // bs), fmt, n_blocks=-(-500 // bs) + 40, budget=budget, max_T=T)
    p.fill(lens, spread=3.0)
    kept, nk = _kept(p, budget, T, lens)
    if (fmt, bs) == (to, to_bs):
        ref = p.ref.sibling()
        dst = p.c.with_sequences(_ints(ref.table), _ints(ref.len))
    else:
        other = Pair(2, 5, 2, d, to_bs, -(-budget // to_bs), to, budget=budget, max_T=T, seed=9)
        ref, dst = other.ref, other.c
    n = nk[0, :, 0]
    assert ref.grow(n) == 0
    if ref.pool is p.ref.pool:
        p.ref.top = ref.top
    p.h.cache8_grow(dst, _ints(n))
    pad = T - np.array(lens, np.int32)
    assert p.ref.compact(ref, pad, kept, nk) == 0
    cp = p.rng.random((2, 5, 2, T)).astype(np.float32)
    co = torch.full((2, 5, 2, budget), 9.0, device="cuda")
    p.h.cache8_compact(p.c, dst, T, _ints(pad), _ints(kept), _ints(nk),
                       credit_post=torch.from_numpy(cp).cuda(), credit_out=co)
    assert p.h.device_status() == 0
    p.same(ref, dst)
    p.same()
    want = np.where(kept >= 0, np.take_along_axis(cp, np.maximum(kept, 0), 3), 0)
    assert np.array_equal(co.cpu().numpy(), want)
    p.h.cache8_compact(p.c, dst, T, _ints(pad), _ints(kept), _ints(nk))
    p.same(ref, dst)


def test_compact_bad_indices():
    budget, T = 20, 60
    p = Pair(1, 4, 2, 64, 16, 8, "int8", budget=budget, max_T=T)
    p.fill([60, 50, 40, 60])
    kept, nk = _kept(p, budget, T, [60, 50, 40, 60])
    kept[0, 0, 0, 3] = -1
    kept[0, 1, 1, 5] = 4          # in the padding
    kept[0, 1, 0, 0] = 10 ** 9
    nk[0, 2, 1] = 19              # not what dst holds: that unit is left alone
    ref = p.ref.sibling()
    dst = p.c.with_sequences(_ints(ref.table), _ints(ref.len))
    n = np.array([20, 20, 20, 20], np.int32)
    ref.grow(n)
    p.ref.top = ref.top
    p.h.cache8_grow(dst, _ints(n))
    ref.table[3, 1] = -3          # nowhere to write
    dst.table.copy_(torch.from_numpy(ref.table))
    ref.ref[ref.table[1, 0]] = 2  # one that another sequence holds as well
    p.c.ref_count.copy_(torch.from_numpy(ref.ref))
    pad = T - p.ref.len
    assert p.ref.compact(ref, pad, kept, nk) == cr.BAD_INDEX
    p.h.cache8_compact(p.c, dst, T, _ints(pad), _ints(kept), _ints(nk))
    assert p.h.device_status() == cr.BAD_INDEX
    p.same(ref, dst)


# ---- pages ----

@pytest.mark.parametrize("bs,B,M", [(4, 8, 12), (16, 40, 6), (1, 1500, 3)])
def test_pages_match_model(bs, B, M):
    """Random grows, forks and frees, refused ones among them; more sequences than one pass takes."""
    p = Pair(2, B, 2, 64, bs, M, "int8", n_blocks=max(30, B * M // 3), seed=bs)
    rng = p.rng
    seen = set()
    for i in range(40):
        what = i % 3
        if what == 0:
            n = rng.integers(0, 2 * bs + 1, B) * rng.integers(0, 2, B)
            seen.add(("grow", p.grow(n)))
        elif what == 1:
            k = int(rng.integers(1, max(2, B // 3)))
            empty = np.flatnonzero(p.ref.len == 0)
            dst = rng.permutation(empty)[:k] if len(empty) and rng.random() < 0.8 else rng.permutation(B)[:k]
            held = np.flatnonzero(p.ref.len > 0)
            src = rng.choice(held if len(held) else np.arange(B), len(dst))
            want = p.ref.fork(src, dst)
            p.h.cache8_fork(p.c, _ints(src), _ints(dst))
            assert p.h.device_status() == want
            seen.add(("fork", want))
        else:
            seqs = rng.permutation(B)[:int(rng.integers(0, B // 2 + 1))]
            want = p.ref.free(seqs)
            p.h.cache8_free(p.c, _ints(seqs))
            assert p.h.device_status() == want
            seen.add(("free", want))
        p.same()
    assert {("grow", 0), ("fork", 0), ("free", 0)} <= seen


@pytest.mark.parametrize("B,M,bs", [(40, 1000, 1), (1300, 6, 2)])
def test_pages_of_large_calls(B, M, bs):
    """More entries than a thread keeps, more sequences than threads; shared blocks freed together."""
    p = Pair(1, B, 1, 64, bs, M, "int8", n_blocks=B * M // 2 + 50, seed=B)
    half = B // 2
    lens = np.zeros(B, int)
    lens[:half] = p.rng.integers(0, M * bs // 2, half)
    assert p.grow(lens) == 0
    src, dst = p.rng.integers(0, half, B - half), half + p.rng.permutation(B - half)
    for want, call, args in ((p.ref.fork, p.h.cache8_fork, (src, dst)),
                             (p.ref.free, p.h.cache8_free, (p.rng.permutation(B)[:B - 3],)),
                             (p.ref.free, p.h.cache8_free, (np.r_[p.rng.permutation(B), 5],)),
                             (p.ref.free, p.h.cache8_free, (p.rng.permutation(B),))):
        code = want(*args)
        call(p.c, *[_ints(a) for a in args])
        assert p.h.device_status() == code
        p.same()
    assert p.ref.top == p.ref.N


def test_pages_refusals_change_nothing():
    p = Pair(1, 6, 1, 64, 16, 4, "e4m3", n_blocks=12)
    p.fill([20, 40, 0, 0, 16, 0])

    def fork(src, dst):
        want = p.ref.fork(src, dst)
        p.h.cache8_fork(p.c, _ints(src), _ints(dst))
        assert p.h.device_status() == want
        p.same()
        return want

    def free(seqs):
        want = p.ref.free(seqs)
        p.h.cache8_free(p.c, _ints(seqs))
        assert p.h.device_status() == want
        p.same()
        return want

    assert p.grow([0, 60, 0, 0, 0, 0]) == cr.BAD_INDEX     # past max_blocks
    assert p.grow([0, -1, 0, 0, 0, 0]) == cr.BAD_INDEX
    assert p.grow([0, 0, 64, 64, 0, 0]) == cr.EXHAUSTED
    p.same()
    assert fork([0, 0], [2, 2]) == cr.BAD_INDEX            # the same new sequence twice
    assert fork([0], [1]) == cr.BAD_INDEX                  # not empty
    assert fork([0, 2], [2, 3]) == cr.BAD_INDEX            # new and source at once
    assert fork([0], [6]) == cr.BAD_INDEX and fork([-1], [2]) == cr.BAD_INDEX
    assert free([1, 1]) == cr.BAD_INDEX and free([6]) == cr.BAD_INDEX and free([0, -2]) == cr.BAD_INDEX
    assert fork([2], [3]) == 0                             # an empty source: an empty sequence
    assert p.grow([60 - 20, 0, 64, 0, 0, 0]) == 0
    assert fork([1, 1], [3, 5]) == cr.EXHAUSTED            # two started blocks, none free
    assert free([0, 2, 3]) == 0
    p.ref.ref[p.ref.table[1, 0]] = 0                       # a count that was lost
    p.sync_up()
    assert free([4, 1]) == cr.BAD_INDEX
    assert fork([1], [5]) == cr.BAD_INDEX
    p.ref.ref[p.ref.table[1, 0]] = 1
    p.ref.free_list[p.ref.top - 1] = p.ref.table[1, 0]     # a stack with a block in use
    p.sync_up()
    assert p.grow([0, 0, 1, 0, 0, 0]) == cr.BAD_INDEX
    assert fork([1], [5]) == cr.BAD_INDEX
    p.ref.free_list[p.ref.top - 1] = 77
    p.sync_up()
    assert p.grow([0, 0, 1, 0, 0, 0]) == cr.BAD_INDEX
    p.ref.top = 13
    p.sync_up()
    for call in (lambda: p.h.cache8_grow(p.c, _ints([0] * 6)), lambda: p.h.cache8_free(p.c, _ints([1])),
                 lambda: p.h.cache8_fork(p.c, _ints([1]), _ints([5]))):
        call()
        assert p.h.device_status() == cr.BAD_INDEX
        p.same()
    p.ref.top = 12                                         # a full stack cannot take blocks back
    p.sync_up()
    assert free([1]) == cr.BAD_INDEX


def test_grow_refuses_a_shared_started_block():
    p = Pair(1, 2, 1, 64, 16, 4, "int8")
    p.fill([20, 0])
    p.ref.ref[p.ref.table[0, 1]] = 2
    p.sync_up()
    assert p.grow([1, 0]) == cr.BAD_INDEX
    p.same()


# ---- refusals of the calls themselves ----

def test_calls_refuse_bad_arguments():
    import eviction_gb300 as kvc
    p = Pair(1, 2, 2, 64, 16, 4, "e4m3", G=2, window=4, budget=16, max_T=64)
    p.fill([10, 20])
    rows = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, out = rows(1, 2, 4, 1, 64), rows(1, 2, 4, 1, 64)

    def refused(code, call, *a, **kw):
        with pytest.raises(kvc.KvcError) as e:
            call(*a, **kw)
        assert e.value.code == code

    h, c = p.h, p.c
    refused(-2, h.cache8_attend, c, rows(1, 2, 4, 5, 64), rows(1, 2, 4, 5, 64))      # n > window
    refused(-3, h.cache8_attend, c, rows(1, 2, 4, 1, 68)[..., 4:], out)              # alignment
    refused(-3, h.cache8_attend, c, rows(1, 2, 4, 1, 68)[..., :64], out)             # strides
    refused(-1, h.cache8_attend, c, q, rows(1, 1, 4, 1, 64).expand(1, 2, 4, 1, 64))  # overlapping rows
    h.cache8_attend(c, rows(1, 1, 4, 1, 64).expand(1, 2, 4, 1, 64), out)             # fine for inputs
    refused(-2, h.cache8_gather, c, 65, _ints([0, 0]), rows(1, 2, 2, 65, 64))        # T > max_T
    refused(-2, h.cache8_append, c, rows(1, 2, 2, 0, 64), rows(1, 2, 2, 0, 64), _ints([0, 0]))
    k16, nk = _ints(np.zeros((1, 2, 2, 16))), _ints(np.zeros((1, 2, 2)))
    refused(-1, h.cache8_compact, c, c, 64, _ints([0, 0]), k16, nk)                  # into itself
    d = c.with_sequences(_ints(np.zeros((2, 4))), _ints([0, 0]))
    refused(-1, h.cache8_compact, c, d, 64, _ints([0, 0]), k16, nk,
            credit_post=torch.zeros((1, 2, 2, 64), device="cuda"))
    for bad in (dict(q=q.float()), dict(q=q[:, :, :, :, ::2]), dict(q=q.cpu()), dict(q=q[:, :1]),
                dict(out=out[:, :, :3]), dict(lse=torch.zeros(1, 2, 4, device="cuda")),
                dict(lse=torch.zeros((1, 2, 4, 1), dtype=torch.float64, device="cuda")),
                dict(n_q=_ints([1])), dict(n_q=_ints([1, 1]).long())):
        with pytest.raises((ValueError, TypeError)):
            h.cache8_attend(c, **{**dict(q=q, out=out), **bad})
    with pytest.raises(ValueError):
        h.cache8_grow(c, _ints([1, 1, 1]))
    with pytest.raises(ValueError):
        h.cache8_fork(c, _ints([0, 1]), _ints([1]))
    with pytest.raises(ValueError):
        kvc.Cache8(c.k_pool, c.v_pool, c.k_scale[:, :-1], c.v_scale, c.table, c.seq_len, c.free_list,
                   c.free_top, c.ref_count)
    with pytest.raises(ValueError):
        c.layers(1)
    other = Pair(1, 3, 2, 64, 16, 4, "e4m3")
    with pytest.raises(ValueError):
        h.cache8_grow(other.c, _ints([0, 0, 0]))
    h.cache8_free(c, _ints([]))
    h.cache8_fork(c, _ints([]), _ints([]))
    assert h.device_status() == 0
    lib = kvc.load_library()
    assert lib.kvc_cache8_grow(h._h, c._ref, None, None) == -1
    assert lib.kvc_cache8_free(h._h, c._ref, -1, None, None) == -1
    assert lib.kvc_cache8_fork(h._h, c._ref, 1, None, None, None) == -1
    assert lib.kvc_cache8_gather(h._h, c._ref, 10, None, None, None, None) == -1
    assert lib.kvc_cache8_attend(h._h, None, None, 1, None, None, None, None) == -1
    assert lib.kvc_cache8_attend(h._h, ctypes.byref(c._c), None, 1, None, None, None, None) == -1
    p.same()


def _strided(shape, strides):
    size = sum((n - 1) * s for n, s in zip(shape, strides)) + 1
    return torch.zeros(size, dtype=torch.bfloat16, device="cuda").as_strided(shape, strides)


@pytest.mark.parametrize("strides,fine", [
    ((0, 256, 64, 64, 1), False),     # heads and tokens at the same place
    ((0, 256, 64, 128, 1), False),    # token 1 of a head in head 2
    ((0, 128, 64, 512, 1), False),    # sequence 1 begins in sequence 0's heads
    ((0, 512, 128, 64, 1), True),     # dense
    ((0, 576, 136, 64, 1), True),     # with gaps
    ((0, 64, 256, 128, 1), True),     # sequences innermost
    ((0, 1024, 64, 512, 1), True),    # token-major
])
def test_attend_refuses_output_rows_that_overlap(strides, fine):
    import eviction_gb300 as kvc
    p = Pair(1, 2, 2, 64, 16, 4, "e4m3", G=2, window=4)
    q = torch.zeros((1, 2, 4, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = _strided((1, 2, 4, 2, 64), strides)
    if fine:
        p.h.cache8_attend(p.c, q, out)
        return
    with pytest.raises(kvc.KvcError) as e:
        p.h.cache8_attend(p.c, q, out)
    assert e.value.code == -1


# ---- together ----

def _steps(p, n_steps, check=True):
    """Decode steps: grow once, then append and attend layer by layer."""
    r, G = p.ref, p.cfg.group
    one = np.ones(r.B, np.int32)
    for _ in range(n_steps):
        assert p.grow(one) == 0
        k, v = p.new_rows(1), p.new_rows(1)
        r.append(k.double().cpu().numpy(), v.double().cpu().numpy(), one)
        q = torch.from_numpy(p.rng.standard_normal((r.L, r.B, r.H * G, 1, r.d))).to(torch.bfloat16).cuda()
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:4], device="cuda")
        for l in range(r.L):
            cl = p.c.layers(l)
            p.h.cache8_append(cl, k[l:l + 1], v[l:l + 1], _ints(one))
            p.h.cache8_attend(cl, q[l:l + 1], out[l:l + 1], lse=lse[l:l + 1])
        if check:
            p.check_attend(q, out, lse)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_loop_with_events(fmt):
    """Prompts in pieces, samples forked, decode steps, a compression event on the cache, more steps
    on what it kept, and sequences given up: the whole life of a cache against the model."""
    import eviction_gb300 as kvc
    L, B, H, G, d, bs, W, budget, T = 2, 5, 2, 3, 64, 16, 8, 64, 140
    p = Pair(L, B, H, d, bs, 10, fmt, n_blocks=80, G=G, window=W, budget=budget, max_T=T, seed=5)
    for n in ([70, 40, 0, 0, 0], [30, 61, 0, 0, 0]):
        p.grow(n)
        p.append(n)
    assert p.ref.fork([0, 0, 1], [2, 3, 4]) == 0
    p.h.cache8_fork(p.c, _ints([0, 0, 1]), _ints([2, 3, 4]))
    p.same()
    _steps(p, 20)
    p.same()
    # the event: dense keys from the cache, the kept set, the rows into new blocks
    k = torch.empty((L, B, H, T, d), dtype=torch.bfloat16, device="cuda")
    pad = torch.empty(B, dtype=torch.int32, device="cuda")
    p.h.cache8_gather(p.c, T, pad, k)
    dense, _, want_pad, _ = p.ref.gather(T)
    assert np.array_equal(k.double().cpu().numpy(), dense) and np.array_equal(pad.cpu().numpy(), want_pad)
    q = torch.randn((L, B, H * G, W, d), device="cuda").to(torch.bfloat16)
    buf, out = p.h.stage_buffers(T), p.h.outputs(T)
    credit = torch.zeros((L, B, H, T), device="cuda")
    p.h.mass_select(q, k, T, pad, p.c.seq_len.clone(), credit, buf["credit_post"], buf["mass"],
                    buf["score"], buf["seg_start"], buf["seg_len"], buf["quota"], buf["n_seg"],
                    out["kept_idx"], out["n_kept"])
    n_kept = out["n_kept"][0, :, 0].contiguous()
    assert n_kept.tolist() == [budget] * B
    new = p.c.with_sequences(torch.full_like(p.c.table, -1), torch.zeros_like(p.c.seq_len))
    p.h.cache8_grow(new, n_kept)
    p.h.cache8_compact(p.c, new, T, pad, out["kept_idx"], out["n_kept"],
                       credit_post=buf["credit_post"], credit_out=out["credit_out"])
    p.h.cache8_free(p.c, _ints(range(B)))
    assert p.h.device_status() == 0
    ref = p.ref.sibling()
    assert ref.grow(n_kept.cpu().numpy()) == 0
    p.ref.compact(ref, want_pad, out["kept_idx"].cpu().numpy(), out["n_kept"].cpu().numpy())
    p.ref.top = ref.top
    assert p.ref.free(range(B)) == 0
    ref.top = p.ref.top
    p.ref, p.c = ref, new
    p.same()
    # the same rows as the dense compaction keeps (requantised: at most half a step off)
    p.h.compact(k, k.clone(), buf["credit_post"], T, out["kept_idx"], out["n_kept"], out["k_out"],
                out["v_out"], torch.empty_like(out["credit_out"]))
    got = ref.gather(T)[0][:, :, :, T - budget:]
    want = out["k_out"].double().cpu().numpy()
    step = 2.0 ** -4 if fmt == "e4m3" else 0
    top = np.abs(want).max()
    assert (np.abs(got - want) <= step * np.abs(want) + top * (2.0 ** -16 if step else 1 / 127)).all()
    _steps(p, 20)
    p.same()
    p.h.cache8_free(p.c, _ints(range(B)))
    assert p.ref.free(range(B)) == 0
    p.same()
    assert p.ref.top == p.ref.N and not p.ref.ref.any()


def test_captured_step_replays():
    """Grow, append and attend in one CUDA graph, replayed with new inputs as the lengths grow; a
    second graph of the same handle in between."""
    p = Pair(1, 3, 2, 128, 16, 20, "e4m3", G=4, window=4)
    p.fill([100, 15, 0])
    one = _ints([1, 1, 1])
    k, v = p.new_rows(1), p.new_rows(1)
    q = torch.randn((1, 3, 8, 1, 128), device="cuda").to(torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:4], device="cuda")
    q3 = torch.randn((1, 3, 8, 3, 128), device="cuda").to(torch.bfloat16)
    out3, lse3 = torch.zeros_like(q3), torch.zeros(q3.shape[:4], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            p.h.cache8_grow(p.c, one)
            p.h.cache8_append(p.c, k, v, one)
            p.h.cache8_attend(p.c, q, out, lse=lse)
        g3 = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g3, stream=s):
            p.h.cache8_attend(p.c, q3, out3, lse=lse3)
    torch.cuda.synchronize()
    p.same()  # capturing ran nothing
    for _ in range(20):
        k.copy_(p.new_rows(1))
        v.copy_(p.new_rows(1))
        q.normal_()
        q3.normal_()
        g.replay()
        g3.replay()
        p.ref.grow([1, 1, 1])
        p.ref.append(k.double().cpu().numpy(), v.double().cpu().numpy(), [1, 1, 1])
        p.check_attend(q, out, lse)
        p.check_attend(q3, out3, lse3)
    p.same()
    assert p.h.device_status() == 0


def test_other_stream_and_tracing():
    p = Pair(1, 2, 1, 64, 16, 8, "int8", G=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.h.profile(True)
    p.h.cache8_grow(p.c, _ints([40, 9]), stream=s)
    torch.cuda.synchronize()
    names = {x["name"]: x["launches"] for x in p.h.profile_read(reset=True) if x["launches"]}
    p.h.profile(False)
    assert names == {"cache8_grow": 1}
    p.ref.grow([40, 9])
    p.same()
    with torch.cuda.stream(s):
        p.append([40, 9])
        p.attend(2)
    p.same()


def test_two_handles_on_two_streams():
    """Each handle has its own workspace: split sequences of both at once, many times."""
    import eviction_gb300 as kvc
    p = Pair(1, 2, 2, 128, 16, 130, "e4m3", G=4, window=64)
    p.fill([2000, 1500])
    h2 = kvc.Handle(p.cfg)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    want, got = [], []
    for n in (1, 40):
        q = torch.randn((1, 2, 8, n, 128), device="cuda").to(torch.bfloat16)
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:4], device="cuda")
        p.h.cache8_attend(p.c, q, out, lse=lse)
        want.append((q, out, lse))
    torch.cuda.synchronize()
    for i in range(40):
        for h, s in zip((p.h, h2), streams):
            q, out, lse = want[i % 2]
            o, l = torch.empty_like(out), torch.empty_like(lse)
            o.record_stream(s), l.record_stream(s)
            s.wait_stream(torch.cuda.current_stream())
            h.cache8_attend(p.c, q, o, lse=l, stream=s)
            got.append((i % 2, o, l))
    torch.cuda.synchronize()
    for k, o, l in got:
        assert torch.equal(o, want[k][1]) and torch.equal(l, want[k][2])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_largest_blocks(fmt):
    """Blocks of 1024 tokens through every call."""
    p = Pair(1, 2, 1, 128, 1024, 3, fmt, G=2, window=40, budget=1030, max_T=2100)
    p.fill([2100, 1])
    p.grow([30, 1023])
    p.append([30, 1023], spread=3.0, token_major=True)
    p.same()
    p.attend(1)
    p.attend(40)
    T = 2130
    k, v, pad, _ = cr.RefCache.gather(p.ref, T)
    import eviction_gb300 as kvc
    big = kvc.Handle(kvc.Config(1, 2, 1, 2, 128, T, 1030, window=40, n_recent=0))
    ko, po = torch.zeros((1, 2, 1, T, 128), dtype=torch.bfloat16, device="cuda"), _ints([0, 0])
    big.cache8_gather(p.c, T, po, ko)
    assert np.array_equal(ko.double().cpu().numpy(), k) and np.array_equal(po.cpu().numpy(), pad)
    kept, nk = _kept(p, 1030, T, [2130, 1024])
    other = Pair(1, 2, 1, 128, 1024, 2, fmt, budget=1030, max_T=T, seed=4)
    other.grow(nk[0, :, 0])
    assert p.ref.compact(other.ref, pad, kept, nk) == 0
    big.cache8_compact(p.c, other.c, T, po, _ints(kept), _ints(nk))
    other.same()


@pytest.mark.parametrize("G,n", [(100, 1), (33, 8), (512, 8)])
def test_attend_large_groups(G, n):
    p = Pair(1, 2, 1, 64, 16, 4, "int8", G=G, window=8)
    p.fill([60, 7])
    p.attend(n)


def test_attend_many_short_sequences():
    """More sequences than a CTA keeps the lengths of, most of them short or empty."""
    p = Pair(1, 3000, 1, 64, 16, 2, "e4m3", G=1, window=2)
    lens = p.rng.integers(0, 4, 3000)
    lens[::97] = 30
    p.fill(lens.tolist())
    p.attend(1)
    p.attend(2, n_q=p.rng.integers(0, 3, 3000))


def test_pools_past_32_bits():
    """A pool of over 2^32 bytes in which the last blocks are used."""
    import eviction_gb300 as kvc
    L, B, H, d, bs, N = 1, 1, 2, 128, 64, 280_000
    cfg = kvc.Config(L, B, H, 1, d, 256, 64, window=1, n_recent=0)
    c = kvc.Cache8.allocate(cfg, N, bs, 4)
    h = kvc.Handle(cfg)
    assert c.k_pool.numel() > 2 ** 32
    c.free_list.copy_(torch.arange(N, device="cuda"))  # the top of the stack: the last blocks
    n = _ints([200])
    h.cache8_grow(c, n)
    k = torch.randn((L, B, H, 200, d), device="cuda").to(torch.bfloat16)
    v = torch.randn((L, B, H, 200, d), device="cuda").to(torch.bfloat16)
    h.cache8_append(c, k, v, n)
    assert c.table.tolist() == [[N - 4, N - 3, N - 2, N - 1]]
    kd, vd, pad = torch.empty_like(k), torch.empty_like(v), _ints([-1])
    h.cache8_gather(c, 200, pad, kd, vd)
    assert ((kd - k).float().abs() <= 2.0 ** -4 * k.float().abs() + 2.0 ** -10 * 5).all()
    q = torch.randn((L, B, H, 1, d), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    h.cache8_attend(c, q, out)
    z = (q.double() @ kd.double().transpose(-1, -2)) * d ** -0.5
    want = torch.softmax(z, -1) @ vd.double()
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9).all()
    assert h.device_status() == 0
