"""The 8-bit paged cache at the ends of what its scales and queries may hold, and calls that reach the
attention kernel for many queries, within the per-token bound of tests/cache8_bounds.py."""
import numpy as np
import pytest
import torch

from tests import cache8_bounds as cb
from tests import cache8_ref as cr
from tests.test_gpu_cache8 import Pair, _ints

pytestmark = pytest.mark.gpu

# (queries, room in the table): few rows; many rows on the kernel for few; on the one for many
KERNELS = [(1, 1), (40, 1), (40, 512)]


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def _check(p, q, n_q=None, absent=None, status=0):
    """Attend with q (numpy, [1, B, Hq, n, d]) and compare."""
    qt = torch.from_numpy(q).to(torch.bfloat16).cuda()
    out = torch.full_like(qt, 7.0)
    lse = torch.full(qt.shape[:4], 7.0, device="cuda")
    p.h.cache8_attend(p.c, qt, out, lse=lse, n_q=None if n_q is None else _ints(n_q))
    assert p.h.device_status() == status
    want, wl, tol, ltol = cb.attend(p.ref, qt.double().cpu().numpy(), p.scale, n_q, absent)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - want) - tol
    assert (off <= 0).all(), (off.max(), np.argwhere(off > 0)[:3])
    seen = np.isfinite(wl)
    assert np.array_equal(np.isneginf(gl), ~seen)
    assert (np.abs(gl[seen] - wl[seen]) <= ltol[seen]).all()
    return got, gl


def _outlier_cache(n, room, fmt, bs, tokens, d=64):
    """A cache of ordinary rows whose keys have no first component, and queries that have one: a
    block whose keys are given a first component gets logits of that product alone on top."""
    p = Pair(1, len(tokens), 1, d, bs, -(-max(tokens) // bs), fmt, G=2, window=64, room=room, seed=n + bs)
    p.fill(tokens)
    p.ref.pool[0][..., 0] = 0
    q = p.rng.standard_normal((1, len(tokens), 2, n, d))
    q[..., 0] = 4.0
    return p, q


def _first(value, fmt):
    return cr.encode(np.array([float(value)]), fmt)[0]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("far", [12, 30, 60, 100])
@pytest.mark.parametrize("n,room", KERNELS)
def test_value_scale_outlier_without_weight(n, room, far, fmt):
    """One block's value scale is 2^far above the others'; its tokens' logits are far below the others',
    so it does not count, wherever it lies."""
    p, q = _outlier_cache(n, room, fmt, 8, [600, 420, 131])
    for b, i in ((0, 20), (1, 0), (2, 8)):   # tile 1, the very first block, tile 0
        blk = p.ref.table[b, i]
        p.ref.pool[0][0, blk, 0, :, 1:] = 0
        p.ref.pool[0][0, blk, 0, :, 0] = _first(-100, fmt)
        p.ref.scale[0][0, blk, 0] = 2.0 ** 5  # logit -100 2^5 4 / 8 = -1600
        p.ref.scale[1][0, blk, 0] *= 2.0 ** far
    p.ref.scale[1] *= np.float32(2.0 ** -min(far // 2, 50))
    p.sync_up()
    _check(p, q)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("far", [30, 100])
@pytest.mark.parametrize("n,room", KERNELS[1:])
def test_value_scale_outlier_among_masked_tokens(n, room, far, fmt):
    """The outlier is the block of the newest tokens: later queries see it, with all the weight there
    is, and earlier ones must not notice."""
    p, q = _outlier_cache(n, room, fmt, 8, [600, 424])
    for b in range(2):
        blk = p.ref.table[b, p.ref.blocks(p.ref.len[b]) - 1]
        p.ref.scale[1][0, blk, 0] *= 2.0 ** far
    p.ref.scale[1] *= np.float32(2.0 ** -(far // 2))
    p.sync_up()
    _check(p, q)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("where", ["middle", "newest"])
@pytest.mark.parametrize("n,room", KERNELS)
def test_key_scale_outlier(n, room, where, fmt):
    """Two blocks' key scales lie 2^9 to 2^67 above the others', whose logits are the usual ones;
    theirs are far below (or, for the newest tokens, above, where a query sees them)."""
    for far in (4, 11, 15, 16, 19, 20, 35, 62):
        p, q = _outlier_cache(n, room, fmt, 8, [600, 420, 131])
        for b in range(3):
            last = p.ref.blocks(p.ref.len[b]) - 1
            for i in ((1, last // 2) if where == "middle" else (last - 1, last)):
                blk = p.ref.table[b, i]
                p.ref.pool[0][0, blk, 0, :, 1:] = 0
                sign = 1 if where == "newest" and b == 1 else -1
                p.ref.pool[0][0, blk, 0, :, 0] = [_first(sign * x, fmt) for x in range(80, 112, 4)]
                p.ref.scale[0][0, blk, 0] = 2.0 ** far
        p.sync_up()
        _check(p, q)


@pytest.mark.parametrize("n,room", KERNELS)
def test_small_key_blocks_beside_large_ones(n, room):
    """Key blocks of every scale from 2^-40 to 2^8 at random, small values in all of them."""
    p, q = _outlier_cache(n, room, "int8", 8, [600, 420, 131])
    p.ref.scale[0][:] = 2.0 ** p.rng.integers(-40, -2, p.ref.scale[0].shape)
    p.ref.scale[0][0, ::7] = 2.0 ** 8
    p.ref.pool[0][:, ::7, :, :, 1:] = 0
    p.ref.pool[0][:, ::7, :, :, 0] = _first(-90, "int8")
    p.sync_up()
    _check(p, q)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("exp", [116, 126, 127, -100, -126, -133])
@pytest.mark.parametrize("n,room", KERNELS)
def test_largest_and_smallest_finite_queries(n, room, exp, fmt):
    """Query rows of one magnitude 2^exp: keys with nothing but a first component, all different, so
    that the softmax picks one token (or, of tiny queries, weighs all alike)."""
    d, tokens = 64, 96
    p = Pair(1, 1, 1, d, 16, 6, fmt, G=2, window=64, room=room * 2, seed=n)
    p.fill([tokens])
    p.ref.pool[0][:] = 0
    order = p.rng.permutation(tokens)
    # 96 different codes of one sign each, in e4m3 as in int8
    codes = (np.arange(96) + 8).astype(np.uint8)
    for t in range(tokens):
        p.ref.pool[0][0, p.ref.table[0, t // 16], 0, t % 16, 0] = codes[order[t]]
    p.ref.scale[0][:] = 2.0 ** -64
    p.sync_up()
    q = np.zeros((1, 1, 2, n, d))
    q[..., 0] = 1.5 * 2.0 ** exp if exp > -133 else 2.0 ** exp
    q[:, :, 1] *= -1
    got, lse = _check(p, q)
    if exp > 100:   # one token each: the bound above is wide there, this is not
        keys = cr.decode(codes, fmt)[order]
        v = p.ref.rows(1, 0, 0, 0)
        for j in range(n):
            see = tokens - n + j + 1
            for g, t in ((0, keys[:see].argmax()), (1, keys[:see].argmin())):
                assert (np.abs(got[0, 0, g, j] - v[t]) <= 2.0 ** -8 * np.abs(v[t])).all()
                z = q[0, 0, g, j, 0] * keys[t] * 2.0 ** -64 * p.scale   # (a few fp32 roundings)
                assert abs(lse[0, 0, g, j] - z) <= 2.0 ** -20 * abs(z)


@pytest.mark.parametrize("n,room", KERNELS)
def test_zero_keys_under_large_queries(n, room):
    """Codes of zero give a logit of zero whatever the query's and the block's scales are."""
    p = Pair(1, 1, 1, 64, 16, 16, "e4m3", G=2, window=64, room=room, seed=n)
    p.fill([250])
    p.ref.pool[0][:] = 0
    p.ref.scale[0][:] = 2.0 ** p.rng.choice([-64, 0, 64], p.ref.scale[0].shape)
    p.sync_up()
    q = np.full((1, 1, 2, n, 64), 1.75 * 2.0 ** 127)
    q[:, :, 1, :, ::2] *= -1
    _check(p, q)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n,room", KERNELS)
def test_logits_of_any_size(n, room, fmt):
    """Logits from 2^13 to 2^62 that are all but equal (a few of fp32's steps apart, one step is 2^16
    and more of a weight from 2^27 on): the output stays within the values, and lse with the logits."""
    d, tokens = 64, 3000
    p = Pair(1, 1, 1, d, 16, 188, fmt, G=2, window=64, room=room, seed=n)
    p.fill([tokens])
    p.ref.pool[0][:] = 0
    p.ref.pool[0][..., 0] = _first(96, fmt)
    codes = cr.encode(p.rng.integers(-100, 101, p.ref.pool[0].shape[:-1]).astype(float), fmt)
    p.ref.pool[0][..., 1] = codes
    v = p.ref.rows(1, 0, 0, 0)
    for exp in range(7, 57):
        p.ref.scale[0][:] = 2.0 ** (exp - 3)
        p.sync_up()
        for sign in (1, -1):
            q = np.zeros((1, 1, 2, n, d))
            q[..., 0], q[..., 1] = sign * 8 * 1.25, 8 * 2.0 ** -21
            q[:, :, 1, :, 0] *= 1.5
            qt = torch.from_numpy(q).to(torch.bfloat16).cuda()
            out = torch.full_like(qt, 7.0)
            lse = torch.full(qt.shape[:4], 7.0, device="cuda")
            p.h.cache8_attend(p.c, qt, out, lse=lse)
            got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
            assert np.isfinite(got).all() and np.isfinite(gl).all(), exp
            # (a mean of values, each weight off by 2^-11, rounded to bf16)
            room_for = 2.0 ** -7 * np.abs(v).max(0)
            assert (got <= v.max(0) + room_for).all() and (got >= v.min(0) - room_for).all(), exp
            z = q[..., 0] * 96 * 2.0 ** (exp - 3) * p.scale
            assert (np.abs(gl - z) <= 2.0 ** -16 * np.abs(z) + np.log(tokens)).all(), exp


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("room", [1, 256])
def test_bad_pages_are_absent_for_many_queries(room, fmt):
    """Tokens of a block out of range do not count, wherever it lies; limits stay where they were."""
    n, lens = 40, [60, 200, 333, 50]
    p = Pair(1, 4, 1, 64, 16, 21, fmt, G=2, window=64, room=room)
    p.fill(lens)
    good = p.ref.table.copy()
    absent = np.zeros((4, 400), bool)
    for b, i, what in ((0, 3, 10 ** 7), (1, 0, -1), (2, 8, p.ref.N), (2, 20, -5), (3, 0, -1), (3, 1, -1),
                       (3, 2, -1)):
        p.ref.table[b, i] = what
        absent[b, i * 16:(i + 1) * 16] = True
    p.sync_up()
    p.ref.table[:] = good
    q = p.rng.standard_normal((1, 4, 2, n, 64))
    _check(p, q, absent=absent, status=cr.BAD_INDEX)


@pytest.mark.parametrize("scale", [0.03, 1.0, 3.5])
@pytest.mark.parametrize("n,room", KERNELS)
def test_softmax_scale_of_the_configuration(n, room, scale):
    p = Pair(1, 3, 2, 128, 16, 30, "e4m3", G=3, window=64, room=room, softmax_scale=scale)
    p.scale = float(np.float32(scale))
    p.fill([450, 33, n])
    _check(p, p.rng.standard_normal((1, 3, 6, n, 128)))


def test_split_heads_of_many_queries_on_two_streams():
    """Two handles at once, both with heads cut into parts and a second launch that joins them."""
    import eviction_gb300 as kvc
    p = Pair(1, 2, 2, 128, 16, 130, "e4m3", G=4, window=64, room=64)
    p.fill([2000, 1500])
    h2 = kvc.Handle(p.cfg)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    want, got = [], []
    for n in (40, 64):
        q, out, lse = p.attend(n)
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
def test_largest_blocks_of_many_queries(fmt):
    p = Pair(1, 2, 1, 128, 1024, 3, fmt, G=2, window=40, room=64)
    p.fill([2100, 1025])
    p.attend(40)


def test_large_group_of_many_queries():
    p = Pair(1, 2, 1, 64, 16, 4, "int8", G=512, window=8, room=64)
    p.fill([60, 7])
    p.attend(8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,room", [(1, 1), (3, 1), (40, 1), (40, 512)])
def test_output_in_the_queries_place(n, room, d):
    """out may be q itself, also where a head's tokens are cut into parts."""
    p = Pair(1, 2, 2, d, 16, 130, "e4m3", G=4, window=64, room=room)
    p.fill([2000, 77])
    q, out, lse = p.attend(n)
    l2 = torch.zeros_like(lse)
    p.h.cache8_attend(p.c, q, q, lse=l2)
    assert torch.equal(q, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("n,room", KERNELS)
def test_captured_attention_of_growing_sequences(n, room):
    """One graph, replayed while the sequences grow past what they were at its capture."""
    p = Pair(1, 3, 2, 64, 16, 60, "int8", G=2, window=64, room=room)
    p.fill([n, 100, 0])
    q = torch.randn((1, 3, 4, n, 64), device="cuda").to(torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:4], device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            p.h.cache8_attend(p.c, q, out, lse=lse)
    torch.cuda.synchronize()
    for more in ([0, 0, 0], [1, 300, 17], [500, 5, 128], [3, 400, 600]):
        assert p.grow(more) == 0
        if max(more):
            p.append(more)
        q.normal_()
        g.replay()
        p.check_attend(q, out, lse)
    assert p.h.device_status() == 0


# ---- compaction between formats ----

@pytest.mark.parametrize("bs,to_bs", [(16, 16), (5, 64)])
def test_compact_to_int8_at_the_largest_scale(bs, to_bs):
    """e4m3 codes above 127 at the scale 2^64, beyond which int8's scale cannot grow: they become the
    largest code, with their sign."""
    lens, budget, T = [90, 30], 45, 90
    p = Pair(1, 2, 2, 64, bs, -(-T // bs), "e4m3", budget=budget, max_T=T)
    p.grow(lens)
    k, v = p.new_rows(T), p.new_rows(T)
    k[:, 0] *= 2.0 ** 72
    v[:, 1, 1] *= 2.0 ** 75
    v[:, 0, 0, ::3] *= 2.0 ** 71
    p.append(lens, rows=(k, v))
    p.same()
    other = Pair(1, 2, 2, 64, to_bs, -(-budget // to_bs), "int8", budget=budget, max_T=T, seed=9)
    kept, nk = np.full((1, 2, 2, budget), -1, np.int32), np.zeros((1, 2, 2), np.int32)
    for b, n in enumerate(lens):
        m = min(budget, n)
        nk[:, b] = m
        for h in range(2):
            kept[0, b, h, :m] = np.sort(p.rng.permutation(n)[:m]) + T - n
    assert other.grow(nk[0, :, 0]) == 0
    pad = T - np.array(lens, np.int32)
    assert p.ref.compact(other.ref, pad, kept, nk) == 0
    assert any((np.abs(x.view(np.int8)) == 127).any() for x in other.ref.pool)
    p.h.cache8_compact(p.c, other.c, T, _ints(pad), _ints(kept), _ints(nk))
    assert p.h.device_status() == 0
    other.same()
