"""The per-token bound of tests/cache8_bounds.py without a GPU: it agrees with the model, admits the
arithmetic that the library promises, and does not admit lost keys or lost weights."""
import numpy as np
import pytest

from tests import cache8_bounds as cb
from tests import cache8_ref as cr

SCALE = 0.125


def _cache(fmt, lens, bs=8, d=64, seed=0):
    rng = np.random.default_rng(seed)
    M = -(-max(lens) // bs)
    c = cr.RefCache(1, len(lens), 1, d, len(lens) * M, bs, M, fmt)
    assert c.grow(lens) == 0
    k, v = rng.standard_normal((2, 1, len(lens), 1, max(lens), d))
    c.append(k, v, lens)
    q = rng.standard_normal((1, len(lens), 2, 3, d))
    return c, (q.astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)


def _kernel(c, q, b, g, j, nq, keys=lambda k, ks: k, drop=0.0):
    """One row in fp32 with fp16 weights.  keys: what is done to the keys before the products;
    drop: log2 by which the weights' reference lies too high."""
    m = int(c.len[b])
    see = m - nq + j + 1
    pos = np.arange(see)
    blk = c.table[b, pos // c.bs]
    ks, vs = (c.scale[w][0, blk, 0].astype(np.float32) for w in (0, 1))
    k = cr.decode(c.pool[0][0, blk, 0, pos % c.bs], c.fmt).astype(np.float32)
    v = cr.decode(c.pool[1][0, blk, 0, pos % c.bs], c.fmt).astype(np.float32)
    z = keys(k, ks) @ q[0, b, g, j].astype(np.float32) * ks * np.float32(SCALE * 1.4426950408889634)
    e = np.log2(vs)
    x = (z + e).astype(np.float32)
    w = np.exp2(x - x.max()).astype(np.float32)
    total = (w * np.exp2(-e)).sum(dtype=np.float32)
    w16 = (w * np.float32(2.0 ** -drop)).astype(np.float16).astype(np.float32)
    out = (w16 @ v) / total * np.float32(2.0 ** drop)
    return out.astype(np.float64), (x.max() + np.log2(total)) * np.log(2.0)


def _inside(c, q, **kw):
    out, lse, tol, ltol = cb.attend(c, q, SCALE)
    ok = True
    for b in range(c.B):
        for g in range(2):
            for j in range(3):
                o, l = _kernel(c, q, b, g, j, 3, **kw)
                ok = ok and (np.abs(o - out[0, b, g, j]) <= tol[0, b, g, j]).all()
                ok = ok and abs(l - lse[0, b, g, j]) <= ltol[0, b, g, j]
    return ok


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_agrees_with_the_model(fmt):
    c, q = _cache(fmt, [100, 3, 41])
    out, lse, _, _ = cb.attend(c, q, SCALE, [3, 3, 0])
    want, wl, _, _ = c.attend(q, SCALE, [3, 3, 0])
    assert np.allclose(out, want, rtol=1e-12, atol=1e-13)
    assert np.allclose(lse, wl, rtol=1e-12)
    # tokens that do not count: as a cache without them, where they are the oldest
    absent = np.zeros((3, 100), bool)
    absent[0, :40] = True
    got = cb.attend(c, q, SCALE, absent=absent)[0][:, 0]
    c.table[0, :8] = c.table[0, 5:13]
    c.len[0] = 60
    assert np.allclose(got, c.attend(q, SCALE)[0][:, 0], rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_admits_the_promised_arithmetic(fmt):
    c, q = _cache(fmt, [200, 3, 41])
    assert _inside(c, q)
    c.scale[1][0, ::5] *= 2.0 ** 40
    c.scale[1] *= np.float32(2.0 ** -20)
    assert _inside(c, q)


def test_does_not_admit_lost_keys():
    """Keys of ordinary scale beside a few of a large one, with no weight: all set to zero."""
    c, q = _cache("int8", [200, 77, 41])
    c.pool[0][..., 0] = 0
    q[..., 0] = 4.0
    for b in range(3):
        c.pool[0][0, c.table[b, 2], 0] = 0
        c.pool[0][0, c.table[b, 2], 0, :, 0] = np.uint8(256 - 100)
        c.scale[0][0, c.table[b, 2]] = 2.0 ** 30
    assert _inside(c, q)
    assert not _inside(c, q, keys=lambda k, ks: np.where(ks[:, None] < 1, 0, k))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_does_not_admit_lost_weights(fmt):
    c, q = _cache(fmt, [200, 77, 41])
    assert not _inside(c, q, drop=20)
