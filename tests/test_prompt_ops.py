"""Rotary positions, prompt attention, gathered weight and the choice of the heaviest tokens without
a GPU: frequencies, refusals that need no device, the plain forms' own checks and the kernels'
sources."""
import ctypes
import glob
import math
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import prompt_ref as pr
from tests.test_cache8_sources import _code, _kernels

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "eviction_gb300", "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("rotary.cu", "prompt_attend.cu", "weigh.cu", "weigh_many.cu", "weigh.cuh", "heaviest.cu", "prompt.cuh")]


@pytest.fixture(scope="module")
def lib():
    from eviction_gb300 import build
    build.build()
    import eviction_gb300
    return eviction_gb300.load_library()


@pytest.mark.parametrize("kw", [
    dict(dim=128), dict(dim=16, base=500000.0), dict(dim=64, scaling="linear", factor=4.0),
    dict(dim=96, scaling="ntk", factor=8.0), dict(dim=128, base=500000.0, scaling="bands", factor=8.0, original=8192.0),
    dict(dim=64, scaling="bands", factor=2.0, low=0.0, high=32.0, original=100.0, base=1.0)])
def test_frequencies(lib, kw):
    """Turns per token in 2^-64 of a turn: within 2^-51 of the value (a few roundings of doubles)."""
    import eviction_gb300 as kvc
    r = kvc.Rope(**kw)
    want = pr.frequencies(**kw)
    for i, f in enumerate(want):
        t = f / (2 * math.pi)
        assert abs(r._c.turn[i] / 2.0 ** 64 - t) <= 2.0 ** -51 * t + 2.0 ** -64
    assert (r._c.dim, r._c.magnitude) == (kw["dim"], 1.0)


def test_far_positions_keep_their_angle(lib):
    """The kernel's integer angle at far positions against exact fractions of the held frequency."""
    import eviction_gb300 as kvc
    r = kvc.Rope(128)
    for i in (0, 3, 40, 63):
        for pos in (1, 131071, 2 ** 31 - 1, -5, -2 ** 31):
            held = Fraction(r._c.turn[i], 2 ** 64) * pos
            got = Fraction(((r._c.turn[i] * pos) % 2 ** 64) >> 32, 2 ** 32)
            off = (held - got) % 1
            assert 0 <= off < Fraction(1, 2 ** 32)


@pytest.mark.parametrize("kw", [
    dict(dim=0), dict(dim=24), dict(dim=144), dict(dim=-16), dict(dim=64, base=0.5), dict(dim=64, base=math.inf),
    dict(dim=64, base=math.nan), dict(dim=64, factor=0.0), dict(dim=64, factor=-1.0), dict(dim=64, factor=math.nan),
    dict(dim=64, magnitude=0.0), dict(dim=64, magnitude=math.inf),
    dict(dim=64, scaling="bands", factor=2.0), dict(dim=64, scaling="bands", original=8.0, low=4.0, high=4.0),
    dict(dim=64, scaling="bands", original=8.0, low=-1.0), dict(dim=64, scaling="bands", original=8.0, high=math.nan)])
def test_rope_refuses(lib, kw):
    import eviction_gb300 as kvc
    with pytest.raises(kvc.KvcError, match="KVC_ERR_ARG"):
        kvc.Rope(**kw)


def test_rope_refuses_other_scalings(lib):
    import eviction_gb300 as kvc
    with pytest.raises(ValueError, match="scaling"):
        kvc.Rope(64, scaling="other")


def test_null_arguments(lib):
    import eviction_gb300.kvc as k
    assert lib.kvc_rope_init(None, None) == -1
    cfg = k._RopeConfig(64, 0, 0, 1e4, 1, 1, 4, 0, 1)
    assert lib.kvc_rope_init(ctypes.byref(cfg), None) == -1
    for interleaved, scaling in ((2, 0), (0, 4), (0, -1)):
        cfg.interleaved, cfg.scaling = interleaved, scaling
        assert lib.kvc_rope_init(ctypes.byref(cfg), ctypes.byref(k._CRope())) == -1
    assert lib.kvc_rotary(None, None, None, None, None, None, 1, 1, 1, None, None, None) == -1
    assert lib.kvc_prompt_attend(None, None, None, None, 1, 1, None, None, None, None, None) == -1
    assert lib.kvc_cache8_weigh(None, None, None, 1, None, None, None, 1.0, None, 1, None) == -1
    assert lib.kvc_keep_heaviest(None, None, 1, 1, None, None, None, None, None) == -1


def test_packed_append_without_a_handle(lib):
    assert lib.kvc_cache8_append_packed(None, None, None, None, 1, None, None, None) == -1


def test_plain_rotation_is_a_rotation():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((3, 5, 64), generator=g, dtype=torch.float64)
    pos = torch.tensor([0, 1, 7, 100000, 2 ** 30])
    for inter in (False, True):
        f = pr.frequencies(32)
        y, _ = pr.rotary(x, pos, f, inter)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-12)
        assert torch.equal(y[..., 32:], x[..., 32:]) and torch.equal(y[:, 0], x[:, 0])
        # products of two turned rows depend on the distance of their positions alone
        a, b = (pr.rotary(x[0, :1], torch.tensor([p]), f, inter)[0] for p in (1007, 7))
        c, d = (pr.rotary(x[0, :1], torch.tensor([p]), f, inter)[0] for p in (1000, 0))
        assert torch.allclose(a @ b.T, c @ d.T, rtol=1e-9)


def test_plain_attention_and_weights_agree():
    """Weights gathered with attention()'s lse sum to the number of queries and are its weights."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn((20, 16), generator=g, dtype=torch.float64) for _ in "qkv")
    out, lse, _, _ = pr.attention(q, k, v, 0.25)
    w, _ = pr.weigh(q[None], k, lse[None], torch.zeros(20), 1.0, 0.25)
    assert abs(w.sum() - 20) < 1e-12
    one = torch.stack([torch.softmax((q[j] @ k[:j + 1].T) * 0.25, -1) @ v[:j + 1] for j in range(20)])
    assert torch.allclose(out, one, rtol=1e-12)


@pytest.mark.parametrize("w,length,budget,sink,recent,want", [
    ([5, 1, 2, 2, 9, 0], 6, 3, 1, 1, [0, 4, 5]), ([0, 1, 2, 2, 2, 0], 6, 3, 1, 1, [0, 2, 5]),
    ([1, 2, 3], 3, 5, 1, 1, [0, 1, 2]), ([1, 2, 3], 0, 5, 1, 1, []),
    ([9, 8, 7, 1, 1, 1], 6, 2, 4, 8, [4, 5]), ([9, 8, 7, 1, 1, 1], 6, 3, 4, 2, [0, 4, 5]),
    ([math.nan, -math.inf, 1, math.nan, 0, 0], 6, 3, 0, 0, [2, 4, 5]),
    ([math.nan, -math.inf, math.nan, -math.inf], 4, 3, 0, 0, [0, 1, 3]),
    ([-0.0, 0.0, -0.0, 1.0], 4, 2, 0, 0, [0, 3])])
def test_plain_choice(w, length, budget, sink, recent, want):
    assert pr.heaviest(w, length, budget, sink, recent) == want


def test_no_load_through_the_read_only_path():
    for path in SOURCES:
        assert not re.search(r"__ldg\b|\.global\.nc\b|__restrict__", _code(path)), path


def test_every_kernel_waits_before_it_reads():
    found = 0
    for path in SOURCES:
        for name, body in _kernels(_code(path)):
            found += 1
            assert body.count("before_all();") == 1, name
            ahead = body[:body.index("before_all();")]
            assert not re.search(r"\ba\.(pos|n_tok|first|lse|w|seq_len|status|n_q)\b\s*\[|atomic|\breturn\b", ahead), name
    assert found >= 4
