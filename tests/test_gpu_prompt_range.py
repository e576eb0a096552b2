"""Prompt attention and rotary positions on the GPU where values, logits and angles are large, against
64 bits: as far as include/kvc.h says that they hold."""
import math

import numpy as np
import pytest
import torch

from tests import prompt_ref as pr
from tests.test_gpu_prompt import Prompts, _handle, _ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rise", [7.5, 13.5, 20.0, 31.0])
@pytest.mark.parametrize("at", [[130], [140, 290, 530], [699], list(range(128, 700))], ids=["second", "some", "last", "all"])
def test_prompt_large_values_of_later_keys(at, rise, d):
    """Keys behind the first tile whose logits lie `rise` (in base 2) above all of its own, and values that
    2^31 of fp32's exponents are too many for: the output is a mean of values all the same."""
    p = Prompts([700], 1, 2, d, False, v_scale=1e30, gap=0)
    p.q = torch.ones_like(p.q)
    p.k = torch.zeros_like(p.k)
    p.k[:, :, at] = rise * math.log(2) / math.sqrt(d)
    p.run()
    p.check()


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_logits_of_any_size(d):
    """Logits of 2^13 to 2^100 that are all but equal (a few of fp32's steps apart, one step is 2^16 and
    more of a weight from 2^27 on): the output stays within the values, and lse with the logits."""
    n = 400
    p = Prompts([n], 1, 2, d, False, gap=0)
    steps = torch.randint(-100, 101, (n,), generator=torch.Generator().manual_seed(d)).cuda()
    v = p.v.double()[0, 0]
    low, high = v.cummin(0).values, v.cummax(0).values
    room = 2.0 ** -7 * v.abs().cummax(0).values  # (weights and the result are rounded to bf16)
    for exp in range(10, 98):
        for sign in (1.0, -1.0):
            p.q, p.k = torch.zeros_like(p.q), torch.zeros_like(p.k)
            p.q[..., 0], p.q[..., 1] = sign * 8 * 1.25, 8 * 2.0 ** -21
            p.q[:, 1, :, 0] *= 1.5
            p.k[..., 0], p.k[..., 1] = 1.5 * 2.0 ** exp, steps * 2.0 ** exp
            out, lse = p.run()
            assert p.h.device_status() == 0
            for g in (0, 1):
                got, gl = out[0, g].double(), lse[0, g].double()
                assert torch.isfinite(got).all() and torch.isfinite(gl).all(), exp
                assert ((got <= high + room) & (got >= low - room)).all(), exp
                z = float(p.q[0, g, 0, 0]) * 1.5 * 2.0 ** exp * d ** -0.5
                assert ((gl - z).abs() <= 2.0 ** -12 * abs(z) + math.log(n)).all(), exp


@pytest.mark.parametrize("scale", [0.03, 1.0, 3.5])
@pytest.mark.parametrize("packed", [True, False])
def test_prompt_softmax_scale_of_the_configuration(packed, scale):
    p = Prompts([150, 1, 333], 2, 3, 128, packed, q_scale=1.0)
    p.h = _handle(2, 3, 128, softmax_scale=scale)
    out, lse = p.run()
    assert p.h.device_status() == 0
    for b in range(3):
        for hq in range(6):
            w, l, tol, ltol = pr.attention(p.rows(b, p.q, hq), p.rows(b, p.k, hq // 3), p.rows(b, p.v, hq // 3),
                                           float(np.float32(scale)))
            assert ((p.rows(b, out, hq).double() - w).abs() <= tol).all()
            assert ((p.rows(b, lse[..., None], hq)[..., 0].double() - l).abs() <= ltol).all()


@pytest.mark.parametrize("near,most", [(2.0 ** -14, 2 ** 20), (2.0 ** -18, 2 ** 22)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_angle_is_as_good_as_stated(interleaved, near, most):
    """Sines of angles next to whole half turns, so that the result's own rounding (bf16 has 8 bits: half a
    step is 2^-8 of a value of at most `near`) is no larger than the angle's: off by pi 2^-25 where the angle, up to
    half a turn, is rounded to fp32, by 2^-28 and 2^-49 of itself before; then a step of a sine next to 0 (below 2^-37)."""
    import eviction_gb300 as kvc
    d, f = 64, pr.frequencies(64)
    pos, pair = [], []
    at = np.arange(1, most, dtype=np.float64)
    for i in (1, 2, 3, 5, 8, 13):
        found = at[np.abs(np.sin(at * f[i])) < near].astype(int)
        assert len(found) > 2
        pos += found.tolist() + (-found).tolist()
        pair += [i] * (2 * len(found))
    n = len(pos)
    h = _handle(1, 1, d)
    x = torch.zeros((1, 1, 1, n, d), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    first, second = (lambda i: 2 * i, lambda i: 2 * i + 1) if interleaved else (lambda i: i, lambda i: i + d // 2)
    rows = torch.arange(n)
    i = torch.tensor(pair)
    x[0, 0, 0, rows, first(i)] = 1.0
    h.rotary(kvc.Rope(d, interleaved=interleaved), _ints([pos]), k=x, k_out=y)
    a = torch.tensor(pos, dtype=torch.float64) * torch.tensor(f, dtype=torch.float64)[i]
    got = y[0, 0, 0, rows, second(i)].double().cpu()
    bound = math.pi * 2.0 ** -25 + 2.0 ** -28 + 2.0 ** -49 * a.abs() + 2.0 ** -8 * a.sin().abs() + 2.0 ** -37
    off = (got - a.sin()).abs()
    assert (off <= bound).all(), float((off / bound).max())
