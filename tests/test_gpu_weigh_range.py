"""Gathered attention weight and the choice of the heaviest on the GPU: queries that see nothing, room
far beyond the lengths, other scales, other company, and the sizes at which kernels change."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_weigh import Weigh, _check_choice

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,G,n,packed", [(64, 2, 1, False), (128, 4, 3, False), (128, 7, 4, True), (64, 2, 60, False),
                                          (128, 7, 200, True), (128, 16, 300, False), (64, 3, 70, True)])
def test_weigh_rows_that_see_nothing_may_hold_anything(d, G, n, packed, fmt):
    """A query whose lse is not finite gives no token anything, whatever its row holds."""
    lens = [400, 300, 310]
    p = Weigh(1, 3, 2, d, 16, 26, fmt, G=G, seed=n, max_T=64, window=1)
    p.fill(lens)
    p.prepare(n, [n, max(n - 1, 1), n], packed=packed)
    g = torch.Generator(device="cuda").manual_seed(n)
    blind = torch.rand(p.lse.shape, generator=g, device="cuda") < 0.3
    if n > 1 and not packed:
        blind[:, 1] = False  # (one sequence without any)
    p.lse[blind] = torch.where(torch.rand(int(blind.sum()), generator=g, device="cuda") < 0.5, -math.inf, math.inf)
    odd = torch.tensor([math.nan, math.inf, -math.inf, 3e38], device="cuda").to(torch.bfloat16)
    rows = int(blind.sum())
    p.q[blind] = odd[torch.randint(0, 4, (rows, d), generator=g, device="cuda")]
    p.run(0.5)
    p.q[blind] = 0
    p.check(0.5)


@pytest.mark.parametrize("scale", [0.03, 1.0, 3.5])
@pytest.mark.parametrize("n", [1, 5, 100])
def test_weigh_softmax_scale_of_the_configuration(n, scale):
    p = Weigh(1, 3, 2, 128, 16, 30, "e4m3", G=3, max_T=64, window=1, softmax_scale=scale)
    p.scale = float(np.float32(scale))
    p.fill([450, 133, 100])
    p.prepare(n)
    p.run(0.9)
    p.check(0.9)


@pytest.mark.parametrize("cap,blocks", [(523, 1200), (14400, 1200), (70000, 1200), (70000, 33)])
@pytest.mark.parametrize("n", [1, 4, 20, 257])
def test_weigh_room_beyond_the_lengths(n, cap, blocks):
    """Weights and tables with room for far longer sequences."""
    lens = [520, 0, 300, 257]
    p = Weigh(1, 4, 1, 128, 16, blocks, "int8", n_blocks=100, G=16, max_T=64, window=1)
    p.fill(lens)
    p.prepare(n, [min(n, m) for m in lens], cap=cap)
    p.run(0.5)
    p.check(0.5)


@pytest.mark.parametrize("packed", [False, True])
def test_weigh_parts_of_many_sequences(packed):
    """More sequences than are sorted by their lengths, and queries cut into parts."""
    B = 140
    lens = [(37 * b) % 71 for b in range(B)]
    lens[3], lens[100], lens[139] = 256, 250, 129
    p = Weigh(1, B, 1, 64, 16, 16, "e4m3", n_blocks=600, G=16, max_T=64, window=1)
    p.fill(lens)
    p.prepare(256, lens, packed=packed, cap=256)
    p.run(0.5)
    p.check(0.5)


def test_weigh_in_other_company():
    """A sequence's weights with other sequences beside it and with other room: the same within the
    bounds (the order of a token's sum goes by the call's sizes), and the same bits at the same sizes."""
    lens = [520, 300, 257]
    for n, G in ((1, 4), (8, 4), (300, 16)):
        calls = []
        for some, cap in ((lens, 523), (lens, 523), (lens, 9000), ([520, 0, 0], 523)):
            p = Weigh(1, 3, 1, 128, 16, 33, "e4m3", G=G, max_T=64, window=1)
            p.fill(lens)
            counts = [min(n, m) for m in some]
            p.prepare(n, [min(n, m) for m in lens], cap=cap)
            p.counts = counts
            calls.append(p.run()[0, 0, :, :520].clone())
            p.check()
        assert torch.equal(calls[0], calls[1])


@pytest.mark.parametrize("cap", [2047, 2048, 2049, 8191, 8192, 8193, 32767, 32768, 32769])
def test_heaviest_where_kernels_change(cap):
    """The largest units of each kernel and the smallest of the next, random weights and ties, also in place."""
    g = torch.Generator(device="cuda").manual_seed(cap)
    w = torch.rand((1, 2, 2, cap), generator=g, device="cuda").log().neg().square()
    w[0, :, 1] = torch.randint(0, 4, (2, cap), generator=g, device="cuda").float()
    _check_choice(w, [cap, cap - 1], cap // 8, 4, 64)
    _check_choice(w, [cap, cap - 1], cap - 3, 0, 0)


@pytest.mark.parametrize("cap", [8000, 32768, 50000])
def test_heaviest_room_beyond_the_lengths(cap):
    g = torch.Generator(device="cuda").manual_seed(cap)
    w = torch.rand((1, 4, 2, cap), generator=g, device="cuda")
    _check_choice(w, [1536, 700, 3, 0], 512, 4, 64)
