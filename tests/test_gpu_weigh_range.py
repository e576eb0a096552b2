"""Gathered attention weight and the choice of the heaviest on the GPU: queries that see nothing."""
import math

import pytest
import torch

from tests.test_gpu_weigh import Weigh

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
