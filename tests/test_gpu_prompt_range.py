"""Prompt attention and rotary positions on the GPU where values, logits and angles are large, against
64 bits: as far as include/kvc.h says that they hold."""
import math

import pytest
import torch

from tests.test_gpu_prompt import Prompts

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
