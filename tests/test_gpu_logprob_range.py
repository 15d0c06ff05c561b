"""vegas_token_logprobs on logits at both ends of fp32's range in one row.

The plain fp64 form and its tolerance are test_gpu_logprobs.py's.  a (x - m) is formed from
numbers whose difference may pass fp32's largest although its product with a < 1 does not.
"""
import math

import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_logprobs import check, run  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [3, 40, 5000, 70000])
@pytest.mark.parametrize("inv_t", [2.0 ** -100, 1e-20, 0.3, 0.7, 1.0, 4.0])
def test_lowest_values_beside_large_ones(dtype, V, inv_t):
    g = torch.Generator(device=DEV).manual_seed(V)
    x = torch.randn((5, V), generator=g, device=DEV).to(dtype)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    tok = torch.zeros(5, dtype=torch.int32, device=DEV)
    x[0] = low                                   # the lowest value everywhere but in one place
    x[0, V // 2] = high
    x[1, :] = low
    x[1, V - 1] = 1e37
    x[2, 0], x[2, 1] = low, high / 2             # among ordinary ones
    x[3] = -math.inf
    x[3, 1], x[3, 2] = low, 3e38
    tok[3] = 1
    x[4, ::2] = low
    x[4, 1] = 2.0 ** 110
    check(run(x, tok, 5, inv_t), x, tok, 5, inv_t)
    want = (float(low) - float(high)) * float(np.float32(inv_t))
    if V == 3 and inv_t < 0.4:                   # the point of it: a finite answer
        assert math.isfinite(want) and math.isfinite(float(run(x, tok, 0, inv_t)["logprob"][0]))
