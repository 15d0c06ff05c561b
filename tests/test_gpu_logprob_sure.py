"""vegas_token_logprobs where one token has nearly all the probability: ln Z = ln(1 + r) of a small r.

Other tokens lie 6 to 20 nats below (a = 1), the given one in a 16-byte chunk of its own, so that
its thread holds nothing else and r is summed apart from the 1.  A term of r is 2^y with
|y| <= 29 from three rounded factors (3 * 29 * ln 2 * 2^-24 = 3.6e-6), moved from a reference at
most 8 powers of two off (1e-6, and 2^-22 for either hardware exponential), and summed over fewer
than 24 roundings (1.5e-6): r is off by less than 2^-17 of itself, and so is ln(1 + r) < r.  The
entropy adds r_i times a distance of 6 or more, moved once (twice that): 2^-15 of itself.
"""
import math

import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402
from test_gpu_logprobs import run  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 64), (torch.bfloat16, 4000), (torch.float32, 2000),
                                     (torch.bfloat16, 60000), (torch.float32, 30000)])
@pytest.mark.parametrize("gap", [6.0, 12.0, 18.0])
def test_a_sure_token(dtype, V, gap):
    rows, step = 6, 128 // torch.finfo(dtype).bits       # logits of a chunk
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (-gap - 2 * torch.rand((rows, V), generator=g, device=DEV)).to(dtype)
    tok = (torch.arange(rows, device=DEV) * (V // step // rows) * step).to(torch.int32)
    chunk = torch.arange(V, device=DEV) // step
    for r in range(rows):
        at = int(tok[r])
        x[r, chunk % 512 == at // step % 512] = -math.inf    # whatever its thread may hold beside it
        x[r, at] = 0.0
    x[4] += 40                                               # the level does not count
    out = run(x, tok, 2)
    for r in range(rows):
        v = x[r].double()
        others = v[(v > -math.inf) & (torch.arange(V, device=DEV) != int(tok[r]))] - v.max()
        rest = float(others.exp().sum())
        lnz = math.log1p(rest)
        ent = lnz + float((others.exp() * -others).sum()) / (1 + rest)
        got = float(out["logprob"][r])
        assert abs(got + lnz) <= 2.0 ** -17 * lnz, (r, got, -lnz)
        assert float(out["lps"][r, 0]) == got and int(out["ids"][r, 0]) == int(tok[r])
        assert abs(float(out["entropy"][r]) - ent) <= 2.0 ** -15 * ent, (r, float(out["entropy"][r]), ent)
    vg.vegas_read_device_status()
