"""vegas_prompt_attn and vegas_rope_append where a call once went wrong or could have.

The plain fp64 form, its tolerance and the packed batches are test_gpu_prompt.py's.
"""
import math

import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402
from test_gpu_prompt import Prompt  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("rows,ctx", [([1, 3], [6000, 900]), ([300], [1500]), ([700, 2, 40], [0, 3000, 129])])
@pytest.mark.parametrize("level", [2.0 ** 21, -2.0 ** 21])
def test_tiles_taken_again_leave_their_second_probabilities(hq, hkv, d, rows, ctx, level):
    """Logits past 2^20: every tile's P is stored twice, at first from a reference that gives NaN.

    Logits are level + 0 .. -6 for every key, exact in fp32, so the result is that of the small
    numbers alone: the difference m - s is exact, an exponent is off by less than
    6 * 1.45 * 3 * 2^-24 < 2^-19 and the exponential and the fp32 sums by 2^-16 more: 2^-14 A
    beside the roundings of P (2^-8 A) and of the output (2^-8 |o|).
    """
    c = Prompt(hq, hkv, d, rows, ctx, seed=31, pad=1)
    c.scale = 1.0
    g = torch.Generator(device=DEV).manual_seed(32)
    c.q.zero_()
    c.q.view(c.total, -1, d)[:, :, :2] = 1
    small = []
    for b, n in enumerate(rows):
        L = ctx[b] + n
        pos = torch.arange(L, device=DEV)
        pg = torch.from_numpy(c.table[b].astype("int64")).to(DEV)[pos // 16]
        kk = torch.zeros((L, hkv, d), device=DEV)
        kk[:, :, 0] = level
        kk[:, :, 1] = -torch.randint(0, 7, (L, hkv), generator=g, device=DEV).float()
        c.k[pg, :, pos % 16] = kk.bfloat16()
        small.append((kk[:, :, 1].double(), c.v[pg, :, pos % 16].double()))
    first = c.run().clone()
    at = 0
    for b, n in enumerate(rows):
        x, v = small[b]
        seen = torch.arange(ctx[b] + n, device=DEV)[None] <= (ctx[b] + torch.arange(n, device=DEV))[:, None]
        for h in range(hq):
            kh = h // (hq // hkv)
            p = torch.softmax(torch.where(seen, x[:, kh][None], -math.inf), -1)
            ref, A = p @ v[:, kh], p @ v[:, kh].abs()
            got = first[at:at + n, h].double()
            assert torch.isfinite(got).all(), (b, h)
            tol = 1.01 * 2.0 ** -8 * (ref.abs() + A) + 2.0 ** -14 * A
            assert ((got - ref).abs() <= tol).all(), (b, h)
        at += n
    for _ in range(20):
        c.out[:c.used] = 0
        assert torch.equal(c.run(), first)
    vg.vegas_read_device_status()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128)])
@pytest.mark.parametrize("rows,ctx", [([1], [40000]), ([600], [9000]), ([300, 1, 2], [700, 9000, 4100])])
def test_shared_items_leave_the_counters_at_zero(hq, hkv, d, rows, ctx):
    c = Prompt(hq, hkv, d, rows, ctx, seed=33)
    counters = c.workspace()[:2 * torch.cuda.get_device_properties(0).multi_processor_count * 4]
    for _ in range(3):
        c.out[:c.used] = 0
        c.run()
        assert not counters.any()
    c.check(heads=(0, hq - 1), rows=24)
