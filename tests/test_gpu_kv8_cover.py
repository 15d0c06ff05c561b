"""The 8-bit verify's kernels one by one: every width with and without captured scores against the oracle,
scores of rows of unlike size, the whole of the tickets.  Tolerances as in test_gpu_kv8.py."""
import math

import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import kv8_case as k8  # noqa: E402
import self_speculative_sparse_paged_gb300 as vg  # noqa: E402
from test_gpu_kv8 import VERIFIES, Cache, check_verify, dev, queries, run_verify, spoil_unused  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def check_case(hq, hkv, d, gamma, mask, ctx, seed):
    rng = np.random.default_rng(seed)
    t = gamma + 1
    c = Cache(rng, [(n + t + 15) // 16 for n in ctx], hq, hkv, d)
    spoil_unused(c, ctx, t)
    c.upload()
    q = queries(rng, (len(ctx), t, hq, d))
    scale = 1 / math.sqrt(d)
    out, scores = run_verify(c, q, ctx, gamma, mask, scale, stride=max(max(ctx), 1) + 3)
    check_verify(c, q, out, scores, ctx, gamma, mask, scale)


@pytest.mark.parametrize("hq,hkv,d,gamma,mask,ctx", [v for v in VERIFIES if v[4]])
def test_verify_without_scores(hq, hkv, d, gamma, mask, ctx):
    check_case(hq, hkv, d, gamma, 0, ctx, hq * 100 + d + gamma + 1)


# every width of columns (8, 16, ... 64; 40 at head_dim 128), full and short of it by some
WIDTHS = [(d, cols, short) for d in (64, 128) for cols in range(8, 72 if d == 64 else 48, 8) for short in (0, 3)]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("d,cols,short", WIDTHS)
def test_verify_of_every_width(d, cols, short, captured):
    nq = cols - short
    t = max(n for n in range(1, 17) if nq % n == 0)
    mask = 1 | 1 << (t - 1) if captured else 0
    check_case(2 * nq // t, 2, d, t - 1, mask, [700, 0, 131], 10 * cols + d + short)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread", [3, 30])
def test_scores_of_rows_of_unlike_size(d, spread):
    """Query rows up to 2^(4 spread) apart, all captured: a score is off by what its terms allow."""
    rng = np.random.default_rng(d + spread)
    n, gamma, hq, hkv, scale = 700, 4, 8, 2, 0.1
    c = Cache(rng, [45], hq, hkv, d)
    c.upload()
    size = 2.0 ** -rng.integers(0, 4 * spread, (1, gamma + 1, hq, 1)).astype(np.float64)
    q = (queries(rng, (1, gamma + 1, hq, d)).double() * torch.from_numpy(size)).bfloat16()
    q[0, 2, 3] = 0
    _, scores = run_verify(c, q, [n], gamma, 0b11111, scale)
    got = scores.double().cpu().numpy()[0]
    for h in range(hkv):
        k = k8.gather(c.codes["k"], c.scale["k"], c.table[0], h, n)
        qq = q[0, :, 4 * h:4 * h + 4].double().numpy().reshape(-1, d)
        tol = 2.0 ** -17 * scale * (np.abs(qq) @ np.abs(k).T).sum(0)
        assert (np.abs(got[h] - scale * (qq @ k.T).sum(0)) <= tol + 1e-30).all()


@pytest.mark.parametrize("ctx", [[5000], [1275, 0, 900], [60 + 37 * i for i in range(50)], [40000, 3]])
def test_every_ticket_is_zero_again(ctx):
    """The workspace begins with a ticket for each CTA; shared units' tickets lie anywhere among them."""
    rng = np.random.default_rng(len(ctx))
    hq, hkv, d, gamma = 8, 2, 128, 4
    c = Cache(rng, [(n + 5 + 15) // 16 for n in ctx], hq, hkv, d)
    c.upload()
    q = queries(rng, (len(ctx), gamma + 1, hq, d)).to(DEV)
    out = torch.empty_like(q)
    size = vg.vegas_verify_kv8_workspace_size(c.kv, len(ctx), gamma)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        vg.vegas_verify_attn_kv8(c.kv, q, out, None, 0, dev(np.array(ctx, np.int32)), len(ctx), gamma, 0, 0.1, ws,
                                 size)
        assert not ws[:192 * 4].any()                  # (192: more CTAs than any call has)
        assert ws[192 * 4:].any()                      # units were shared
    vg.vegas_read_device_status()
