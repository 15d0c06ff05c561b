"""Attention over the 8-bit cache with V's scales at the ends of their range, 2^120 apart.

A row's sum takes every position by its logit alone, whatever its block's scale: positions whose values
are 2^-120 of the largest move the output by what they weigh.  The tolerances are those of test_gpu_kv8.py.
"""
import math

import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import kv8_case as k8  # noqa: E402
import self_speculative_sparse_paged_gb300 as vg  # noqa: E402
from test_gpu_kv8 import P_PARTS, dev, queries  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
LN2 = float(np.float32(math.log(2)))      # the softmax scale: logits in binades


class Logits:
    """One KV head whose keys are (x, 0, 0, ...) and whose queries begin with 1: position i has x[i]
    for its logit, in binades, and page j has 2^e[j] for V's scale."""

    def __init__(self, rng, x, e, d, hq):
        n, pages = len(x), (len(x) + 15) // 16
        codes = np.zeros((pages, 1, 16, d), np.uint8)
        codes.reshape(-1, d)[:n, 0] = k8.encode(np.asarray(x, np.float64))
        assert np.array_equal(k8.VALUE[codes.reshape(-1, d)[:n, 0]], x)
        self.codes, self.d, self.hq, self.n = codes, d, hq, n
        self.v_codes = k8.encode(rng.uniform(100, 448, (pages, 1, 16, d)) * rng.choice([-1, 1], (pages, 1, 16, d)))
        self.k_scale = np.full((pages, 1), 127, np.uint8)
        self.v_scale = (np.asarray(e, np.int64)[:, None] + 127).astype(np.uint8)
        self.v = k8.gather(self.v_codes, self.v_scale, np.arange(pages), 0, n)
        self.k = k8.gather(codes, self.k_scale, np.arange(pages), 0, n)

    def kv(self, batch):
        """The cache for `batch` sequences of the same pages."""
        self.held = [dev(a) for a in (self.codes, self.v_codes, self.k_scale, self.v_scale,
                                      np.tile(np.arange(len(self.codes), dtype=np.int32), (batch, 1)))]
        return vg.paged_kv8(*self.held, self.hq)

    def check(self, q, got, at, parts):
        """Rows of queries q (rows, d) with outputs `got`, over the positions `at`."""
        want, mag, _ = k8.attend(q, self.k[at], self.v[at], LN2)
        grid = 2.0 ** -17 * np.abs(q).max() * np.abs(self.k).sum(-1).max() if parts else 0.0
        d_logit = LN2 * (grid + 2.0 ** -20 * (np.abs(q) @ np.abs(self.k[at]).T).max())
        tol = 2.0 ** -8 * np.abs(want) + (parts + 2.0 ** -11 + 2 * d_logit + 2.0 ** -16) * mag
        err = np.abs(got - want)
        assert (err <= tol).all(), float((err / tol).max())


def one_heavy(n, at, lead):
    """Position `at` leads by `lead` binades, its page's scale is the largest and all others' the
    smallest; the other positions of its page weigh nothing."""
    x, e = np.zeros(n), np.full((n + 15) // 16, -60)
    x[at // 16 * 16:at // 16 * 16 + 16] = -96
    x[at], e[at // 16] = lead, 60
    return x, e


def by_rank(rng, n, rising):
    """Logits that fall along shuffled pages, with the scales rising as they fall, or falling with them."""
    pages = (n + 15) // 16
    rank = rng.permutation(pages)
    e = np.round(-60 + 120 * rank / (pages - 1)).astype(int)
    x = np.repeat(np.round((pages - 1 - rank if rising else rank) / (pages - 1) * 12), 16)[:n]
    return x, e


def anyhow(rng, n):
    return rng.integers(-7, 8, n).astype(float), rng.integers(-60, 61, (n + 15) // 16)


CASES = {
    "leads at the beginning": lambda rng, n: one_heavy(n, 3, 7),
    "leads at the end": lambda rng, n: one_heavy(n, n - 2, 7),
    "leads in the middle": lambda rng, n: one_heavy(n, n * 5 // 8, 7),
    "leads by far": lambda rng, n: one_heavy(n, 3, 18),
    "small scales where the weight is": lambda rng, n: by_rank(rng, n, True),
    "large scales where the weight is": lambda rng, n: by_rank(rng, n, False),
    "scales and logits anyhow": anyhow,
}


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("hq,d,n,batch", [(4, 128, 65536, 1), (8, 64, 65536, 1), (4, 128, 1999, 3), (3, 64, 300, 1),
                                          (24, 64, 40000, 1), (2, 128, 16384, 160), (1, 64, 16384, 160)])
def test_verify_sums_whatever_the_scales(hq, d, n, batch, case):
    """One sequence in pieces, short ones, and batches whose units one CTA holds from end to end."""
    rng = np.random.default_rng(n + hq)
    gamma = 1
    c = Logits(rng, *CASES[case](rng, n), d, hq)
    kv = c.kv(batch)
    q = queries(rng, (1, 2, hq, d))
    q[..., 0] = 1
    ctx = n - gamma - 1
    dq = q.to(DEV).expand(batch, 2, hq, d).contiguous()
    out = torch.full_like(dq, float("nan"))
    ws = torch.zeros(vg.vegas_verify_kv8_workspace_size(kv, batch, gamma), dtype=torch.uint8, device=DEV)
    vg.vegas_verify_attn_kv8(kv, dq, out, None, 0, dev(np.full(batch, ctx, np.int32)), batch, gamma, 0, LN2, ws,
                             ws.numel())
    vg.vegas_read_device_status()
    for got in out.double().cpu().numpy()[::max(1, batch // 8)]:
        for t in range(2):
            c.check(q[0, t].double().numpy(), got[t], np.arange(ctx + t + 1), P_PARTS)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("hq,d,n,batch", [(4, 128, 20000, 1), (8, 64, 20000, 1), (16, 128, 6000, 3), (3, 64, 300, 1),
                                          (16, 64, 20000, 4), (2, 128, 4000, 200), (1, 64, 4000, 200)])
def test_drafts_sum_whatever_the_scales(hq, d, n, batch, case):
    """Lists over one cluster, over a few CTAs, and of one CTA each."""
    rng = np.random.default_rng(n + hq)
    c = Logits(rng, *CASES[case](rng, n), d, hq)
    kv = c.kv(batch)
    q = queries(rng, (1, hq, d))
    q[..., 0] = 1
    k, tail = n - 20, 4
    dq = q.to(DEV).expand(batch, hq, d).contiguous()
    out = torch.full_like(dq, float("nan"))
    idx = dev(np.tile(np.arange(k, dtype=np.int32), (batch, 1, 1)))
    vg.vegas_sparse_decode_attn_kv8(kv, dq, out, idx, k, dev(np.full(batch, k, np.int32)),
                                    dev(np.full(batch, n - tail, np.int32)), dev(np.full(batch, tail, np.int32)), tail,
                                    batch, LN2)
    vg.vegas_read_device_status()
    at = np.concatenate([np.arange(k), n - tail + np.arange(tail)])
    for got in out.double().cpu().numpy()[::max(1, batch // 8)]:
        c.check(q[0].double().numpy(), got, at, 0.0)
