"""vegas_token_logprobs against a plain fp64 implementation.

Tolerance: a thread sums at most E = ceil(V / 512) + 10 terms in fp32 before a tree
of 14 levels, each term off by 2^-21 (hardware exponential, fp32 argument up to 2^5):
Z and sum e y are off by at most (E + 24) 2^-24 + 2^-21 =: eps, relative to the sum of
magnitudes.  Then |logprob| is off by eps + 2^-22 |logprob|, and the entropy by
eps (2 + ln Z + H) for terms of magnitude y.  Ids and ranks are whole numbers.
"""
import math

import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(x, tokens, top, inv_t=1.0, vocab=None, stride=None, stream=None, fill=9):
    rows = x.shape[0]
    vocab = x.shape[1] if vocab is None else vocab
    stride = x.stride(0) if stride is None else stride
    out = dict(logprob=torch.full((rows,), float(fill), device=DEV),
               entropy=torch.full((rows,), float(fill), device=DEV),
               rank=torch.full((rows,), fill, dtype=torch.int32, device=DEV),
               ids=torch.full((rows, top), fill, dtype=torch.int32, device=DEV),
               lps=torch.full((rows, top), float(fill), device=DEV))
    dtype = vg.VEGAS_BF16 if x.dtype == torch.bfloat16 else vg.VEGAS_FP32
    vg.vegas_token_logprobs(x, dtype, stride, tokens, rows, vocab, inv_t, out["logprob"],
                            out["entropy"], out["rank"], top, out["ids"] if top else None,
                            out["lps"] if top else None, stream=stream)
    return out


def check(out, x, tokens, top, inv_t=1.0):
    V = x.shape[1]
    inv_t = float(np.float32(inv_t))
    eps = (V / 512 + 34) * 2.0 ** -24 + 2.0 ** -21
    for r in range(x.shape[0]):
        v = x[r].double().cpu().numpy()
        tok = int(tokens[r])
        m = v.max()
        if m == -math.inf:
            lnz, ent, y = 0.0, 0.0, np.full(V, -math.inf)
        else:
            y = (v - m) * inv_t
            e = np.exp(y)
            z = e.sum()
            lnz = math.log(z)
            p = e / z
            ent = -float((p[p > 0] * np.log(p[p > 0])).sum())

        def lp(i):
            # as fp32 holds it: below -3.4028e38 (the largest finite fp32 is 2^128 (1 - 2^-24))
            # that is -inf, which a lowest-value logit times 1.7 reaches
            with np.errstate(over="ignore"):
                return float(np.float32(y[i] - lnz))

        got = float(out["logprob"][r])
        if tok < 0:
            assert got == 0 and int(out["rank"][r]) == -1
        else:
            want = lp(tok)
            assert got == want or abs(got - want) <= eps + 2.0 ** -22 * abs(want), (r, got, want)
            rank = int((v > v[tok]).sum() + (v[:tok] == v[tok]).sum())
            assert int(out["rank"][r]) == rank, (r, int(out["rank"][r]), rank)
        assert abs(float(out["entropy"][r]) - ent) <= eps * (2 + abs(lnz) + ent), r
        order = np.argsort(-v, kind="stable")[:top]
        ids = [int(i) if v[i] > -math.inf else -1 for i in order] + [-1] * (top - len(order))
        assert out["ids"][r].tolist() == ids, r
        for j, i in enumerate(ids):
            g = float(out["lps"][r, j])
            assert (g == -math.inf) if i < 0 else (g == lp(i) or abs(g - lp(i)) <= eps + 2.0 ** -22 * abs(lp(i)))
    vg.vegas_read_device_status()


def logits(rows, V, dtype, seed, spread=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn((rows, V), generator=g, device=DEV) * spread).to(dtype)
    tok = torch.randint(0, V, (rows,), generator=g, device=DEV, dtype=torch.int32)
    best = x.float().argmax(1).to(torch.int32)
    return x, torch.where(torch.arange(rows, device=DEV) % 2 == 0, best, tok)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 9, 31, 100, 511, 1000, 4097, 32000, 50257, 151936])
@pytest.mark.parametrize("rows,top", [(1, 1), (5, 20), (37, 0), (3, 32)])
def test_sizes(dtype, V, rows, top):
    x, tok = logits(rows, V, dtype, V + rows)
    check(run(x, tok, top, 0.8), x, tok, top, 0.8)


@pytest.mark.parametrize("rows", [1, 2, 10, 20, 40, 80, 160, 400])
def test_every_cluster_size(rows):
    x, tok = logits(rows, 70001, torch.bfloat16, rows)
    check(run(x, tok, 4), x, tok, 4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_unaligned_rows(dtype):
    wide, _ = logits(9, 5003, dtype, 1)
    for off, V in ((1, 4999), (3, 5000), (0, 4096), (5, 17)):
        x = wide[:, off:off + V]
        _, tok = logits(9, V, dtype, 2)
        check(run(x, tok, 7), x, tok, 7)


def test_masks_empty_rows_and_padding_tokens():
    x, tok = logits(8, 6000, torch.float32, 3)
    g = torch.Generator(device=DEV).manual_seed(4)
    x[torch.rand(x.shape, generator=g, device=DEV) < 0.6] = -math.inf
    x[1] = -math.inf                                  # nothing left
    x[2] = -math.inf
    x[2, 4321] = -5.0                                 # one token left
    x[3] = torch.finfo(torch.float32).min             # the lowest value is not a mask
    x[4, :3000] = torch.finfo(torch.float32).min
    x[5, 17] = torch.finfo(torch.float32).max
    tok[0] = -1
    tok[1] = 777
    tok[2] = 4321
    tok[6] = int((x[6] == -math.inf).nonzero()[5])    # a masked token given
    x[7] = -math.inf                                  # lowest values among masked ones
    x[7, 100:140] = torch.finfo(torch.float32).min
    for t in (1.0, 1.7, 0.3):
        check(run(x, tok, 6, t), x, tok, 6, t)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1500, 40000])
def test_ties_go_to_the_lower_index(dtype, V):
    x = torch.zeros((6, V), dtype=dtype, device=DEV)
    x[1] = (torch.arange(V, device=DEV) % 3).to(dtype)
    x[2, ::2] = -0.0                                  # equal to +0
    x[3, V // 2:] = 1
    x[4] = torch.arange(V, device=DEV).div(200, rounding_mode="floor").to(dtype)
    x[5] = -x[4]
    tok = torch.tensor([V - 1, 5, V // 3, V - 1, V // 2, 3], dtype=torch.int32, device=DEV)
    check(run(x, tok, 32), x, tok, 32)


def test_large_row_offsets():
    """Rows whose offsets pass 2^31 elements."""
    stride = 2 ** 30 + 16
    big = torch.empty(4 * stride + 3000, dtype=torch.bfloat16, device=DEV)
    x, tok = logits(4, 2999, torch.bfloat16, 6)
    view = torch.as_strided(big, (4, 2999), (stride, 1))
    view.copy_(x)
    check(run(view, tok, 5), x, tok, 5)


def test_outputs_may_be_left_out_and_graphs_replay():
    x, tok = logits(6, 8000, torch.bfloat16, 7)
    want = run(x, tok, 3)
    ent = torch.empty(6, device=DEV)
    vg.vegas_token_logprobs(x, vg.VEGAS_BF16, 8000, None, 6, 8000, 1.0, None, ent, None, 0, None,
                            None)
    assert torch.equal(ent, want["entropy"])
    lp = torch.empty(6, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vg.vegas_token_logprobs(x, vg.VEGAS_BF16, 8000, tok, 6, 8000, 1.0, lp, None, None, 0, None,
                                None)
    for _ in range(2):
        lp.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lp, want["logprob"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run(x, tok, 3, stream=side)
    side.synchronize()
    for k in want:
        assert torch.equal(again[k], want[k])


def test_a_token_outside_the_vocabulary_is_recorded():
    x, tok = logits(3, 500, torch.float32, 8)
    tok[1] = 500
    out = run(x, tok, 1)
    with pytest.raises(vg.VegasError) as ei:
        vg.vegas_read_device_status()
    assert ei.value.status == 5
    assert float(out["logprob"][1]) == 0 and int(out["rank"][1]) == -1


@pytest.mark.parametrize("inv_t", [2.0 ** -100, 1e-20, 1e20, 2.0 ** 100])
def test_temperatures_at_the_ends_of_the_range(inv_t):
    x, tok = logits(4, 9000, torch.float32, 10)
    x[1, 100:5000] = -math.inf
    x[2, 100:5000] = torch.finfo(torch.float32).min
    x[3, 7] = 1e38
    check(run(x, tok, 5, inv_t), x, tok, 5, inv_t)
