"""The prompt calls and the token log probabilities as a serving step uses them: a prompt is
rotated into the paged cache and attended, a second chunk follows it, the last rows are
attended again by the verify kernel, and the drafted tokens are judged from the logits."""
import math

import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rotated(x, pos, inv_freq):
    ang = pos[:, None].double() * inv_freq.double()
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x.double().chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).bfloat16()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 2, 64)])
@pytest.mark.parametrize("captured", [False, True])
def test_prompt_then_verify_then_judge(hq, hkv, d, captured):
    gamma, batch = 4, 3
    first, second = [130, 17, 400], [33, 64, 5]           # two chunks; the last rows are the window
    g = torch.Generator(device=DEV).manual_seed(hq)
    lens = [a + b for a, b in zip(first, second)]
    pages = [(n + 15) // 16 for n in lens]
    perm = torch.randperm(sum(pages), generator=g, device=DEV).cpu().numpy()
    table = np.zeros((batch, max(pages)), dtype=np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    bt = torch.from_numpy(table).to(DEV)
    kc = torch.full((sum(pages), hkv, 16, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    kv = vg.paged_kv(kc, vc, bt, hq)
    inv_freq = (1e4 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().to(DEV)
    scale = 1 / math.sqrt(d)
    width = (hq + 2 * hkv) * d
    chunks = []
    for rows, ctx in ((first, [0] * batch), (second, first)):
        total = sum(rows)
        chunks.append(dict(
            rows=rows, total=total, ctx=torch.tensor(ctx, dtype=torch.int32, device=DEV),
            start=torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=DEV),
            qkv=torch.randn((total, width), generator=g, device=DEV).bfloat16(),
            q=torch.empty((total, hq, d), dtype=torch.bfloat16, device=DEV),
            out=torch.empty((total, hq, d), dtype=torch.bfloat16, device=DEV)))
    need = max(vg.vegas_prompt_workspace_size(kv, c["total"], batch) for c in chunks)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    vws = torch.zeros(max(256, vg.vegas_verify_workspace_size(kv, batch, gamma)), dtype=torch.uint8,
                      device=DEV)
    vocab = 997
    head = torch.randn((hq * d, vocab), generator=g, device=DEV) / math.sqrt(hq)
    window = torch.empty((batch, gamma + 1, hq, d), dtype=torch.bfloat16, device=DEV)
    window_out = torch.empty_like(window)
    window_ctx = torch.tensor([n - gamma - 1 for n in lens], dtype=torch.int32, device=DEV)
    tokens = torch.randint(0, vocab, (batch * (gamma + 1),), generator=g, device=DEV, dtype=torch.int32)
    n = tokens.numel()
    lp, rank = torch.empty(n, device=DEV), torch.empty(n, dtype=torch.int32, device=DEV)
    ids, lps = torch.empty((n, 3), dtype=torch.int32, device=DEV), torch.empty((n, 3), device=DEV)
    logits = torch.empty((n, vocab), device=DEV)

    def step():
        for c in chunks:
            w = c["qkv"].stride(0)
            vg.vegas_rope_append(kv, c["qkv"], w, c["qkv"][:, hq * d:], w, c["qkv"][:, (hq + hkv) * d:], w,
                                 c["q"], c["start"], c["ctx"], None, None, 1, inv_freq, d, False, 1.0,
                                 c["total"], batch)
            vg.vegas_prompt_attn(kv, c["q"], hq * d, c["out"], c["start"], c["ctx"], c["total"], batch,
                                 scale, ws, ws.numel())
        ends = chunks[1]["start"][1:].long()
        back = torch.arange(-gamma - 1, 0, device=DEV)
        window.copy_(chunks[1]["q"][ends[:, None] + back])
        vg.vegas_verify_attn_capture(kv, window, window_out, None, 1, window_ctx, batch, gamma, 0, gamma,
                                     scale, vws, vws.numel())
        torch.matmul(window_out.view(n, hq * d).float(), head, out=logits)
        vg.vegas_token_logprobs(logits, vg.VEGAS_FP32, vocab, tokens, n, vocab, 1.0, lp, None, rank, 3,
                                ids, lps)

    step()
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t in (kc, vc):
            t.fill_(float("nan"))
        for c in chunks:
            c["out"].zero_()
        window_out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    vg.vegas_read_device_status()

    # every row of both chunks against fp64 over the whole sequence's rotated keys
    for b in range(batch):
        qs, ks, vs, got = [], [], [], []
        for c in chunks:
            lo, hi = int(c["start"][b]), int(c["start"][b + 1])
            pos = torch.arange(lo, hi, device=DEV) - lo + int(c["ctx"][b])
            x = c["qkv"][lo:hi].view(hi - lo, hq + 2 * hkv, d)
            qs.append(rotated(x[:, :hq], pos, inv_freq))
            ks.append(rotated(x[:, hq:hq + hkv], pos, inv_freq))
            vs.append(x[:, hq + hkv:])
            got.append(c["out"][lo:hi])
        q, k, v, o = (torch.cat(t).double() for t in (qs, ks, vs, got))
        L = lens[b]
        k, v = (t.repeat_interleave(hq // hkv, 1) for t in (k, v))
        x = torch.einsum("qhd,khd->hqk", q, k) * scale
        x.masked_fill_(torch.ones((L, L), dtype=torch.bool, device=DEV).triu(1), -math.inf)
        p = torch.softmax(x, -1)
        ref = torch.einsum("hqk,khd->qhd", p, v)
        size = torch.einsum("hqk,khd->qhd", p, v.abs())
        # bf16 output and probabilities (half a step each), and rotated queries and keys that may
        # round to the neighbouring bf16 number: a logit moves by at most 2^-8 (|q| . |k|) scale
        # for those few, bounded here by one such element of the largest product
        moved = 2.0 ** -7 * float((q.abs().amax() * k.abs().amax())) * scale
        tol = 1.01 * 2.0 ** -8 * (ref.abs() + size) + 2 * moved * size
        assert ((o - ref).abs() <= tol).all()
        # the verify kernel's rows over the same cache
        w = window_out[b].double()
        assert ((w - ref[-gamma - 1:]).abs() <= tol[-gamma - 1:] + 2.0 ** -8 * size[-gamma - 1:]).all()

    full = torch.log_softmax(logits.double(), -1)
    want = full.gather(1, tokens.long()[:, None])[:, 0]
    assert (lp.double() - want).abs().max() <= 1e-5 * (1 + want.abs().max())
    mine = logits.gather(1, tokens.long()[:, None])
    assert torch.equal(rank.long(), (logits > mine).sum(1))
    top = torch.topk(logits, 3, dim=-1)
    assert torch.equal(ids.long(), top.indices)
    assert (lps.double() - full.gather(1, top.indices)).abs().max() <= 1e-5 * (1 + full.gather(1, top.indices).abs().max())
    # greedy acceptance: the drafted tokens before the first one that is not the model's choice
    accepted = (rank.view(batch, gamma + 1)[:, :gamma] == 0).long().cumprod(1).sum(1)
    best = logits.argmax(1).view(batch, gamma + 1)
    again = (best[:, :gamma] == tokens.view(batch, gamma + 1)[:, :gamma]).long().cumprod(1).sum(1)
    assert torch.equal(accepted, again)
