"""The prompt calls and the token log probabilities on a stream of their own and in a captured
graph, with everything they write cleared in between: each call has to be there, and to run in
its stream's order."""
import math

import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402
from test_gpu_rope import Rope  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Step:
    """A chunk of rows behind a cached prefix: rotated in, attended, judged."""

    def __init__(self, hq, hkv, d, seed=51):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rows, ctx = [1, 130, 0, 40], [3000, 20, 5, 700]
        self.hq, self.hkv, self.d, self.batch, self.total = hq, hkv, d, 4, sum(rows)
        pages = [(c + n + 15) // 16 for c, n in zip(ctx, rows)]
        table = np.zeros((4, max(pages)), dtype=np.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = np.arange(at, at + n)
            at += n
        self.bt = torch.from_numpy(table).to(DEV)
        shape = (at, hkv, 16, d)
        self.k0 = torch.randn(shape, generator=g, device=DEV).bfloat16()
        self.v0 = torch.randn(shape, generator=g, device=DEV).bfloat16()
        self.k, self.v = self.k0.clone(), self.v0.clone()
        self.kv = vg.paged_kv(self.k, self.v, self.bt, hq)
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=DEV)
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        self.qkv = torch.randn((self.total, (hq + 2 * hkv) * d), generator=g, device=DEV).bfloat16()
        self.freq = (1e4 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().to(DEV)
        self.vocab = 2311
        self.head = torch.randn((hq * d, self.vocab), generator=g, device=DEV) / math.sqrt(hq)
        self.tokens = torch.randint(0, self.vocab, (self.total,), generator=g, device=DEV,
                                    dtype=torch.int32)
        self.ws = torch.zeros(vg.vegas_prompt_workspace_size(self.kv, self.total, 4), dtype=torch.uint8,
                              device=DEV)
        n = self.total
        bf, i32 = torch.bfloat16, torch.int32
        self.out = dict(q=torch.empty((n, hq, d), dtype=bf, device=DEV),
                        attn=torch.empty((n, hq, d), dtype=bf, device=DEV),
                        logits=torch.empty((n, self.vocab), device=DEV),
                        lp=torch.empty(n, device=DEV), ent=torch.empty(n, device=DEV),
                        rank=torch.empty(n, dtype=i32, device=DEV),
                        ids=torch.empty((n, 4), dtype=i32, device=DEV),
                        lps=torch.empty((n, 4), device=DEV))

    def clear(self):
        """What the calls write holds nothing of an earlier run."""
        self.k.copy_(self.k0)
        self.v.copy_(self.v0)
        for t in self.out.values():
            t.fill_(float("nan") if t.is_floating_point() else -77)

    def run(self, stream=None):
        o, w, hq, hkv, d = self.out, self.qkv.stride(0), self.hq, self.hkv, self.d
        vg.vegas_rope_append(self.kv, self.qkv, w, self.qkv[:, hq * d:], w, self.qkv[:, (hq + hkv) * d:], w,
                             o["q"], self.start, self.ctx, None, None, 1, self.freq, d, False, 1.0,
                             self.total, self.batch, stream=stream)
        vg.vegas_prompt_attn(self.kv, o["q"], hq * d, o["attn"], self.start, self.ctx, self.total,
                             self.batch, 1 / math.sqrt(d), self.ws, self.ws.numel(), stream=stream)
        torch.matmul(o["attn"].view(self.total, hq * d).float(), self.head, out=o["logits"])
        vg.vegas_token_logprobs(o["logits"], vg.VEGAS_FP32, self.vocab, self.tokens, self.total,
                                self.vocab, 1.0, o["lp"], o["ent"], o["rank"], 4, o["ids"], o["lps"],
                                stream=stream)

    def written(self):
        return {**{k: t.clone() for k, t in self.out.items()}, "k": self.k.clone(), "v": self.v.clone()}


def same(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 2, 64)])
def test_a_replayed_step_writes_everything_again(hq, hkv, d):
    s = Step(hq, hkv, d)
    s.clear()
    s.run()
    torch.cuda.synchronize()
    want = s.written()
    for k in ("q", "attn", "logits", "lp", "ent", "lps"):
        assert torch.isfinite(want[k]).all(), k
    assert (want["rank"] >= 0).all() and (want["ids"] >= 0).all()
    assert not torch.equal(want["k"], s.k0) and not torch.equal(want["v"], s.v0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(3):
        s.clear()
        graph.replay()
        torch.cuda.synchronize()
        same(want, s.written())
    vg.vegas_read_device_status()


@pytest.mark.parametrize("given", [False, True])
def test_a_step_on_a_stream_of_its_own(given):
    """The stream as torch's current one, and as the calls' argument."""
    s = Step(32, 8, 128)
    s.clear()
    s.run()
    torch.cuda.synchronize()
    want = s.written()
    side = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(side):       # the clearing is on it too, just before
            s.clear()
            s.run(stream=side if given else None)
        side.synchronize()
        same(want, s.written())
    vg.vegas_read_device_status()


def test_log_probabilities_follow_what_their_stream_did_before():
    side = torch.cuda.Stream()
    g = torch.Generator(device=DEV).manual_seed(52)
    x = torch.randn((6, 8000), generator=g, device=DEV).bfloat16()
    tok = torch.randint(0, 8000, (6,), generator=g, device=DEV, dtype=torch.int32)
    torch.cuda.synchronize()
    full = torch.log_softmax(x.double(), -1)
    want = full.gather(1, tok.long()[:, None])[:, 0]
    ids = x.float().sort(dim=-1, descending=True, stable=True).indices[:, :3].to(torch.int32)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):           # logits and outputs are made on the stream itself
        y = torch.zeros_like(x)
        lp = torch.full((6,), 9.0, device=DEV)
        top = torch.full((6, 3), 9, dtype=torch.int32, device=DEV)
        lps = torch.full((6, 3), 9.0, device=DEV)
        y.copy_(x)
    vg.vegas_token_logprobs(y, vg.VEGAS_BF16, 8000, tok, 6, 8000, 1.0, lp, None, None, 3, top, lps,
                            stream=side)
    side.synchronize()
    assert torch.equal(top, ids)
    assert (lp.double() - want).abs().max() <= 1e-5 * (1 + want.abs().max())


def test_the_rotary_append_replayed_and_on_another_stream():
    rng = np.random.default_rng(0)
    rows = [int(x) for x in rng.integers(0, 4, 300)]
    c = Rope(8, 2, 64, rows, [int(x) for x in rng.integers(0, 90, 300)], rot=64, seed=53, pad=1)

    def clear():
        c.k_cache.copy_(c.before[0])
        c.v_cache.copy_(c.before[1])
        c.q_out.fill_(7)

    c.run()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(2):
        clear()
        graph.replay()
        torch.cuda.synchronize()
        c.check()
    side = torch.cuda.Stream()
    clear()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    c.check()
