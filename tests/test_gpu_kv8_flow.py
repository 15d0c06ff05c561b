"""The 8-bit cache as a serving step uses it: prompts appended to it in chunks, read back and
attended by the prompt call, windows verified with captured scores, positions selected and
drafted from; eagerly, on a stream of its own, from a graph, and two of them at once."""
import math

import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Step:
    """Two prompt chunks and a window of each sequence, then one draft step, over an 8-bit cache;
    the bf16 calls do the same over what is read back."""

    def __init__(self, hq, hkv, d, seed):
        self.gamma, self.batch, self.hq, self.hkv, self.d = 3, 3, hq, hkv, d
        chunks = [[130, 17, 400], [33, 64, 5], [4, 4, 4]]
        g = torch.Generator(device=DEV).manual_seed(seed)
        lens = np.sum(chunks, 0)
        pages = [(n + 15) // 16 for n in lens]
        perm = torch.randperm(sum(pages), generator=g, device=DEV).cpu().numpy()
        table, at = np.zeros((3, max(pages)), np.int32), 0
        for b, n in enumerate(pages):
            table[b, :n] = perm[at:at + n]
            at += n
        shape = (sum(pages), hkv, 16, d)
        self.bt, self.to_bt = torch.from_numpy(table).to(DEV), torch.from_numpy(
            (sum(pages) - 1 - table).astype(np.int32)).to(DEV)
        self.k8 = torch.full(shape, 0x7f, dtype=torch.uint8, device=DEV)       # NaN codes
        self.v8, self.ks = self.k8.clone(), torch.zeros(shape[:2], dtype=torch.uint8, device=DEV)
        self.vs = self.ks.clone()
        self.kv8 = vg.paged_kv8(self.k8, self.v8, self.ks, self.vs, self.bt, hq)
        self.k16 = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)
        self.v16 = self.k16.clone()
        self.kv16 = vg.paged_kv(self.k16, self.v16, self.to_bt, hq)
        self.inv = (1e4 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().to(DEV)
        self.scale = 1 / math.sqrt(d)
        self.chunks, ctx = [], np.zeros(3, np.int64)
        for rows in chunks:
            total = sum(rows)
            self.chunks.append(dict(
                total=total, ctx=ints(ctx.tolist()), upto=ints((ctx + rows).tolist()),
                start=ints([0] + np.cumsum(rows).tolist()),
                qkv=torch.randn((total, (hq + 2 * hkv) * d), generator=g, device=DEV).bfloat16(),
                q=torch.empty((total, hq, d), dtype=torch.bfloat16, device=DEV),
                out=torch.empty((total, hq, d), dtype=torch.bfloat16, device=DEV)))
            ctx = ctx + rows
        self.window_ctx = self.chunks[2]["ctx"]
        self.stride = int(self.window_ctx.max())
        need = max(vg.vegas_prompt_workspace_size(self.kv16, c["total"], 3) for c in self.chunks)
        self.pws = torch.zeros(need, dtype=torch.uint8, device=DEV)
        self.ws8 = torch.zeros(vg.vegas_verify_kv8_workspace_size(self.kv8, 3, 3), dtype=torch.uint8, device=DEV)
        self.ws16 = torch.zeros(max(256, vg.vegas_verify_workspace_size(self.kv16, 3, 3)), dtype=torch.uint8,
                                device=DEV)
        w = (3, 4, hq, d)
        self.out8, self.out16 = (torch.empty(w, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.s8, self.s16 = (torch.zeros((3, hkv, self.stride), device=DEV) for _ in range(2))
        self.k = ints([16, 8, 20])
        self.idx = torch.empty((3, hkv, 20), dtype=torch.int32, device=DEV)
        self.qd = torch.randn((3, hq, d), generator=g, device=DEV).bfloat16()
        self.d8, self.d16 = torch.empty_like(self.qd), torch.empty_like(self.qd)
        self.tail = ints([4, 4, 4])

    def run(self):
        hq, hkv, d = self.hq, self.hkv, self.d
        for c in self.chunks:
            x, w = c["qkv"], c["qkv"].stride(0)
            vg.vegas_rope_append_kv8(self.kv8, x, w, x[:, hq * d:], w, x[:, (hq + hkv) * d:], w, c["q"],
                                     c["start"], c["ctx"], None, None, 1, self.inv, d, False, 1.0,
                                     c["total"], 3)
            # the whole prefix again: a first page's codes may have been raised by this chunk
            vg.vegas_kv8_read(self.kv8, self.kv16, None, c["upto"], 3)
            vg.vegas_prompt_attn(self.kv16, c["q"], hq * d, c["out"], c["start"], c["ctx"], c["total"], 3,
                                 self.scale, self.pws, self.pws.numel())
        q = self.chunks[2]["q"]                       # (4 rows of each sequence: the window)
        vg.vegas_verify_attn_kv8(self.kv8, q, self.out8, self.s8, self.stride, self.window_ctx, 3, 3,
                                 0b1001, self.scale, self.ws8, self.ws8.numel())
        vg.vegas_verify_attn_capture(self.kv16, q, self.out16, self.s16, self.stride, self.window_ctx, 3,
                                     3, 0, 3, self.scale, self.ws16, self.ws16.numel())
        vg.vegas_select_topk(self.s8, self.stride, self.window_ctx, self.k, self.idx, 3, hkv, 20)
        for call, kv, out in ((vg.vegas_sparse_decode_attn_kv8, self.kv8, self.d8),
                              (vg.vegas_sparse_decode_attn, self.kv16, self.d16)):
            call(kv, self.qd, out, self.idx, 20, self.k, self.window_ctx, self.tail, 4, 3, self.scale)

    def results(self):
        return [t.clone() for t in (self.k8, self.v8, self.ks, self.vs, self.k16.nan_to_num(), self.out8,
                                    self.s8, self.idx, self.d8, self.chunks[1]["out"])]

    def clear(self):
        for t in (self.k8, self.v8):
            t.fill_(0x7f)
        for t in (self.k16, self.v16, self.out8, self.out16, self.d8, self.d16):
            t.fill_(float("nan"))
        for t in (self.ks, self.vs, self.idx):
            t.zero_()
        self.s8.zero_()
        self.s16.zero_()

    def check(self):
        """Both verifies attend the same numbers (the read back is exact), as does the prompt call over
        the window's rows: outputs differ by their roundings (2^-8 each), those of P (2^-8 in the
        bf16 calls, 2^-11 here) and of logits, all of them times magnitudes of a few."""
        for a, b in ((self.out8, self.out16), (self.d8, self.d16),
                     (self.out8, self.chunks[2]["out"].view(3, 4, self.hq, self.d))):
            a, b = a.double(), b.double()
            assert torch.isfinite(a).all()
            assert (a - b).norm() <= 2.0 ** -7 * b.norm()
        assert (self.s8 - self.s16).abs().max() <= 2.0 ** -13 * self.s16.abs().max()
        # the selected positions are those of the scores that this cache's verify captured
        for b, (n, k) in enumerate(zip(self.window_ctx.tolist(), self.k.tolist())):
            order = torch.sort(self.s8[b, :, :n], dim=-1, descending=True, stable=True).indices[:, :k]
            assert torch.equal(order.sort(-1).values.int(), self.idx[b, :, :k])


SHAPES = [(32, 8, 128), (16, 2, 64)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_step(hq, hkv, d):
    s = Step(hq, hkv, d, hq)
    s.run()
    vg.vegas_read_device_status()
    s.check()


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_step_on_a_stream_and_from_a_graph(hq, hkv, d):
    s = Step(hq, hkv, d, hq + 1)
    s.run()
    torch.cuda.synchronize()
    want = s.results()
    side = torch.cuda.Stream()
    s.clear()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(s.results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.run()
    for _ in range(3):
        s.clear()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.results(), want))
    vg.vegas_read_device_status()
    s.check()


def test_two_steps_at_once():
    """Two steps of their own buffers and workspaces on two streams, and the same alone."""
    steps = [Step(32, 8, 128, 5), Step(16, 2, 64, 6)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append(s.results())
        s.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    vg.vegas_read_device_status()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w))


def test_replays_follow_the_lengths():
    """A captured verify and draft step goes by the lengths that the buffers hold when it runs, with
    one workspace for all of them."""
    rng = np.random.default_rng(3)
    hq, hkv, d, gamma = 8, 2, 128, 4
    pages = 80
    k8 = torch.from_numpy(rng.integers(0, 126, (2 * pages, hkv, 16, d), dtype=np.uint8)).to(DEV)
    v8 = torch.from_numpy(rng.integers(0, 126, (2 * pages, hkv, 16, d), dtype=np.uint8)).to(DEV)
    ks = torch.full((2 * pages, hkv), 118, dtype=torch.uint8, device=DEV)
    vs = torch.full((2 * pages, hkv), 120, dtype=torch.uint8, device=DEV)
    bt = torch.from_numpy(rng.permutation(2 * pages).astype(np.int32).reshape(2, pages)).to(DEV)
    kv = vg.paged_kv8(k8, v8, ks, vs, bt, hq)
    q = torch.from_numpy(rng.standard_normal((2, gamma + 1, hq, d))).bfloat16().to(DEV)
    ctx = ints([1, 1])
    out = torch.empty_like(q)
    ws = torch.zeros(vg.vegas_verify_kv8_workspace_size(kv, 2, gamma), dtype=torch.uint8, device=DEV)
    scores = torch.empty((2, hkv, 1280), device=DEV)

    def call():
        vg.vegas_verify_attn_kv8(kv, q, out, scores, 1280, ctx, 2, gamma, 0b10001, 0.05, ws, ws.numel())

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([1275, 0], [5, 900], [0, 0], [128, 123], [700, 1275]):
        ctx.copy_(ints(lens))
        scores.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), scores.clone()
        scores.fill_(-1)
        out.fill_(float("nan"))
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], scores)
        assert not out.isnan().any()
        for b, n in enumerate(lens):
            assert (scores[b, :, n:] == -1).all()
    vg.vegas_read_device_status()
    assert not ws[:16].any()                          # the tickets are at zero again


def test_one_workspace_for_calls_of_many_sizes():
    """Batches and windows of every size through one workspace in turn, against workspaces of their
    own: what one call leaves there is not another's counter."""
    rng = np.random.default_rng(8)
    hq, hkv, d, pages = 8, 2, 128, 64
    cache = [torch.from_numpy(rng.integers(0, 126, (60 * pages, hkv, 16, d), dtype=np.uint8)).to(DEV)
             for _ in range(2)]
    scales = [torch.full((60 * pages, hkv), b, dtype=torch.uint8, device=DEV) for b in (118, 120)]
    bt = torch.from_numpy(rng.permutation(60 * pages).astype(np.int32).reshape(60, pages)).to(DEV)
    kv = vg.paged_kv8(*cache, *scales, bt, hq)
    cases = [(1, 4, [900]), (60, 0, [11 * i for i in range(60)]), (3, 9, [1000, 1, 500]), (60, 4, [1000] * 60),
             (2, 4, [1000, 1000]), (17, 1, [63 * i for i in range(17)])]
    one = torch.zeros(max(vg.vegas_verify_kv8_workspace_size(kv, b, g) for b, g, _ in cases),
                      dtype=torch.uint8, device=DEV)
    for batch, gamma, lens in cases + cases[::-1]:
        q = torch.from_numpy(rng.standard_normal((batch, gamma + 1, hq, d))).bfloat16().to(DEV)
        outs = []
        for ws in (one, torch.zeros_like(one)):
            out = torch.full_like(q, float("nan"))
            vg.vegas_verify_attn_kv8(kv, q, out, None, 0, ints(lens), batch, gamma, 0, 0.05, ws, ws.numel())
            outs.append(out)
        vg.vegas_read_device_status()
        assert not outs[1].isnan().any()
        assert torch.equal(*outs), (batch, gamma)
