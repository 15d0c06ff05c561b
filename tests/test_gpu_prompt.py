"""vegas_prompt_attn against a plain fp64 implementation.

Tolerance, element by element, for o = sum_i p_i v_i / l with A = sum_i p_i |v_i| / l:
the output is rounded to bf16 (half a step, 2^-8 |o|), the probabilities are rounded
to bf16 before the second product (2^-8 A), and a logit of fp32 sums over d products
is off by at most delta = d * 2^-23 * max sum_j |q_j k_j| * scale, which moves every
p_i / l by at most a factor 1 +- 2 delta.  Second-order terms: 1 %.
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


class Prompt:
    """A packed batch; every cache slot outside the sequences holds NaN."""

    def __init__(self, hq, hkv, d, rows, ctx, seed=0, pad=0, q_extra=0, spare_pages=2, heavy=True,
                 num_pages=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.hq, self.hkv, self.d, self.rows, self.ctx = hq, hkv, d, rows, ctx
        self.batch, self.used = len(rows), sum(rows)
        self.total = self.used + pad
        pages = [(c + n + 15) // 16 if n else 0 for c, n in zip(ctx, rows)]
        self.max_pages = max(max((c + n + 15) // 16 for c, n in zip(ctx, rows)), 1) + 1
        self.num_pages = num_pages or sum(pages) + spare_pages
        shape = (self.num_pages, hkv, 16, d)
        if num_pages:
            self.k = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
            self.v = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
            order = np.arange(self.num_pages - sum(pages), self.num_pages)
        else:
            self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)
            self.v = self.k.clone()
            order = rng.permutation(self.num_pages)
        # entries past a sequence's pages must not be followed
        self.table = np.full((self.batch, self.max_pages), 2 ** 30, dtype=np.int32)
        at = 0
        u = torch.randn((d,), generator=g, device=DEV)
        u /= u.norm()
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
            L = ctx[b] + rows[b]
            if n == 0:
                continue
            kk = torch.randn((L, hkv, d), generator=g, device=DEV)
            if heavy:
                hit = torch.rand((L, hkv, 1), generator=g, device=DEV) < 0.05
                kk = torch.where(hit, 4 * u + 0.3 * kk, kk)
            vv = torch.randn((L, hkv, d), generator=g, device=DEV)
            pos = torch.arange(L, device=DEV)
            pg = torch.from_numpy(self.table[b].astype(np.int64)).to(DEV)[pos // 16]
            self.k[pg, :, pos % 16] = kk.bfloat16()
            self.v[pg, :, pos % 16] = vv.bfloat16()
        self.q_stride = hq * d + q_extra
        q = torch.randn((self.total, self.q_stride), generator=g, device=DEV)
        q[:, :hq * d] += (2 * u).repeat(hq)
        self.q = q.bfloat16()
        self.out = torch.full((self.total, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
        self.row_start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32,
                                      device=DEV)
        self.ctx_t = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        self.bt = torch.from_numpy(self.table).to(DEV)
        self.kv = vg.paged_kv(self.k, self.v, self.bt, hq)
        self.scale = 1 / math.sqrt(d)
        self.ws = None

    def workspace(self):
        if self.ws is None:
            n = vg.vegas_prompt_workspace_size(self.kv, self.total, self.batch)
            self.ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
        return self.ws

    def run(self, stream=None, ws=None):
        ws = self.workspace() if ws is None else ws
        vg.vegas_prompt_attn(self.kv, self.q, self.q_stride, self.out, self.row_start, self.ctx_t,
                             self.total, self.batch, self.scale, ws, ws.numel(), stream=stream)
        return self.out

    def check(self, heads=None, rows=None):
        """Every row (or a sample of each sequence's) against fp64."""
        at = 0
        g = self.hq // self.hkv
        for b, n in enumerate(self.rows):
            L = self.ctx[b] + n
            pick = torch.arange(n, device=DEV)
            if rows is not None and n > rows:
                pick = torch.unique(torch.cat([pick[:3], pick[-3:], torch.linspace(
                    0, n - 1, rows, device=DEV).long()]))
            pg = torch.from_numpy(self.table[b, :(L + 15) // 16].astype(np.int64)).to(DEV)
            for h in range(self.hq) if n else []:
                if heads is not None and h not in heads:
                    continue
                k = self.k[pg, h // g].reshape(-1, self.d)[:L].double()
                v = self.v[pg, h // g].reshape(-1, self.d)[:L].double()
                q = self.q[at + pick, h * self.d:(h + 1) * self.d].double()
                x = q @ k.t() * self.scale
                seen = torch.arange(L, device=DEV)[None] <= (self.ctx[b] + pick)[:, None]
                x = torch.where(seen, x, -math.inf)
                p = torch.softmax(x, -1)
                ref, A = p @ v, p @ v.abs()
                delta = self.d * 2.0 ** -23 * float((q.abs() @ k.abs().t()).max()) * self.scale
                tol = 1.01 * 2.0 ** -8 * (ref.abs() + A) + 2 * delta * A
                got = self.out[at + pick, h].double()
                assert torch.isfinite(got).all(), (b, h)
                worst = ((got - ref).abs() / tol).max()
                assert worst <= 1, (b, h, float(worst))
            at += n
        assert (self.out[self.used:] == 7).all()       # rows behind the last sequence
        vg.vegas_read_device_status()


SHAPES = [(8, 2, 64), (32, 8, 128), (4, 4, 128), (5, 1, 128), (12, 4, 64), (16, 1, 64), (14, 2, 128)]


@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_small_ragged_batches(hq, hkv, d):
    c = Prompt(hq, hkv, d, [1, 0, 17, 130, 33, 1, 0], [0, 5, 0, 15, 111, 300, 0], seed=hq, pad=2)
    c.run()
    c.check()


@pytest.mark.parametrize("n,ctx", [(1, 0), (1, 127), (1, 128), (2, 126), (16, 112), (64, 0),
                                   (65, 63), (127, 1), (128, 128), (129, 0), (300, 1000)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 2, 128)])
def test_one_sequence_at_tile_and_page_edges(hq, hkv, d, n, ctx):
    c = Prompt(hq, hkv, d, [n], [ctx], seed=n)
    c.run()
    c.check()


@pytest.mark.parametrize("hq,hkv,d", [(64, 1, 64), (64, 1, 128), (33, 1, 128), (3, 3, 64)])
def test_group_sizes(hq, hkv, d):
    c = Prompt(hq, hkv, d, [5, 70], [260, 3], seed=7, heavy=False)
    c.run()
    c.check()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (64, 8, 64)])
def test_decode_rows_with_long_caches_split_over_the_sms(hq, hkv, d):
    c = Prompt(hq, hkv, d, [1, 3, 1, 40], [9000, 4097, 1, 20000], seed=3)
    c.run()
    c.check()
    first = c.out.clone()
    for _ in range(3):                       # the workspace's counters are back at zero
        c.out[:c.used] = 0
        c.run()
        assert torch.equal(first, c.out)     # and the joins are in a fixed order


def test_long_prompt_and_chunk():
    c = Prompt(32, 8, 128, [4096, 1000], [0, 9000], seed=5)
    c.run()
    c.check(heads=(0, 13, 31), rows=300)


def test_many_short_sequences():
    rng = np.random.default_rng(2)
    rows = [int(x) for x in rng.integers(0, 60, 300)]
    ctx = [int(x) for x in rng.integers(0, 200, 300)]
    c = Prompt(8, 2, 64, rows, ctx, seed=6)
    c.run()
    c.check(heads=(0, 5))


def test_sharp_and_flat_rows():
    """Logits thousands apart, rising over the cache so that the maximum moves late."""
    c = Prompt(8, 2, 128, [200], [1500], seed=8)
    ramp = torch.linspace(0.01, 30, c.num_pages * 16, device=DEV)
    pg = torch.from_numpy(c.table[0, :107].astype(np.int64)).to(DEV)
    pos = torch.arange(1700, device=DEV)
    k = c.k[pg[pos // 16], :, pos % 16].float() * ramp[pos][:, None, None]
    c.k[pg[pos // 16], :, pos % 16] = k.bfloat16()
    c.run()
    c.check()


def test_strided_queries_and_rows_left_alone():
    c = Prompt(8, 2, 64, [77, 50], [10, 0], seed=9, pad=6, q_extra=2 * 2 * 64)
    c.run()
    c.check()


def test_workspace_serves_calls_of_other_sizes():
    big = Prompt(32, 8, 128, [1, 500], [12000, 2000], seed=10)
    small = Prompt(8, 2, 128, [1], [700], seed=11)
    ws = big.workspace()
    for c in (small, big, small, big):
        c.out[:c.used] = 0
        c.run(ws=ws)
        c.check(heads=(0, 7))


def test_on_another_stream_and_in_a_graph():
    c = Prompt(8, 2, 128, [1, 90], [5000, 30], seed=12)
    c.run()
    first = c.out.clone()
    side = torch.cuda.Stream()
    c.out[:c.used] = 0
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    assert torch.equal(first, c.out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(3):
        c.out[:c.used] = 0
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, c.out)
    # a replay reads the lengths as they are then
    c.ctx_t.copy_(torch.tensor([4000, 30], dtype=torch.int32))
    c.ctx = [4000, 30]
    graph.replay()
    c.check()


def test_lengths_that_do_not_fit_are_recorded_and_skipped():
    c = Prompt(8, 2, 64, [20, 30], [100, 50], seed=13)
    c.ctx_t[0] = c.max_pages * 16 - 19           # one position too many
    c.run()
    with pytest.raises(vg.VegasError) as ei:
        vg.vegas_read_device_status()
    assert ei.value.status == 5
    assert (c.out[:20] == 7).all() and not (c.out[20:] == 7).all()
    c.ctx_t[0] = 100
    c.run()
    c.check()


def test_a_page_outside_the_cache_is_recorded():
    c = Prompt(8, 2, 64, [20], [100], seed=14)
    good = c.bt.clone()
    c.bt[0, 2] = c.num_pages
    c.run()
    with pytest.raises(vg.VegasError) as ei:
        vg.vegas_read_device_status()
    assert ei.value.status == 5
    c.bt.copy_(good)
    c.run()
    c.check()


def test_empty_batches():
    c = Prompt(8, 2, 64, [0, 0], [10, 0], seed=15, pad=3)
    c.run()
    assert (c.out == 7).all()
    vg.vegas_read_device_status()


def test_cache_beyond_32_bit_offsets():
    c = Prompt(8, 8, 128, [60, 1], [100, 2000], seed=16, num_pages=140000)
    assert c.k.numel() > 2 ** 31
    c.run()
    c.check()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (64, 8, 64), (8, 8, 128)])
@pytest.mark.parametrize("batch", [1, 7, 31, 32, 33, 150])
def test_decode_batches(hq, hkv, d, batch):
    """One to three rows each: items whose tiles both softmax groups share, many a CTA."""
    rng = np.random.default_rng(batch)
    rows = [int(x) for x in rng.integers(1, 4, batch)]
    ctx = [int(x) for x in rng.integers(0, 1500, batch)]
    c = Prompt(hq, hkv, d, rows, ctx, seed=batch)
    c.run()
    c.check(heads=(0, hq // 2, hq - 1))
    first = c.out.clone()
    for _ in range(2):
        c.out[:c.used] = 0
        c.run()
        assert torch.equal(first, c.out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,ctx", [([600], [7000]), ([128, 1], [30000, 30000]), ([90, 33], [5000, 12345])])
def test_items_of_many_rows_split_over_ctas(d, rows, ctx):
    c = Prompt(8, 2, d, rows, ctx, seed=rows[0])
    c.run()
    c.check(heads=(1, 6))
    first = c.out.clone()
    for _ in range(4):
        c.out[:c.used] = 0
        c.run()
        assert torch.equal(first, c.out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("jump", [40.0, 400.0, 1e4])
def test_late_large_logits(d, jump):
    """Keys that exceed all earlier ones by far, in either half of a tile and in the rows' own
    positions: rows raise their reference once most of their cache has been summed."""
    c = Prompt(8, 2, d, [200], [900], seed=17, heavy=False)
    pg = torch.from_numpy(c.table[0].astype(np.int64)).to(DEV)
    for pos in (300, 440, 777, 950, 1010, 1099):
        u = c.q[:, :8 * d].float().view(-1, 8, d).mean((0, 1))
        c.k[pg[pos // 16], :, pos % 16] = (u / u.norm() * jump).bfloat16()
    c.run()
    c.check()


def test_very_low_logits_are_no_mask():
    c = Prompt(4, 2, 64, [70], [100], seed=18, heavy=False)
    c.q.copy_(torch.full_like(c.q, 1e17))
    pg = torch.from_numpy(c.table[0].astype(np.int64)).to(DEV)
    pos = torch.arange(170, device=DEV)
    c.k[pg[pos // 16], :, pos % 16] = -1e17          # every logit about -8e34
    c.run()
    mean = torch.cumsum(c.v[pg[pos // 16], :, pos % 16].double(), 0) / (pos + 1).double()[:, None, None]
    got = c.out.double().view(70, 2, 2, 64)
    ref = mean[100:, :, None, :]
    assert ((got - ref).abs() <= 2.0 ** -7 * (ref.abs() + 1)).all()
    vg.vegas_read_device_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,ctx", [([40], [900]), ([1, 1], [9000, 700]), ([600], [5000]), ([200, 3], [0, 2000])])
@pytest.mark.parametrize("levels", [(0, 2 ** 19), (2 ** 21, 0), (-2 ** 22, -2 ** 22), (2 ** 22, 2 ** 22),
                                    (2 ** 20, 2 ** 19, 2 ** 22), (-2 ** 21, -2 ** 19)])
def test_references_of_any_size(d, rows, ctx, levels):
    """Logits level + 0 .. -20, exact in fp32, the level changing every 150 positions.

    Only the greatest level seen counts; there |s - m| <= 20, so an exponent (rounded scale and
    log2 e, one fused step) is off by less than 20 * 1.45 * 3 * 2^-24 < 2^-17, the exponential and
    the fp32 sums by 2^-16 more: 2^-14 A beside the roundings of P and of the output.
    """
    c = Prompt(8, 2, d, rows, ctx, seed=11)
    c.scale = 1.0
    g = torch.Generator(device=DEV).manual_seed(12)
    c.q.zero_()
    c.q.view(c.total, -1, d)[:, :, :2] = 1
    for b, n in enumerate(rows):
        L = ctx[b] + n
        pos = torch.arange(L, device=DEV)
        pg = torch.from_numpy(c.table[b].astype(np.int64)).to(DEV)[pos // 16]
        kk = torch.zeros((L, 2, d), device=DEV)
        kk[:, :, 0] = torch.tensor(levels, device=DEV, dtype=torch.float32)[(pos // 150) % len(levels)][:, None]
        kk[:, :, 1] = -torch.randint(0, 21, (L, 2), generator=g, device=DEV).float()
        c.k[pg, :, pos % 16] = kk.bfloat16()
    c.run()
    at = 0
    for b, n in enumerate(rows):
        L = ctx[b] + n
        pg = torch.from_numpy(c.table[b, :(L + 15) // 16].astype(np.int64)).to(DEV)
        for h in (0, 7):
            k = c.k[pg, h // 4].reshape(-1, d)[:L].double()
            v = c.v[pg, h // 4].reshape(-1, d)[:L].double()
            x = c.q[at:at + n, h * d:(h + 1) * d].double() @ k.t()
            seen = torch.arange(L, device=DEV)[None] <= (ctx[b] + torch.arange(n, device=DEV))[:, None]
            p = torch.softmax(torch.where(seen, x, -math.inf), -1)
            ref, A = p @ v, p @ v.abs()
            worst = ((c.out[at:at + n, h].double() - ref).abs() /
                     (1.01 * 2.0 ** -8 * (ref.abs() + A) + 2.0 ** -14 * A)).max()
            assert worst <= 1, (b, h, float(worst))
        at += n
    vg.vegas_read_device_status()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 2, 64)])
@pytest.mark.parametrize("rows,ctx", [
    ([300, 1, 0, 1, 3], [700, 9000, 3, 5000, 4100]),       # a part of the CTAs for each kind
    ([1, 1, 900, 2, 33], [20, 60, 0, 4000, 6000]),
    ([1] * 40 + [200] + [1] * 9, [1000 + 77 * i for i in range(40)] + [500] + [9] * 9),
    ([500, 400, 1], [0, 0, 0]),                            # next to nothing of the one kind
    ([9, 1, 1], [0, 30000, 12000]),
])
def test_decode_rows_beside_prompts(hq, hkv, d, rows, ctx):
    c = Prompt(hq, hkv, d, rows, ctx, seed=21, pad=1)
    c.run()
    c.check(heads=(0, hq // 2, hq - 1), rows=24)
    first = c.out.clone()
    c.out[:c.used] = 0
    c.run()
    assert torch.equal(first, c.out)
