"""vegas_rope_append against a plain fp64 implementation.

Tolerance: the rotated element is rounded to bf16 (half a step, 2^-8 |y|) from fp32;
sine and cosine of an angle reduced in fp64 are off by at most 2^-21, the three fp32
operations by 2^-22 of |x| + |y| together: 2^-20 scale (|a| + |b|) covers both.
Values, pass-through elements and every other slot are copied: bit for bit.
"""
import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Rope:
    def __init__(self, hq, hkv, d, rows, ctx, rot, axes=1, interleaved=False, pad=0, scale=1.0,
                 seed=0, positions=None, fused=True, num_pages=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.__dict__.update(hq=hq, hkv=hkv, d=d, rows=rows, ctx=ctx, rot=rot, axes=axes,
                             interleaved=interleaved, scale=scale)
        self.batch, self.used = len(rows), sum(rows)
        self.total = self.used + pad
        pages = [(c + n + 15) // 16 for c, n in zip(ctx, rows)]
        self.max_pages = max(pages) + 1
        self.num_pages = num_pages or sum(pages) + 2
        order = (np.arange(self.num_pages)[::-1] if num_pages else rng.permutation(self.num_pages))
        self.table = np.full((self.batch, self.max_pages), 2 ** 30, dtype=np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.num_pages, hkv, 16, d)

        def cache():
            if num_pages:
                return torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
            return torch.randn(shape, generator=g, device=DEV).bfloat16()

        self.k_cache, self.v_cache = cache(), cache()
        if fused:
            qkv = torch.randn((self.total, (hq + 2 * hkv) * d), generator=g, device=DEV).bfloat16()
            self.q, self.k, self.v = qkv, qkv[:, hq * d:], qkv[:, (hq + hkv) * d:]
            self.strides = (qkv.stride(0),) * 3
        else:
            self.q = torch.randn((self.total, hq * d), generator=g, device=DEV).bfloat16()
            self.k = torch.randn((self.total, hkv * d + 8), generator=g, device=DEV).bfloat16()
            self.v = torch.randn((self.total, hkv * d + 24), generator=g, device=DEV).bfloat16()
            self.strides = (self.q.stride(0), self.k.stride(0), self.v.stride(0))
        self.q_out = torch.full((self.total, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
        half = rot // 2
        self.inv_freq = (1e6 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().to(DEV)
        self.positions = positions
        self.pair_axis = None
        if axes > 1:
            if positions is None:
                self.positions = torch.randint(-50, 10 ** 6, (axes, self.total), generator=g,
                                               device=DEV, dtype=torch.int32)
            self.pair_axis = torch.randint(0, axes, (half,), generator=g, device=DEV,
                                           dtype=torch.int32)
        self.row_start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32,
                                      device=DEV)
        self.ctx_t = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        self.bt = torch.from_numpy(self.table).to(DEV)
        self.kv = vg.paged_kv(self.k_cache, self.v_cache, self.bt, hq)
        self.before = None if num_pages else (self.k_cache.clone(), self.v_cache.clone())

    def run(self, q_out=None, stream=None):
        vg.vegas_rope_append(self.kv, self.q, self.strides[0], self.k, self.strides[1], self.v,
                             self.strides[2], self.q_out if q_out is None else q_out,
                             self.row_start, self.ctx_t, self.positions, self.pair_axis, self.axes,
                             self.inv_freq if self.rot else None, self.rot, self.interleaved,
                             self.scale, self.total, self.batch, stream=stream)

    def turned(self, x, p):
        """fp64 rotation of x [n][heads][d] at positions p [n][half], and |a| + |b|."""
        y, mag = x.clone(), torch.zeros_like(x)
        if self.rot:
            ang = p * self.inv_freq.double()
            cos, sin = ang.cos()[:, None] * self.scale, ang.sin()[:, None] * self.scale
            first = slice(0, self.rot, 2) if self.interleaved else slice(0, self.rot // 2)
            second = slice(1, self.rot, 2) if self.interleaved else slice(self.rot // 2, self.rot)
            a, b = x[..., first], x[..., second]
            y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
            mag[..., first] = mag[..., second] = (a.abs() + b.abs()) * abs(self.scale)
        return y, mag

    def check(self, q=None):
        q = self.q if q is None else q
        n = self.used
        seq = torch.from_numpy(np.repeat(np.arange(self.batch), self.rows)).to(DEV)
        start = self.row_start[:-1].long()
        pos = torch.arange(n, device=DEV) - start[seq] + self.ctx_t.long()[seq]
        half = self.rot // 2
        if self.positions is None:
            p = pos[:, None].expand(n, half).double()
        else:
            ax = torch.zeros(half, dtype=torch.long, device=DEV) if self.pair_axis is None else self.pair_axis.long()
            p = self.positions[ax][:, :n].t().double()

        def close(got, src):
            ref, mag = self.turned(src.double(), p)
            tol = 2.0 ** -8 * ref.abs() * 1.001 + 2.0 ** -20 * mag
            bad = (got.double() - ref).abs() > tol
            assert not bad.any(), float(((got.double() - ref).abs() - tol).max())
            assert torch.equal(got[..., self.rot:], src[..., self.rot:])

        page = torch.from_numpy(self.table.astype(np.int64)).to(DEV)[seq, pos // 16]
        close(self.q_out[:n], q[:n, :self.hq * self.d].reshape(n, self.hq, self.d))
        close(self.k_cache[page, :, pos % 16], self.k[:n, :self.hkv * self.d].reshape(n, self.hkv, self.d))
        v = self.v[:n, :self.hkv * self.d].reshape(n, self.hkv, self.d)
        assert torch.equal(self.v_cache[page, :, pos % 16], v)
        if self.before is not None:      # no other slot changed
            left = torch.ones(self.k_cache.shape[:1] + (16,), dtype=torch.bool, device=DEV)
            left[page, pos % 16] = False
            for now, old in zip((self.k_cache, self.v_cache), self.before):
                assert torch.equal(now.transpose(1, 2)[left], old.transpose(1, 2)[left])
        assert (self.q_out[n:] == 7).all()
        vg.vegas_read_device_status()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (5, 5, 128), (7, 1, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot_of", [0, 16, 48, 1])
def test_shapes_and_rotary_widths(hq, hkv, d, interleaved, rot_of):
    c = Rope(hq, hkv, d, [1, 0, 33, 16, 100], [0, 7, 15, 1000, 3], rot=d if rot_of == 1 else rot_of,
             interleaved=interleaved, pad=3, seed=hq)
    c.run()
    c.check()


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_several_axes(axes, interleaved):
    c = Rope(8, 2, 128, [40, 1, 300], [0, 9, 31], rot=128, axes=axes, interleaved=interleaved,
             scale=1.25, seed=axes)
    c.run()
    c.check()


def test_far_positions_are_as_exact_as_near_ones():
    far = torch.tensor([[0, 1, 131071, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, -131072, 12345678]],
                       dtype=torch.int32, device=DEV)
    c = Rope(4, 2, 128, [8], [40], rot=128, positions=far)
    c.run()
    c.check()


def test_large_cache_positions_of_text():
    c = Rope(4, 2, 64, [20], [150000], rot=64, seed=3)
    c.run()
    c.check()


def test_separate_tensors_and_in_place_queries():
    c = Rope(8, 2, 64, [50, 3], [2, 2], rot=32, fused=False, seed=4)
    src = c.q.clone()
    c.run(q_out=c.q)
    c.q_out[:c.used] = c.q.view(-1, 8, 64)[:c.used]
    c.check(q=src)


def test_many_sequences_and_a_graph_on_another_stream():
    rng = np.random.default_rng(0)
    rows = [int(x) for x in rng.integers(0, 4, 700)]
    c = Rope(8, 2, 64, rows, [int(x) for x in rng.integers(0, 90, 700)], rot=64, seed=5, pad=1)
    c.run()
    c.check()
    want = c.k_cache.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    c.k_cache.copy_(c.before[0])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.k_cache, want)
    side = torch.cuda.Stream()
    c.k_cache.copy_(c.before[0])
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    assert torch.equal(c.k_cache, want)


def test_bad_lengths_pages_and_axes_are_recorded():
    c = Rope(8, 2, 64, [20, 30], [100, 50], rot=64, seed=6)
    c.ctx_t[0] = c.max_pages * 16 - 19
    c.run()
    with pytest.raises(vg.VegasError) as ei:
        vg.vegas_read_device_status()
    assert ei.value.status == 5
    assert (c.q_out[:20] == 7).all() and not (c.q_out[20:] == 7).all()
    c = Rope(8, 2, 64, [20], [100], rot=64, seed=7)
    c.bt[0, 6] = -1                      # positions 96 .. 111
    c.run()
    with pytest.raises(vg.VegasError) as ei:
        vg.vegas_read_device_status()
    assert ei.value.status == 5
    c = Rope(8, 2, 64, [20], [100], rot=64, axes=2, seed=8)
    c.pair_axis[3] = 2
    c.run()
    with pytest.raises(vg.VegasError) as ei:
        vg.vegas_read_device_status()
    assert ei.value.status == 5


def test_cache_beyond_32_bit_offsets():
    c = Rope(8, 8, 128, [60, 1], [100, 2000], rot=128, seed=9, num_pages=140000)
    assert c.k_cache.numel() > 2 ** 31
    c.run()
    c.check()
