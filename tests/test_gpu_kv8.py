"""The 8-bit cache's calls on a GPU against their definitions in 64 bits.

Tolerances: an output's own rounding is half a step of bf16, 2^-8 of it.  A softmax weight is
off by f16's half step 2^-11 and by the error d of its logit (twice that, numerator and sum), so
an output by at most (2^-11 + 2 d + 2^-16) sum_i p_i |v_i| more; in verify attention by 2^-9 more
for the weights' three e5m2 parts (of p in [2^e, 2^(e + 1)) the first cut leaves less than 2^(e - 2),
the second, of a leading bit of 2^(e - 3) at most, less than 2^(e - 5), and the last part, of a
leading bit of 2^(e - 6) at most, is rounded by half a step, 2^(e - 9)) and 2^-13 for weights below
their grid (2^-28 of the largest, of up to 2^15 positions); where d = 2^-17 times the unit's
largest |q| times the largest sum_j |k_ij| (the grid of the queries' two parts; 0 for drafts),
plus 2^-20 sum_j |q_j k_ij| (fp32 sums), times the softmax scale.  A captured score is off by
2^-17 of its terms' magnitudes: the fp32 sum of up to 64 query rows (63 * 2^-24), the tensor cores'
sum of 128 products (2^-22) and a few roundings.
"""
import math

import numpy as np
import pytest
import torch

import kv8_case as k8

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def tables(rng, pages, extra=2):
    """Shuffled pages for sequences of so many pages each; unused entries lie outside the pool."""
    num = sum(pages) + extra
    perm = rng.permutation(num).astype(np.int32)
    table = np.full((len(pages), max(max(pages), 1)), 1 << 30, dtype=np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, num


class Cache:
    def __init__(self, rng, pages, hq, hkv, d, **kw):
        self.table, num = tables(rng, pages)
        self.codes = {n: None for n in "kv"}
        self.scale = {}
        for n in "kv":
            self.codes[n], self.scale[n] = k8.random_cache(rng, num, hkv, d, **kw)
        self.hq, self.hkv, self.d, self.num = hq, hkv, d, num

    def upload(self):
        self.dk, self.dv = dev(self.codes["k"]), dev(self.codes["v"])
        self.dks, self.dvs = dev(self.scale["k"]), dev(self.scale["v"])
        self.dt = dev(self.table)
        self.kv = vg.paged_kv8(self.dk, self.dv, self.dks, self.dvs, self.dt, self.hq)
        return self.kv


# ------------------------------------------------------------------ append
APPENDS = [
    # hq, hkv, d, rot, interleaved, rows, ctx, pad
    (8, 2, 64, 64, False, [1], [0], 0),
    (8, 2, 64, 64, True, [1, 1, 1], [15, 16, 17], 2),
    (4, 4, 128, 128, False, [33, 0, 5, 16], [0, 7, 30, 16], 0),
    (32, 8, 128, 128, True, [5, 5, 5, 5, 5], [11, 12, 13, 1000, 0], 3),
    (6, 2, 128, 64, False, [100], [3], 1),
    (5, 1, 64, 32, True, [17, 31], [31, 1], 0),
    (3, 3, 64, 0, False, [40, 2], [5, 14], 0),
    (64, 8, 64, 16, False, [300], [250], 0),
    (1, 1, 128, 128, False, [1] * 70, [i % 33 for i in range(70)], 0),
]


def run_append(rng, case, qkv=None, positions=None, pair_axis=None, axes=1, scale=1.0):
    """The call and its bf16 counterpart on the same rows; returns the cache before and after,
    and the bf16 cache that the counterpart wrote."""
    hq, hkv, d, rot, inter, rows, ctx, pad = case
    used = sum(rows)
    total = used + pad
    c = Cache(rng, [(a + n + 15) // 16 for n, a in zip(rows, ctx)], hq, hkv, d)
    c.upload()
    if qkv is None:
        size = 2.0 ** rng.uniform(-3, 6, (total, hq + 2 * hkv, 1))
        qkv = torch.from_numpy(rng.standard_normal((total, hq + 2 * hkv, d)) * size).bfloat16()
    qkv = qkv.reshape(total, -1).to(DEV)
    start = dev(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32))
    dctx = dev(np.array(ctx, np.int32))
    inv = dev((1e4 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32))
    w = qkv.stride(0)
    args = (qkv, w, qkv[:, hq * d:], w, qkv[:, (hq + hkv) * d:], w)
    rest = (start, dctx, positions, pair_axis, axes, inv, rot, inter, scale, total, len(rows))
    q8 = torch.full((total, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    q16 = q8.clone()
    vg.vegas_rope_append_kv8(c.kv, *args, q8, *rest)
    kc = torch.zeros((c.num, hkv, 16, d), dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    vg.vegas_rope_append(vg.paged_kv(kc, vc, c.dt, hq), *args, q16, *rest)
    vg.vegas_read_device_status()
    assert torch.equal(q8, q16)                  # the same turning, rows behind the last left alone
    return c, {"k": kc, "v": vc}, qkv


def expect_append(c, case, bf16):
    """c's host copy after the oracle's append of the rows that the bf16 cache holds."""
    _, hkv, d, _, _, rows, ctx, _ = case
    want = {}
    for n in "kv":
        codes, scale = c.codes[n].copy(), c.scale[n].copy()
        x = bf16[n].double().cpu().numpy()
        for b, (r, a) in enumerate(zip(rows, ctx)):
            if r:
                pos = np.arange(a, a + r)
                k8.append(codes, scale, x[c.table[b, pos // 16], :, pos % 16], c.table[b], a)
        want[n] = codes, scale
    return want


@pytest.mark.parametrize("case", APPENDS)
def test_append(case):
    rng = np.random.default_rng(len(case[5]) + case[2])
    c, bf16, _ = run_append(rng, case)
    want = expect_append(c, case, bf16)
    for n, codes, scale in (("k", c.dk, c.dks), ("v", c.dv, c.dvs)):
        assert np.array_equal(scale.cpu().numpy(), want[n][1])
        assert np.array_equal(codes.cpu().numpy(), want[n][0])    # untouched slots and pages too


def test_append_turns_by_the_angles():
    """Against an independent rotation in 64 bits: a code is at most a step off, where the turned
    key's bf16 rounding went the other way."""
    rng = np.random.default_rng(5)
    hq, hkv, d, rows, ctx = 4, 2, 128, [200], [100000]
    x = torch.from_numpy(rng.standard_normal((200, hq + 2 * hkv, d))).bfloat16()
    c, _, _ = run_append(rng, (hq, hkv, d, d, False, rows, ctx, 0), qkv=x)
    inv = (1e4 ** (-np.arange(d // 2) / (d // 2))).astype(np.float32).astype(np.float64)
    ang = (np.arange(200) + 100000)[:, None] * inv
    cos, sin = np.cos(ang)[:, None], np.sin(ang)[:, None]
    k = x[:, hq:hq + hkv].double().numpy()
    a, b = k[..., :d // 2], k[..., d // 2:]
    y = torch.from_numpy(np.concatenate([a * cos - b * sin, b * cos + a * sin], -1)).bfloat16()
    codes, scale = c.codes["k"].copy(), c.scale["k"].copy()
    k8.append(codes, scale, y.double().numpy(), c.table[0], 100000)
    got = k8.decode(c.dk.cpu().numpy(), c.dks.cpu().numpy())
    want = k8.decode(codes, scale)
    off = got != want
    assert off.mean() < 1e-3 and np.all(np.abs(got - want)[off] <= np.abs(want)[off] / 8 + 2.0 ** -8)


def test_append_given_positions():
    rng = np.random.default_rng(6)
    rows, ctx = [21, 40], [9, 0]
    pos = dev(rng.integers(0, 1 << 20, (3, 61)).astype(np.int32))
    axis = dev((np.arange(64) % 3).astype(np.int32))
    case = (8, 2, 128, 128, False, rows, ctx, 0)
    c, bf16, _ = run_append(rng, case, positions=pos, pair_axis=axis, axes=3, scale=1.25)
    want = expect_append(c, case, bf16)
    assert np.array_equal(c.dk.cpu().numpy(), want["k"][0])
    assert np.array_equal(c.dks.cpu().numpy(), want["k"][1])


def test_append_odd_values():
    """Blocks of zeros, of infinities and NaN among numbers, and of numbers beyond either end of
    the scales."""
    rng = np.random.default_rng(7)
    hq, hkv, d, rows, ctx = 8, 8, 64, [20], [0]
    x = rng.standard_normal((20, hq + 2 * hkv, d))
    x[:, hq + 0] = 0
    x[:, hq + 1] *= 1e38
    x[:, hq + 2] *= 1e-38
    x[3, hq + 3, 5], x[4, hq + 3, 6], x[5, hq + 3, 7] = np.inf, -np.inf, np.nan
    x[:, hq + 4] = np.nan
    x[:, hq + 5] = np.inf
    x[:, hq + 6] = -0.0
    x[:, hq + hkv:] = x[:, hq:hq + hkv]
    case = (hq, hkv, d, 0, False, rows, ctx, 0)
    c, bf16, _ = run_append(rng, case, qkv=torch.from_numpy(x).bfloat16())
    want = expect_append(c, case, bf16)
    assert np.array_equal(c.dk.cpu().numpy(), want["k"][0])
    assert np.array_equal(c.dks.cpu().numpy(), want["k"][1])
    assert np.array_equal(c.dv.cpu().numpy(), want["v"][0])


@pytest.mark.parametrize("step", [1, 3])
def test_append_in_steps(step):
    """A sequence grown a few rows a call, rows of rising and falling size, some written over."""
    rng = np.random.default_rng(step)
    hq, hkv, d = 4, 2, 64
    c = Cache(rng, [4], hq, hkv, d)
    c.upload()
    codes = {n: c.codes[n].copy() for n in "kv"}
    scale = {n: c.scale[n].copy() for n in "kv"}
    at = 0
    for i in range(30):
        if at + step > 64:
            break
        x = torch.from_numpy(rng.standard_normal((step, hq + 2 * hkv, d)) *
                             2.0 ** rng.uniform(-12, 12)).bfloat16()
        dx = x.reshape(step, -1).to(DEV)
        q = torch.empty((step, hq, d), dtype=torch.bfloat16, device=DEV)
        w = dx.stride(0)
        vg.vegas_rope_append_kv8(c.kv, dx, w, dx[:, hq * d:], w, dx[:, (hq + hkv) * d:], w, q,
                                 dev(np.array([0, step], np.int32)), dev(np.array([at], np.int32)),
                                 None, None, 1, None, 0, False, 1.0, step, 1)
        for n, lo in (("k", hq), ("v", hq + hkv)):
            k8.append(codes[n], scale[n], x[:, lo:lo + hkv].double().numpy(), c.table[0], at)
        at += step if i % 4 != 3 else 0          # (every fourth call is written over)
    for n, dc, ds in (("k", c.dk, c.dks), ("v", c.dv, c.dvs)):
        assert np.array_equal(ds.cpu().numpy(), scale[n])
        assert np.array_equal(dc.cpu().numpy(), codes[n])


def test_append_faults_are_recorded():
    rng = np.random.default_rng(8)
    hq, hkv, d = 2, 1, 64
    x = torch.randn((6, 4 * d), device=DEV).bfloat16()
    q = torch.zeros((6, hq, d), dtype=torch.bfloat16, device=DEV)

    def call(c, start, ctx):
        before = c.dk.clone()
        w = x.stride(0)
        vg.vegas_rope_append_kv8(c.kv, x, w, x[:, 2 * d:], w, x[:, 3 * d:], w, q,
                                 dev(np.array(start, np.int32)), dev(np.array(ctx, np.int32)), None,
                                 None, 1, None, 0, False, 1.0, 6, len(ctx))
        with pytest.raises(vg.VegasError) as e:
            vg.vegas_read_device_status()
        assert e.value.status == 5
        return before

    for start, ctx in (([0, 6], [-1]), ([0, 6], [27]), ([0, 7], [0]), ([4, 2], [0])):
        c = Cache(rng, [2], hq, hkv, d)
        c.upload()
        assert torch.equal(call(c, start, ctx), c.dk)      # skipped
    c = Cache(rng, [2], hq, hkv, d)
    c.table[0, 1] = c.num                                  # the second page lies outside the pool
    c.upload()
    before = call(c, [0, 6], [13])
    ok = c.table[0, 0]
    assert not torch.equal(before[ok, :, 13:], c.dk[ok, :, 13:])
    assert torch.equal(before[[p for p in range(c.num) if p != ok]], c.dk[[p for p in range(c.num) if p != ok]])


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("hkv,d,first,upto", [
    (1, 64, [0], [1]), (2, 64, [0, 5, 40], [700, 5, 41]), (8, 128, [0, 16, 31, 0], [33, 32, 200, 0]),
    (3, 128, None, [100, 16]), (5, 64, [15, 0], [17, 300]),
    (1, 64, [0] * 63 + [37], [5 * i for i in range(63)] + [6001])])         # a long one among many
def test_read(hkv, d, first, upto):
    rng = np.random.default_rng(d + hkv)
    c = Cache(rng, [(u + 15) // 16 for u in upto], hkv, hkv, d, wild=True, spread=110)
    c.scale["k"][0, 0] = 255                 # (bytes out of range are the nearest end)
    c.upload()
    to_table, num = tables(rng, [(u + 15) // 16 + 2 for u in upto])
    want = {n: rng.standard_normal((num, hkv, 16, d)) for n in "kv"}
    to = {n: torch.from_numpy(want[n]).bfloat16().to(DEV) for n in "kv"}
    want = {n: to[n].double().cpu().numpy() for n in "kv"}
    dto = dev(to_table)                      # (a descriptor keeps no tensor alive)
    vg.vegas_kv8_read(c.kv, vg.paged_kv(to["k"], to["v"], dto, hkv),
                      None if first is None else dev(np.array(first, np.int32)),
                      dev(np.array(upto, np.int32)), len(upto))
    vg.vegas_read_device_status()
    for n in "kv":
        x = k8.decode(c.codes[n], c.scale[n])
        for b, u in enumerate(upto):
            pos = np.arange(first[b] if first else 0, u)
            want[n][to_table[b, pos // 16], :, pos % 16] = x[c.table[b, pos // 16], :, pos % 16]
        assert np.array_equal(to[n].double().cpu().numpy(), want[n])


def test_read_faults_are_recorded():
    rng = np.random.default_rng(1)
    for first, upto, spoil in (([-1], [5], None), ([0], [33], None), ([0], [20], "from"), ([0], [20], "to")):
        c = Cache(rng, [2], 2, 2, 64)
        table = np.array([[1, 0]], np.int32)
        if spoil:
            (c.table if spoil == "from" else table)[0, 1] = -3
        c.upload()
        k = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16, device=DEV)
        v = torch.zeros_like(k)
        dto = dev(table)
        vg.vegas_kv8_read(c.kv, vg.paged_kv(k, v, dto, 2), dev(np.array(first, np.int32)),
                          dev(np.array(upto, np.int32)), 1)
        with pytest.raises(vg.VegasError) as e:
            vg.vegas_read_device_status()
        assert e.value.status == 5
        assert not k[0].any() and bool(k[1].any()) == (spoil is not None)


# ------------------------------------------------------------------ verify
def queries(rng, shape, size=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * size).bfloat16()


P_PARTS = 2.0 ** -9 + 2.0 ** -13      # of the weights in verify attention


def check_verify(c, q, out, scores, ctx, gamma, mask, scale):
    batch, t, hq, d = q.shape
    g = hq // c.hkv
    qd, od = q.double().numpy(), out.double().cpu().numpy()
    sd = None if scores is None else scores.double().cpu().numpy()
    rows = [i for i in range(t) if mask >> i & 1]
    for b, n in enumerate(ctx):
        pages = c.table[b, :(n + t + 15) // 16]
        for h in range(c.hkv):
            k = k8.gather(c.codes["k"], c.scale["k"], pages, h, n + t)
            v = k8.gather(c.codes["v"], c.scale["v"], pages, h, n + t)
            qq = qd[b, :, h * g:(h + 1) * g]
            grid = 2.0 ** -17 * np.abs(qq).max() * np.abs(k).sum(-1).max()
            for i in range(t):
                want, mag, _ = k8.attend(qq[i], k[:n + i + 1], v[:n + i + 1], scale)
                terms = (np.abs(qq[i]) @ np.abs(k[:n + i + 1]).T).max()
                d_logit = abs(scale) * (grid + 2.0 ** -20 * terms)
                tol = 2.0 ** -8 * np.abs(want) + (P_PARTS + 2.0 ** -11 + 2 * d_logit + 2.0 ** -16) * mag + 1e-30
                err = np.abs(od[b, i, h * g:(h + 1) * g] - want)
                assert (err <= tol).all(), (b, h, i, float((err / tol).max()))
            if sd is not None:
                x = (qq[rows].reshape(-1, d) @ k[:n].T).sum(0) * scale
                tol = 2.0 ** -17 * (np.abs(qq[rows]).reshape(-1, d) @ np.abs(k[:n]).T).sum(0) * abs(scale)
                err = np.abs(sd[b, h, :n] - x)
                assert (err <= tol + 1e-30).all(), (b, h, float((err / tol).max()))
                assert (sd[b, h, n:] == -5).all()        # nothing past the prefix


def run_verify(c, q, ctx, gamma, mask, scale, stride=None):
    batch = len(ctx)
    out = torch.full_like(q, float("nan"), device=DEV)
    stride = stride or max(max(ctx), 1)
    scores = torch.full((batch, c.hkv, stride), -5.0, device=DEV) if mask else None
    n = vg.vegas_verify_kv8_workspace_size(c.kv, batch, gamma)
    ws = torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV)
    dctx = dev(np.array(ctx, np.int32))
    dq = q.to(DEV)
    for _ in range(2):                                    # (the workspace is left as it was)
        vg.vegas_verify_attn_kv8(c.kv, dq, out, scores, stride, dctx, batch, gamma, mask, scale, ws,
                                 ws.numel())
    vg.vegas_read_device_status()
    return out, scores


def spoil_unused(c, ctx, t):
    """NaN codes in every slot that no window row may see."""
    for b, n in enumerate(ctx):
        last, used = c.table[b, (n + t - 1) // 16], (n + t - 1) % 16 + 1
        for x in "kv":
            c.codes[x][last, :, used:] = 0x7f
    own = {p for b, n in enumerate(ctx) for p in c.table[b, :(n + t + 15) // 16]}
    for p in set(range(c.num)) - own:
        for x in "kv":
            c.codes[x][p] = 0xff
            c.scale[x][p] = 255


VERIFIES = [
    # hq, hkv, d, gamma, mask, ctx
    (1, 1, 64, 0, 0, [0]), (1, 1, 128, 0, 1, [1]), (2, 2, 128, 0, 0, [0, 15, 16, 17]),
    (8, 2, 64, 4, 0b10001, [2048]), (32, 8, 128, 4, 0b10001, [1000, 127, 128]),
    (4, 4, 128, 3, 0b1111, [130, 3]), (8, 2, 128, 9, 1 << 9, [300]), (6, 2, 64, 2, 0b010, [5000, 77]),
    (16, 1, 64, 3, 0b1001, [900]), (8, 1, 64, 5, 0b100001, [640, 0, 2]), (14, 2, 64, 7, 0b11, [257]),
    (8, 1, 64, 4, 0b10001, [700]), (2, 1, 128, 15, 0xffff, [513]), (10, 2, 128, 6, 0b1000001, [33, 4097]),
    (40, 8, 128, 7, 0b10000001, [400]), (64, 8, 64, 6, 0b1000001, [1500, 20]), (3, 1, 128, 4, 0, [20000]),
    (4, 1, 64, 3, 0b1, [30000]), (32, 8, 128, 0, 0, [0, 1, 15, 400, 277, 810, 129, 64, 555, 103, 16, 301]),
    (8, 4, 64, 1, 0b11, [60 + 37 * i for i in range(50)]), (16, 4, 128, 4, 0b10001, [9] * 40),
]


@pytest.mark.parametrize("hq,hkv,d,gamma,mask,ctx", VERIFIES)
def test_verify(hq, hkv, d, gamma, mask, ctx):
    rng = np.random.default_rng(hq * 100 + d + gamma)
    t = gamma + 1
    c = Cache(rng, [(n + t + 15) // 16 for n in ctx], hq, hkv, d)
    spoil_unused(c, ctx, t)
    c.upload()
    q = queries(rng, (len(ctx), t, hq, d))
    scale = 1 / math.sqrt(d)
    out, scores = run_verify(c, q, ctx, gamma, mask, scale, stride=max(max(ctx), 1) + 3)
    check_verify(c, q, out, scores, ctx, gamma, mask, scale)


def test_verify_many_sequences():
    """More sequences than the lengths' first pass takes at once, most of them short."""
    rng = np.random.default_rng(21)
    ctx = [int(x) for x in rng.integers(0, 40, 900)]
    ctx[500], ctx[899] = 1000, 300
    c = Cache(rng, [(n + 2 + 15) // 16 for n in ctx], 2, 1, 64)
    spoil_unused(c, ctx, 2)
    c.upload()
    q = queries(rng, (900, 2, 2, 64))
    out, scores = run_verify(c, q, ctx, 1, 0b11, 0.125)
    check_verify(c, q, out, scores, ctx, 1, 0b11, 0.125)


def test_verify_long_table_short_sequence():
    """A table with far more pages than the sequences have: most splits are empty."""
    rng = np.random.default_rng(4)
    ctx, gamma = [40, 333], 4
    c = Cache(rng, [3, 22], 8, 2, 128)
    c.table = np.concatenate([c.table, np.full((2, 4000), -1, np.int32)], 1)
    c.upload()
    q = queries(rng, (2, 5, 8, 128))
    out, scores = run_verify(c, q, ctx, gamma, 17, 0.09)
    check_verify(c, q, out, scores, ctx, gamma, 17, 0.09)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread", [3, 30])
def test_verify_rows_of_unlike_size(d, spread):
    """Query rows up to 2^(4 spread) apart: each keeps bits of its own.  (The grid of a row is
    that of its own largest element once the rows are more than 2^4 apart.)"""
    rng = np.random.default_rng(d)
    ctx, gamma, hq, hkv = [700], 4, 8, 2
    c = Cache(rng, [45], hq, hkv, d)
    c.upload()
    q = queries(rng, (1, 5, hq, d))
    small = 2.0 ** -rng.integers(0, 4 * spread, (1, 5, hq, 1)).astype(np.float64)
    small[0, 0, 0] = 1
    small[0, 1, 0] = 2.0 ** (-4 * spread)
    q = (q.double() * torch.from_numpy(small)).bfloat16()
    q[0, 2, 3] = 0                                            # a row of zeros: the mean of V
    out, scores = run_verify(c, q, ctx, gamma, 0b11111, 0.1)
    # row by row: the grid is the row's own
    for i in range(5):
        for h in range(hq):
            k = k8.gather(c.codes["k"], c.scale["k"], c.table[0], h // 4, 705)
            v = k8.gather(c.codes["v"], c.scale["v"], c.table[0], h // 4, 705)
            qq = q[0, i, h:h + 1].double().numpy()
            want, mag, _ = k8.attend(qq, k[:700 + i + 1], v[:700 + i + 1], 0.1)
            d_logit = 0.1 * (2.0 ** -17 * np.abs(qq).max() * np.abs(k).sum(-1).max()
                             + 2.0 ** -20 * (np.abs(qq) @ np.abs(k).T).max())
            tol = 2.0 ** -8 * np.abs(want) + (P_PARTS + 2.0 ** -11 + 2 * d_logit + 2.0 ** -16) * mag
            assert (np.abs(out[0, i, h].double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("d", [64, 128])
def test_verify_scales_of_every_size(d):
    """Blocks whose values differ by up to 2^100, with the heaviest weights on the smallest."""
    rng = np.random.default_rng(d + 1)
    ctx, gamma, hq, hkv = [900], 2, 4, 2
    c = Cache(rng, [57], hq, hkv, d)
    c.scale["v"][:] = rng.integers(127 - 50, 127 + 51, c.scale["v"].shape)
    c.upload()
    q = queries(rng, (1, 3, hq, d))
    out, scores = run_verify(c, q, ctx, gamma, 0b101, 0.3)
    check_verify(c, q, out, scores, ctx, gamma, 0b101, 0.3)


def test_verify_sharp_softmax():
    """Large logits: one position takes all, references are raised from tile to tile."""
    rng = np.random.default_rng(9)
    ctx, gamma, hq, hkv, d = [3000], 3, 4, 1, 128
    c = Cache(rng, [188], hq, hkv, d)
    order = np.argsort(c.table[0])
    for j in range(188):                          # keys grow along the sequence
        c.scale["k"][c.table[0, j]] = 127 - 8 + j // 32
    c.upload()
    q = queries(rng, (1, 4, hq, d))
    out, scores = run_verify(c, q, ctx, gamma, 0b1, 1.0)
    check_verify(c, q, out, scores, ctx, gamma, 0b1, 1.0)
    assert order.size == 188


def test_verify_one_position_is_its_value():
    """With one position the output is its value, whatever the logits: exact."""
    rng = np.random.default_rng(10)
    c = Cache(rng, [1, 1], 4, 2, 64, wild=True)
    c.upload()
    q = queries(rng, (2, 1, 4, 64), size=30)
    out, _ = run_verify(c, q, [0, 0], 0, 0, 0.5)
    for b in range(2):
        v = k8.decode(c.codes["v"], c.scale["v"])[c.table[b, 0], :, 0]
        assert np.array_equal(out[b, 0].double().cpu().numpy(), np.repeat(v, 2, 0))


def test_verify_faults_are_recorded():
    rng = np.random.default_rng(11)
    for ctx, spoil in (([-1], False), ([44], False), ([30], True)):
        c = Cache(rng, [3], 4, 2, 64)
        if spoil:
            c.table[0, 1] = c.num
        c.upload()
        q = queries(rng, (1, 5, 4, 64)).to(DEV)
        out = torch.zeros_like(q)
        ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
        vg.vegas_verify_attn_kv8(c.kv, q, out, None, 0, dev(np.array(ctx, np.int32)), 1, 4, 0, 0.1, ws,
                                 ws.numel())
        with pytest.raises(vg.VegasError) as e:
            vg.vegas_read_device_status()
        assert e.value.status == 5


# ------------------------------------------------------------------ sparse drafts
DRAFTS = [
    # hq, hkv, d, ctx, k, tail
    (1, 1, 64, [0], [0], [1]), (8, 2, 64, [100], [1], [1]), (4, 4, 128, [500, 20], [77, 0], [3, 9]),
    (32, 8, 128, [4000], [205], [6]), (16, 1, 64, [333, 40], [40, 40], [2, 17]), (9, 1, 128, [90], [17], [4]),
    (16, 1, 128, [2500], [1300], [5]), (64, 8, 64, [3000, 2999], [90, 93], [8, 11]),
    (5, 1, 64, [70] * 40, [11] * 40, [1] * 40), (2, 1, 128, [40000], [32000], [16]),
    (16, 1, 128, [9000], [6000], [3]), (16, 2, 64, [9000], [7000], [9]),    # long lists, wide groups
    (8, 8, 128, [3500] * 10, [3000] * 10, [5] * 10),                        # one CTA a list
]


@pytest.mark.parametrize("hq,hkv,d,ctx,k,tail", DRAFTS)
def test_draft(hq, hkv, d, ctx, k, tail):
    rng = np.random.default_rng(hq + d + len(ctx))
    c = Cache(rng, [(n + t + 15) // 16 for n, t in zip(ctx, tail)], hq, hkv, d, spread=20)
    spoil_unused(c, [n + t - 1 for n, t in zip(ctx, tail)], 1)
    c.upload()
    batch, k_max, g = len(ctx), max(k), hq // hkv
    idx = np.full((batch, hkv, max(k_max, 1)), -1, np.int32)
    for b in range(batch):
        for h in range(hkv):
            idx[b, h, :k[b]] = np.sort(rng.choice(ctx[b], k[b], replace=False)) if k[b] else []
    q = queries(rng, (batch, hq, d))
    q[0, 0] *= 2.0 ** 20 if hq > 1 else 1                        # heads keep bits of their own
    out = torch.full_like(q, float("nan"), device=DEV)
    scale = 1 / math.sqrt(d)
    vg.vegas_sparse_decode_attn_kv8(c.kv, q.to(DEV), out, dev(idx), k_max, dev(np.array(k, np.int32)),
                                    dev(np.array(ctx, np.int32)), dev(np.array(tail, np.int32)),
                                    max(tail), batch, scale)
    vg.vegas_read_device_status()
    for b in range(batch):
        pages = c.table[b, :(ctx[b] + tail[b] + 15) // 16]
        for h in range(hkv):
            at = np.concatenate([idx[b, h, :k[b]], ctx[b] + np.arange(tail[b])])
            kk = k8.gather(c.codes["k"], c.scale["k"], pages, h, ctx[b] + tail[b])[at]
            vv = k8.gather(c.codes["v"], c.scale["v"], pages, h, ctx[b] + tail[b])[at]
            qq = q[b, h * g:(h + 1) * g].double().numpy()
            want, mag, _ = k8.attend(qq, kk, vv, scale)
            d_logit = scale * 2.0 ** -20 * (np.abs(qq) @ np.abs(kk).T).max(-1, keepdims=True)
            tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * d_logit + 2.0 ** -16) * mag + 1e-30
            err = np.abs(out[b, h * g:(h + 1) * g].double().cpu().numpy() - want)
            assert (err <= tol).all(), (b, h, float((err / tol).max()))


def test_draft_scales_of_every_size():
    rng = np.random.default_rng(12)
    c = Cache(rng, [40], 4, 2, 128)
    c.scale["v"][:] = rng.integers(127 - 50, 127 + 51, c.scale["v"].shape)
    c.upload()
    idx = np.sort(rng.choice(600, (1, 2, 200)), -1).astype(np.int32)      # repeats count twice
    q = queries(rng, (1, 4, 128))
    out = torch.empty_like(q, device=DEV)
    vg.vegas_sparse_decode_attn_kv8(c.kv, q.to(DEV), out, dev(idx), 200, dev(np.array([200], np.int32)),
                                    dev(np.array([610], np.int32)), dev(np.array([4], np.int32)), 4, 1, 0.2)
    vg.vegas_read_device_status()
    for h in range(2):
        at = np.concatenate([idx[0, h], 610 + np.arange(4)])
        kk = k8.gather(c.codes["k"], c.scale["k"], c.table[0], h, 640)[at]
        vv = k8.gather(c.codes["v"], c.scale["v"], c.table[0], h, 640)[at]
        qq = q[0, 2 * h:2 * h + 2].double().numpy()
        want, mag, _ = k8.attend(qq, kk, vv, 0.2)
        d_logit = 0.2 * 2.0 ** -20 * (np.abs(qq) @ np.abs(kk).T).max()
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * d_logit + 2.0 ** -16) * mag
        assert (np.abs(out[0, 2 * h:2 * h + 2].double().cpu().numpy() - want) <= tol).all()


def test_draft_faults_are_recorded():
    rng = np.random.default_rng(13)
    for bad in (-1, 48, None):
        c = Cache(rng, [3], 4, 2, 64)
        idx = np.array([[[1, 5, 20]] * 2], np.int32)
        if bad is None:
            c.table[0, 1] = -1
        else:
            idx[0, 1, 2] = bad
        c.upload()
        q = queries(rng, (1, 4, 64)).to(DEV)
        vg.vegas_sparse_decode_attn_kv8(c.kv, q, torch.empty_like(q), dev(idx), 3, dev(np.array([3], np.int32)),
                                        dev(np.array([40], np.int32)), dev(np.array([2], np.int32)), 2, 1, 0.1)
        with pytest.raises(vg.VegasError) as e:
            vg.vegas_read_device_status()
        assert e.value.status == 5
