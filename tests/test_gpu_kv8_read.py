"""The read back of large batches and long tables, where a bounded grid takes turns on the pages that the
sequences have; exact, and nothing else is written."""
import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import kv8_case as k8  # noqa: E402
import self_speculative_sparse_paged_gb300 as vg  # noqa: E402
from test_gpu_kv8 import Cache, dev  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def read_back(c, to_table, first, upto, to_pages, faults=False):
    shape = (to_pages, c.hkv, 16, c.d)
    to = [torch.full(shape, -3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    to_t = dev(to_table)
    kv16 = vg.paged_kv(to[0], to[1], to_t, c.hq)
    vg.vegas_read_device_status()
    vg.vegas_kv8_read(c.kv, kv16, None if first is None else dev(np.array(first, np.int32)),
                      dev(np.array(upto, np.int32)), len(upto))
    if faults:
        with pytest.raises(vg.VegasError) as e:
            vg.vegas_read_device_status()
        assert e.value.status == 5
    vg.vegas_read_device_status()
    return [t.float().cpu().numpy() for t in to]


def expect(c, to_table, first, upto, to_pages, skip=()):
    want = []
    for x in "kv":
        w = np.full((to_pages, c.hkv, 16, c.d), -3.0, np.float32)
        values = k8.decode(c.codes[x], c.scale[x]).astype(np.float32)
        for b, n in enumerate(upto):
            if b in skip:
                continue
            lo = 0 if first is None else first[b]
            for j in range(lo // 16, (n + 15) // 16):
                a, z = max(lo - 16 * j, 0), min(n - 16 * j, 16)
                if z > a:
                    w[to_table[b, j], :, a:z] = values[c.table[b, j], :, a:z]
        want.append(w)
    return want


CASES = [
    # hkv, d, lengths, pages of the table, given beginnings
    (2, 64, [9] * 300, 40, False), (1, 128, [0, 33] * 400, 30, False), (3, 64, [500] + [20] * 900, 40, True),
    (8, 128, [7000] + [0] * 20 + [16, 17, 1], 500, True), (2, 128, [16 * i for i in range(40)] * 7, 50, True),
    (1, 64, [5000] * 40, 400, False), (2, 64, [1] * 20000, 1, False), (16, 64, [40, 0, 3000], 5000, True),
]


@pytest.mark.parametrize("hkv,d,lengths,pages,begun", CASES)
def test_read_in_turns(hkv, d, lengths, pages, begun):
    rng = np.random.default_rng(len(lengths) + pages)
    c = Cache(rng, [(n + 15) // 16 for n in lengths], hkv, hkv, d, wild=True)
    table = np.full((len(lengths), pages), -1, np.int32)
    table[:, :c.table.shape[1]] = np.where(c.table >= c.num, -1, c.table)
    c.table = table
    c.upload()
    assert pages * len(lengths) > 8192
    first = [int(rng.integers(0, n + 3)) for n in lengths] if begun else None
    # another order of pages in the bf16 cache
    to_table = np.where(table >= 0, c.num - 1 - table, -1).astype(np.int32)
    got = read_back(c, to_table, first, lengths, c.num)
    for a, b in zip(got, expect(c, to_table, first, lengths, c.num)):
        assert np.array_equal(a, b)


def test_faults_of_a_large_batch():
    """Ranges and pages that do not exist are recorded and skipped, the others read."""
    rng = np.random.default_rng(5)
    lengths = [30] * 700
    c = Cache(rng, [2] * 700, 2, 2, 64)
    c.table = np.concatenate([c.table, np.full((700, 30), -1, np.int32)], 1)
    c.upload()
    to_table = c.table.copy()
    good = expect(c, to_table, None, lengths, c.num, skip=(3, 300, 699))
    for bad in (32 * 16 + 1, 2 ** 31 - 1):                        # past the tables' capacity
        upto = list(lengths)
        upto[3] = upto[300] = upto[699] = bad
        for a, b in zip(read_back(c, to_table, None, upto, c.num, faults=True), good):
            assert np.array_equal(a, b)
    first = [0] * 700
    first[3] = first[300] = first[699] = -1
    for a, b in zip(read_back(c, to_table, first, lengths, c.num, faults=True), good):
        assert np.array_equal(a, b)
    upto = list(lengths)
    upto[3] = upto[300] = upto[699] = 0
    to_table[5, 1], to_table[600, 0] = c.num, -1                  # pages outside the pool
    want = expect(c, np.clip(to_table, 0, c.num - 1), None, lengths, c.num, skip=(3, 300, 699, 5, 600))
    values = {x: k8.decode(c.codes[x], c.scale[x]).astype(np.float32) for x in "kv"}
    for w, x in zip(want, "kv"):
        w[to_table[5, 0]] = values[x][c.table[5, 0]]
        w[to_table[600, 1], :, :14] = values[x][c.table[600, 1], :, :14]
    for a, b in zip(read_back(c, to_table, None, upto, c.num, faults=True), want):
        assert np.array_equal(a, b)


def test_a_large_batch_of_short_sequences_goes_by_its_pages():
    """1024 sequences of 100 positions in tables of 64K and in tables of 112: the long tables cost little
    (a CTA for each of their pages: three times as much)."""
    n, hkv, d = 1024, 8, 128
    k = torch.zeros((7 * n, hkv, 16, d), dtype=torch.uint8, device=DEV)
    s = torch.full((7 * n, hkv), 127, dtype=torch.uint8, device=DEV)
    to = torch.empty((7 * n, hkv, 16, d), dtype=torch.bfloat16, device=DEV)
    upto = torch.full((n,), 100, dtype=torch.int32, device=DEV)
    times = []
    for pages in (7, 4096):
        bt = torch.zeros((n, pages), dtype=torch.int32, device=DEV)
        bt[:, :7] = torch.arange(7 * n, dtype=torch.int32, device=DEV).view(n, 7)
        kv8, kv16 = vg.paged_kv8(k, k, s, s, bt, hkv), vg.paged_kv(to, to, bt, hkv)
        best = float("inf")
        for _ in range(12):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                vg.vegas_kv8_read(kv8, kv16, None, upto, n)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    vg.vegas_read_device_status()
    assert times[1] < 2 * times[0], times
