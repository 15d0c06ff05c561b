"""Lengths that no table holds, in the 8-bit cache's calls: recorded and clamped, and the sequences
beside them are answered as if they were alone.  (What the test of lengths gives near 2^31 is checked on
the host first, in test_lengths_cpu.py.)"""
import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402
from test_gpu_kv8 import Cache, check_verify, dev, queries  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOP = 2 ** 31 - 1


@pytest.mark.parametrize("masked", [0, 0b10001])
@pytest.mark.parametrize("ctx", [[TOP], [TOP - 4], [TOP - 5], [-2 ** 31, TOP - 1], [40, TOP, 75], [TOP] * 40,
                                 [2 ** 30, 7, TOP - 2], [5 * i for i in range(16)] + [TOP - 3]])
def test_verify_records_a_length_that_no_table_holds(ctx, masked):
    rng = np.random.default_rng(len(ctx))
    hq, hkv, d, gamma, pages = 8, 2, 128, 4, 6
    t, cap = gamma + 1, 16 * pages
    c = Cache(rng, [pages] * len(ctx), hq, hkv, d)
    c.upload()
    held = [min(max(n, 0), cap - t) for n in ctx]           # what a length is clamped to
    q = queries(rng, (len(ctx), t, hq, d))
    dq, out = q.to(DEV), torch.full_like(q, float("nan"), device=DEV)
    scores = torch.full((len(ctx), hkv, cap), -5.0, device=DEV) if masked else None
    ws = torch.zeros(vg.vegas_verify_kv8_workspace_size(c.kv, len(ctx), gamma), dtype=torch.uint8, device=DEV)

    def call(lengths):
        vg.vegas_verify_attn_kv8(c.kv, dq, out, scores, cap, dev(np.array(lengths, np.int32)), len(ctx), gamma,
                                 masked, 0.1, ws, ws.numel())

    vg.vegas_read_device_status()
    call(ctx)
    with pytest.raises(vg.VegasError) as e:
        vg.vegas_read_device_status()
    assert e.value.status == 5
    check_verify(c, q, out, scores, held, gamma, masked, 0.1)
    first = out.clone()
    call(held)                                              # the workspace serves the next call
    vg.vegas_read_device_status()
    assert torch.equal(first, out)


@pytest.mark.parametrize("long_tail", [7, 200, TOP - 11, TOP])
@pytest.mark.parametrize("d", [64, 128])
def test_draft_records_a_tail_longer_than_the_calls(d, long_tail):
    """A tail above max_tail is recorded and cut to it (its sum with the list may pass 2^31), and the
    sequence beside it is answered as if it were alone."""
    rng = np.random.default_rng(d)
    hq, hkv, max_tail = 8, 2, 6
    c = Cache(rng, [10, 10], hq, hkv, d)
    c.upload()
    q = queries(rng, (2, hq, d)).to(DEV)
    idx = dev(np.sort(rng.choice(100, (2, hkv, 12)), -1).astype(np.int32))
    k = dev(np.array([12, 12], np.int32))
    results = []
    for tails in ([4, long_tail], [4, max_tail]):
        out = torch.full_like(q, float("nan"))
        vg.vegas_read_device_status()
        vg.vegas_sparse_decode_attn_kv8(c.kv, q, out, idx, 12, k, dev(np.array([100, 100], np.int32)),
                                        dev(np.array(tails, np.int32)), max_tail, 2, 0.1)
        if tails[1] != max_tail:
            with pytest.raises(vg.VegasError) as e:
                vg.vegas_read_device_status()
            assert e.value.status == 5
        vg.vegas_read_device_status()
        results.append(out)
    assert torch.isfinite(results[0]).all() and torch.equal(*results)
