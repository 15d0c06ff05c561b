"""Lengths that no table holds, in the bf16 verify: recorded, and answered as the nearest one that a
table holds.  (What the test of lengths gives near 2^31 is checked on the host first, in
test_lengths_cpu.py.)"""
import numpy as np
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402
from vegas_case import Case, to_dev  # noqa: E402
from workload import configs  # noqa: E402

pytestmark = pytest.mark.gpu
TOP = 2 ** 31 - 1


@pytest.mark.parametrize("capture", [False, True])
@pytest.mark.parametrize("length", [-1, TOP, TOP - 3, TOP - 40])
@pytest.mark.parametrize("gamma", [4, 10])                # 20 query rows on the tensor cores' kernel, 44 on the other
def test_verify_records_a_length_that_no_table_holds(gamma, length, capture):
    c = Case(configs.QWEN3_8B_B1_32K.with_(gamma=gamma, ctx_lo=500, ctx_hi=500))
    cap = 16 * c.pm.block_table.shape[1]
    nearest = 0 if length < 0 else cap - gamma - 1
    scores = torch.full((1, c.w.hkv, cap), -5.0, device="cuda")
    c.stride = cap
    results = []
    for n in (length, nearest):
        vg.vegas_read_device_status()
        c.lens_t.copy_(to_dev(np.array([n], np.int32)))
        scores.fill_(-5)
        out, _ = c.verify(capture=capture, scores=scores if capture else None)
        if n == length:
            with pytest.raises(vg.VegasError) as e:
                vg.vegas_read_device_status()
            assert e.value.status == 5
        vg.vegas_read_device_status()
        results.append((out.clone(), scores.clone()))
    assert torch.isfinite(results[0][0]).all()
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
