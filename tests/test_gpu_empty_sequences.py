"""Sequences without rows in a packed batch: inactive slots, whose cached length may hold anything."""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import self_speculative_sparse_paged_gb300 as vg  # noqa: E402
from test_gpu_prompt import Prompt  # noqa: E402
from test_gpu_rope import Rope  # noqa: E402

pytestmark = pytest.mark.gpu

STALE = (-1, -2 ** 31, 2 ** 31 - 1, 10 ** 6)


def empty_slots(c):
    """Lengths that no sequence could have, in the slots without rows."""
    lens = list(c.ctx)
    for i, b in enumerate(b for b, n in enumerate(c.rows) if n == 0):
        lens[b] = STALE[i % len(STALE)]
    c.ctx_t.copy_(torch.tensor(lens, dtype=torch.int32))


@pytest.mark.parametrize("rows", [[0, 1, 0, 30, 0, 0], [0, 0, 700, 0, 2], [0, 0], [0] * 40 + [5, 0, 300]])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_ignores_their_lengths(rows, d):
    c = Prompt(8, 2, d, rows, [0 if n == 0 else 40 + 977 * (i % 3) for i, n in enumerate(rows)], seed=41,
               pad=2)
    vg.vegas_read_device_status()
    want = c.run().clone()
    c.out[:c.used] = 0
    empty_slots(c)
    c.run()
    vg.vegas_read_device_status()                     # nothing to record
    assert torch.equal(c.out, want)
    c.check(heads=(0, 7), rows=40)


@pytest.mark.parametrize("rows", [[0, 1, 0, 30, 0, 0], [0, 0, 700, 0, 2], [0, 0]])
def test_the_rotary_append_ignores_their_lengths(rows):
    c = Rope(8, 2, 64, rows, [0 if n == 0 else 40 + 977 * (i % 3) for i, n in enumerate(rows)], rot=64,
             seed=42, pad=2)
    vg.vegas_read_device_status()
    empty_slots(c)
    c.run()
    vg.vegas_read_device_status()
    lens = torch.tensor(c.ctx, dtype=torch.int32)
    c.ctx_t.copy_(lens)
    c.check()


def test_rows_that_do_not_fit_are_still_recorded():
    for length in (-1, 10 ** 6):
        c = Prompt(8, 2, 64, [0, 20, 5], [0, 100, 3], seed=43)
        c.ctx_t.copy_(torch.tensor([length, length, 3], dtype=torch.int32))
        c.run()
        with pytest.raises(vg.VegasError) as ei:
            vg.vegas_read_device_status()
        assert ei.value.status == 5
        assert (c.out[:20] == 7).all() and not (c.out[20:] == 7).all()
