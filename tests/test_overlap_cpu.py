"""Refusal of outputs that lie partly over their call's inputs.

Made-up addresses, so this runs only where no GPU is visible.
"""
import pytest

from test_abi_cpu import vg  # noqa: F401  (the fixture)
from test_prompt_abi_cpu import _refused


def _not_refused_for_it(call):
    """Past the argument checks: without a GPU the next step fails."""
    from self_speculative_sparse_paged_gb300 import VegasError
    with pytest.raises(VegasError) as ei:
        call()
    assert "lies over" not in ei.value.detail and " is q" not in ei.value.detail, ei.value


def test_rotated_queries_over_the_projections(vg):  # noqa: F811
    # 8 + 2 + 2 heads of 64: rows of 768 elements, 1536 bytes; 5 rows of q_out take 5120 bytes
    kv = vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 64, 4)
    base = 1 << 20
    good = dict(kv=kv, q=base, q_stride=768, k=base + 1024, k_stride=768, v=base + 1280, v_stride=768,
                q_out=1 << 16, row_start=16, ctx_lens=16, positions=None, pair_axis=None, num_axes=1,
                inv_freq=16, rot_dim=64, interleaved=False, rope_scale=1.0, total_rows=5, batch=1,
                stream=0)
    _not_refused_for_it(lambda: vg.vegas_rope_append(**good))
    last = base + 4 * 1536
    for change in (dict(q_out=base + 16), dict(q_out=base + 1536), dict(q_out=base - 5104),
                   dict(q_out=last + 1520),                        # the last value row's end
                   dict(q=base + 512, k=base, v=base + 256, q_out=base),   # keys first
                   dict(q=1 << 24, q_stride=512, k=1 << 25, v=1 << 26, q_out=(1 << 24) + 1024),
                   dict(q=1 << 24, k=1 << 25, q_out=(1 << 25) - 64),
                   dict(q=1 << 24, v=1 << 25, q_out=(1 << 25) + 64)):
        _refused(lambda: vg.vegas_rope_append(**{**good, **change}), 1, "q_out lies over")
    for change in (dict(q_out=base - 5120), dict(q_out=last + 1536),
                   dict(q=1 << 24, q_stride=512, k=1 << 25, v=1 << 26, q_out=1 << 24)):   # in place
        _not_refused_for_it(lambda: vg.vegas_rope_append(**{**good, **change}))


def test_attention_output_over_the_queries(vg):  # noqa: F811
    kv = vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 64, 4)
    q = 1 << 20
    good = dict(kv=kv, q=q, q_stride=512, out=1 << 16, row_start=16, ctx_lens=16, total_rows=5, batch=1,
                softmax_scale=0.1, workspace=1 << 28, workspace_bytes=1 << 30, stream=0)
    for out, stride in ((q + 1024, 512), (q + 32, 512), (q - 5088, 512), (q + 5120, 1024),
                        (q + 4 * 2048 + 992, 1024)):
        _refused(lambda: vg.vegas_prompt_attn(**{**good, "out": out, "q_stride": stride}), 1,
                 "out lies over")
    for out, stride in ((q + 5120, 512), (q - 5120, 512), (q + 4 * 2048 + 1024, 1024)):
        _not_refused_for_it(lambda: vg.vegas_prompt_attn(**{**good, "out": out, "q_stride": stride}))
