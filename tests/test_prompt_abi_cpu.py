"""Host-side refusals of the prompt calls and of the token log probabilities.

Made-up addresses, so these run only where no GPU is visible.
"""
import pytest

from test_abi_cpu import vg  # noqa: F401  (the fixture)


def _refused(call, status, word=""):
    from self_speculative_sparse_paged_gb300 import VegasError
    with pytest.raises(VegasError) as ei:
        call()
    assert ei.value.status == status, ei.value
    assert word in ei.value.detail


def test_rope_append_refusals(vg):  # noqa: F811
    kv = vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 64, 4)
    good = dict(kv=kv, q=16, q_stride=768, k=16, k_stride=768, v=16, v_stride=768, q_out=16,
                row_start=16, ctx_lens=16, positions=None, pair_axis=None, num_axes=1, inv_freq=16,
                rot_dim=64, interleaved=False, rope_scale=1.0, total_rows=5, batch=1, stream=0)
    for change, status, word in (
            (dict(kv=vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 96, 4)), 2, "head_dim"),
            (dict(q=None), 1, "q is NULL"), (dict(k=24), 1, "k must be 16-byte"),
            (dict(v=8), 1, "v must be 16-byte"), (dict(q_stride=504), 1, "q_stride"),
            (dict(k_stride=130), 2, "k_stride"), (dict(v_stride=1 << 33), 2, "v_stride"),
            (dict(q_out=None), 1, "q_out"), (dict(q_out=8), 1, "q_out"),
            (dict(row_start=None), 1, "row_start"), (dict(ctx_lens=None), 1, "ctx_lens"),
            (dict(rot_dim=80), 1, "rot_dim"), (dict(rot_dim=-16), 1, "rot_dim"),
            (dict(rot_dim=24), 2, "multiple of 16"), (dict(inv_freq=None), 1, "inv_freq"),
            (dict(num_axes=0), 1, "num_axes"),
            (dict(num_axes=3, positions=16), 1, "pair_axis"),
            (dict(rope_scale=float("nan")), 1, "rope_scale"),
            (dict(total_rows=-1), 1, "total_rows"), (dict(batch=-1), 1, "batch"),
            (dict(total_rows=1 << 24), 2, "total_rows"), (dict(batch=(1 << 16) + 1), 2, "batch")):
        _refused(lambda: vg.vegas_rope_append(**{**good, **change}), status, word)
    vg.vegas_rope_append(**{**good, "total_rows": 0})       # nothing to do
    vg.vegas_rope_append(**{**good, "batch": 0})


def test_prompt_attn_refusals(vg):  # noqa: F811
    kv = vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 64, 4)
    good = dict(kv=kv, q=16, q_stride=512, out=32, row_start=16, ctx_lens=16, total_rows=5,
                batch=1, softmax_scale=0.1, workspace=256, workspace_bytes=1 << 30, stream=0)
    for change, status, word in (
            (dict(kv=vg.PagedKV(16, 16, 16, 4, 8, 8, 2, 64, 4)), 2, "page_size"),
            (dict(kv=vg.PagedKV(16, 16, 16, 4, 16, 65, 1, 64, 4), q_stride=65 * 64), 2, "group"),
            (dict(q=None), 1, "q is NULL"), (dict(q=8), 1, "16-byte"),
            (dict(q_stride=511), 1, "q_stride"), (dict(q_stride=516), 2, "q_stride"),
            (dict(out=None), 1, "out"), (dict(out=48), 1, "out"),
            (dict(row_start=None), 1, "row_start"), (dict(ctx_lens=None), 1, "ctx_lens"),
            (dict(total_rows=-2), 1, "total_rows"), (dict(batch=-1), 1, "batch"),
            (dict(total_rows=1 << 24), 2, "total_rows"), (dict(batch=(1 << 16) + 1), 2, "batch"),
            (dict(kv=vg.PagedKV(16, 16, 16, 4, 16, 64 * 999, 999, 64, 4), q_stride=64 * 64 * 999,
                  total_rows=(1 << 24) - 1), 2, "too many"),
            (dict(softmax_scale=0.0), 1, "softmax_scale"),
            (dict(softmax_scale=-0.5), 1, "softmax_scale"),
            (dict(softmax_scale=float("inf")), 1, "softmax_scale")):
        _refused(lambda: vg.vegas_prompt_attn(**{**good, **change}), status, word)
    vg.vegas_prompt_attn(**{**good, "total_rows": 0, "workspace": None, "workspace_bytes": 0})
    vg.vegas_prompt_attn(**{**good, "batch": 0})


def test_prompt_workspace_size(vg):  # noqa: F811
    kv = vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 64, 4)
    assert vg.vegas_prompt_workspace_size(kv, 10, 2) > 0
    big = vg.PagedKV(16, 16, 16, 4096, 16, 32, 8, 128, 4096)
    assert vg.vegas_prompt_workspace_size(big, 8192, 4) >= vg.vegas_prompt_workspace_size(big, 1, 1)
    bad = vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 80, 4)
    assert vg.vegas_prompt_workspace_size(bad, 10, 2) == 0
    assert vg.vegas_prompt_workspace_size(kv, -1, 2) == 0


def test_token_logprobs_refusals(vg):  # noqa: F811
    good = dict(logits=16, dtype=vg.VEGAS_BF16, row_stride=100, tokens=16, rows=3, vocab=100,
                inv_temperature=1.0, logprob=16, entropy=16, rank=16, top_n=2, top_ids=16,
                top_logprobs=16, stream=0)
    for change, status, word in (
            (dict(dtype=2), 2, "dtype"), (dict(logits=None), 1, "logits"),
            (dict(logits=17), 1, "aligned"), (dict(logits=18, dtype=vg.VEGAS_FP32), 1, "aligned"),
            (dict(rows=-1), 1, "rows"), (dict(vocab=0), 1, "vocab"),
            (dict(row_stride=99), 1, "row_stride"),
            (dict(inv_temperature=0.0), 1, "inv_temperature"),
            (dict(inv_temperature=float("nan")), 1, "inv_temperature"),
            (dict(tokens=None), 1, "tokens"), (dict(top_n=33), 2, "top_n"),
            (dict(top_n=-1), 2, "top_n"), (dict(top_ids=None), 1, "top_ids"),
            (dict(top_logprobs=None), 1, "top_logprobs"),
            (dict(rows=(1 << 26) + 1), 2, "rows"),
            (dict(vocab=(1 << 28) + 1, row_stride=1 << 30), 2, "vocab"),
            (dict(logprob=None, entropy=None, rank=None, top_n=0), 1, "no output")):
        _refused(lambda: vg.vegas_token_logprobs(**{**good, **change}), status, word)
    vg.vegas_token_logprobs(**{**good, "rows": 0})


def test_scales_whose_exponents_overflow_are_refused(vg):  # noqa: F811
    good = dict(logits=16, dtype=vg.VEGAS_BF16, row_stride=100, tokens=16, rows=0, vocab=100,
                inv_temperature=1.0, logprob=16, entropy=16, rank=16, top_n=2, top_ids=16,
                top_logprobs=16, stream=0)
    for t in (1e-38, 2.0 ** -101, 2.0 ** 101, 3e38):
        _refused(lambda: vg.vegas_token_logprobs(**{**good, "inv_temperature": t}), 2,
                 "inv_temperature")
    for t in (2.0 ** -100, 2.0 ** 100):
        vg.vegas_token_logprobs(**{**good, "inv_temperature": t})
    kv = vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 64, 4)
    good = dict(kv=kv, q=16, q_stride=512, out=32, row_start=16, ctx_lens=16, total_rows=0,
                batch=1, softmax_scale=0.1, workspace=256, workspace_bytes=1 << 30, stream=0)
    _refused(lambda: vg.vegas_prompt_attn(**{**good, "softmax_scale": 3e38}), 2, "softmax_scale")
    vg.vegas_prompt_attn(**{**good, "softmax_scale": 2.0 ** 100})


def test_outputs_over_inputs_are_refused(vg):  # noqa: F811
    kv = vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 64, 4)
    _refused(lambda: vg.vegas_prompt_attn(
        kv=kv, q=512, q_stride=512, out=512, row_start=16, ctx_lens=16, total_rows=5, batch=1,
        softmax_scale=0.1, workspace=256, workspace_bytes=1 << 30, stream=0), 1, "out is q")
    _refused(lambda: vg.vegas_rope_append(
        kv=kv, q=16, q_stride=768, k=1040, k_stride=768, v=1296, v_stride=768, q_out=16,
        row_start=16, ctx_lens=16, positions=None, pair_axis=None, num_axes=1, inv_freq=16,
        rot_dim=64, interleaved=False, rope_scale=1.0, total_rows=5, batch=1, stream=0),
        1, "q_out is q")
