"""The 8-bit cache without a GPU: its oracle against itself and torch, and the calls' refusals."""
import numpy as np
import pytest

import kv8_case as k8
from test_abi_cpu import vg  # noqa: F401  (the fixture)
from test_prompt_abi_cpu import _refused


def test_oracle_codes_are_torchs():
    torch = pytest.importorskip("torch")
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(every, k8.VALUE, equal_nan=True)
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 9, 4000),
                        (k8.VALUE[:126] + k8.VALUE[1:127]) / 2, -k8.VALUE[:127]]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(k8.encode(x), want)
    assert list(k8.encode([np.inf, -np.inf, 1e9])) == [126, 254, 126]


def test_oracle_exponents():
    assert k8.exponent(0.0) == -60 and k8.exponent(448.0) == 0 and k8.exponent(449.0) == 1
    assert k8.exponent(1e30) == 60 and k8.exponent(1e-30) == -60
    for a in (1e-3, 0.5, 1.75, 1.76, 300.0, 7e5):
        e = k8.exponent(a)
        assert a <= 448 * 2.0 ** e and a > 448 * 2.0 ** (e - 1)


def test_oracle_append_raises_a_held_page():
    codes, scale = np.zeros((2, 1, 16, 4), np.uint8), np.zeros((2, 1), np.uint8)
    first = np.array([[[1.0, -2, 448, 2 ** -9]], [[3.0, 5, 7, 9]]])
    k8.append(codes, scale, first, [1, 0], 0)
    assert scale[1, 0] == 127 and k8.VALUE[codes[1, 0, 0, 3]] == 2 ** -9
    k8.append(codes, scale, np.full((1, 1, 4), 1000.0), [1, 0], 2)
    assert scale[1, 0] == 129                                  # 448 * 4 holds 1000
    got = k8.decode(codes[1:2], scale[1:2])[0, 0]
    assert np.array_equal(got[0], [1.0, -2, 448, 0]) and np.array_equal(got[1], [3.0, 5, 7, 9])
    k8.append(codes, scale, np.full((1, 1, 4), 1e-3), [1, 0], 2)   # written over: stays raised
    assert scale[1, 0] == 129


def _kv(mod, **change):
    f = dict(k_cache=16, v_cache=16, k_scale=1, v_scale=1, block_table=16, num_pages=4, page_size=16,
             num_q_heads=8, num_kv_heads=2, head_dim=64, max_pages_per_seq=4)
    return mod.PagedKV8(**{**f, **change})


BAD_CACHES = ((dict(k_cache=None), 1, "NULL cache"), (dict(v_cache=None), 1, "NULL cache"),
              (dict(k_cache=8), 1, "16-byte"), (dict(k_scale=None), 1, "NULL scales"),
              (dict(v_scale=None), 1, "NULL scales"), (dict(block_table=None), 1, "block table"),
              (dict(page_size=32), 2, "page_size"), (dict(head_dim=96), 2, "head_dim"),
              (dict(num_q_heads=7), 1, "heads"), (dict(num_pages=0), 1, "num_pages"),
              (dict(num_pages=1 << 27), 2, "cache rows"),
              (dict(max_pages_per_seq=1 << 20), 2, "capacity"))


def test_append_refusals(vg):  # noqa: F811
    good = dict(kv=_kv(vg), q=16, q_stride=768, k=16, k_stride=768, v=16, v_stride=768, q_out=16,
                row_start=16, ctx_lens=16, positions=None, pair_axis=None, num_axes=1, inv_freq=16,
                rot_dim=64, interleaved=False, rope_scale=1.0, total_rows=5, batch=1, stream=0)
    changes = [(dict(kv=_kv(vg, **c)), s, w) for c, s, w in BAD_CACHES]
    changes += [
        (dict(q=None), 1, "q is NULL"), (dict(k=24), 1, "k must be 16-byte"), (dict(v=8), 1, "v must be"),
        (dict(q_stride=504), 1, "q_stride"), (dict(k_stride=130), 2, "k_stride"),
        (dict(v_stride=1 << 33), 2, "v_stride"), (dict(q_out=None), 1, "q_out"),
        (dict(row_start=None), 1, "row_start"), (dict(ctx_lens=None), 1, "ctx_lens"),
        (dict(rot_dim=80), 1, "rot_dim"), (dict(rot_dim=24), 2, "multiple of 16"),
        (dict(inv_freq=None), 1, "inv_freq"), (dict(num_axes=0), 1, "num_axes"),
        (dict(num_axes=3, positions=16), 1, "pair_axis"),
        (dict(rope_scale=float("inf")), 1, "rope_scale"), (dict(total_rows=-1), 1, "total_rows"),
        (dict(batch=-1), 1, "batch"), (dict(total_rows=1 << 24), 2, "total_rows"),
        (dict(batch=(1 << 16) + 1), 2, "batch"),
        (dict(q=1 << 20, q_out=(1 << 20) + 1024), 1, "lies over"),
        (dict(q_out=16), 1, "q_out is q")]
    for change, status, word in changes:
        _refused(lambda: vg.vegas_rope_append_kv8(**{**good, **change}), status, word)
    vg.vegas_rope_append_kv8(**{**good, "total_rows": 0})       # nothing to do
    vg.vegas_rope_append_kv8(**{**good, "batch": 0})


def test_read_refusals(vg):  # noqa: F811
    to = vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 64, 4)
    good = dict(kv=_kv(vg), to=to, first=None, upto=16, batch=1, stream=0)
    changes = [(dict(kv=_kv(vg, **c)), s, w) for c, s, w in BAD_CACHES]
    changes += [(dict(to=vg.PagedKV(16, 16, 16, 4, 16, 8, 4, 64, 4)), 1, "differ"),
                (dict(to=vg.PagedKV(16, 16, 16, 4, 16, 8, 2, 128, 4)), 1, "differ"),
                (dict(to=vg.PagedKV(16, None, 16, 4, 16, 8, 2, 64, 4)), 1, "NULL cache"),
                (dict(upto=None), 1, "upto"), (dict(batch=-1), 1, "batch"),
                (dict(batch=65536), 2, "batch")]
    for change, status, word in changes:
        _refused(lambda: vg.vegas_kv8_read(**{**good, **change}), status, word)
    vg.vegas_kv8_read(**{**good, "batch": 0})


def test_verify_refusals(vg):  # noqa: F811
    good = dict(kv=_kv(vg), q=16, out=16, scores=16, score_stride=64, ctx_lens=16, batch=1, gamma=4,
                capture_row_mask=17, softmax_scale=0.1, workspace=256, workspace_bytes=1 << 30, stream=0)
    changes = [(dict(kv=_kv(vg, **c)), s, w) for c, s, w in BAD_CACHES]
    changes += [
        (dict(q=None), 1, "NULL q"), (dict(out=None), 1, "NULL q"), (dict(ctx_lens=None), 1, "NULL q"),
        (dict(q=8), 1, "16-byte"), (dict(out=24), 1, "16-byte"), (dict(batch=-1), 1, "batch"),
        (dict(batch=(1 << 16) + 1), 2, "batch"),
        (dict(gamma=-1), 2, "gamma"), (dict(gamma=16), 2, "gamma"),
        (dict(gamma=16, scores=None), 2, "gamma"), (dict(capture_row_mask=0), 1, "mask"),
        (dict(capture_row_mask=32), 1, "mask"), (dict(score_stride=0), 1, "score_stride"),
        (dict(softmax_scale=float("nan")), 1, "softmax_scale"),
        (dict(softmax_scale=2.0 ** 21), 2, "softmax_scale"),
        (dict(kv=_kv(vg, num_q_heads=32), gamma=4), 2, "query rows"),          # 80 columns
        (dict(kv=_kv(vg, head_dim=128, num_q_heads=18), gamma=4), 2, "query rows")]   # 45
    for change, status, word in changes:
        _refused(lambda: vg.vegas_verify_attn_kv8(**{**good, **change}), status, word)
    vg.vegas_verify_attn_kv8(**{**good, "batch": 0})
    vg.vegas_verify_attn_kv8(**{**good, "batch": 0, "scores": None, "capture_row_mask": 0})


def test_verify_workspace_size(vg):  # noqa: F811
    many = _kv(vg, num_pages=1 << 16, max_pages_per_seq=4096, num_q_heads=32, num_kv_heads=8, head_dim=128)
    assert vg.vegas_verify_kv8_workspace_size(many, 64, 4) > 0
    assert vg.vegas_verify_kv8_workspace_size(many, 64, 16) == 0
    assert vg.vegas_verify_kv8_workspace_size(many, -1, 4) == 0
    assert vg.vegas_verify_kv8_workspace_size(_kv(vg, head_dim=80), 4, 4) == 0
    assert vg.vegas_verify_kv8_workspace_size(_kv(vg, num_q_heads=64), 4, 4) == 0


def test_sparse_refusals(vg):  # noqa: F811
    good = dict(kv=_kv(vg), q=16, out=16, idx=16, k_max=8, k_per_seq=16, tail_start=16, tail_len=16,
                max_tail=2, batch=1, softmax_scale=0.1, stream=0)
    changes = [(dict(kv=_kv(vg, **c)), s, w) for c, s, w in BAD_CACHES]
    changes += [
        (dict(batch=-1), 1, "batch"), (dict(k_max=-1), 1, "k_max"), (dict(k_max=0, max_tail=0), 1, "empty"),
        (dict(q=None), 1, "NULL"), (dict(out=None), 1, "NULL"), (dict(idx=None), 1, "NULL"),
        (dict(k_per_seq=None), 1, "NULL"), (dict(q=8), 1, "16-byte"),
        (dict(softmax_scale=float("inf")), 1, "softmax_scale"),
        (dict(softmax_scale=-2.0 ** 21), 2, "softmax_scale"),
        (dict(kv=_kv(vg, num_q_heads=34)), 2, "group"), (dict(k_max=40000), 2, "exceeds")]
    for change, status, word in changes:
        _refused(lambda: vg.vegas_sparse_decode_attn_kv8(**{**good, **change}), status, word)
    vg.vegas_sparse_decode_attn_kv8(**{**good, "batch": 0})
