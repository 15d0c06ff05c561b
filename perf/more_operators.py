"""Measured cases of the paged cache in 8 bits: the append that quantises keys and values as
they are written, the read back into a bf16 cache, verify attention with its captured scores
and a sparse draft step over it.

A block is one page (16 positions) of one KV head: e4m3 codes and one power-of-two scale each
for K and V, held as a byte e + 127.

With ``own`` false every operator runs in its plain form (elementary torch operations in
32 bits, angles in 64); with ``own`` true through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
PAGE = 16
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
E_MIN, E_MAX, E_BIAS = -60, 60, 127   # exponents of a block's scale, and its byte's offset


# ------------------------------------------------------------------ cases
def listed():
    return [
        # Rotary positions, quantised append.
        # One drafted token each of 32 running sequences: latency counts, most pages partly filled.
        dict(name="append8_step_32", op="append", hq=32, hkv=8, d=128, rows=_lens([1] * 32),
             ctx=_lens([37 + 53 * i for i in range(32)]), rot=128, interleaved=False, pad=0),
        # The windows (gamma 4) of 48 sequences, 64-wide heads in a group of eight.
        dict(name="append8_windows_d64", op="append", hq=64, hkv=8, d=64, rows=_lens([5] * 48),
             ctx=_lens([1000 + 37 * i for i in range(48)]), rot=64, interleaved=True, pad=3),
        # A prefill batch with ragged prompts, one of them behind a cached prefix.
        dict(name="append8_prefill_16k", op="append", hq=32, hkv=8, d=128,
             rows=_lens([8192, 5001, 0, 2095, 1096]), ctx=_lens([0, 0, 9, 515, 0]), rot=128,
             interleaved=False, pad=0),
        # Reading back.
        # The 700 positions of a short prefix, ahead of a prompt chunk.
        dict(name="read8_prefix_700", op="read", hq=8, hkv=2, d=64, first=_lens([0]),
             upto=_lens([700])),
        # Eight long sequences; two of them were partly read back before.
        dict(name="read8_batch_8", op="read", hq=32, hkv=8, d=128,
             first=_lens([0, 0, 4099, 0, 0, 0, 16000, 0]),
             upto=_lens([16384, 9001, 12289, 0, 31000, 777, 16001, 24576])),
        # Verify attention with the captured scores of window rows.
        # A short context of a small layer: the smallest call.
        dict(name="verify8_short", op="verify", hq=8, hkv=2, d=64, ctx=_lens([2048]), gamma=4,
             mask=0b10001),
        # Single tokens of a ragged batch, an empty prefix among them, nothing captured.
        dict(name="verify8_token_ragged", op="verify", hq=32, hkv=8, d=128,
             ctx=_lens([0, 1, 15, 4000, 2777, 8100, 129, 640, 5555, 1031, 16, 3001]), gamma=0, mask=0),
        # One long sequence.
        dict(name="verify8_32k", op="verify", hq=32, hkv=8, d=128, ctx=_lens([32768]), gamma=4,
             mask=0b10001),
        # Four very long sequences of 64-wide heads in a group of eight: many query columns.
        dict(name="verify8_128k_d64", op="verify", hq=64, hkv=8, d=64, ctx=_lens([131072] * 4),
             gamma=6, mask=0b1000001),
        # A batch of long sequences: the largest call.
        dict(name="verify8_batch_8", op="verify", hq=32, hkv=8, d=128,
             ctx=_lens([49152, 65536, 53001, 60007, 51111, 64000, 57345, 62003]), gamma=5,
             mask=0b100001),
        # Draft steps over the selected positions (5% and 3% of the prefix) and the dense tail.
        dict(name="draft8_32k", op="draft", hq=32, hkv=8, d=128, ctx=_lens([32768]),
             k=_lens([1639]), tail=_lens([6])),
        dict(name="draft8_128k_d64", op="draft", hq=64, hkv=8, d=64, ctx=_lens([131072] * 4),
             k=_lens([3933, 3933, 3001, 3933]), tail=_lens([8, 9, 8, 11])),
    ]


def _lens(v):
    return ",".join(str(int(x)) for x in v)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "verify", "draft"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 8] if d == 128 else [1, 2, 4, 5, 8, 16])
    case = dict(op=op, hq=hkv * g, hkv=hkv, d=d)
    batch = _log_int(rng, 1, 12)
    if op == "append":
        total = _log_int(rng, max(4, batch), 16384)
        rows = _split(rng, total, batch)
        ctx = [rng.choice([0, _log_int(rng, 1, 2000)]) for _ in rows]
        case.update(rows=_lens(rows), ctx=_lens(ctx), rot=rng.choice([d, d, d // 2, 32, 0]),
                    interleaved=rng.random() < 0.4, pad=rng.choice([0, 0, 3]))
        return case
    ctx = [rng.choice([0, 1, _log_int(rng, 1, 65536), _log_int(rng, 1, 65536)]) for _ in range(batch)]
    while sum(ctx) * hkv * d > 110000 * 8 * 128:     # (the largest listed read moves about as much)
        ctx = [c // 2 for c in ctx]
    if op == "read":
        ctx[0] = max(ctx[0], 1)
        first = [0] + [rng.choice([0, 0, rng.randrange(c + 1)]) for c in ctx[1:]]
        case.update(first=_lens(first), upto=_lens(ctx))
        return case
    if op == "verify":
        most = min(15, (40 if d == 128 else 64) // g - 1)
        gamma = rng.choice([0, most, rng.randrange(most + 1), min(4, most)])
        while len(ctx) * max(ctx) * hkv * max(d, (gamma + 1) * g) > 8 * 65536 * 8 * 128:
            ctx = [c // 2 for c in ctx]
        mask = rng.choice([0, 1 | 1 << gamma, 1 | 1 << gamma, (1 << (gamma + 1)) - 1,
                           1 << rng.randrange(gamma + 1)])
        case.update(ctx=_lens(ctx), gamma=gamma, mask=mask)
        return case
    k = [min(c, rng.choice([c // 20, c // 33, _log_int(rng, 1, 6000), 0])) for c in ctx]
    case.update(ctx=_lens(ctx), k=_lens(k), tail=_lens([rng.randrange(1, 12) for _ in ctx]))
    return case


def _split(rng, total, batch):
    cut = sorted(rng.randrange(total + 1) for _ in range(batch - 1))
    rows = [b - a for a, b in zip([0] + cut, cut + [total])]
    return rows if max(rows) else [total] + rows[1:]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    return {"append": _prepare_append, "read": _prepare_read, "verify": _prepare_verify,
            "draft": _prepare_draft}[case["op"]](case, gen)


def _two_to(e):
    """2^e of 32-bit integers, from the bits (a power function may round)."""
    return (e + 127 << 23).view(FP32)


def _codes(x, e):
    """The e4m3 codes of x for a scale of 2^e."""
    return (x * _two_to(-e)).clamp_(-448.0, 448.0).to(E4M3)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, within the scales' range (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(torch.int32)
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _cache(case, lens, gen, s):
    """Pages of `lens` positions a sequence lie shuffled in the pool; each block holds values
    quantised with a scale of its own."""
    hkv, d = case["hkv"], case["d"]
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    max_pages = max(max(pages), 1)
    num_pages = sum(pages) + 3
    perm = torch.randperm(num_pages, generator=gen, device=DEV, dtype=torch.int64).cpu().numpy()
    table, at = np.zeros((len(lens), max_pages), dtype=np.int32), 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    s.update(case=case, batch=len(lens), num_pages=num_pages, max_pages=max_pages, table=table,
             block_table=torch.from_numpy(table).to(DEV))
    shape = (num_pages, hkv, PAGE, d)
    # a few keys lie along a direction that the queries share (heavy hitters); values differ in
    # size from page to page
    u = torch.randn((d,), generator=gen, device=DEV)
    u = u / u.norm()
    x = torch.randn(shape, generator=gen, device=DEV)
    heavy = torch.rand((num_pages, hkv, PAGE, 1), generator=gen, device=DEV) < 0.02
    x = torch.where(heavy, 3 * u + 0.3 * x, x).to(BF16).float()
    e = _exponent(x.abs().amax((2, 3)))
    s["k_cache"], s["k_scale"] = _codes(x, e[:, :, None, None]), (e + E_BIAS).to(torch.uint8)
    del x
    x = torch.randn(shape, generator=gen, device=DEV)
    x *= torch.exp2(torch.rand((num_pages, hkv, 1, 1), generator=gen, device=DEV) * 3 - 2)
    x = x.to(BF16).float()
    e = _exponent(x.abs().amax((2, 3)))
    s["v_cache"], s["v_scale"] = _codes(x, e[:, :, None, None]), (e + E_BIAS).to(torch.uint8)
    return u


def _prepare_append(case, gen):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows, ctx = _ints(case["rows"]), _ints(case["ctx"])
    used = sum(rows)
    total = used + case["pad"]
    s = {"total": total, "used": used}
    _cache(case, [c + n for c, n in zip(ctx, rows)], gen, s)
    s["row_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)).to(DEV)
    s["ctx_lens"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    # what a host scheduler knows: each packed row's sequence and position, and the first pages
    # that hold rows already
    seq = np.repeat(np.arange(len(rows)), rows)
    pos = np.concatenate([np.arange(n) + c for n, c in zip(rows, ctx)] + [np.zeros(0)])
    s["row_seq"] = torch.from_numpy(seq.astype(np.int64)).to(DEV)
    s["row_pos"] = torch.from_numpy(pos.astype(np.int64)).to(DEV)
    held = [b for b, (n, c) in enumerate(zip(rows, ctx)) if n and c % PAGE]
    s["held_page"] = torch.tensor([int(s["table"][b, ctx[b] // PAGE]) for b in held],
                                  dtype=torch.int64, device=DEV)
    s["held_rows"] = torch.tensor([ctx[b] % PAGE for b in held], dtype=torch.int64, device=DEV)
    # heads and rows differ in size, so scales differ and some first pages have to be raised
    size = torch.exp2(torch.rand((total, hq + 2 * hkv, 1), generator=gen, device=DEV) * 4 - 2)
    s["qkv"] = (torch.randn((total, hq + 2 * hkv, d), generator=gen, device=DEV) * size).to(BF16).flatten(1)
    s["q_out"] = torch.randn((total, hq, d), generator=gen, device=DEV).to(BF16)
    half = case["rot"] // 2
    s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).to(FP32).to(DEV)
    return s


def _prepare_read(case, gen):
    first, upto = _ints(case["first"]), _ints(case["upto"])
    s = {}
    _cache(case, upto, gen, s)
    s["first"] = torch.tensor(first, dtype=torch.int32, device=DEV)
    s["upto"] = torch.tensor(upto, dtype=torch.int32, device=DEV)
    seq = np.repeat(np.arange(len(upto)), [n - f for f, n in zip(first, upto)])
    pos = np.concatenate([np.arange(f, n) for f, n in zip(first, upto)] + [np.zeros(0)])
    s["row_seq"] = torch.from_numpy(seq.astype(np.int64)).to(DEV)
    s["row_pos"] = torch.from_numpy(pos.astype(np.int64)).to(DEV)
    # the bf16 cache that is written, with a table of its own
    perm = torch.randperm(s["num_pages"], generator=gen, device=DEV, dtype=torch.int32)
    s["to_table"] = perm[s["block_table"].long()].contiguous()
    shape = (s["num_pages"], case["hkv"], PAGE, case["d"])
    s["to_k"] = torch.zeros(shape, dtype=BF16, device=DEV)
    s["to_v"] = torch.zeros(shape, dtype=BF16, device=DEV)
    return s


def _queries(case, shape, u, gen):
    """Queries that share the heavy keys' direction; heads differ somewhat in size."""
    q = torch.randn(shape, generator=gen, device=DEV) + 2 * u
    return (q * torch.exp2(torch.rand(shape[:-1] + (1,), generator=gen, device=DEV) - 0.5)).to(BF16)


def _prepare_verify(case, gen):
    ctx, t = _ints(case["ctx"]), case["gamma"] + 1
    s = {}
    u = _cache(case, [c + t for c in ctx], gen, s)
    s["ctx_lens"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    s["q"] = _queries(case, (len(ctx), t, case["hq"], case["d"]), u, gen)
    s["out"] = torch.zeros_like(s["q"])
    s["scale"] = 1.0 / math.sqrt(case["d"])
    s["stride"] = max(max(ctx), 1)
    s["scores"] = torch.zeros((len(ctx), case["hkv"], s["stride"]), device=DEV) if case["mask"] else None
    bits = [i for i in range(t) if case["mask"] >> i & 1]
    s["captured"] = torch.tensor(bits, dtype=torch.int64, device=DEV)
    return s


def _prepare_draft(case, gen):
    ctx, k, tail = _ints(case["ctx"]), _ints(case["k"]), _ints(case["tail"])
    s = {}
    u = _cache(case, [c + t for c, t in zip(ctx, tail)], gen, s)
    s["k_max"], s["max_tail"] = max(max(k), 1), max(tail)
    idx = torch.full((len(ctx), case["hkv"], s["k_max"]), -1, dtype=torch.int32, device=DEV)
    for b, (c, n) in enumerate(zip(ctx, k)):
        if n:
            got = torch.rand((case["hkv"], c), generator=gen, device=DEV).topk(n, dim=-1).indices
            idx[b, :, :n] = got.sort(dim=-1).values.to(torch.int32)
    s["idx"] = idx
    for name, v in (("ctx_lens", ctx), ("k", k), ("tail", tail)):
        s[name] = torch.tensor(v, dtype=torch.int32, device=DEV)
    s["q"] = _queries(case, (len(ctx), case["hq"], case["d"]), u, gen)
    s["out"] = torch.zeros_like(s["q"])
    s["scale"] = 1.0 / math.sqrt(case["d"])
    return s


# ------------------------------------------------------------------ passes
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "read": _own_read, "verify": _own_verify,
                "draft": _own_draft}[op](state)
    return {"append": _plain_append, "read": _plain_read, "verify": _plain_verify,
            "draft": _plain_draft}[op](state)


def _kv8(state):
    """The cache's descriptor, which a program makes once."""
    import self_speculative_sparse_paged_gb300 as vg
    if "kv8" not in state:
        state["kv8"] = vg.paged_kv8(state["k_cache"], state["v_cache"], state["k_scale"],
                                    state["v_scale"], state["block_table"], state["case"]["hq"])
    return vg, state["kv8"]


def _own_append(s):
    c = s["case"]
    vg, kv = _kv8(s)
    qkv, d = s["qkv"], c["d"]
    stride = qkv.stride(0)
    vg.vegas_rope_append_kv8(kv, qkv, stride, qkv[:, c["hq"] * d:], stride,
                             qkv[:, (c["hq"] + c["hkv"]) * d:], stride, s["q_out"],
                             s["row_start"], s["ctx_lens"], None, None, 1, s["inv_freq"],
                             c["rot"], c["interleaved"], 1.0, s["total"], s["batch"])
    return {n: s[n] for n in ("q_out", "k_cache", "k_scale", "v_cache", "v_scale")}


def _own_read(s):
    vg, kv = _kv8(s)
    if "to" not in s:
        s["to"] = vg.paged_kv(s["to_k"], s["to_v"], s["to_table"], s["case"]["hq"])
    vg.vegas_kv8_read(kv, s["to"], s["first"], s["upto"], s["batch"])
    return {"k": s["to_k"], "v": s["to_v"]}


def _own_verify(s):
    c = s["case"]
    vg, kv = _kv8(s)
    if "workspace" not in s:
        n = vg.vegas_verify_kv8_workspace_size(kv, s["batch"], c["gamma"])
        s["workspace"] = torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV)
    ws = s["workspace"]
    vg.vegas_verify_attn_kv8(kv, s["q"], s["out"], s["scores"], s["stride"], s["ctx_lens"],
                             s["batch"], c["gamma"], c["mask"], s["scale"], ws, ws.numel())
    return {"out": s["out"]} if s["scores"] is None else {"out": s["out"], "scores": s["scores"]}


def _own_draft(s):
    vg, kv = _kv8(s)
    vg.vegas_sparse_decode_attn_kv8(kv, s["q"], s["out"], s["idx"], s["k_max"], s["k"],
                                    s["ctx_lens"], s["tail"], s["max_tail"], s["batch"], s["scale"])
    return s["out"]


def _plain_append(s):
    c = s["case"]
    hq, hkv, d, rot, used = c["hq"], c["hkv"], c["d"], c["rot"], s["used"]
    x = s["qkv"][:used].view(used, hq + 2 * hkv, d)
    angle = s["row_pos"][:, None].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    y = x[:, :hq + hkv].float()
    half = rot // 2
    if c["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    y = torch.cat([turned, y[..., rot:]], dim=-1).to(BF16)
    s["q_out"][:used] = y[:, :hq]
    _plain_quantise(s, "k", y[:, hq:].float())
    _plain_quantise(s, "v", x[:, hq + hkv:].float())
    return {n: s[n] for n in ("q_out", "k_cache", "k_scale", "v_cache", "v_scale")}


def _plain_quantise(s, which, y):
    """Rows y (used, hkv, d) to their pages: the largest element of a page's new rows sets its
    scale; a first page that holds rows keeps the larger of this and its own, its rows requantised."""
    codes, scale = s[which + "_cache"].view(torch.uint8), s[which + "_scale"]
    page = s["block_table"].long()[s["row_seq"], s["row_pos"] // PAGE]
    slot = s["row_pos"] % PAGE
    amax = torch.full(scale.shape, -1.0, device=DEV)
    amax.scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]), y.abs().amax(-1), "amax")
    old = scale.to(torch.int32) - E_BIAS
    e = torch.where(amax >= 0, _exponent(amax), old)
    hp = s["held_page"]
    e[hp] = torch.maximum(e[hp], old[hp])
    held = s["k_cache" if which == "k" else "v_cache"].view(torch.uint8)[hp]
    again = _codes(held.view(E4M3).float(), (e[hp] - old[hp])[:, :, None, None]).view(torch.uint8)
    keep = torch.arange(PAGE, device=DEV) < s["held_rows"][:, None]
    codes[hp] = torch.where(keep[:, None, :, None], again, held)
    codes[page, :, slot] = _codes(y, e[page][:, :, None]).view(torch.uint8)
    scale.copy_((e + E_BIAS).to(torch.uint8))


def _values(s, which):
    """The numbers that the cache's codes stand for."""
    e = (s[which + "_scale"].to(torch.int32) - E_BIAS)[:, :, None, None]
    return s[which + "_cache"].float() * _two_to(e)


def _plain_read(s):
    at, slot = s["row_pos"] // PAGE, s["row_pos"] % PAGE
    page = s["block_table"].long()[s["row_seq"], at]
    to = s["to_table"].long()[s["row_seq"], at]
    s["to_k"][to, :, slot] = _values(s, "k")[page, :, slot].to(BF16)
    s["to_v"][to, :, slot] = _values(s, "v")[page, :, slot].to(BF16)
    return {"k": s["to_k"], "v": s["to_v"]}


def _plain_verify(s):
    c = s["case"]
    hq, hkv, d, batch, t = c["hq"], c["hkv"], c["d"], s["batch"], c["gamma"] + 1
    g, n = hq // hkv, s["max_pages"] * PAGE
    table = s["block_table"].long()
    k = _values(s, "k")[table].permute(0, 2, 1, 3, 4).reshape(batch, hkv, n, d)
    q = s["q"].float().view(batch, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, t * g, d)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(batch, hkv, t, g, n)
    del k
    ctx = s["ctx_lens"].long()
    pos = torch.arange(n, device=DEV)
    if s["scores"] is not None:
        got = x[:, :, s["captured"]].sum((2, 3))[..., :s["stride"]]
        inside = pos[None, :got.shape[-1]] < ctx[:, None]
        m = s["scores"][..., :got.shape[-1]]
        m.copy_(torch.where(inside[:, None, :], got, m))
    ahead = pos > (ctx[:, None] + torch.arange(t, device=DEV))[:, None, :, None, None]
    x.masked_fill_(ahead, -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    v = _values(s, "v")[table].permute(0, 2, 1, 3, 4).reshape(batch, hkv, n, d)
    o = torch.matmul(x.view(batch, hkv, t * g, n), v).view(batch, hkv, t, g, d)
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(batch, t, hq, d))
    return {"out": s["out"]} if s["scores"] is None else {"out": s["out"], "scores": s["scores"]}


def _plain_draft(s):
    c = s["case"]
    hq, hkv, d, batch = c["hq"], c["hkv"], c["d"], s["batch"]
    g, n = hq // hkv, s["k_max"] + s["max_tail"]
    # the list of a sequence and head: the selected positions, then the tail
    j = torch.arange(n, device=DEV)
    k = s["k"].long()[:, None]
    listed_at = torch.nn.functional.pad(s["idx"].long(), (0, s["max_tail"]))
    pos = torch.where((j < k)[:, None], listed_at, (s["ctx_lens"].long()[:, None] + j - k)[:, None])
    there = j < k + s["tail"].long()[:, None]
    pos = torch.where(there[:, None], pos, 0)
    page = s["block_table"].long()[torch.arange(batch, device=DEV)[:, None, None], pos // PAGE]
    head, slot = torch.arange(hkv, device=DEV)[None, :, None], pos % PAGE
    ek = (s["k_scale"][page, head].to(torch.int32) - E_BIAS)[..., None]
    ev = (s["v_scale"][page, head].to(torch.int32) - E_BIAS)[..., None]
    kk = s["k_cache"].view(torch.uint8)[page, head, slot].view(E4M3).float() * _two_to(ek)
    vv = s["v_cache"].view(torch.uint8)[page, head, slot].view(E4M3).float() * _two_to(ev)
    x = torch.matmul(s["q"].float().view(batch, hkv, g, d), kk.transpose(-1, -2)).mul_(s["scale"])
    x.masked_fill_(~there[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    s["out"].copy_(torch.matmul(x, vv).view(batch, hq, d))
    return s["out"]


# ------------------------------------------------------------------ what a pass needs
def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        used = sum(_ints(case["rows"]))
        return {"bytes": used * d * (2 * (hq + 2 * hkv) + 2 * hq + 2 * hkv) + 2 * case["rot"],
                "flops": used * (hq + hkv) * case["rot"] * 3 + used * hkv * d * 4}
    if case["op"] == "read":
        n = sum(u - f for f, u in zip(_ints(case["first"]), _ints(case["upto"])))
        return {"bytes": n * hkv * (6 * d + 2 / PAGE), "flops": 2 * n * hkv * d}
    ctx = _ints(case["ctx"])
    if case["op"] == "verify":
        t = case["gamma"] + 1
        n = sum(c + t for c in ctx)
        pairs = sum(t * c + t * (t + 1) // 2 for c in ctx)
        scores = 4 * sum(ctx) * hkv if case["mask"] else 0
        return {"bytes": n * hkv * (2 * d + 2 / PAGE) + scores + 4 * len(ctx) * t * hq * d,
                "flops": 4 * pairs * hq * d}
    k, tail = _ints(case["k"]), _ints(case["tail"])
    n = sum(k) + sum(tail)
    return {"bytes": n * hkv * (2 * d + 2) + 4 * sum(k) * hkv + 4 * len(ctx) * hq * d,
            "flops": 4 * n * hq * d}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "verify": _exact_verify,
            "draft": _exact_draft}[case["op"]](s)


def _decode(codes, scale):
    """c * 2^e of whole blocks (..., PAGE, d) with scale bytes (...), from the bits of the codes:
    sign, four bits of exponent (bias 7), three of fraction."""
    bits = codes.view(torch.uint8).long()
    ex, frac = bits >> 3 & 15, (bits & 7).double() / 8
    size = torch.where(ex > 0, (1 + frac) * 2.0 ** (ex.double() - 7), frac * 2.0 ** -6)
    return torch.where(bits > 127, -size, size) * 2.0 ** (scale.double() - 127)[..., None, None]


def _exact_append(s):
    c = s["case"]
    hq, hkv, d, rot = c["hq"], c["hkv"], c["d"], c["rot"]
    q, src, at, half = s["q_out"].double(), s["qkv"].double(), 0, rot // 2
    for n, ctx in zip(_ints(c["rows"]), _ints(c["ctx"])):
        x = src[at:at + n].view(n, hq + 2 * hkv, d)[:, :hq].clone()
        p = torch.arange(ctx, ctx + n, device=DEV, dtype=torch.float64)[:, None].expand(n, half)
        turn = torch.polar(torch.ones_like(p), p * s["inv_freq"].double())[:, None, :]
        first = slice(0, rot, 2) if c["interleaved"] else slice(0, half)
        second = slice(1, rot, 2) if c["interleaved"] else slice(half, rot)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        x[..., first], x[..., second] = z.real, z.imag
        q[at:at + n] = x
        at += n
    # (codes and their scales are choices, not computed numbers)
    return {"q_out": q, "k_cache": None, "k_scale": None, "v_cache": None, "v_scale": None}


def _exact_read(s):
    out = {}
    for n in ("k", "v"):
        to = s["to_" + n].double()
        for b, (f, u) in enumerate(zip(_ints(s["case"]["first"]), _ints(s["case"]["upto"]))):
            if u <= f:
                continue
            pages = s["block_table"][b, :(u + PAGE - 1) // PAGE].long()
            x = _decode(s[n + "_cache"].view(torch.uint8)[pages], s[n + "_scale"][pages])     # (pages, hkv, PAGE, d)
            pos = torch.arange(f, u, device=DEV)
            to[s["to_table"][b].long()[pos // PAGE], :, pos % PAGE] = x[pos // PAGE, :, pos % PAGE]
        out[n] = to
    return out


def _exact_verify(s):
    c = s["case"]
    hq, hkv, d, t = c["hq"], c["hkv"], c["d"], c["gamma"] + 1
    g, out = hq // hkv, s["out"].double()
    scores = None if s["scores"] is None else s["scores"].double()
    bits = [i for i in range(t) if c["mask"] >> i & 1]
    for b, ctx in enumerate(_ints(c["ctx"])):
        pages = s["block_table"][b, :(ctx + t + PAGE - 1) // PAGE].long()
        for h in range(hkv):
            k = _decode(s["k_cache"].view(torch.uint8)[pages, h], s["k_scale"][pages, h]).reshape(-1, d)[:ctx + t]
            v = _decode(s["v_cache"].view(torch.uint8)[pages, h], s["v_scale"][pages, h]).reshape(-1, d)[:ctx + t]
            x = s["q"][b, :, h * g:(h + 1) * g].double() @ k.t() / math.sqrt(d)      # (t, g, positions)
            if scores is not None:
                scores[b, h, :ctx] = x[bits].sum((0, 1))[:ctx]
            for i in range(t):
                out[b, i, h * g:(h + 1) * g] = torch.softmax(x[i, :, :ctx + i + 1], -1) @ v[:ctx + i + 1]
    return {"out": out} if scores is None else {"out": out, "scores": scores}


def _exact_draft(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g, out = hq // hkv, s["out"].double()
    for b, (ctx, k, tail) in enumerate(zip(_ints(c["ctx"]), _ints(c["k"]), _ints(c["tail"]))):
        for h in range(hkv):
            pos = torch.cat([s["idx"][b, h, :k].long(), torch.arange(ctx, ctx + tail, device=DEV)])
            page = s["block_table"][b].long()[pos // PAGE]
            kk = _decode(s["k_cache"].view(torch.uint8)[page, h, pos % PAGE][:, None], s["k_scale"][page, h])[:, 0]
            vv = _decode(s["v_cache"].view(torch.uint8)[page, h, pos % PAGE][:, None], s["v_scale"][page, h])[:, 0]
            x = s["q"][b, h * g:(h + 1) * g].double() @ kk.t() / math.sqrt(d)
            out[b, h * g:(h + 1) * g] = torch.softmax(x, -1) @ vv
    return out
