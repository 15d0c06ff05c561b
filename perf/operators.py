"""Measured cases of the operators around a decode iteration: rotary positions with the
cache append, attention over whole prompts, and log probabilities of given tokens.

With ``own`` false every operator runs in its plain form (elementary torch operations in
32 bits, angles in 64); with ``own`` true through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
PAGE = 16
BF16, FP32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ cases
def listed():
    return [
        # Rotary positions and cache append.
        # One new token each of 32 running sequences: a decode step, where latency counts.
        dict(name="rope_decode_32", op="rope", hq=32, hkv=8, d=128, rows=_lens([1] * 32),
             ctx=_lens([37 + 53 * i for i in range(32)]), rot=128, axes=1, interleaved=False, pad=0),
        # Ragged prompts packed into one batch, 64-wide heads in a group of eight.
        dict(name="rope_ragged_d64", op="rope", hq=64, hkv=8, d=64,
             rows=_lens([1, 777, 0, 2049, 130, 64]), ctx=_lens([500, 0, 9, 33, 0, 1]), rot=64,
             axes=1, interleaved=True, pad=5),
        # A video prompt: three position axes (time, height, width), some chunk of it cached before.
        dict(name="rope_video_3axes", op="rope", hq=32, hkv=8, d=128, rows=_lens([6001, 2100]),
             ctx=_lens([0, 515]), rot=128, axes=3, interleaved=False, pad=0),
        # A full prefill batch.
        dict(name="rope_prefill_32k", op="rope", hq=32, hkv=8, d=128,
             rows=_lens([16384, 9001, 4095, 3288]), ctx=_lens([0, 0, 0, 0]), rot=128, axes=1,
             interleaved=False, pad=0),
        # Attention over whole prompts.
        # A short question: the smallest call.
        dict(name="prompt_short", op="prompt", hq=8, hkv=2, d=64, rows=_lens([45]),
             ctx=_lens([0]), pad=0),
        # Chunked prefill next to running sequences: a few decode tokens and one prompt chunk.
        dict(name="prompt_mixed_step", op="prompt", hq=32, hkv=8, d=128,
             rows=_lens([1, 1, 5, 509, 1, 0]), ctx=_lens([4000, 15, 8100, 1031, 2777, 40]), pad=2),
        # One 1000-token chunk of a long document whose first 31K tokens are cached.
        dict(name="prompt_chunk_at_31k", op="prompt", hq=32, hkv=8, d=128, rows=_lens([1000]),
             ctx=_lens([31768]), pad=0),
        # Ragged prompts packed into one batch, 64-wide heads in a group of eight.
        dict(name="prompt_packed_d64", op="prompt", hq=64, hkv=8, d=64,
             rows=_lens([2500, 31, 1777, 640, 2051, 129]), ctx=_lens([0, 0, 0, 64, 0, 7]), pad=0),
        # One long prompt at once.
        dict(name="prompt_16k", op="prompt", hq=32, hkv=8, d=128, rows=_lens([16384]),
             ctx=_lens([0]), pad=0),
        # Log probabilities of given tokens.
        # The verify rows of one sequence (gamma 4): the drafted tokens and the bonus row.
        dict(name="logprobs_verify_5", op="logprobs", rows=5, vocab=151936, bf16=True, top=1,
             temperature=1.0, stride_pad=0, masked=0.0),
        # The verify rows of 48 sequences in 32 bits, an odd vocabulary, some tokens masked.
        dict(name="logprobs_masked_240", op="logprobs", rows=240, vocab=50257, bf16=False, top=5,
             temperature=0.7, stride_pad=0, masked=0.3),
        # Scoring a prompt with its alternatives.
        dict(name="logprobs_prompt_1000", op="logprobs", rows=1000, vocab=151936, bf16=True, top=20,
             temperature=1.0, stride_pad=0, masked=0.0),
    ]


def _lens(v):
    return ",".join(str(int(x)) for x in v)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "logprobs"])
    if op == "logprobs":
        rows, vocab = _log_int(rng, 1, 1000), _log_int(rng, 300, 151936)
        return dict(op=op, rows=rows, vocab=vocab, bf16=rng.random() < 0.5,
                    top=rng.choice([0, 1, 2, 5, 8, 20, 32]),
                    temperature=round(rng.uniform(0.5, 1.5), 3),
                    stride_pad=rng.choice([0, 0, 1, 7, 64]), masked=rng.choice([0.0, 0.0, 0.5, 0.98]))
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8] if d == 128 else [1, 2, 4, 5, 8, 16])
    hq = min(hq, 64 // hkv * hkv)
    pad = rng.choice([0, 0, 3])
    batch = _log_int(rng, 1, 12)
    if op == "rope":
        total = _log_int(rng, max(8, batch), 16384)
        rows = _split(rng, total, batch)
        ctx = [rng.choice([0, _log_int(rng, 1, 2000)]) for _ in rows]
        rot = rng.choice([d, d, d // 2, 32])
        return dict(op=op, hq=hq, hkv=hkv, d=d, rows=_lens(rows), ctx=_lens(ctx), rot=rot,
                    axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4, pad=pad)
    total = _log_int(rng, max(4, batch), 8192)
    rows = _split(rng, total, batch)
    ctx = [rng.choice([0, _log_int(rng, 1, 16000)]) for _ in rows]
    # the padded score matrix of the plain form, and with it the largest listed case, bounds a draw
    while len(rows) * max(rows) * max(n + c for n, c in zip(rows, ctx)) * hq > (1 << 32):
        rows, ctx = [max(1, n // 2) for n in rows], [c // 2 for c in ctx]
    return dict(op=op, hq=hq, hkv=hkv, d=d, rows=_lens(rows), ctx=_lens(ctx), pad=pad)


def _split(rng, total, batch):
    cut = sorted(rng.randrange(total + 1) for _ in range(batch - 1))
    rows = [b - a for a, b in zip([0] + cut, cut + [total])]
    return rows if max(rows) else [total] + rows[1:]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    if case["op"] == "logprobs":
        return _prepare_logprobs(case, gen)
    return _prepare_cache_case(case, gen)


def _prepare_cache_case(case, gen):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows, ctx = _ints(case["rows"]), _ints(case["ctx"])
    batch, used = len(rows), sum(rows)
    total = used + case["pad"]
    pages = [(c + n + PAGE - 1) // PAGE for c, n in zip(ctx, rows)]
    max_pages = max(max(pages), 1)
    num_pages = sum(pages) + 3
    s = {"case": case, "batch": batch, "total": total, "used": used, "max_pages": max_pages}
    # pages of the sequences lie shuffled in the pool; unused table entries point at page 0
    perm = torch.randperm(num_pages, generator=gen, device=DEV, dtype=torch.int64).cpu().numpy()
    table, at = np.zeros((batch, max_pages), dtype=np.int32), 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    row_start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    s["block_table"] = torch.from_numpy(table).to(DEV)
    s["row_start"] = torch.from_numpy(row_start).to(DEV)
    s["ctx_lens"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    shape = (num_pages, hkv, PAGE, d)
    s["k_cache"] = torch.randn(shape, generator=gen, device=DEV).to(BF16)
    s["v_cache"] = torch.randn(shape, generator=gen, device=DEV).to(BF16)
    # what a host scheduler knows of each packed row: its sequence and its cache position
    seq = np.repeat(np.arange(batch), rows)
    pos = np.concatenate([np.arange(n) + c for n, c in zip(rows, ctx)] + [np.zeros(0)])
    s["row_seq"] = torch.from_numpy(seq.astype(np.int64)).to(DEV)
    s["row_pos"] = torch.from_numpy(pos.astype(np.int64)).to(DEV)
    if case["op"] == "rope":
        s["qkv"] = torch.randn((total, (hq + 2 * hkv) * d), generator=gen, device=DEV).to(BF16)
        s["q_out"] = torch.randn((total, hq, d), generator=gen, device=DEV).to(BF16)
        half = case["rot"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).to(FP32).to(DEV)
        if case["axes"] > 1:
            # the image or video starts somewhere in a long document: time steps on slowly,
            # height and width run over a 34-wide grid
            t = pos.astype(np.int64)
            grid = [t // 680 + 100003, t // 34 % 20 + 100003, t % 34 + 100003][:case["axes"]]
            p = np.zeros((case["axes"], total), dtype=np.int32)
            p[:, :used] = np.stack(grid)
            s["positions"] = torch.from_numpy(p).to(DEV)
            s["pair_axis"] = (torch.arange(half, device=DEV) * case["axes"] // half).to(torch.int32)
        else:
            s["positions"] = s["pair_axis"] = None
    else:
        # a few keys lie along a direction that the queries share: heavy hitters
        u = torch.randn((d,), generator=gen, device=DEV)
        u = u / u.norm()
        heavy = torch.rand((num_pages, hkv, PAGE, 1), generator=gen, device=DEV) < 0.02
        s["k_cache"] = torch.where(heavy, (3 * u + 0.3 * s["k_cache"].float()).to(BF16), s["k_cache"])
        s["q"] = (torch.randn((total, hq, d), generator=gen, device=DEV) + 2 * u).to(BF16)
        s["out"] = torch.randn((total, hq, d), generator=gen, device=DEV).to(BF16)
        s["scale"] = 1.0 / math.sqrt(d)
        n_max, kv_max = max(rows), max_pages * PAGE
        s["n_max"], s["kv_max"] = n_max, kv_max
        s["row_slot"] = s["row_pos"] - s["ctx_lens"].long()[s["row_seq"]]
    return s


def _prepare_logprobs(case, gen):
    rows, vocab = case["rows"], case["vocab"]
    dtype = BF16 if case["bf16"] else FP32
    stride = vocab + case["stride_pad"]
    x = torch.randn((rows, stride), generator=gen, device=DEV) * 2.5
    # a handful of likely tokens a row
    hot = torch.randint(0, vocab, (rows, 6), generator=gen, device=DEV)
    x.scatter_add_(1, hot, torch.rand((rows, 6), generator=gen, device=DEV) * 12)
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device=DEV, dtype=torch.int32)
    likely = torch.rand((rows,), generator=gen, device=DEV) < 0.7
    tokens = torch.where(likely, hot[:, 0].to(torch.int32), tokens)
    if case["masked"] > 0:
        gone = torch.rand((rows, stride), generator=gen, device=DEV) < case["masked"]
        x.masked_fill_(gone, -math.inf)
        if rows > 3:
            x[3] = -math.inf          # a row whose mask leaves nothing
            tokens[2] = -1            # a padding row
    logits = x.to(dtype)
    top = case["top"]
    return {"case": case, "logits": logits, "tokens": tokens, "stride": stride,
            "inv_t": float(np.float32(1.0 / case["temperature"])),
            "logprob": torch.zeros((rows,), device=DEV), "entropy": torch.zeros((rows,), device=DEV),
            "rank": torch.zeros((rows,), dtype=torch.int32, device=DEV),
            "top_ids": torch.zeros((rows, top), dtype=torch.int32, device=DEV),
            "top_logprobs": torch.zeros((rows, top), device=DEV)}


# ------------------------------------------------------------------ passes
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "prompt": _own_prompt, "logprobs": _own_logprobs}[op](state)
    return {"rope": _plain_rope, "prompt": _plain_prompt, "logprobs": _plain_logprobs}[op](state)


def _kv(state):
    """The cache's descriptor, which a program makes once."""
    import self_speculative_sparse_paged_gb300 as vg
    if "kv" not in state:
        state["kv"] = vg.paged_kv(state["k_cache"], state["v_cache"], state["block_table"],
                                  state["case"]["hq"])
    return vg, state["kv"]


def _own_rope(s):
    c = s["case"]
    vg, kv = _kv(s)
    qkv, d = s["qkv"], c["d"]
    stride = qkv.stride(0)
    vg.vegas_rope_append(kv, qkv, stride, qkv[:, c["hq"] * d:], stride,
                         qkv[:, (c["hq"] + c["hkv"]) * d:], stride, s["q_out"], s["row_start"],
                         s["ctx_lens"], s["positions"], s["pair_axis"], c["axes"], s["inv_freq"],
                         c["rot"], c["interleaved"], 1.0, s["total"], s["batch"])
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _own_prompt(s):
    c = s["case"]
    vg, kv = _kv(s)
    if "workspace" not in s:
        n = vg.vegas_prompt_workspace_size(kv, s["total"], s["batch"])
        s["workspace"] = torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV)
    ws = s["workspace"]
    vg.vegas_prompt_attn(kv, s["q"], c["hq"] * c["d"], s["out"], s["row_start"], s["ctx_lens"],
                         s["total"], s["batch"], s["scale"], ws, ws.numel())
    return s["out"]


def _own_logprobs(s):
    import self_speculative_sparse_paged_gb300 as vg
    c, top = s["case"], s["case"]["top"]
    vg.vegas_token_logprobs(s["logits"], vg.VEGAS_BF16 if c["bf16"] else vg.VEGAS_FP32, s["stride"],
                            s["tokens"], c["rows"], c["vocab"], s["inv_t"], s["logprob"],
                            s["entropy"], s["rank"], top, s["top_ids"] if top else None,
                            s["top_logprobs"] if top else None)
    return {k: s[k] for k in ("logprob", "entropy", "rank", "top_ids", "top_logprobs")}


def _plain_rope(s):
    c = s["case"]
    hq, hkv, d, rot, used = c["hq"], c["hkv"], c["d"], c["rot"], s["used"]
    x = s["qkv"][:used].view(used, hq + 2 * hkv, d)
    if s["positions"] is None:
        p = s["row_pos"][:, None].double()
    else:
        p = s["positions"][:, :used].t()[:, s["pair_axis"].long()].double()
    angle = p * s["inv_freq"].double()
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
    page = s["block_table"].long()[s["row_seq"], s["row_pos"] // PAGE]
    slot = s["row_pos"] % PAGE
    s["k_cache"][page, :, slot] = y[:, hq:]
    s["v_cache"][page, :, slot] = x[:, hq + hkv:]
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _plain_prompt(s):
    c = s["case"]
    hq, hkv, d, used, batch, n, kvn = c["hq"], c["hkv"], c["d"], s["used"], s["batch"], s["n_max"], s["kv_max"]
    g = hq // hkv
    table = s["block_table"].long()
    k = s["k_cache"][table].permute(0, 2, 1, 3, 4).reshape(batch, hkv, kvn, d).float()
    v = s["v_cache"][table].permute(0, 2, 1, 3, 4).reshape(batch, hkv, kvn, d).float()
    q = torch.zeros((batch, n, hq, d), device=DEV)
    q[s["row_seq"], s["row_slot"]] = s["q"][:used].float()
    q = q.view(batch, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, g * n, d)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    last = s["ctx_lens"].long()[:, None] + torch.arange(n, device=DEV)
    ahead = torch.arange(kvn, device=DEV) > last[:, None, None, :, None]
    x = x.view(batch, hkv, g, n, kvn).masked_fill_(ahead, -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    o = torch.matmul(x.view(batch, hkv, g * n, kvn), v)
    o = o.view(batch, hkv, g, n, d).permute(0, 3, 1, 2, 4).reshape(batch, n, hq, d)
    s["out"][:used] = o[s["row_seq"], s["row_slot"]].to(BF16)
    return s["out"]


def _plain_logprobs(s):
    c = s["case"]
    vocab, top = c["vocab"], c["top"]
    x = s["logits"][:, :vocab].float()
    m = x.amax(-1, keepdim=True)
    some = m > -math.inf                       # rows whose mask leaves something
    t = torch.where(x > -math.inf, (x - m) * s["inv_t"], -math.inf)
    e = t.exp()
    z = e.sum(-1, keepdim=True)
    log_z = torch.where(some, z.log(), 0.0)
    entropy = log_z - torch.where(e > 0, e * t, 0.0).sum(-1, keepdim=True) / torch.where(some, z, 1.0)
    tok = s["tokens"].long()[:, None]
    given = tok >= 0
    tok = tok.clamp_min(0)
    x_tok = x.gather(1, tok)
    logprob = torch.where(given, t.gather(1, tok) - log_z, 0.0)
    before = torch.arange(vocab, device=DEV)[None, :] < tok
    rank = (x > x_tok).sum(-1, keepdim=True) + ((x == x_tok) & before).sum(-1, keepdim=True)
    rank = torch.where(given, rank, -1)
    got, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    got, ids = got[:, :top], ids[:, :top]
    finite = got > -math.inf
    top_lp = torch.where(finite, (got - m) * s["inv_t"] - log_z, -math.inf)
    return {"logprob": logprob[:, 0], "entropy": entropy[:, 0], "rank": rank[:, 0].to(torch.int32),
            "top_ids": torch.where(finite, ids, -1).to(torch.int32), "top_logprobs": top_lp}


# ------------------------------------------------------------------ what a pass needs
def work(case):
    if case["op"] == "logprobs":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2 if case["bf16"] else 4) + case["rows"] * (16 + 8 * case["top"]),
                "flops": 6 * n}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows, ctx = _ints(case["rows"]), _ints(case["ctx"])
    used = sum(rows)
    if case["op"] == "rope":
        per_row = 2 * (hq + 2 * hkv) * d * 2
        return {"bytes": used * per_row + 4 * case["rot"] // 2,
                "flops": used * (hq + hkv) * case["rot"] * 3}
    kv = sum(c + n for c, n in zip(ctx, rows) if n)
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, rows))
    return {"bytes": 2 * used * hq * d * 2 + 2 * kv * hkv * d * 2, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "prompt": _exact_prompt, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    hq, hkv, d, rot = c["hq"], c["hkv"], c["d"], c["rot"]
    rows, ctx = _ints(c["rows"]), _ints(c["ctx"])
    q, k, v = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
    src, at, half = s["qkv"].double(), 0, rot // 2
    for b, n in enumerate(rows):
        if n == 0:
            continue
        x = src[at:at + n].view(n, hq + 2 * hkv, d)
        if s["positions"] is None:
            p = torch.arange(ctx[b], ctx[b] + n, device=DEV, dtype=torch.float64)[:, None].expand(n, half)
        else:
            p = torch.stack([s["positions"][s["pair_axis"][j].item(), at:at + n] for j in range(half)], 1).double()
        turn = torch.polar(torch.ones_like(p), p * s["inv_freq"].double())[:, None, :]
        y = x[:, :hq + hkv].clone()
        first = slice(0, rot, 2) if c["interleaved"] else slice(0, half)
        second = slice(1, rot, 2) if c["interleaved"] else slice(half, rot)
        z = torch.complex(x[:, :hq + hkv, first].contiguous(), x[:, :hq + hkv, second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        q[at:at + n] = y[:, :hq]
        pos = torch.arange(ctx[b], ctx[b] + n, device=DEV)
        page = s["block_table"][b].long()[pos // PAGE]
        k[page, :, pos % PAGE] = y[:, hq:]
        v[page, :, pos % PAGE] = x[:, hq + hkv:]
        at += n
    return {"q": q, "k": k, "v": v}


def _exact_prompt(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    rows, ctx = _ints(c["rows"]), _ints(c["ctx"])
    out, at = s["out"].double(), 0
    for b, n in enumerate(rows):
        total = ctx[b] + n
        pages = s["block_table"][b, :(total + PAGE - 1) // PAGE].long()
        for h in range(hq if n else 0):
            k = s["k_cache"][pages, h // (hq // hkv)].reshape(-1, d)[:total].double()
            v = s["v_cache"][pages, h // (hq // hkv)].reshape(-1, d)[:total].double()
            for lo in range(0, n, 4096):
                hi = min(n, lo + 4096)
                seen = ctx[b] + hi
                x = s["q"][at + lo:at + hi, h].double() @ k[:seen].t() / math.sqrt(d)
                x.masked_fill_(torch.ones_like(x, dtype=torch.bool).triu_(ctx[b] + lo + 1), -math.inf)
                out[at + lo:at + hi, h] = torch.softmax(x, -1) @ v[:seen]
        at += n
    return out


def _exact_logprobs(s):
    c = s["case"]
    lp, ent, tops = [], [], []
    for r in range(0, c["rows"], 64):
        x = s["logits"][r:r + 64, :c["vocab"]].double() * s["inv_t"]
        tok = s["tokens"][r:r + 64].long()
        y = x - torch.logsumexp(x, -1, keepdim=True)
        y = torch.where(x.amax(-1, keepdim=True) > -math.inf, y, -math.inf)
        got = y.gather(1, tok.clamp_min(0)[:, None])[:, 0]
        lp.append(torch.where(tok >= 0, got, 0.0))
        ent.append(-torch.where(y > -math.inf, y.exp() * y, 0.0).sum(-1))
        k = min(c["top"], c["vocab"])
        tops.append(torch.topk(y, k, dim=-1).values if k else y[:, :0])
    return {"logprob": torch.cat(lp), "entropy": torch.cat(ent), "rank": None, "top_ids": None,
            "top_logprobs": torch.cat(tops)}
