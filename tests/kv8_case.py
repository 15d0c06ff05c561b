"""The 8-bit cache in 64 bits, for its tests: the code table, the rounding to codes, the append's
scales and attention over decoded blocks.  Shares no code with the library."""
import numpy as np

PAGE = 16


def _table():
    v = np.empty(256)
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = (1 + f / 8) * 2.0 ** (e - 7) if e else f / 8 * 2.0 ** -6
        v[c] = np.nan if c & 127 == 127 else x
        if c > 127:
            v[c] = -v[c]
    return v


VALUE = _table()                       # of each of the 256 codes
_POS = VALUE[:127]                     # 0 .. 448, ascending


def encode(x):
    """Codes of x (float64): nearest, ties to the even code, saturating at 448, NaN to 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_POS, np.where(np.isnan(a), 0.0, a))      # first code >= a
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POS[hi] - a, a - _POS[lo]
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    c = np.where(up, hi, lo).astype(np.uint8)
    c = np.where(np.isnan(x), np.uint8(127), c | np.where(np.signbit(x), 128, 0).astype(np.uint8))
    return c.astype(np.uint8)


def exponent(amax):
    """Least e in [-60, 60] with amax <= 448 * 2^e (60 where none is enough)."""
    for e in range(-60, 61):
        if amax <= 448 * 2.0 ** e:
            return e
    return 60


def decode(codes, scale):
    """Blocks (..., 16, d) of codes with scale bytes (...) as float64."""
    e = np.clip(scale.astype(np.int64) - 127, -60, 60)
    return VALUE[codes] * (2.0 ** e)[..., None, None]


def append(codes, scale, y, page_of, ctx):
    """One sequence's rows y (n, hkv, d) at positions ctx.. into codes (pages, hkv, 16, d) and
    scale (pages, hkv), in place; page_of[j] is the pool page of the sequence's j-th page."""
    n, hkv, _ = y.shape
    for j in range(ctx // PAGE, (ctx + n - 1) // PAGE + 1 if n else 0):
        lo, hi = max(0, j * PAGE - ctx), min(n, (j + 1) * PAGE - ctx)
        held = max(0, ctx - j * PAGE)
        pg = page_of[j]
        for g in range(hkv):
            new = y[lo:hi, g]
            mag = np.abs(new[np.isfinite(new)])
            e = exponent(mag.max() if mag.size else 0.0)
            old = int(np.clip(int(scale[pg, g]) - 127, -60, 60))
            if held and old >= e:
                e = old
            elif held:
                codes[pg, g, :held] = encode(VALUE[codes[pg, g, :held]] * 2.0 ** (old - e))
            at = ctx + lo - j * PAGE
            codes[pg, g, at:at + hi - lo] = encode(new * 2.0 ** -e)
            scale[pg, g] = e + 127


def gather(codes, scale, pages, g, n):
    """The first n positions of head g over `pages` as (n, d) float64."""
    return decode(codes[pages, g], scale[pages, g]).reshape(-1, codes.shape[-1])[:n]


def attend(q, k, v, scale):
    """(rows, d) queries over (n, d): output, its weighted magnitudes sum p |v|, logits."""
    x = q @ k.T * scale
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    return p @ v, p @ np.abs(v), x


def random_cache(rng, num_pages, hkv, d, spread=6, wild=False):
    """Codes and scale bytes: random values quantised block by block, exponents spread over
    `spread` binades; wild: any finite code."""
    if wild:
        codes = rng.integers(0, 256, (num_pages, hkv, PAGE, d), dtype=np.uint8)
        codes = np.where((codes & 127) == 127, codes ^ 1, codes)
    else:
        codes = encode(rng.standard_normal((num_pages, hkv, PAGE, d)) * 100)
    scale = (127 - 7 - rng.integers(0, spread + 1, (num_pages, hkv))).astype(np.uint8)
    return codes, scale
