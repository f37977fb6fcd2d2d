"""Plain 64-bit NumPy definitions of the sequence calls: the quantised paged
cache (bytes included) and attention over sequences of different lengths.

Nothing here is shared with the CUDA path.  Rows are [..., d]; the formats are
named "e4m3", "int8" and "int4".
"""
import numpy as np

LEAST = 2.0 ** -96  # rows whose largest magnitude is below this are stored as zeros
TOP = {"e4m3": 448.0, "int8": 127.0, "int4": 3136.0}


def e4m3_grid():
    """Every finite e4m3 value by its code 0..255 (NaN codes hold NaN)."""
    v = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (e == 15 and m == 7) else (-x if s else x)
    return v


_GRID = e4m3_grid()
_POS = _GRID[:127]  # codes 0..126: 0 .. 448, ascending


def e4m3_codes(x):
    """Nearest code, ties to the even mantissa, saturating; the sign of zero is kept."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POS[hi] - a, a - _POS[lo]
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def e4m3_values(codes):
    return _GRID[codes]


def quantise(fmt, x):
    """Rows as (code bytes [..., row], scale records [..., 4 or 8])."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    amax = np.abs(x).max(-1, keepdims=True)
    amax = np.where(amax < LEAST, 0.0, amax)
    div = np.where(amax > 0, amax, np.inf)
    scale = (amax.astype(np.float32) / np.float32(TOP[fmt])).astype("<f4")
    rec = np.ascontiguousarray(scale).view(np.uint8)
    if fmt == "int4":
        groups = x.reshape(*x.shape[:-1], d // 32, 32)
        g = e4m3_codes(448.0 * np.abs(groups).max(-1) / div)
        over = np.where(amax > 0, amax, 1.0)[..., None] * e4m3_values(g)[..., None]
        n = 3136.0 * groups / np.where(over > 0, over, np.inf)
        n = (np.clip(np.rint(n), -7, 7) + 8).astype(np.uint8).reshape(x.shape)
        tail = np.zeros((*g.shape[:-1], 4), np.uint8)
        tail[..., :d // 32] = g
        return n[..., 0::2] | (n[..., 1::2] << 4), np.concatenate([rec, tail], -1)
    y = TOP[fmt] * x / div
    if fmt == "int8":
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8), rec
    y = np.where(np.isfinite(div), y, 0.0)
    return e4m3_codes(y), rec


def dequantise(fmt, codes, rec):
    """The fp32 values that bytes stand for: code * scale, or n * (s * g), each product rounded to fp32."""
    s = np.ascontiguousarray(rec[..., :4]).view("<f4")
    if fmt == "int4":
        n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1]).astype(np.float32) - np.float32(8)
        g = e4m3_values(rec[..., 4:4 + n.shape[-1] // 32]).astype(np.float32)
        return (n.reshape(*n.shape[:-1], n.shape[-1] // 32, 32) * (s * g)[..., None]).reshape(n.shape)
    v = codes.view(np.int8).astype(np.float32) if fmt == "int8" else e4m3_values(codes).astype(np.float32)
    return v * s


class Cache:
    """The bytes of one layer's cache: sections [pages, H_kv, page_tokens, row] on multiples of 256."""

    def __init__(self, fmt, H_kv, d, page, pages, fill=0):
        self.fmt, self.H_kv, self.d, self.page, self.pages = fmt, H_kv, d, page, pages
        row, rec = (d // 2, 8) if fmt == "int4" else (d, 4)
        rows, at = pages * H_kv * page, [0]
        for size in (row, row, rec, rec):
            at.append(at[-1] + (rows * size + 255) // 256 * 256)
        self.buf = np.full(at[-1], fill, np.uint8)
        self.parts = [self.buf[a:a + rows * size].reshape(pages, H_kv, page, size)
                      for a, size in zip(at, (row, row, rec, rec))]

    def put(self, table, pos, k, v):
        """Rows k, v [n, H_kv, d] at positions pos of the sequence with this table row."""
        for i, p in enumerate(pos):
            page, place = table[p // self.page], p % self.page
            for which, x in ((0, k), (1, v)):
                codes, rec = quantise(self.fmt, x[i])
                self.parts[which][page, :, place] = codes
                self.parts[2 + which][page, :, place] = rec

    def get(self, table, pos):
        """(k, v) fp32 [n, H_kv, d] at positions pos."""
        pos = np.asarray(pos, np.int64)
        page, place = np.asarray(table)[pos // self.page], pos % self.page
        return tuple(dequantise(self.fmt, self.parts[w][page, :, place], self.parts[2 + w][page, :, place])
                     for w in (0, 1))


def attention(q, k, v, causal, scale=None, keep=None):
    """One sequence: q [n, H, d] over k, v [len, H_kv, d] in 64 bits.

    Returns o [n, H, d], lse [n, H], and per (query, head) what error bounds
    need: sum of weight * |v| [n, H, d] and the largest sum |q_i k_i| * scale.
    keep [len]: keys taken into account (None: all)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, H, d = q.shape
    length, H_kv = k.shape[:2]
    G = H // H_kv
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    o, lse = np.zeros((n, H, d)), np.full((n, H), -np.inf)
    absv, size = np.zeros((n, H, d)), np.zeros((n, H))
    if length == 0 or n == 0:
        return o, lse, absv, size
    seen = np.ones((n, length), bool)
    if causal:
        seen = np.arange(length)[None, :] <= np.arange(n)[:, None] + (length - n)
    if keep is not None:
        seen = seen & np.asarray(keep, bool)[None, :]
    for h in range(H):
        s = np.where(seen, scale * (q[:, h] @ k[:, h // G].T), -np.inf)
        m = s.max(-1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        p = np.exp(s - m)
        total = p.sum(-1, keepdims=True)
        some = total[:, 0] > 0
        w = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
        o[:, h] = w @ v[:, h // G]
        absv[:, h] = w @ np.abs(v[:, h // G])
        lse[some, h] = (m + np.log(np.where(total > 0, total, 1.0)))[some, 0]
        size[:, h] = np.where(seen, scale * (np.abs(q[:, h]) @ np.abs(k[:, h // G]).T), 0.0).max(-1)
    return o, lse, absv, size
