"""The serving operators around a quantised, paged KV cache, as measured work.

Four operators, each with a plain form in elementary torch operations and the
library call that does the same work:

  write   new keys and values quantised into the pages of a cache (fp8 e4m3,
          int8 or int4), then the written rows read back
  read    whole sequences of such a cache read back in 16 bits
  attn    attention of the newest tokens of each sequence (one, or a few) over
          its cache, quantised as it lies in the pages
  prompt  attention of whole prompts, packed sequences of different lengths,
          over 16-bit keys and values (causal, or every key)

The cache of one layer is one buffer of bytes: the codes of K, the codes of V,
the scales of K, the scales of V, each section [pages, Hkv, page, row] and
starting on a multiple of 256 bytes.  A row holds one token of one head:
  e4m3, int8  d codes; scale: one float, amax / 448 or amax / 127
  int4        d / 2 bytes, channel 2j in the low nibble of byte j, nibble = value + 8;
              scale record of 8 bytes: one float s = amax / 3136, then one e4m3
              factor g per 32 channels (2 or 4 of them, the rest zero); value = n s g
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
FMT = ("e4m3", "int8", "int4")


# ---------------------------------------------------------------------------------------- cases
def listed():
    """Cases in the shapes of this framework's layers (12 and 40 heads of 128, 1560 tokens a
    frame, chunks of 3 frames) and in generic ones with grouped heads."""
    return [
        # one decoding step of a batch: every sequence adds one token (latency)
        case("write", "write_step_b64_int8", B=64, new=(1, 1), past=(100, 4000), H=32, Hkv=8, d=128, fmt="int8", page=16),
        # a chunk of three frames of the 12-head layer goes into a 4-bit history
        case("write", "write_chunk_4680_int4", B=1, new=(4680, 4680), past=(1560, 1560), H=12, Hkv=12, d=128, fmt="int4", page=64),
        # 15 frames of history of the 12-head layer are read back for a recalibration
        case("read", "read_history_23400_int4", B=1, new=(23400, 23400), H=12, Hkv=12, d=128, fmt="int4", page=64),
        # prefixes of a batch of ragged prompts are read back for their next chunk
        case("read", "read_ragged_b37_e4m3_d64", B=37, new=(1, 3000), H=16, Hkv=2, d=64, fmt="e4m3", page=32, dtype="fp16"),
        # one user, a short context (latency)
        case("attn", "attn_b1_999_int8", B=1, new=(1, 1), past=(998, 998), H=32, Hkv=8, d=128, fmt="int8", page=16),
        # an ordinary batch of users at different lengths
        case("attn", "attn_b48_ragged_e4m3", B=48, new=(1, 1), past=(200, 16000), H=32, Hkv=8, d=128, fmt="e4m3", page=32),
        # one token over the longest history of the 40-head layer, 66 frames in 4 bits
        case("attn", "attn_b1_102960_h40_int4", B=1, new=(1, 1), past=(102959, 102959), H=40, Hkv=40, d=128, fmt="int4", page=256),
        # several drafted or pending tokens a sequence, small heads
        case("attn", "attn_b16_new7_int8_d64", B=16, new=(2, 7), past=(500, 9000), H=16, Hkv=2, d=64, fmt="int8", page=16, dtype="fp16"),
        # many short prompts packed into one call
        case("prompt", "prompt_b24_short_d64", B=24, new=(1, 300), H=16, Hkv=2, d=64, dtype="fp16"),
        # a batch of ragged prompts with grouped heads
        case("prompt", "prompt_b6_ragged_gqa", B=6, new=(400, 4000), H=32, Hkv=8, d=128),
        # one long prompt
        case("prompt", "prompt_8192_gqa", B=1, new=(8192, 8192), H=32, Hkv=8, d=128),
        # a chunk of the 12-head layer over its whole context, every key in sight
        case("prompt", "prompt_chunk_4680_over_32760", B=1, new=(4680, 4680), past=(28080, 28080), H=12, Hkv=12, d=128, causal=False),
    ]


def case(op, name, B, new, H, Hkv, d, past=(0, 0), fmt="", page=0, dtype="bf16", causal=True, mix=1, pad=0, empty=0):
    """new, past: ranges of the tokens that a sequence adds and of those before them; mix seeds the
    lengths; pad: rows behind the last sequence; empty: sequences without a token."""
    c = dict(op=op, B=B, new_lo=new[0], new_hi=new[1], past_lo=past[0], past_hi=past[1], H=H, Hkv=Hkv, d=d, fmt=fmt,
             page=page, dtype=dtype, causal=causal, mix=mix, pad=pad, empty=empty)
    if name:
        c["name"] = name
    return c


def draw(rng):
    lg = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    span = lambda lo, hi: tuple(sorted((lg(lo, hi), lg(lo, hi))))  # noqa: E731
    op = rng.choice(["write", "read", "attn", "prompt"])
    Hkv, d = rng.choice([1, 2, 3, 5, 8, 12]), rng.choice([64, 128])
    H = Hkv * rng.choice([1, 2, 3, 4, 7, 8, 16] if Hkv <= 3 else [1, 2, 4, 5])
    fmt, page, dtype = rng.choice(FMT), rng.choice([16, 32, 64, 128, 256]), rng.choice(["bf16", "fp16"])
    mix, pad, empty = rng.randrange(1 << 30), rng.choice([0, 0, 1, 37]), rng.choice([0, 0, 1, 2])
    both = dict(H=H, Hkv=Hkv, d=d, dtype=dtype, mix=mix, pad=pad, empty=empty)
    if op == "write":
        B = lg(1, 128)
        return case(op, "", B=B, new=rng.choice([(1, 1), span(1, 20000 // B)]), past=span(1, 3000), fmt=fmt, page=page, **both)
    if op == "read":
        B = lg(1, 64)
        return case(op, "", B=B, new=span(1, max(2, 60000 // B)), fmt=fmt, page=page, **both)
    if op == "attn":
        B = lg(1, 128)
        return case(op, "", B=B, new=rng.choice([(1, 1), (1, 1), span(1, 16)]), past=span(1, min(65000, 1500000 // (B * Hkv))),
                    fmt=fmt, page=page, **both)
    causal = rng.random() < 0.75
    B = lg(1, 48)
    top = max(8, min(8192, int(math.sqrt(1.2e9 / (B * H)))))  # the plain form holds B * H * new * keys scores
    new = span(1, top)
    past = rng.choice([(0, 0), (0, 0), span(1, max(2, top - new[1] + 1)), (-3, -1)])
    return case("prompt", "", B=B, new=new, past=past, causal=causal, **both)


def lengths(c):
    """New and past tokens of each sequence (a negative past leaves fewer keys than queries)."""
    r = random.Random(c["mix"])

    def one(lo, hi):
        return r.randint(lo, hi) if lo < 1 or hi < 10 * lo else int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))

    new = [one(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    past = [one(c["past_lo"], c["past_hi"]) for _ in range(c["B"])]
    for i in range(min(c["empty"], c["B"] - 1)):  # from the second sequence on
        new[1 + i] = 0
        past[1 + i] = 0
    return new, [max(p, -n) for n, p in zip(new, past)]


def work(c):
    new, past = lengths(c)
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    n, total = sum(new), sum(new) + sum(past)
    row = record(c)[0] + record(c)[1] if c["fmt"] else 0
    rows16 = 2 * Hkv * d * 2  # K and V of one token in 16 bits
    if c["op"] == "write":  # read, quantised and written, read again, written back
        return {"bytes": n * (2 * rows16 + 2 * 2 * Hkv * row), "flops": n * 2 * Hkv * d * 4}
    if c["op"] == "read":
        return {"bytes": n * (rows16 + 2 * Hkv * row), "flops": n * 2 * Hkv * d}
    pairs = sum(sum(max(0, min(k, k - q + i + 1)) for i in range(q)) if c["causal"] else q * k
                for q, k in ((a, a + b) for a, b in zip(new, past)))
    io = n * H * (2 * 2 * d + 4)  # queries, outputs, log-sum-exp
    keys = total * (2 * Hkv * row if c["op"] == "attn" else rows16)
    return {"bytes": io + keys, "flops": 4 * d * H * pairs}


# ------------------------------------------------------------------------------- the cache's bytes
def record(c):
    """Bytes of a row's codes and of its scale record."""
    return (c["d"] // 2, 8) if c["fmt"] == "int4" else (c["d"], 4)


def sections(c, pages):
    """Where the codes of K and V and the scales of K and V start, and the buffer's size."""
    rows, (code, scale) = pages * c["Hkv"] * c["page"], record(c)
    at = [0]
    for size in (code, code, scale, scale):
        at.append(at[-1] + (rows * size + 255) // 256 * 256)
    return at


def views(c, kvq, pages):
    """[codes of K, of V, scales of K, of V] as byte tensors [pages, Hkv, page, row]."""
    at, rows = sections(c, pages), pages * c["Hkv"] * c["page"]
    return [kvq[a:a + rows * size].view(pages, c["Hkv"], c["page"], size)
            for a, size in zip(at, record(c)[:1] * 2 + record(c)[1:] * 2)]


LEAST = 2.0 ** -96  # rows whose largest magnitude is below this are stored as zeros


def quantise(fmt, x):
    """Rows x [..., d] as (codes, scale record), both bytes."""
    x = x.float()
    amax = x.abs().amax(-1, keepdim=True)
    amax = torch.where(amax >= LEAST, amax, torch.zeros_like(amax))
    safe = torch.where(amax > 0, amax, torch.ones_like(amax))
    # Every quotient below has exact operands (powers of two keep them in range), so that its one
    # rounding cannot move a value onto or over a border between two codes.
    if fmt == "int4":
        groups = x.view(*x.shape[:-1], -1, 32)
        g8 = ((groups.abs().amax(-1) * 0.875) / safe * 512.0).to(torch.float8_e4m3fn)  # 448 amax of the group / amax
        step = safe * (g8.float() / 512.0)  # amax g / 512
        over = torch.where(step > 0, step, torch.ones_like(step))[..., None]
        n = (groups * (49.0 / 64.0)) / over * 8.0  # 3136 x / (amax g)
        n = torch.where((step > 0)[..., None], n, torch.zeros_like(n))
        n = (torch.round(n).clamp(-7, 7) + 8).to(torch.uint8).view(x.shape)
        n = torch.where(amax > 0, n, torch.full_like(n, 8))
        g8 = torch.where(amax > 0, g8.view(torch.uint8), torch.zeros_like(g8.view(torch.uint8)))
        codes = n[..., 0::2] | (n[..., 1::2] << 4)
        tail = torch.zeros(*g8.shape[:-1], 4, dtype=torch.uint8, device=x.device)
        tail[..., :g8.shape[-1]] = g8
        return codes, torch.cat([(amax / 3136.0).view(torch.uint8), tail], -1)
    top, unit = (448.0, 512.0) if fmt == "e4m3" else (127.0, 128.0)
    y = (x * (top / unit)) / safe * unit
    y = torch.where(amax > 0, y, torch.zeros_like(y))
    codes = y.clamp(-448, 448).to(torch.float8_e4m3fn) if fmt == "e4m3" else torch.round(y).clamp(-127, 127).to(torch.int8)
    return codes.view(torch.uint8), (amax / top).view(torch.uint8)


def dequantise(fmt, codes, scale):
    """The fp32 values that rows of bytes stand for."""
    s = scale[..., :4].contiguous().view(torch.float32)
    if fmt == "int4":
        n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8.0
        g = scale[..., 4:4 + n.shape[-1] // 32].contiguous().view(torch.float8_e4m3fn).float()
        return (n.view(*n.shape[:-1], -1, 32) * (s * g)[..., None]).view(n.shape)
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float() * s


# ---------------------------------------------------------------------------------------- inputs
def keys_values(gen, n, heads, d, dtype):
    """Rows as a projection leaves them: a few channels of each head are much larger than the rest."""
    x = torch.randn(n, heads, d, generator=gen, device="cuda")
    return x.mul_(torch.where(torch.arange(d, device="cuda") % 16 == 5, 4.0, 1.0)).to(dtype)


def starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    new, past = lengths(c)
    total = [a + b for a, b in zip(new, past)]
    B, H, Hkv, d, dtype = c["B"], c["H"], c["Hkv"], c["d"], DT[c["dtype"]]
    n, rows = sum(new), sum(new) + c["pad"]
    st = {"case": c, "n": n, "max_new": max(new), "max_len": max(total), "cu_new": ints(starts(new)), "lens": ints(total)}
    empty = lambda *shape, t=dtype: torch.zeros(shape, dtype=t, device="cuda")  # noqa: E731
    if c["op"] == "prompt":
        st["cu_k"] = ints(starts(total))
        st["q"] = torch.randn(rows, H, d, generator=gen, device="cuda").to(dtype)
        keys = sum(total) + c["pad"]
        st["k"] = keys_values(gen, keys, Hkv, d, dtype)
        st["v"] = torch.randn(keys, Hkv, d, generator=gen, device="cuda").to(dtype)
        if c["past_lo"] == c["past_hi"] == 0:  # one projection's output holds all three
            fused = torch.cat([st["q"], st["k"], st["v"]], 1)
            st["q"], st["k"], st["v"] = fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:]
    else:
        page = c["page"]
        need = [-(-t // page) for t in total]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        table = torch.full((B, max(need) + 1), -1, dtype=torch.int32, device="cuda")
        for b, at in enumerate(starts(need)[:-1]):
            table[b, :need[b]] = order[at:at + need[b]]
        kvq = torch.zeros(sections(c, pages)[-1], dtype=torch.uint8, device="cuda")
        st |= {"pages": pages, "table": table, "kvq": kvq, "begin": ints(past)}
        st["k_scale"], st["v_scale"] = (x[..., :4].view(torch.float32) if c["fmt"] != "int4" else x.view(torch.float32)[..., :1]
                                        for x in views(c, kvq, pages)[2:])
        if c["op"] == "write":
            fused = torch.cat([torch.randn(rows, H, d, generator=gen, device="cuda").to(dtype),
                               keys_values(gen, rows, 2 * Hkv, d, dtype)], 1)
            st["k"], st["v"] = fused[:, H:H + Hkv], fused[:, H + Hkv:]
        else:  # the cache holds every token already
            cu = ints(starts(total))
            for x, at in ((keys_values(gen, sum(total), Hkv, d, dtype), 0),
                          (torch.randn(sum(total), Hkv, d, generator=gen, device="cuda").to(dtype), 1)):
                store(c, st, cu, ints([0] * B), sum(total), x, at)
        if c["op"] == "attn":
            st["q"] = torch.randn(rows, H, d, generator=gen, device="cuda").to(dtype)
        else:
            st["k_back"], st["v_back"] = empty(rows, Hkv, d), empty(rows, Hkv, d)
    if c["op"] in ("attn", "prompt"):
        st["o"], st["lse"] = empty(rows, H, d), empty(rows, H, t=torch.float32)
    if own:  # the descriptors and the workspace that a program keeps beside its cache
        import kv_cache_compression_two_b200 as ispa
        code = {"bf16": ispa.ISPA_BF16, "fp16": ispa.ISPA_F16}[c["dtype"]]
        if c["fmt"]:
            fmt = {"e4m3": ispa.ISPA_KVQ_E4M3, "int8": ispa.ISPA_KVQ_INT8, "int4": ispa.ISPA_KVQ_INT4}[c["fmt"]]
            st["cache"] = ispa.kvq_desc(Hkv, d, c["page"], st["pages"], fmt)
        if c["op"] in ("attn", "prompt"):
            st["attn"] = ispa.attn_seq_desc(B, H, Hkv, d, code, code, causal=c["causal"])
            size = ispa.ispa_attn_kvq_workspace_bytes(st["attn"], st["cache"]) if c["op"] == "attn" else ispa.ispa_attn_prompt_workspace_bytes(st["attn"])
            st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------------ one pass
def run(st):
    c = st["case"]
    if own:
        import kv_cache_compression_two_b200 as ispa
        if c["op"] == "write":
            ispa.ispa_kvq_write(st["cache"], st["k"], st["v"], st["table"], st["lens"], st["cu_new"], st["kvq"])
        if c["op"] in ("write", "read"):
            ispa.ispa_kvq_read(st["cache"], st["kvq"], st["table"], st["cu_new"], st["k_back"], st["v_back"],
                               seq_begin=st["begin"])
        if c["op"] == "attn":
            ispa.ispa_attn_kvq(st["attn"], st["cache"], st["q"], st["kvq"], st["table"], st["lens"], st["cu_new"],
                               st["o"], st["lse"], workspace=st["ws"])
        if c["op"] == "prompt":
            ispa.ispa_attn_prompt(st["attn"], st["q"], st["k"], st["v"], st["cu_new"], st["cu_k"], st["o"], st["lse"],
                                  workspace=st["ws"])
    else:
        if c["op"] == "write":
            store(c, st, st["cu_new"], st["begin"], st["n"], st["k"], 0)
            store(c, st, st["cu_new"], st["begin"], st["n"], st["v"], 1)
        if c["op"] in ("write", "read"):
            load(c, st, 0, st["k_back"])
            load(c, st, 1, st["v_back"])
        if c["op"] in ("attn", "prompt"):
            attention(c, st)
    if c["op"] == "write":
        return {"k": st["k_back"], "v": st["v_back"], "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    return {"k": st["k_back"], "v": st["v_back"]} if c["op"] == "read" else {"o": st["o"], "lse": st["lse"]}


def places(c, st, cu, begin, n):
    """Page and place in it of each of n packed tokens."""
    t = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    pos = begin.long()[b] + t - cu.long()[b]
    return st["table"].long()[b, pos // c["page"]], pos % c["page"]


def store(c, st, cu, begin, n, x, which):
    page, place = places(c, st, cu, begin, n)
    parts = views(c, st["kvq"], st["pages"])
    codes, scale = quantise(c["fmt"], x[:n])
    parts[which][page, :, place] = codes
    parts[2 + which][page, :, place] = scale


def load(c, st, which, out):
    page, place = places(c, st, st["cu_new"], st["begin"], st["n"])
    parts = views(c, st["kvq"], st["pages"])
    out[:st["n"]] = dequantise(c["fmt"], parts[which][page, :, place], parts[2 + which][page, :, place]).to(out.dtype)


def attention(c, st):
    """Padded to the longest sequence: queries [B, Hkv, group * new, d], keys [B, Hkv, len, d]."""
    B, H, Hkv, d, n = c["B"], c["H"], c["Hkv"], c["d"], st["n"]
    mq, mk, G = st["max_new"], max(1, st["max_len"]), H // Hkv
    cu, lens = st["cu_new"].long(), st["lens"].long()
    news = cu[1:] - cu[:-1]
    i, j = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    q = st["q"][(cu[:-1, None] + i).clamp_(max=max(0, n - 1))].float()
    if c["op"] == "prompt":
        at = (st["cu_k"].long()[:-1, None] + j).clamp_(max=max(0, st["k"].shape[0] - 1))
        k, v = st["k"][at].float(), st["v"][at].float()
    else:
        parts = views(c, st["kvq"], st["pages"])
        page, place = st["table"].long()[:, j // c["page"]].clamp_(min=0), j % c["page"]
        k, v = (dequantise(c["fmt"], parts[x][page, :, place], parts[2 + x][page, :, place]) for x in (0, 1))
    q = q.view(B, mq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * mq, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(d)).view(B, Hkv, G, mq, mk)
    seen = (j < lens[:, None])[:, None, :].expand(B, mq, mk)
    if c["causal"]:
        seen = seen & (j <= (i + (lens - news)[:, None])[:, :, None])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * mq, mk), v.transpose(1, 2)).view(B, Hkv, G, mq, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + total.log()).squeeze(-1)
    b = torch.searchsorted(cu[1:], torch.arange(n, device="cuda"), right=True)
    t = torch.arange(n, device="cuda") - cu[b]
    st["o"][:n] = o[b, :, :, t].reshape(n, H, d).to(st["o"].dtype)
    st["lse"][:n] = lse[b, :, :, t].reshape(n, H)


# ------------------------------------------------------------------- the definitions in 64 bits
def _round_codes(fmt, y):
    """Nearest code of y in 64 bits: whole numbers, or the e4m3 grid."""
    if fmt != "e4m3":
        return y.round()
    e = torch.frexp(y)[1].double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return ((y / step).round() * step).clamp(-448, 448)


def _row_values(fmt, x):
    """(values that the stored rows stand for, scales) of rows x, by the definition."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    amax[amax < LEAST] = 0
    div = torch.where(amax > 0, amax, math.inf)
    if fmt == "int4":
        parts = []
        for part in x.split(32, -1):
            g = _round_codes("e4m3", 448 * part.abs().amax(-1, keepdim=True) / div)
            n = (3136 * part / torch.where(g > 0, div * g, math.inf)).round().clamp(-7, 7)
            parts.append(n * g * (amax / 3136))
        return torch.cat(parts, -1), amax / 3136
    top = 448 if fmt == "e4m3" else 127
    return _round_codes(fmt, top * x / div) * (amax / top), amax / top


def _stored(c, st, b, length):
    """K and V of sequence b, [length, Hkv, d] in 64 bits, out of the cache's bytes."""
    pos = torch.arange(length, device="cuda")
    page, place = st["table"][b].long()[pos // c["page"]], pos % c["page"]
    kc, vc, ks, vs = (x[page, :, place] for x in views(c, st["kvq"], st["pages"]))
    out = []
    for code, scale in ((kc, ks), (vc, vs)):
        s = scale[..., :4].contiguous().view(torch.float32).double()
        if c["fmt"] == "int4":
            val = torch.empty(*code.shape[:-1], c["d"], dtype=torch.float64, device="cuda")
            val[..., 0::2] = (code % 16).double() - 8
            val[..., 1::2] = torch.div(code, 16, rounding_mode="floor").double() - 8
            for g in range(c["d"] // 32):
                val[..., 32 * g:32 * g + 32] *= scale[..., 4 + g:5 + g].contiguous().view(torch.float8_e4m3fn).double()
        elif c["fmt"] == "int8":
            val = code.double()
            val = torch.where(val > 127, val - 256, val)
        else:
            val = code.contiguous().view(torch.float8_e4m3fn).double()
        out.append(val * s)
    return out


def exact(c, seed):
    st = prepare(c, seed)
    new, past = lengths(c)
    cu = starts(new)
    if c["op"] == "read":
        back = [torch.zeros(st["k_back"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
        for b, length in enumerate(new):
            for x, y in zip(back, _stored(c, st, b, length)):
                x[cu[b]:cu[b + 1]] = y
        return {"k": back[0], "v": back[1]}
    if c["op"] == "write":
        got = {}
        for key in ("k", "v"):
            back = torch.zeros(st["k_back"].shape, dtype=torch.float64, device="cuda")
            pool = torch.zeros(st["k_scale"].shape, dtype=torch.float64, device="cuda")
            back[:cu[-1]], scale = _row_values(c["fmt"], st[key][:cu[-1]])
            for b in range(c["B"]):
                pos = past[b] + torch.arange(new[b], device="cuda")
                pool[st["table"][b].long()[pos // c["page"]], :, pos % c["page"]] = scale[cu[b]:cu[b + 1]]
            got |= {key: back, key + "_scale": pool}
        return got
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    G, ck = c["H"] // c["Hkv"], starts([a + b for a, b in zip(new, past)])
    for b in range(c["B"]):
        length, n = new[b] + past[b], new[b]
        if not n:
            continue
        k, v = (st["k"][ck[b]:ck[b + 1]].double(), st["v"][ck[b]:ck[b + 1]].double()) if c["op"] == "prompt" else _stored(c, st, b, length)
        if not length:
            lse[cu[b]:cu[b + 1]] = -math.inf
            continue
        hidden = torch.arange(length, device="cuda") > torch.arange(n, device="cuda")[:, None] + past[b]
        for h in range(c["H"]):
            s = st["q"][cu[b]:cu[b + 1], h].double() @ k[:, h // G].T / math.sqrt(c["d"])
            if c["causal"]:
                s[hidden] = -math.inf
            part = torch.logsumexp(s, -1)
            lse[cu[b]:cu[b + 1], h] = part
            weights = torch.exp(s - torch.where(part > -math.inf, part, 0.0)[:, None])
            o[cu[b]:cu[b + 1], h] = weights @ v[:, h // G]
    return {"o": o, "lse": lse}
