"""GPU tests of the sequence calls: the quantised paged cache, attention over it
and over packed prompts, against plain 64-bit NumPy (bounds in seq_helpers)."""
import itertools

import numpy as np
import pytest
import torch

import kv_cache_compression_two_b200 as ispa
from oracle import seq_oracle as so
from seq_helpers import DT, HALF, check_attention, f64, paged, rand16, starts

pytestmark = pytest.mark.gpu
FMT = {"e4m3": ispa.ISPA_KVQ_E4M3, "int8": ispa.ISPA_KVQ_INT8, "int4": ispa.ISPA_KVQ_INT4}
CODE = {torch.bfloat16: ispa.ISPA_BF16, torch.float16: ispa.ISPA_F16, torch.float32: ispa.ISPA_F32}


def cuda(x, dtype=None):
    t = torch.as_tensor(x) if isinstance(x, (np.ndarray, list)) else x
    return t.to("cuda", dtype) if dtype else t.cuda()


def ints(x):
    return cuda(np.asarray(x, np.int32))


def make_cache(rng, fmt, H_kv, d, page, lens, dtype, wide=False):
    """An oracle cache filled with random rows, its device copy, table and descriptor."""
    table, pages = paged(rng, lens, page)
    c = so.Cache(fmt, H_kv, d, page, pages, fill=0x7F)  # unwritten bytes are NaN codes
    for b, n in enumerate(lens):
        if n:
            k, v = (f64(rand16(rng, (n, H_kv, d), dtype, wide)) for _ in range(2))
            c.put(table[b], np.arange(n), k, v)
    return c, cuda(c.buf), ints(table), ispa.kvq_desc(H_kv, d, page, pages, FMT[fmt]), table


def attn_ws(a, c):
    return torch.empty(ispa.ispa_attn_kvq_workspace_bytes(a, c), dtype=torch.uint8, device="cuda")


def prompt_ws(a):
    return torch.empty(ispa.ispa_attn_prompt_workspace_bytes(a), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ cache: write and read
@pytest.mark.parametrize("fmt,d,dtype,page,H_kv", [
    (f, d, t, p, h) for (f, d), (t, p, h) in zip(
        itertools.product(["e4m3", "int8", "int4"], [64, 128]),
        [("bf16", 16, 1), ("fp16", 32, 3), ("bf16", 64, 5), ("fp16", 16, 8), ("bf16", 256, 2), ("fp16", 128, 12)])] + [
    ("int4", 128, "bf16", 16, 7), ("int8", 128, "bf16", 16, 4), ("e4m3", 128, "fp16", 32, 4)])
def test_write_and_read_are_exact(fmt, d, dtype, page, H_kv):
    """Codes, scales and the values read back, bit for bit; bytes and rows that the calls do not own stay."""
    rng = np.random.default_rng([d, page, H_kv, len(fmt)])
    new, past = [1, 0, 37, 2, 130, 1], [0, 9, 3, 0, 259, page - 1]
    total = [a + b for a, b in zip(new, past)]
    T, pad, H = sum(new), 5, 3
    table, pages = paged(rng, total, page)
    rows = rand16(rng, (T + pad, H + 2 * H_kv, d), DT[dtype], wide=True)  # a fused projection's output
    rows[0] = 0                                   # rows of zeros
    rows[1, :, 1:] = 0                            # a single value
    rows[2] *= 2.0 ** -14                         # (subnormals in fp16)
    x = cuda(rows)
    k, v = x[:, H:H + H_kv], x[:, H + H_kv:]
    c = so.Cache(fmt, H_kv, d, page, pages, fill=0xAB)
    kvq = cuda(c.buf.copy())
    desc = ispa.kvq_desc(H_kv, d, page, pages, FMT[fmt])
    assert ispa.ispa_kvq_bytes(desc) == c.buf.size
    cu = starts(new)
    ispa.ispa_kvq_write(desc, k, v, ints(table), ints(total), ints(cu), kvq)
    ispa.ispa_check_device_error()
    hk, hv = f64(k), f64(v)
    for b in range(len(new)):
        c.put(table[b], np.arange(past[b], total[b]), hk[cu[b]:cu[b + 1]], hv[cu[b]:cu[b + 1]])
    assert np.array_equal(kvq.cpu().numpy(), c.buf)
    # the new rows, and then a window that begins inside them
    for skip in (0, 1):
        n = [max(0, a - skip) for a in new]
        begin = [p + skip for p in past]
        cu2, T2 = starts(n), sum(n)
        out = [torch.full((T2 + pad, H_kv, d), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
        ispa.ispa_kvq_read(desc, kvq, ints(table), ints(cu2), *out, seq_begin=ints(begin))
        ispa.ispa_check_device_error()
        for b in range(len(n)):
            if n[b]:
                for got, want in zip(out, c.get(table[b], np.arange(begin[b], begin[b] + n[b]))):
                    want = torch.from_numpy(want).to(DT[dtype])
                    assert torch.equal(got[cu2[b]:cu2[b + 1]].cpu(), want)
        for got in out:
            assert torch.all(got[T2:] == 7.0)


def test_write_extremes_of_the_types():
    """The largest and smallest rows of bf16: no overflow, rows below 2^-96 are zeros."""
    desc = ispa.kvq_desc(1, 64, 16, 1, ispa.ISPA_KVQ_INT8)
    for fmt in FMT:
        desc.fmt = FMT[fmt]
        c = so.Cache(fmt, 1, 64, 16, 1)
        rows = torch.randn(6, 1, 64).to(torch.bfloat16)
        rows[0] = 3.38e38
        rows[1] *= 2.0 ** 120
        rows[2] *= 2.0 ** -90
        rows[3] *= 2.0 ** -110
        rows[4] = -0.0
        rows[5, 0, ::2] = 2.0 ** -96
        kvq = torch.zeros(c.buf.size, dtype=torch.uint8, device="cuda")
        x = rows.cuda()
        ispa.ispa_kvq_write(desc, x, x, ints([[0]]), ints([6]), ints([0, 6]), kvq)
        c.put([0], np.arange(6), f64(rows), f64(rows))
        got = kvq.cpu().numpy()
        if fmt == "e4m3":  # the sign of a zero code is free
            n = c.parts[0].size
            for a in (got, c.buf):
                a[:2 * ((n + 255) // 256 * 256)] = np.where(a[:2 * ((n + 255) // 256 * 256)] == 128, 0, a[:2 * ((n + 255) // 256 * 256)])
        assert np.array_equal(got, c.buf), fmt


def test_pages_beyond_four_gib():
    """Offsets past 32 bits: the last pages of a large cache."""
    desc = ispa.kvq_desc(8, 128, 256, 20000, ispa.ISPA_KVQ_INT8)
    kvq = torch.empty(ispa.ispa_kvq_bytes(desc), dtype=torch.uint8, device="cuda")
    assert kvq.numel() > 2 * 2 ** 32
    rng = np.random.default_rng(4)
    n = 300
    k, v = (rand16(rng, (n, 8, 128), torch.bfloat16) for _ in range(2))
    table = ints([[19999, 4]])
    ispa.ispa_kvq_write(desc, k.cuda(), v.cuda(), table, ints([n]), ints([0, n]), kvq)
    ko, vo = (torch.empty_like(k, device="cuda") for _ in range(2))
    ispa.ispa_kvq_read(desc, kvq, table, ints([0, n]), ko, vo)
    kk, vv = (so.dequantise("int8", *so.quantise("int8", f64(x))) for x in (k, v))
    assert torch.equal(ko.cpu(), torch.from_numpy(kk).to(torch.bfloat16))
    assert torch.equal(vo.cpu(), torch.from_numpy(vv).to(torch.bfloat16))
    q = rand16(rng, (1, 16, 128), torch.bfloat16)
    a = ispa.attn_seq_desc(1, 16, 8, 128, ispa.ISPA_BF16, ispa.ISPA_F32)
    o, lse = torch.empty(1, 16, 128, device="cuda"), torch.empty(1, 16, device="cuda")
    ispa.ispa_attn_kvq(a, desc, q.cuda(), kvq, table, ints([n]), ints([0, 1]), o, lse, workspace=attn_ws(a, desc))
    ref = so.attention(f64(q), kk, vv, True)
    check_attention(o, lse, ref, 2.0 ** -11, 128, n, np.abs(vv).max() * 2 ** 7)
    ispa.ispa_check_device_error()


# ------------------------------------------------------------------ attention over the cache
def run_attn_kvq(rng, fmt, d, dtype, out, G, H_kv, page, new, lens, causal=True, pad=0, wide=False, scale=0.0):
    c, kvq, table, cd, htable = make_cache(rng, fmt, H_kv, d, page, lens, DT[dtype], wide)
    B, H, T = len(new), G * H_kv, sum(new)
    q = rand16(rng, (T + pad, H, d), DT[dtype])
    a = ispa.attn_seq_desc(B, H, H_kv, d, CODE[DT[dtype]], CODE[out], causal, scale)
    o = torch.full((T + pad, H, d), 7.0, dtype=out, device="cuda")
    lse = torch.full((T + pad, H), 7.0, device="cuda")
    ispa.ispa_attn_kvq(a, cd, q.cuda(), kvq, table, ints(lens), ints(starts(new)), o, lse, workspace=attn_ws(a, cd))
    ispa.ispa_check_device_error()
    cu = starts(new)
    for b in range(B):
        k, v = c.get(htable[b], np.arange(lens[b]))
        part = slice(cu[b], cu[b + 1])
        if new[b]:
            ref = so.attention(f64(q[part]), k, v, causal, scale or None)
            vmax = np.abs(v).max() * 2.0 ** 7 if lens[b] else 0.0
            check_attention(o[part], lse[part], ref, 2.0 ** -11, d, lens[b], vmax, f"sequence {b}")
    assert torch.all(o[T:] == 7.0) and torch.all(lse[T:] == 7.0)


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("d,dtype,out,G,H_kv,page", [
    (128, "bf16", torch.bfloat16, 4, 2, 16), (64, "fp16", torch.float16, 7, 3, 32), (128, "fp16", torch.float32, 1, 5, 64),
    (64, "bf16", torch.float32, 16, 1, 256), (128, "bf16", torch.float32, 33, 1, 128)])
def test_cached_attention_one_token(fmt, d, dtype, out, G, H_kv, page):
    lens = [1, 15, 16, 17, 31, 32, 33, 300, 1025, 2]
    run_attn_kvq(np.random.default_rng([d, G]), fmt, d, dtype, out, G, H_kv, page, [1] * len(lens), lens, pad=2)


@pytest.mark.parametrize("fmt,d", [("e4m3", 64), ("int8", 128), ("int4", 128), ("int4", 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_cached_attention_several_tokens(fmt, d, causal):
    """Ragged counts, none at all, more queries than tokens in the cache."""
    run_attn_kvq(np.random.default_rng(d), fmt, d, "bf16", torch.float32, 3, 2, 16, [2, 0, 7, 1, 16, 3, 40],
                 [2, 50, 200, 0, 700, 1, 64], causal, pad=1)


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
def test_cached_attention_split_over_sms(fmt):
    """Few sequences, long caches: every item is joined from the parts of many SMs."""
    run_attn_kvq(np.random.default_rng(8), fmt, 128, "bf16", torch.float32, 4, 1, 64, [1, 5], [9001, 4097])


@pytest.mark.parametrize("fmt,d,dtype,G", [("int8", 64, "bf16", 1), ("e4m3", 128, "fp16", 3), ("int4", 64, "fp16", 13)])
def test_cached_attention_from_few_to_many_parts(fmt, d, dtype, G):
    """Items of about 6, 18, 36 and 70 parts, whose merge one, two or four CTAs share; one alone of 150."""
    rng = np.random.default_rng([12, d])
    run_attn_kvq(rng, fmt, d, dtype, torch.float32, G, 1, 32, [1] * 4, [700, 2300, 4600, 9000])
    run_attn_kvq(rng, fmt, d, dtype, torch.float32, G, 1, 256, [2], [19001])


@pytest.mark.parametrize("fmt,d", [("e4m3", 128), ("int8", 64), ("int4", 128)])
def test_cached_attention_wide_scales(fmt, d):
    """Token scales over ten powers of two, and a sharp softmax."""
    run_attn_kvq(np.random.default_rng(9), fmt, d, "fp16", torch.float32, 2, 2, 32, [1, 3], [777, 123], wide=True)
    run_attn_kvq(np.random.default_rng(10), fmt, d, "bf16", torch.float32, 2, 2, 32, [1, 3], [777, 123], scale=1.0)


def test_cached_attention_many_sequences():
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(1, 40, 700)]
    run_attn_kvq(rng, "int8", 64, "bf16", torch.bfloat16, 2, 1, 16, [1] * 700, lens)


# ------------------------------------------------------------------ prompts
def run_prompt(rng, d, dtype, out, G, H_kv, nq, nk, causal, pad=0, fused=False, scale=0.0):
    B, H, Tq, Tk = len(nq), G * H_kv, sum(nq), sum(nk)
    cq, ck = starts(nq), starts(nk)
    if fused:
        rows = rand16(rng, (Tq + pad, H + 2 * H_kv, d), DT[dtype])
        x = rows.cuda()
        (q, k, v), (dq, dk, dv) = (((y[:, :H], y[:, H:H + H_kv], y[:, H + H_kv:])) for y in (rows, x))
    else:
        q = rand16(rng, (Tq + pad, H, d), DT[dtype])
        k, v = (rand16(rng, (Tk + pad, H_kv, d), DT[dtype]) for _ in range(2))
        if pad:
            k[Tk:], v[Tk:] = float("nan"), float("inf")
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    a = ispa.attn_seq_desc(B, H, H_kv, d, CODE[DT[dtype]], CODE[out], causal, scale)
    o = torch.full((Tq + pad, H, d), 7.0, dtype=out, device="cuda")
    lse = torch.full((Tq + pad, H), 7.0, device="cuda")
    ispa.ispa_attn_prompt(a, dq, dk, dv, ints(cq), ints(ck), o, lse, workspace=prompt_ws(a))
    ispa.ispa_check_device_error()
    for b in range(B):
        pq, pk = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        if nq[b]:
            ref = so.attention(f64(q[pq]), f64(k[pk]), f64(v[pk]), causal, scale or None)
            vmax = np.abs(f64(v[pk])).max() if nk[b] else 0.0
            check_attention(o[pq], lse[pq], ref, HALF[DT[dtype]], d, nk[b], vmax, f"sequence {b}")
    assert torch.all(o[Tq:] == 7.0) and torch.all(lse[Tq:] == 7.0)


@pytest.mark.parametrize("d,dtype,out", [(128, "bf16", torch.bfloat16), (64, "fp16", torch.float16),
                                         (128, "fp16", torch.float32), (64, "bf16", torch.float32)])
@pytest.mark.parametrize("G,H_kv", [(1, 3), (4, 2), (3, 1), (8, 1), (128, 1), (100, 1)])
def test_prompts_causal(d, dtype, out, G, H_kv):
    n = [1, 16, 17, 127, 128, 129, 0, 260, 5] if G < 100 else [1, 3, 0, 20]
    run_prompt(np.random.default_rng([d, G]), d, dtype, out, G, H_kv, n, n, True, pad=3, fused=True)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_with_more_or_fewer_keys(d, dtype, causal):
    """A chunk after a prefix, no key at all, fewer keys than queries (their first rows see nothing)."""
    run_prompt(np.random.default_rng(d), d, dtype, torch.float32, 2, 2, [1, 40, 130, 7, 300, 3, 200],
               [1000, 553, 131, 0, 45, 2, 199], causal, pad=4)


@pytest.mark.parametrize("d,dtype,causal", [(128, "bf16", False), (64, "fp16", True), (128, "fp16", True)])
def test_prompts_split_over_sms(d, dtype, causal):
    """Few queries over many keys: items are joined from the parts of many SMs."""
    run_prompt(np.random.default_rng(2), d, dtype, torch.float32, 1, 1, [33, 300], [12011, 5001], causal)


@pytest.mark.parametrize("d,B,H_kv,nq,nk", [(64, 2, 9, 2300, 515), (128, 1, 13, 3001, 2100), (128, 3, 1, 300, 700),
                                            (64, 2, 3, 50, 0)])
def test_prompts_alike_over_every_key(d, B, H_kv, nq, nk):
    """Equal sequences that see every key: more items than SMs (whole rounds, then a cut rest), or fewer."""
    run_prompt(np.random.default_rng(13), d, "bf16", torch.float32, 1, H_kv, [nq] * B, [nk] * B, False)


def test_prompt_long_causal():
    run_prompt(np.random.default_rng(5), 128, "bf16", torch.bfloat16, 4, 1, [3001], [3001], True, fused=True)


def test_prompt_sharp_softmax():
    """Scores far apart: the running maximum moves often and the first product must not lose bits."""
    run_prompt(np.random.default_rng(6), 128, "fp16", torch.float32, 1, 2, [200, 900], [1500, 900], True, scale=1.5)


def test_prompt_output_at_every_alignment_allowed():
    """O 16-byte but not 32-byte aligned gives the same bits as an aligned one."""
    rng = np.random.default_rng(12)
    q, k, v = (rand16(rng, (150, h, 64), torch.bfloat16).cuda() for h in (2, 1, 1))
    cu = ints([0, 150])
    for out in (torch.bfloat16, torch.float32):
        a = ispa.attn_seq_desc(1, 2, 1, 64, ispa.ISPA_BF16, CODE[out])
        got = []
        for shift in (0, 16):
            n = shift // torch.empty(0, dtype=out).element_size()
            buf = torch.full((150 * 2 * 64 + 16,), 7.0, dtype=out, device="cuda")
            o = buf[n:n + 150 * 2 * 64].view(150, 2, 64)
            assert o.data_ptr() % 32 == shift
            ispa.ispa_attn_prompt(a, q, k, v, cu, cu, o, None, workspace=prompt_ws(a))
            assert torch.all(buf[:n] == 7.0) and torch.all(buf[n + 150 * 2 * 64:] == 7.0)
            got.append(o.clone())
        assert torch.equal(*got)
    ispa.ispa_check_device_error()


def test_prompts_many_sequences():
    rng = np.random.default_rng(7)
    n = [int(x) for x in rng.integers(0, 30, 900)]
    run_prompt(rng, 64, "bf16", torch.bfloat16, 2, 1, n, n, True)


def test_values_of_other_sequences_do_not_matter():
    """Infinities and NaN in a neighbour's rows, right behind a ragged end."""
    rng = np.random.default_rng(11)
    n = [70, 33, 90]
    cu = starts(n)
    q, k, v = (rand16(rng, (sum(n), 1, 128), torch.bfloat16) for _ in range(3))
    bad_k, bad_v = k.clone(), v.clone()
    bad_k[cu[1]:cu[2]], bad_v[cu[1]:cu[2]] = float("nan"), float("inf")
    a = ispa.attn_seq_desc(3, 1, 1, 128, ispa.ISPA_BF16, ispa.ISPA_F32, False)
    got = []
    for kk, vv in ((k, v), (bad_k, bad_v)):
        o = torch.empty(sum(n), 1, 128, device="cuda")
        ispa.ispa_attn_prompt(a, q.cuda(), kk.cuda(), vv.cuda(), ints(cu), ints(cu), o, None, workspace=prompt_ws(a))
        got.append(o.cpu())
    for part in (slice(0, 70), slice(103, 193)):
        assert torch.equal(got[0][part], got[1][part])


# ------------------------------------------------------------------ as they are used together
@pytest.mark.parametrize("fmt,dtype", [("int4", "bf16"), ("e4m3", "fp16"), ("int8", "bf16")])
def test_serving_run(fmt, dtype):
    """Prompts, then decoding steps, then a second chunk over the cache read back, and a merge of two groups."""
    rng = np.random.default_rng(21)
    H, H_kv, d, page, t = 8, 2, 128, 16, DT[dtype]
    first, steps = [45, 7, 130], 3
    B = len(first)
    chunk = [20, 33, 1]
    total = [n + steps + c for n, c in zip(first, chunk)]
    table, pages = paged(rng, total, page)
    cd = ispa.kvq_desc(H_kv, d, page, pages, FMT[fmt])
    kvq = torch.full((ispa.ispa_kvq_bytes(cd),), 0x7F, dtype=torch.uint8, device="cuda")
    oc = so.Cache(fmt, H_kv, d, page, pages)
    code, dt_table = CODE[t], ints(table)
    a = ispa.attn_seq_desc(B, H, H_kv, d, code, code)
    ws = torch.empty(max(ispa.ispa_attn_prompt_workspace_bytes(a), ispa.ispa_attn_kvq_workspace_bytes(a, cd)),
                     dtype=torch.uint8, device="cuda")

    def rows(lens):
        x = rand16(rng, (sum(lens), H + 2 * H_kv, d), t)
        return x, x.cuda(), starts(lens)

    # 1. the prompts attend to themselves and are written
    x, gx, cu = rows(first)
    o = torch.empty(sum(first), H, d, dtype=t, device="cuda")
    ispa.ispa_attn_prompt(a, gx[:, :H], gx[:, H:H + H_kv], gx[:, H + H_kv:], ints(cu), ints(cu), o, None, workspace=ws)
    ispa.ispa_kvq_write(cd, gx[:, H:H + H_kv], gx[:, H + H_kv:], dt_table, ints(first), ints(cu), kvq)
    for b in range(B):
        y = x[cu[b]:cu[b + 1]]
        k, v = f64(y[:, H:H + H_kv]), f64(y[:, H + H_kv:])
        check_attention(o[cu[b]:cu[b + 1]], None, so.attention(f64(y[:, :H]), k, v, True), HALF[t], d, first[b],
                        np.abs(v).max())
        oc.put(table[b], np.arange(first[b]), k, v)
    # 2. steps of one token
    lens = list(first)
    for _ in range(steps):
        x, gx, cu = rows([1] * B)
        lens = [n + 1 for n in lens]
        o, lse = torch.empty(B, H, d, dtype=t, device="cuda"), torch.empty(B, H, device="cuda")
        ispa.ispa_kvq_write(cd, gx[:, H:H + H_kv], gx[:, H + H_kv:], dt_table, ints(lens), ints(cu), kvq)
        ispa.ispa_attn_kvq(a, cd, gx[:, :H], kvq, dt_table, ints(lens), ints(cu), o, lse, workspace=ws)
        for b in range(B):
            y = x[b:b + 1]
            oc.put(table[b], [lens[b] - 1], f64(y[:, H:H + H_kv]), f64(y[:, H + H_kv:]))
            k, v = oc.get(table[b], np.arange(lens[b]))
            check_attention(o[b:b + 1], lse[b:b + 1], so.attention(f64(y[:, :H]), k, v, True), 2.0 ** -11, d, lens[b],
                            np.abs(v).max() * 2 ** 7)
    # 3. a second chunk: written, the whole context read back, attended to
    x, gx, cu = rows(chunk)
    lens = [n + c for n, c in zip(lens, chunk)]
    ck = starts(lens)
    ispa.ispa_kvq_write(cd, gx[:, H:H + H_kv], gx[:, H + H_kv:], dt_table, ints(lens), ints(cu), kvq)
    kb, vb = (torch.empty(sum(lens), H_kv, d, dtype=t, device="cuda") for _ in range(2))
    ispa.ispa_kvq_read(cd, kvq, dt_table, ints(ck), kb, vb)
    o = torch.empty(sum(chunk), H, d, dtype=t, device="cuda")
    ispa.ispa_attn_prompt(a, gx[:, :H], kb, vb, ints(cu), ints(ck), o, None, workspace=ws)
    for b in range(B):
        y = x[cu[b]:cu[b + 1]]
        oc.put(table[b], np.arange(lens[b] - chunk[b], lens[b]), f64(y[:, H:H + H_kv]), f64(y[:, H + H_kv:]))
        k, v = (f64(torch.from_numpy(z).to(t)) for z in oc.get(table[b], np.arange(lens[b])))
        assert np.array_equal(f64(kb[ck[b]:ck[b + 1]]), k) and np.array_equal(f64(vb[ck[b]:ck[b + 1]]), v)
        check_attention(o[cu[b]:cu[b + 1]], None, so.attention(f64(y[:, :H]), k, v, True), HALF[t], d, lens[b],
                        np.abs(v).max())
    # 4. the first page's tokens and the rest as two groups, merged by their log-sum-exp
    a32 = ispa.attn_seq_desc(B, H, H_kv, d, code, ispa.ISPA_F32, False)
    q = rand16(rng, (B, H, d), t)
    rest = [n - page if n > page else 0 for n in lens]
    head = [min(n, page) for n in lens]
    parts = [(dt_table, lens), (dt_table, head), (ints(np.roll(table, -1, 1)), rest)]
    got = []
    for tab, n in parts:
        o, lse = torch.empty(B, H, d, device="cuda"), torch.empty(B, H, device="cuda")
        ispa.ispa_attn_kvq(a32, cd, q.cuda(), kvq, tab, ints(n), ints(starts([1] * B)), o, lse, workspace=ws)
        got.append((o, lse))
    mo, ml = torch.empty_like(got[0][0]), torch.empty_like(got[0][1])
    ispa.ispa_lse_merge(B, H, d, ispa.ISPA_F32, *got[1], *got[2], mo, ml)
    for b in range(B):
        k, v = oc.get(table[b], np.arange(lens[b]))
        ref = so.attention(f64(q[b:b + 1]), k, v, False)
        check_attention(mo[b:b + 1], ml[b:b + 1], ref, 2.0 ** -11, d, lens[b], np.abs(v).max() * 2 ** 7)
    ispa.ispa_check_device_error()


def test_graph_of_a_step_replayed_as_the_sequences_grow():
    """One captured step (write, attend) on a stream of its own, replayed with longer lengths; twice the same bits."""
    rng = np.random.default_rng(31)
    H, H_kv, d, page, t = 8, 2, 64, 16, torch.bfloat16
    lens = [30, 1, 300]
    B = len(lens)
    table, pages = paged(rng, [n + 8 for n in lens], page)
    cd = ispa.kvq_desc(H_kv, d, page, pages, ispa.ISPA_KVQ_INT8)
    oc = so.Cache("int8", H_kv, d, page, pages)
    for b, n in enumerate(lens):
        oc.put(table[b], np.arange(n), f64(rand16(rng, (n, H_kv, d), t)), f64(rand16(rng, (n, H_kv, d), t)))
    kvq, dt_table, dl, cu = cuda(oc.buf), ints(table), ints(lens), ints(starts([1] * B))
    x = torch.zeros(B, H + 2 * H_kv, d, dtype=t, device="cuda")
    a = ispa.attn_seq_desc(B, H, H_kv, d, ispa.ISPA_BF16, ispa.ISPA_F32)
    o, lse, ws = torch.empty(B, H, d, device="cuda"), torch.empty(B, H, device="cuda"), attn_ws(a, cd)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ispa.ispa_kvq_write(cd, x[:, H:H + H_kv], x[:, H + H_kv:], dt_table, dl, cu, kvq)
        ispa.ispa_attn_kvq(a, cd, x[:, :H], kvq, dt_table, dl, cu, o, lse, workspace=ws)
    for step in range(4):
        y = rand16(rng, (B, H + 2 * H_kv, d), t)
        lens = [n + 1 for n in lens]
        x.copy_(y)
        dl.copy_(ints(lens))
        graph.replay()
        torch.cuda.synchronize()
        bits = o.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits, o)
        for b in range(B):
            oc.put(table[b], [lens[b] - 1], f64(y[b:b + 1, H:H + H_kv]), f64(y[b:b + 1, H + H_kv:]))
            k, v = oc.get(table[b], np.arange(lens[b]))
            check_attention(o[b:b + 1], lse[b:b + 1], so.attention(f64(y[b:b + 1, :H]), k, v, True), 2.0 ** -11, d,
                            lens[b], np.abs(v).max() * 2 ** 7)
    ispa.ispa_check_device_error()


def test_two_streams_with_a_workspace_each():
    rng = np.random.default_rng(41)
    a = ispa.attn_seq_desc(1, 4, 1, 128, ispa.ISPA_BF16, ispa.ISPA_F32, False)
    cu_q, cu_k = ints([0, 200]), ints([0, 9000])
    work = []
    for i in range(2):
        q, k, v = (rand16(rng, s, torch.bfloat16).cuda() for s in ((200, 4, 128), (9000, 1, 128), (9000, 1, 128)))
        work.append((torch.cuda.Stream(), q, k, v, torch.empty(200, 4, 128, device="cuda"), prompt_ws(a)))
    alone = []
    for s, q, k, v, o, ws in work:
        ispa.ispa_attn_prompt(a, q, k, v, cu_q, cu_k, o, None, workspace=ws)
        torch.cuda.synchronize()
        alone.append(o.clone())
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for s, q, k, v, o, ws in work:
            ispa.ispa_attn_prompt(a, q, k, v, cu_q, cu_k, o, None, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for (s, q, k, v, o, ws), want in zip(work, alone):
        assert torch.equal(o, want)
    ispa.ispa_check_device_error()


def test_graph_of_a_chunk_replayed_with_other_lengths():
    """Write, read back and prompt attention captured once, replayed as the bounds on the device change."""
    rng = np.random.default_rng(61)
    H, H_kv, d, page, t = 6, 2, 128, 32, torch.bfloat16
    T, Tk = 200, 1500
    cd = ispa.kvq_desc(H_kv, d, page, 64, ispa.ISPA_KVQ_INT4)
    kvq = torch.zeros(ispa.ispa_kvq_bytes(cd), dtype=torch.uint8, device="cuda")
    table = ints(rng.permutation(64).reshape(2, 32))
    x = torch.zeros(T, H + 2 * H_kv, d, dtype=t, device="cuda")
    a = ispa.attn_seq_desc(2, H, H_kv, d, ispa.ISPA_BF16, ispa.ISPA_F32)
    cu_q, cu_k, lens = ints([0, 0, 0]), ints([0, 0, 0]), ints([0, 0])
    kb, vb = (torch.zeros(Tk, H_kv, d, dtype=t, device="cuda") for _ in range(2))
    o, ws = torch.zeros(T, H, d, device="cuda"), prompt_ws(a)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ispa.ispa_kvq_write(cd, x[:, H:H + H_kv], x[:, H + H_kv:], table, lens, cu_q, kvq)
        ispa.ispa_kvq_read(cd, kvq, table, cu_k, kb, vb)
        ispa.ispa_attn_prompt(a, x[:, :H], kb, vb, cu_q, cu_k, o, None, workspace=ws)
    total = np.zeros(2, int)
    oc = so.Cache("int4", H_kv, d, page, 64)
    htab = table.cpu().numpy()
    for new in ([150, 50], [0, 200], [33, 1], [100, 100]):
        y = rand16(rng, (T, H + 2 * H_kv, d), t)
        total = total + new
        cq, ck = starts(new), starts(total)
        x.copy_(y)
        cu_q.copy_(ints(cq)), cu_k.copy_(ints(ck)), lens.copy_(ints(total))
        graph.replay()
        ispa.ispa_check_device_error()
        for b in range(2):
            z = y[cq[b]:cq[b + 1]]
            oc.put(htab[b], np.arange(total[b] - new[b], total[b]), f64(z[:, H:H + H_kv]), f64(z[:, H + H_kv:]))
            k, v = (f64(torch.from_numpy(w).to(t)) for w in oc.get(htab[b], np.arange(total[b])))
            if new[b]:
                check_attention(o[cq[b]:cq[b + 1]], None, so.attention(f64(z[:, :H]), k, v, True), HALF[t], d,
                                total[b], np.abs(v).max())


def test_rows_in_front_of_the_first_sequence_stay():
    """cu[0] > 0: the rows before it belong to no sequence."""
    rng = np.random.default_rng(62)
    k, v = (rand16(rng, (30, 1, 64), torch.bfloat16) for _ in range(2))
    q = rand16(rng, (30, 2, 64), torch.bfloat16)
    cu = ints([7, 12, 25])
    a = ispa.attn_seq_desc(2, 2, 1, 64, ispa.ISPA_BF16, ispa.ISPA_F32)
    o = torch.full((30, 2, 64), 7.0, device="cuda")
    ispa.ispa_attn_prompt(a, q.cuda(), k.cuda(), v.cuda(), cu, cu, o, None, workspace=prompt_ws(a))
    cd = ispa.kvq_desc(1, 64, 16, 3, ispa.ISPA_KVQ_E4M3)
    c = so.Cache("e4m3", 1, 64, 16, 3, fill=0xAB)
    kvq, table = cuda(c.buf.copy()), ints([[2], [0]])
    ispa.ispa_kvq_write(cd, k.cuda(), v.cuda(), table, ints([5, 13]), cu, kvq)
    c.put([2], np.arange(5), f64(k[7:12]), f64(v[7:12]))
    c.put([0], np.arange(13), f64(k[12:25]), f64(v[12:25]))
    assert np.array_equal(kvq.cpu().numpy(), c.buf)
    o2 = torch.full((30, 2, 64), 7.0, device="cuda")
    ispa.ispa_attn_kvq(a, cd, q.cuda(), kvq, table, ints([5, 13]), cu, o2, None, workspace=attn_ws(a, cd))
    for rows, tab in ((slice(7, 12), [2]), (slice(12, 25), [0])):
        n = rows.stop - rows.start
        check_attention(o[rows], None, so.attention(f64(q[rows]), f64(k[rows]), f64(v[rows]), True), 2.0 ** -8, 64, n, 5.0)
        kk, vv = c.get(tab, np.arange(n))
        check_attention(o2[rows], None, so.attention(f64(q[rows]), kk, vv, True), 2.0 ** -11, 64, n, np.abs(vv).max() * 2 ** 7)
    for x in (o, o2):
        assert torch.all(x[:7] == 7.0) and torch.all(x[25:] == 7.0)
    ispa.ispa_check_device_error()


def test_no_rows_and_no_keys():
    a = ispa.attn_seq_desc(1, 2, 1, 64, ispa.ISPA_F16, ispa.ISPA_F16)
    none = torch.zeros(0, 1, 64, dtype=torch.float16, device="cuda")
    q = torch.ones(3, 2, 64, dtype=torch.float16, device="cuda")
    o, lse = torch.full_like(q, 7.0), torch.full((3, 2), 7.0, device="cuda")
    ispa.ispa_attn_prompt(a, q, none, none, ints([0, 3]), ints([0, 0]), o, lse, workspace=prompt_ws(a))
    assert torch.all(o == 0) and torch.all(lse == -float("inf"))
    ispa.ispa_attn_prompt(a, q[:0], none, none, ints([0, 0]), ints([0, 0]), o[:0], lse[:0], workspace=prompt_ws(a))
    cd = ispa.kvq_desc(1, 64, 16, 1, ispa.ISPA_KVQ_INT8)
    kvq = torch.full((ispa.ispa_kvq_bytes(cd),), 9, dtype=torch.uint8, device="cuda")
    ispa.ispa_kvq_write(cd, none, none, ints([[0]]), ints([0]), ints([0, 0]), kvq)
    ispa.ispa_kvq_read(cd, kvq, ints([[0]]), ints([0, 0]), none, none)
    assert torch.all(kvq == 9)
    ispa.ispa_check_device_error()


def test_cached_attention_scales_far_apart():
    """V rows over 2^24 of scale: each keeps its share, whichever comes first."""
    rng = np.random.default_rng(63)
    for order in (1, -1):
        k = rand16(rng, (200, 1, 64), torch.bfloat16)
        v = (rand16(rng, (200, 1, 64), torch.bfloat16).float() * torch.exp2(torch.linspace(-12.0 * order, 12.0 * order, 200))[:, None, None]).to(torch.bfloat16)
        q = rand16(rng, (1, 4, 64), torch.bfloat16)
        for fmt in FMT:
            cd = ispa.kvq_desc(1, 64, 16, 13, FMT[fmt])
            c = so.Cache(fmt, 1, 64, 16, 13)
            c.put(np.arange(13), np.arange(200), f64(k), f64(v))
            a = ispa.attn_seq_desc(1, 4, 1, 64, ispa.ISPA_BF16, ispa.ISPA_F32)
            o = torch.empty(1, 4, 64, device="cuda")
            ispa.ispa_attn_kvq(a, cd, q.cuda(), cuda(c.buf), ints([np.arange(13)]), ints([200]), ints([0, 1]), o, None, workspace=attn_ws(a, cd))
            kk, vv = c.get(np.arange(13), np.arange(200))
            # weights below 2^-14 of fp16's unit are off by 2^-25: at most 2^-31 of the largest V scale times its largest code
            check_attention(o, None, so.attention(f64(q), kk, vv, True), 2.0 ** -11, 64, 200, np.abs(vv).max())
    ispa.ispa_check_device_error()


# ------------------------------------------------------------------ values out of range
def expect_bad_sequence(b):
    # (the exception is not kept: its traceback would hold the caller's tensors in a cycle, to be freed
    # whenever the collector runs, in the middle of a test that counts memory, say)
    status, text = ispa.ISPA_OK, ""
    try:
        ispa.ispa_check_device_error()
    except ispa.IspaError as e:
        status, text = e.status, str(e)
    assert status == ispa.ISPA_ERR_INVALID_ARG and f"sequence {b} " in text
    ispa.ispa_check_device_error()  # cleared


@pytest.mark.parametrize("page_id", [-1, 1 << 30])
def test_bad_pages_are_skipped_and_reported(page_id):
    rng = np.random.default_rng(51)
    H_kv, d, page, lens = 2, 128, 16, [40, 50]
    c, kvq, table, cd, htable = make_cache(rng, "int8", H_kv, d, page, lens, torch.bfloat16)
    htable = htable.copy()
    htable[1, 1] = page_id  # positions 16..31 of sequence 1
    table = ints(htable)
    a = ispa.attn_seq_desc(2, 4, H_kv, d, ispa.ISPA_BF16, ispa.ISPA_F32)
    q = rand16(rng, (2, 4, d), torch.bfloat16)
    o, lse = torch.empty(2, 4, d, device="cuda"), torch.empty(2, 4, device="cuda")
    ispa.ispa_attn_kvq(a, cd, q.cuda(), kvq, table, ints(lens), ints([0, 1, 2]), o, lse, workspace=attn_ws(a, cd))
    expect_bad_sequence(1)
    htable[1, 1] = 0
    keep = np.ones(50, bool)
    keep[16:32] = False
    for b, kp in ((0, None), (1, keep)):
        k, v = c.get(htable[b], np.arange(lens[b]))
        if b == 1:
            k, v = (np.where(kp[:, None, None], z, 0.0) for z in (k, v))
        check_attention(o[b:b + 1], lse[b:b + 1], so.attention(f64(q[b:b + 1]), k, v, True, keep=kp), 2.0 ** -11, d,
                        lens[b], np.abs(v).max() * 2 ** 7)
    # read: rows without a page are zeros; write: they go nowhere
    out = [torch.full((90, H_kv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ispa.ispa_kvq_read(cd, kvq, table, ints([0, 40, 90]), *out)
    expect_bad_sequence(1)
    for got, want in zip(out, c.get(htable[1], np.arange(50))):
        want = torch.from_numpy(np.where(keep[:, None, None], want, 0.0).astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(got[40:].cpu(), want)
    before = kvq.clone()
    rows = rand16(rng, (16, H_kv, d), torch.bfloat16).cuda()
    ispa.ispa_kvq_write(cd, rows, rows, table, ints([0, 32]), ints([0, 0, 16]), kvq)
    expect_bad_sequence(1)
    assert torch.equal(before, kvq)


def test_bad_lengths_and_bounds_are_clamped_and_reported():
    rng = np.random.default_rng(52)
    H_kv, d, page = 1, 64, 16
    c, kvq, table, cd, htable = make_cache(rng, "e4m3", H_kv, d, page, [30, 30], torch.bfloat16)
    a = ispa.attn_seq_desc(2, 2, H_kv, d, ispa.ISPA_BF16, ispa.ISPA_F32)
    q = rand16(rng, (2, 2, d), torch.bfloat16)
    k, v = c.get(htable[0], np.arange(30))
    for lens, cu, bad in (([30, -7], [0, 1, 2], 1), ([30, 5], [0, 1, 900], 1), ([30, 30], [0, 1, -4], 1)):
        o, lse = torch.empty(2, 2, d, device="cuda"), torch.empty(2, 2, device="cuda")
        ispa.ispa_attn_kvq(a, cd, q.cuda(), kvq, table, ints(lens), ints(cu), o, lse, workspace=attn_ws(a, cd))
        if cu[2] != -4:
            expect_bad_sequence(bad)
        else:
            torch.cuda.synchronize()
        check_attention(o[:1], lse[:1], so.attention(f64(q[:1]), k, v, True), 2.0 ** -11, d, 30, np.abs(v).max() * 2 ** 7)
    ap = ispa.attn_seq_desc(2, 2, 1, d, ispa.ISPA_BF16, ispa.ISPA_F32)
    kk, vv = (rand16(rng, (40, 1, d), torch.bfloat16) for _ in range(2))
    q = rand16(rng, (40, 2, d), torch.bfloat16)
    o = torch.empty(40, 2, d, device="cuda")
    ispa.ispa_attn_prompt(ap, q.cuda(), kk.cuda(), vv.cuda(), ints([0, 30, 70]), ints([0, 30, 9999]), o, None,
                          workspace=prompt_ws(ap))
    expect_bad_sequence(1)
    check_attention(o[:30], None, so.attention(f64(q[:30]), f64(kk[:30]), f64(vv[:30]), True), 2.0 ** -8, d, 30, 5.0)


def test_binding_refuses_what_does_not_fit():
    cd = ispa.kvq_desc(2, 64, 16, 4, ispa.ISPA_KVQ_INT8)
    kvq = torch.zeros(ispa.ispa_kvq_bytes(cd), dtype=torch.uint8, device="cuda")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    table, lens, cu = ints([[0, 1]]), ints([3]), ints([0, 3])
    ispa.ispa_kvq_write(cd, k, k, table, lens, cu, kvq)
    bad = [dict(k=k.float()), dict(k=k.cpu()), dict(k=k[:2]), dict(k=k.half()), dict(k=k.transpose(1, 2)),
           dict(k=k[:, :1]), dict(table=table.long()), dict(lens=lens.cpu()), dict(cu=ints([0, 1, 3])),
           dict(kvq=kvq[:100]), dict(kvq=kvq.view(torch.int8)), dict(k=torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda").expand(3, 2, 64))]
    for change in bad:
        args = dict(k=k, v=k, table=table, lens=lens, cu=cu, kvq=kvq) | change
        with pytest.raises((ValueError, TypeError, ispa.IspaError)):
            ispa.ispa_kvq_write(cd, args["k"], args["v"], args["table"], args["lens"], args["cu"], args["kvq"])
    a = ispa.attn_seq_desc(1, 4, 2, 64, ispa.ISPA_BF16, ispa.ISPA_BF16)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    ws = attn_ws(a, cd)
    for kw in (dict(workspace=ws[:64]), dict(workspace=None), dict(workspace=ws, o=q.float())):
        with pytest.raises((ValueError, TypeError, ispa.IspaError)):
            ispa.ispa_attn_kvq(a, cd, q, kvq, table, lens, ints([0, 1]), kw.get("o", torch.empty_like(q)), None,
                               workspace=kw["workspace"])
    torch.cuda.synchronize()


def test_binding_names_an_argument_that_is_no_tensor():
    cd = ispa.kvq_desc(2, 64, 16, 4, ispa.ISPA_KVQ_INT8)
    kvq = torch.zeros(ispa.ispa_kvq_bytes(cd), dtype=torch.uint8, device="cuda")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    table, lens, cu = ints([[0, 1]]), ints([3]), ints([0, 3])
    names = ("k", "v", "block_table", "seq_lens", "cu_new", "kvq")
    for i, name in enumerate(names):
        args = [k, k, table, lens, cu, kvq]
        args[i] = [1, 2, 3]
        with pytest.raises(TypeError, match=name):
            ispa.ispa_kvq_write(cd, *args)
    names = ("kvq", "block_table", "cu_out", "k_out", "v_out", "seq_begin")
    for i, name in enumerate(names):
        args = [kvq, table, cu, torch.empty_like(k), torch.empty_like(k), lens]
        args[i] = [1, 2, 3]
        with pytest.raises(TypeError, match=name):
            ispa.ispa_kvq_read(cd, *args)
    torch.cuda.synchronize()
