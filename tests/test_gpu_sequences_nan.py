"""GPU tests: a query with a NaN is seen in its own outputs, and only there."""
import numpy as np
import pytest
import torch

import kv_cache_compression_two_b200 as ispa
from oracle import seq_oracle as so
from seq_bounds import CODE, FMT, ints, random_rows
from seq_helpers import HALF, check_attention, f64

pytestmark = pytest.mark.gpu
LENS, NEW = [100, 3000], [5, 3]
BAD = [(0, 1), (3, 0), (6, 5)]  # (packed query, head)


def outputs_are_nan_where_queries_are(o, lse, refs, weight_half, d, vmax):
    bad = torch.zeros(o.shape[:2], dtype=torch.bool)
    for t, h in BAD:
        bad[t, h] = True
    assert torch.equal(torch.isnan(lse).cpu(), bad)
    assert torch.equal(torch.isnan(o).cpu(), bad[..., None].expand(o.shape))
    clean_o, clean_lse = torch.where(bad[..., None].cuda(), 0, o), torch.where(bad.cuda(), 0, lse)
    at = 0
    for n, ref, length in zip(NEW, refs, LENS):
        ref = [x.copy() for x in ref]
        for t, h in BAD:
            if at <= t < at + n:
                ref[0][t - at, h] = ref[1][t - at, h] = 0
        check_attention(clean_o[at:at + n], clean_lse[at:at + n], ref, weight_half, d, length, vmax)
        at += n


def poisoned(q):
    x = q.clone()
    for t, h in BAD:
        x[t, h, (5 * t) % x.shape[2]] = float("nan")
    return x.cuda()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16)])
def test_nan_queries_over_the_cache(fmt, d, dtype):
    rng = np.random.default_rng(71)
    q, k, v = random_rows(rng, 8, LENS, 6, 2, d, dtype)
    c = so.Cache(fmt, 2, d, 256, 14)
    table = np.full((2, 12), -1)
    table[0, :1], table[1] = [13], np.arange(12)
    refs = []
    for b, rows in enumerate((slice(0, 100), slice(100, 3100))):
        c.put(table[b], np.arange(LENS[b]), f64(k[rows]), f64(v[rows]))
        kk, vv = c.get(table[b], np.arange(LENS[b]))
        refs.append(so.attention(f64(q[:5] if b == 0 else q[5:]), kk, vv, True))
    cd = ispa.kvq_desc(2, d, 256, 14, FMT[fmt])
    a = ispa.attn_seq_desc(2, 6, 2, d, CODE[dtype], ispa.ISPA_F32)
    o, lse = torch.empty(8, 6, d, device="cuda"), torch.empty(8, 6, device="cuda")
    ws = torch.empty(ispa.ispa_attn_kvq_workspace_bytes(a, cd), dtype=torch.uint8, device="cuda")
    ispa.ispa_attn_kvq(a, cd, poisoned(q), torch.as_tensor(c.buf).cuda(), ints(table), ints(LENS), ints([0, 5, 8]), o, lse,
                       workspace=ws)
    ispa.ispa_check_device_error()
    # (2^-34 of the row's largest weight x |v| a key, which is at most 2^-34 max|v|)
    outputs_are_nan_where_queries_are(o, lse, refs, 2.0 ** -11, d, f64(v).max() * 2.0 ** -9)


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16)])
@pytest.mark.parametrize("causal", [True, False])
def test_nan_queries_of_prompts(d, dtype, causal):
    rng = np.random.default_rng(72)
    q, k, v = random_rows(rng, 8, LENS, 6, 2, d, dtype)
    refs = [so.attention(f64(q[a]), f64(k[b]), f64(v[b]), causal)
            for a, b in ((slice(0, 5), slice(0, 100)), (slice(5, 8), slice(100, 3100)))]
    a = ispa.attn_seq_desc(2, 6, 2, d, CODE[dtype], ispa.ISPA_F32, causal)
    o, lse = torch.empty(8, 6, d, device="cuda"), torch.empty(8, 6, device="cuda")
    ws = torch.empty(ispa.ispa_attn_prompt_workspace_bytes(a), dtype=torch.uint8, device="cuda")
    ispa.ispa_attn_prompt(a, poisoned(q), k.cuda(), v.cuda(), ints([0, 5, 8]), ints([0, 100, 3100]), o, lse, workspace=ws)
    ispa.ispa_check_device_error()
    outputs_are_nan_where_queries_are(o, lse, refs, HALF[dtype], d, f64(v).max() * 2.0 ** -7)


@pytest.mark.parametrize("fmt", list(FMT))
def test_a_scale_times_a_query_below_every_fp32_number(fmt):
    """Scores as good as 0: the mean of the values, with tokens masked in the last tile."""
    rng = np.random.default_rng(73)
    q, k, v = random_rows(rng, 2, [50], 2, 1, 64, torch.bfloat16)
    tiny = (q.float() * 2.0 ** -126).to(torch.bfloat16)
    c = so.Cache(fmt, 1, 64, 64, 1)
    c.put([0], np.arange(50), f64(k), f64(v))
    kk, vv = c.get([0], np.arange(50))
    cd = ispa.kvq_desc(1, 64, 64, 1, FMT[fmt])
    a = ispa.attn_seq_desc(1, 2, 1, 64, ispa.ISPA_BF16, ispa.ISPA_F32, True, 2.0 ** -30)
    o, lse = torch.empty(2, 2, 64, device="cuda"), torch.empty(2, 2, device="cuda")
    ws = torch.empty(ispa.ispa_attn_kvq_workspace_bytes(a, cd), dtype=torch.uint8, device="cuda")
    ispa.ispa_attn_kvq(a, cd, tiny.cuda(), torch.as_tensor(c.buf).cuda(), ints([[0]]), ints([50]), ints([0, 2]), o, lse,
                       workspace=ws)
    ispa.ispa_check_device_error()
    check_attention(o, lse, so.attention(f64(tiny), kk, vv, True, 2.0 ** -30), 2.0 ** -11, 64, 50, np.abs(vv).max() * 2.0 ** -9)
    ap = ispa.attn_seq_desc(1, 2, 1, 64, ispa.ISPA_BF16, ispa.ISPA_F32, True, 2.0 ** -30)
    wp = torch.empty(ispa.ispa_attn_prompt_workspace_bytes(ap), dtype=torch.uint8, device="cuda")
    ispa.ispa_attn_prompt(ap, tiny.cuda(), k.cuda(), v.cuda(), ints([0, 2]), ints([0, 50]), o, lse, workspace=wp)
    ispa.ispa_check_device_error()
    check_attention(o, lse, so.attention(f64(tiny), f64(k), f64(v), True, 2.0 ** -30), 2.0 ** -8, 64, 50, 5.0)
