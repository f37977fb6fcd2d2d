"""GPU tests of the cached attention where items are cut and joined, against a bound that a lost part does not pass."""
import numpy as np
import pytest
import torch

import kv_cache_compression_two_b200 as ispa
from oracle import seq_oracle as so
from seq_bounds import CODE, ints, random_rows, run_cached
from seq_helpers import check_attention, f64, rand16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
def test_items_cut_by_many_sms(fmt):
    rng = np.random.default_rng(8)
    lens, new = [9001, 4097], [1, 5]
    run_cached(rng, fmt, *random_rows(rng, 6, lens, 4, 1, 128, torch.bfloat16, 4.0), lens, new, page=64)


@pytest.mark.parametrize("fmt,d,dtype,G", [("int8", 64, torch.bfloat16, 1), ("e4m3", 128, torch.float16, 3),
                                           ("int4", 64, torch.float16, 13), ("int4", 128, torch.bfloat16, 2)])
def test_items_joined_by_one_two_or_four_ctas(fmt, d, dtype, G):
    """Items of about 6, 18, 36 and 70 parts, and one alone of 150."""
    rng = np.random.default_rng([12, d])
    for lens, new, page in (([700, 2300, 4600, 9000], [1] * 4, 32), ([19001], [2], 256)):
        run_cached(rng, fmt, *random_rows(rng, sum(new), lens, G, 1, d, dtype, 4.0), lens, new, page=page)


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("d,dtype,out,G,H_kv,page", [
    (128, torch.bfloat16, torch.bfloat16, 4, 2, 16), (64, torch.float16, torch.float16, 7, 3, 32),
    (128, torch.float16, torch.float32, 1, 5, 64), (64, torch.bfloat16, torch.float32, 16, 1, 256)])
def test_one_token(fmt, d, dtype, out, G, H_kv, page):
    rng = np.random.default_rng([d, G])
    lens = [1, 15, 16, 17, 31, 32, 33, 300, 1025, 2]
    run_cached(rng, fmt, *random_rows(rng, 10, lens, G * H_kv, H_kv, d, dtype), lens, [1] * 10, out, page=page)


@pytest.mark.parametrize("fmt,d", [("e4m3", 64), ("int8", 128), ("int4", 128), ("int4", 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_several_tokens(fmt, d, causal):
    rng = np.random.default_rng(d)
    lens, new = [2, 50, 200, 0, 700, 1, 64], [2, 0, 7, 1, 16, 3, 40]
    run_cached(rng, fmt, *random_rows(rng, sum(new), lens, 6, 2, d, torch.bfloat16), lens, new, causal=causal, page=16)


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("d,G", [(128, 8), (64, 8), (128, 5)])
def test_a_few_rows_of_padding_change_no_bit(fmt, d, G):
    """A batch of up to 8 rows a sequence takes the same kernel with padding behind it."""
    rng = np.random.default_rng([91, d])
    lens = [int(n) for n in rng.integers(1, 900, 8)]
    q, k, v = random_rows(rng, 8, lens, G, 1, d, torch.bfloat16)
    o, lse = run_cached(np.random.default_rng(0), fmt, q, k, v, lens, [1] * 8)
    more = torch.cat([q, torch.full((3, G, d), float("nan"), dtype=q.dtype)])
    o2, lse2 = run_cached(np.random.default_rng(0), fmt, more, k, v, lens, [1] * 8)
    assert torch.equal(o, o2[:8]) and torch.equal(lse, lse2[:8]) and torch.all(o2[8:] == 7.0) and torch.all(lse2[8:] == 7.0)


def test_prompts_beyond_four_gib():
    """Offsets past 32 bits in q, o, k and v: the last sequence of a call of 4.9 and 4.5 GB tensors."""
    rng = np.random.default_rng(92)
    H, H_kv, d, many_q, many_k, n = 32, 8, 128, 600_000, 2_200_000, 300
    q = torch.zeros(many_q + n, H, d, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(many_k + n, H_kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert 2 * k[:many_k].numel() > 2 ** 32 and q[:many_q].numel() > 2 ** 31
    hq, hk, hv = (rand16(rng, (n, h, d), torch.bfloat16) for h in (H, H_kv, H_kv))
    q[many_q:], k[many_k:], v[many_k:] = hq.cuda(), hk.cuda(), hv.cuda()
    v[:many_k] = 0.5
    a = ispa.attn_seq_desc(3, H, H_kv, d, ispa.ISPA_BF16, ispa.ISPA_BF16)
    o, lse = torch.full_like(q, 7.0), torch.full((many_q + n, H), 7.0, device="cuda")
    ws = torch.empty(ispa.ispa_attn_prompt_workspace_bytes(a), dtype=torch.uint8, device="cuda")
    # one query over 2.2 million keys, many queries without a key, then the sequence that is looked at
    ispa.ispa_attn_prompt(a, q, k, v, ints([0, 1, many_q, many_q + n]), ints([0, many_k, many_k, many_k + n]), o, lse, workspace=ws)
    ispa.ispa_check_device_error()
    check_attention(o[many_q:], lse[many_q:], so.attention(f64(hq), f64(hk), f64(hv), True), 2.0 ** -8, d, n, np.abs(f64(hv)).max())
    assert torch.all(o[1:many_q] == 0) and torch.all(torch.isneginf(lse[1:many_q]))
    # equal scores: the mean of equal values, of weights that are exact
    assert torch.all(o[0] == 0.5) and torch.all((lse[0] - np.log(many_k)).abs() < many_k * 2.0 ** -23)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
def test_joined_prompts_at_every_alignment_allowed(out):
    """O 16-byte but not 32-byte aligned, written by the merge of the parts: the same bits as an aligned one."""
    rng = np.random.default_rng(93)
    dtype = torch.float16 if out is torch.float16 else torch.bfloat16
    q, k, v = (rand16(rng, s, dtype).cuda() for s in ((40, 2, 64), (9000, 1, 64), (9000, 1, 64)))
    a = ispa.attn_seq_desc(1, 2, 1, 64, CODE[dtype], CODE[out])
    ws = torch.empty(ispa.ispa_attn_prompt_workspace_bytes(a), dtype=torch.uint8, device="cuda")
    got = []
    for shift in (0, 16):
        n = shift // torch.empty(0, dtype=out).element_size()
        buf = torch.full((40 * 2 * 64 + 16,), 7.0, dtype=out, device="cuda")
        o = buf[n:n + 40 * 2 * 64].view(40, 2, 64)
        assert o.data_ptr() % 32 == shift
        ispa.ispa_attn_prompt(a, q, k, v, ints([0, 40]), ints([0, 9000]), o, None, workspace=ws)
        assert torch.all(buf[:n] == 7.0) and torch.all(buf[n + 40 * 2 * 64:] == 7.0)
        got.append(o.clone())
    assert torch.equal(*got)
    check_attention(got[0], None, so.attention(f64(q), f64(k), f64(v), True), 2.0 ** -11 if dtype is torch.float16 else 2.0 ** -8,
                    64, 9000, np.abs(f64(v)).max() * 2.0 ** -7)
    ispa.ispa_check_device_error()
