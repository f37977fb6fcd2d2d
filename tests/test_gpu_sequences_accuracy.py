"""GPU tests of the sequence calls' accuracy where values lie far apart: each output against its own query's bound."""
import numpy as np
import pytest
import torch

import kv_cache_compression_two_b200 as ispa
from oracle import seq_oracle as so
from seq_bounds import FMT, ints, random_rows, run_cached
from seq_helpers import check_attention, f64

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ V scales that a query has no use for
@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("d,G,dtype,large,small,nats", [
    (128, 1, torch.bfloat16, 2.0 ** 30, 1.0, 60), (64, 4, torch.bfloat16, 2.0 ** 100, 1.0, 120),
    (128, 16, torch.bfloat16, 2.0 ** 34, 1.0, 60), (64, 3, torch.float16, 2.0 ** 15, 2.0 ** -13, 60)])
@pytest.mark.parametrize("at", [0, 37, 99])
def test_a_large_value_without_weight_takes_no_bits(fmt, d, G, dtype, large, small, nats, at):
    """One token's V is far above the others', and its score far below: it leaves them their bits."""
    rng = np.random.default_rng([d, G, at])
    n = 100
    q, k, v = random_rows(rng, 1, [n], G, 1, d, dtype)
    base = torch.randn(d, generator=torch.Generator().manual_seed(at))
    q = (base + 0.02 * q.float()).to(dtype)
    k = (0.2 * k.float()).to(dtype)
    v = (v.float() * small).to(dtype)
    k[at] = (-nats * d ** 0.5 / float(base @ base) * base).to(dtype)  # a score of about -nats
    v[at] = large
    run_cached(rng, fmt, q, k, v, [n], [1])


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("at", [0, 150, 299])
def test_a_large_value_of_little_weight_beside_the_others(fmt, at):
    """A weight of about 2^-30 on a V of about 2^28: both it and the others count."""
    rng = np.random.default_rng([5, at])
    n, d = 300, 64
    q, k, v = random_rows(rng, 1, [n], 2, 1, d, torch.bfloat16)
    base = torch.randn(d, generator=torch.Generator().manual_seed(at))
    q = (base + 0.02 * q.float()).to(torch.bfloat16)
    k = (0.1 * k.float()).to(torch.bfloat16)
    k[at] = (-21.0 * 8.0 / float(base @ base) * base).to(torch.bfloat16)  # a score of about -21: 2^-30
    v[at] = (v[at].float() * 2.0 ** 28).to(torch.bfloat16)
    run_cached(rng, fmt, q, k, v, [n], [1])


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("G,large", [(1, 2.0 ** 24), (3, 2.0 ** 40)])
def test_a_later_token_takes_no_bits_of_an_earlier_query(fmt, G, large):
    """The newest tokens' V are large: the queries before them do not see them."""
    rng = np.random.default_rng([6, G])
    lens, new = [40, 333, 3, 2000], [4, 6, 3, 2]
    q, k, v = random_rows(rng, sum(new), lens, 2 * G, 2, 128, torch.bfloat16)
    for end in np.cumsum(lens):
        v[end - 1] = (v[end - 1].float() * large).to(torch.bfloat16)
    run_cached(rng, fmt, q, k, v, lens, new)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("order", [1, -1])
def test_values_that_grow_or_shrink_as_the_scores_do(fmt, order):
    """V over 2^80 and scores over 2^60 of weight, with and against each other, in one cache of many tiles."""
    n, d = 1500, 64
    for both in (1, -1):
        rng = np.random.default_rng([7, order + 1, both + 1])
        q, k, v = random_rows(rng, 2, [n], 1, 1, d, torch.bfloat16)
        base = torch.randn(d, generator=torch.Generator().manual_seed(1))
        q = base.expand(2, 1, d).to(torch.bfloat16)
        ramp = torch.linspace(-1.0, 1.0, n)[:, None, None] * order
        k = (ramp * 21.0 * 8.0 / float(base @ base) * base + 0.05 * k.float()).to(torch.bfloat16)
        v = (v.float() * torch.exp2(both * 40.0 * ramp)).to(torch.bfloat16)
        run_cached(rng, fmt, q, k, v, [n], [2])


def test_rows_of_zeros_among_the_values():
    """V rows that are stored as zeros, first, last and alone."""
    rng = np.random.default_rng(8)
    for zero in (slice(0, 64), slice(100, 200), slice(0, 200)):
        q, k, v = random_rows(rng, 1, [200], 2, 1, 64, torch.bfloat16)
        v[zero] = 0
        for fmt in FMT:
            run_cached(rng, fmt, q, k, v, [200], [1])


@pytest.mark.parametrize("fmt", list(FMT))
def test_values_at_the_ends_of_the_type(fmt):
    """All of V near bf16's largest magnitude, or near the least that is stored."""
    rng = np.random.default_rng(9)
    q, k, v = random_rows(rng, 1, [100], 4, 2, 128, torch.bfloat16)
    big = (v.float() / v.float().abs().max() * 2.0 ** 120).to(torch.bfloat16)
    run_cached(rng, fmt, q, k, big, [100], [1])
    o, _ = run_cached(rng, fmt, q, k, (v.float() * 2.0 ** -80).to(torch.bfloat16), [100], [1])
    want, _ = run_cached(rng, fmt, q, k, v, [100], [1])
    assert torch.allclose(o * 2.0 ** 80, want, rtol=2.0 ** -9, atol=2.0 ** -14)


# ------------------------------------------------------------------ prompts: small weights of fp16
@pytest.mark.parametrize("d,first,n,nq", [(64, True, 6000, 3), (128, False, 6000, 300), (128, True, 700, 40), (64, False, 40, 1)])
@pytest.mark.parametrize("log2", [-18, -26])
@pytest.mark.parametrize("causal", [True, False])
def test_small_weights_of_a_prompt_add_up(d, first, n, nq, log2, causal):
    """One key holds nearly all of the weight and no value; many of weight 2^log2 hold the output.

    A weight is off by 2^-11 of itself or by 2^-25 in units in which the row's largest is at least
    2^7: 2^-32 max|v| a key."""
    rng = np.random.default_rng([n, d, -log2])
    q, k, v = random_rows(rng, nq, [n], 2, 1, d, torch.float16)
    base = torch.randn(d, generator=torch.Generator().manual_seed(3))
    q = base.expand(nq, 2, d).to(torch.float16)
    k = (0.02 * k.float() + log2 * np.log(2.0) * d ** 0.5 / float(base @ base) * base).to(torch.float16)
    v = v.float().abs().add(0.5).to(torch.float16)
    one = 0 if first else n - nq
    k[one], v[one] = 0, 0
    a = ispa.attn_seq_desc(1, 2, 1, d, ispa.ISPA_F16, ispa.ISPA_F32, causal)
    o, lse = torch.empty(nq, 2, d, device="cuda"), torch.empty(nq, 2, device="cuda")
    ws = torch.empty(ispa.ispa_attn_prompt_workspace_bytes(a), dtype=torch.uint8, device="cuda")
    ispa.ispa_attn_prompt(a, q.cuda(), k.cuda(), v.cuda(), ints([0, nq]), ints([0, n]), o, lse, workspace=ws)
    ispa.ispa_check_device_error()
    ref = so.attention(f64(q), f64(k), f64(v), causal)
    check_attention(o, lse, ref, 2.0 ** -11, d, n, f64(v).max() * 2.0 ** -7)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,nq", [(300, 1), (3000, 2)])
def test_values_at_the_end_of_fp16_stay_finite(d, n, nq):
    """One late key holds nearly all of the weight, which fp16 rounds up by almost 2^-11: O is still V's largest.

    Weights are 2^7 for the first tile's largest and 2^12 * 1.0005 for the late key (fp16: 2^12 * (1 + 2^-10)),
    so that the mean comes to 65504 (1 + 2^-11.1), above 65520, where rounding to fp16 gives infinity."""
    q, k = torch.zeros(nq, 1, d, dtype=torch.float16), torch.zeros(n, 1, d, dtype=torch.float16)
    q[:, :, 0], k[:, :, 0] = 2.0, -60.0
    k[0, 0, 0], k[n - nq, 0, 0] = 0.0, 4.0
    v = torch.full((n, 1, d), 65504.0, dtype=torch.float16)
    v[:, :, 1::2] *= -1.0
    scale = (5.0 + np.log2(1.0005)) * np.log(2.0) / 8.0
    a = ispa.attn_seq_desc(1, 1, 1, d, ispa.ISPA_F16, ispa.ISPA_F16, False, scale)
    o, ws = torch.empty_like(q, device="cuda"), torch.empty(ispa.ispa_attn_prompt_workspace_bytes(a), dtype=torch.uint8, device="cuda")
    ispa.ispa_attn_prompt(a, q.cuda(), k.cuda(), v.cuda(), ints([0, nq]), ints([0, n]), o, None, workspace=ws)
    ispa.ispa_check_device_error()
    assert torch.equal(o.cpu(), v[:1].expand(nq, 1, d))
