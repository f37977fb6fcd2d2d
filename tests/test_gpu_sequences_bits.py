"""GPU tests: the sequence calls' bits depend on nothing but their own inputs."""
import numpy as np
import pytest
import torch

import kv_cache_compression_two_b200 as ispa
from seq_bounds import CODE, FMT, ints
from seq_helpers import paged, rand16, starts

pytestmark = pytest.mark.gpu


def prompt_call(H, H_kv, d, dtype, lens_q, lens_k, causal, q, k, v):
    a = ispa.attn_seq_desc(len(lens_q), H, H_kv, d, CODE[dtype], ispa.ISPA_F32, causal)
    ws = torch.empty(ispa.ispa_attn_prompt_workspace_bytes(a), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty(sum(lens_q), H, d, device="cuda"), torch.empty(sum(lens_q), H, device="cuda")
    ispa.ispa_attn_prompt(a, q, k, v, ints(starts(lens_q)), ints(starts(lens_k)), o, lse, workspace=ws)
    return o, lse


def leave_large_values(d, dtype):
    """A call whose queries fill every SM's shared memory with values far above those of the calls under test."""
    q = torch.randn(148 * 256, 1, d, device="cuda").mul_(100.0).to(dtype)
    k = torch.randn(300, 1, d, device="cuda").to(dtype)
    prompt_call(1, 1, d, dtype, [q.shape[0]], [300], False, q, k, k)


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16)])
@pytest.mark.parametrize("G", [1, 3, 7, 100])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_do_not_depend_on_earlier_calls(d, dtype, G, causal):
    """Groups that do not divide 128 leave rows of a tile unloaded."""
    rng = np.random.default_rng([81, G])
    nq, nk = [371, 40, 300], [900, 40, 299]
    if G == 100:
        nq = [20, 3, 9]
    q, k, v = (rand16(rng, (n, h, d), dtype).cuda() for n, h in ((sum(nq), 2 * G), (sum(nk), 2), (sum(nk), 2)))
    first = prompt_call(2 * G, 2, d, dtype, nq, nk, causal, q, k, v)
    for _ in range(3):
        leave_large_values(d, dtype)
        again = prompt_call(2 * G, 2, d, dtype, nq, nk, causal, q, k, v)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    ispa.ispa_check_device_error()


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16)])
@pytest.mark.parametrize("factor", [100.0, float("nan"), float("inf")])
def test_prompts_do_not_depend_on_a_neighbours_queries(d, dtype, factor):
    """The rows behind a sequence's last one in its tile are the next sequence's."""
    rng = np.random.default_rng(82)
    nq, nk = [70, 33, 90], [700, 300, 900]
    q, k, v = (rand16(rng, (n, h, d), dtype).cuda() for n, h in ((sum(nq), 2), (sum(nk), 1), (sum(nk), 1)))
    other = q.clone()
    other[70:103] = other[70:103] * factor
    one, two = (prompt_call(2, 1, d, dtype, nq, nk, True, x, k, v) for x in (q, other))
    for rows in (slice(0, 70), slice(103, 193)):
        assert torch.equal(one[0][rows], two[0][rows]) and torch.equal(one[1][rows], two[1][rows])
    ispa.ispa_check_device_error()


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("d,G,dtype", [(128, 3, torch.bfloat16), (64, 7, torch.float16), (128, 1, torch.float16)])
def test_cached_attention_does_not_depend_on_earlier_calls_or_neighbours(fmt, d, G, dtype):
    rng = np.random.default_rng([83, d, G])
    lens, new = [900, 33, 2500, 1], [3, 1, 5, 1]
    H_kv, page = 2, 32
    table, pages = paged(rng, lens, page)
    cd = ispa.kvq_desc(H_kv, d, page, pages, FMT[fmt])
    kvq = torch.empty(ispa.ispa_kvq_bytes(cd), dtype=torch.uint8, device="cuda").fill_(0x7F)
    kv = [rand16(rng, (sum(lens), H_kv, d), dtype).cuda() for _ in range(2)]
    ispa.ispa_kvq_write(cd, *kv, ints(table), ints(lens), ints(starts(lens)), kvq)
    q = rand16(rng, (sum(new), G * H_kv, d), dtype).cuda()
    other = q.clone()
    other[3:4] = float("nan")
    a = ispa.attn_seq_desc(4, G * H_kv, H_kv, d, CODE[dtype], ispa.ISPA_F32)
    ws = torch.empty(ispa.ispa_attn_kvq_workspace_bytes(a, cd), dtype=torch.uint8, device="cuda")
    got = []
    for x in (q, q, other):
        ws.fill_(0xFF)
        leave_large_values(d, dtype)
        o, lse = torch.empty(sum(new), G * H_kv, d, device="cuda"), torch.empty(sum(new), G * H_kv, device="cuda")
        ispa.ispa_attn_kvq(a, cd, x, kvq, ints(table), ints(lens), ints(starts(new)), o, lse, workspace=ws)
        got.append((o, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for rows in (slice(0, 3), slice(4, 10)):
        assert torch.equal(got[0][0][rows], got[2][0][rows]) and torch.equal(got[0][1][rows], got[2][1][rows])
    ispa.ispa_check_device_error()
