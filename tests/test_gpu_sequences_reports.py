"""GPU tests of the sequence calls' reports: bounds out of range are named, and touch nothing that they do not own."""
import numpy as np
import pytest
import torch

import kv_cache_compression_two_b200 as ispa
from oracle import seq_oracle as so
from seq_bounds import ints
from seq_helpers import check_attention, f64, rand16

pytestmark = pytest.mark.gpu


def reported():
    """The sequence in the error word (cleared by this), or None.  (No exception is kept: see the older tests.)"""
    try:
        ispa.ispa_check_device_error()
    except ispa.IspaError as e:
        assert e.status == ispa.ISPA_ERR_INVALID_ARG
        return int(str(e).split("sequence ")[1].split()[0])
    return None


# ------------------------------------------------------------------ prompts
@pytest.mark.parametrize("cu_q,cu_k,bad", [([0, 30, 30, 50], [0, 30, 9999, 9999], (1, 2)), ([0, 30, 70, 70], [0, 30, 35, 40], (1, 2)),
                                           ([0, 30, 35, 20], [0, 30, 35, 40], (2,)), ([-3, 30, 35, 40], [0, 30, 35, 40], (0,)),
                                           ([0, 30, 35, 40], [0, 30, 35, -1], (2,)), ([0, 30, 35, 40], [0, 30, 35, 40], None)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_name_a_bad_bound(cu_q, cu_k, bad, causal):
    rng = np.random.default_rng(52)
    k, v = (rand16(rng, (40, 1, 64), torch.bfloat16) for _ in range(2))
    q = rand16(rng, (40, 2, 64), torch.bfloat16)
    a = ispa.attn_seq_desc(3, 2, 1, 64, ispa.ISPA_BF16, ispa.ISPA_F32, causal)
    ws = torch.empty(ispa.ispa_attn_prompt_workspace_bytes(a), dtype=torch.uint8, device="cuda")
    o = torch.empty(40, 2, 64, device="cuda")
    assert reported() is None
    ispa.ispa_attn_prompt(a, q.cuda(), k.cuda(), v.cuda(), ints(cu_q), ints(cu_k), o, None, workspace=ws)
    got = reported()
    assert got in bad if bad else got is None
    if cu_q[0] == 0 and (not bad or 0 not in bad) and cu_q[3] != 20:  # (a later sequence that overlaps writes there too)
        check_attention(o[:30], None, so.attention(f64(q[:30]), f64(k[:30]), f64(v[:30]), causal), 2.0 ** -8, 64, 30, 5.0)


@pytest.mark.parametrize("lens,cu,bad", [([30, -7, 30], [0, 1, 2, 3], (1,)), ([30, 30, 5], [0, 1, 2, 900], (2,)),
                                         ([30, 30, 30], [0, 1, 2, -4], (2,)), ([30, 33, 30], [0, 1, 2, 3], (1,)),
                                         ([30, 30, 30], [0, 1, 2, 3], None)])
def test_cached_attention_names_a_bad_bound(lens, cu, bad):
    rng = np.random.default_rng(53)
    cd = ispa.kvq_desc(1, 64, 16, 6, ispa.ISPA_KVQ_INT8)
    kvq = torch.zeros(ispa.ispa_kvq_bytes(cd), dtype=torch.uint8, device="cuda")
    a = ispa.attn_seq_desc(3, 2, 1, 64, ispa.ISPA_BF16, ispa.ISPA_F32)
    ws = torch.empty(ispa.ispa_attn_kvq_workspace_bytes(a, cd), dtype=torch.uint8, device="cuda")
    q, o = rand16(rng, (3, 2, 64), torch.bfloat16).cuda(), torch.empty(3, 2, 64, device="cuda")
    assert reported() is None
    ispa.ispa_attn_kvq(a, cd, q, kvq, ints([[0, 1], [2, 3], [4, 5]]), ints(lens), ints(cu), o, None, workspace=ws)
    got = reported()
    assert got in bad if bad else got is None


# ------------------------------------------------------------------ the cache
def test_decreasing_bounds_write_nothing_past_a_sequence():
    """Rows 2..7 lie in no sequence, but a search that takes the bounds as ascending ends at the last one."""
    k = rand16(np.random.default_rng(56), (8, 1, 64), torch.bfloat16).cuda()
    cd = ispa.kvq_desc(1, 64, 16, 3, ispa.ISPA_KVQ_INT8)
    c = so.Cache("int8", 1, 64, 16, 3, fill=0xAB)
    kvq = torch.as_tensor(c.buf.copy()).cuda()
    ispa.ispa_kvq_write(cd, k, k, ints([[0], [1], [2]]), ints([8, 8, 8]), ints([0, 8, 1, 2]), kvq)
    reported()
    c.buf[:] = kvq.cpu().numpy()
    for which in range(4):
        assert np.all(c.parts[which][:, :, 8:] == 0xAB)


BAD_BOUNDS = [([0, 4, 4, 9], (2,)), ([0, 4, 8, 3], (2,)), ([0, 8, 1, 2], (1,)), ([-2, 4, 6, 8], (0,)), ([9, 9, 9, 9], (0, 1, 2)),
              ([0, 8, 8, -1], (2,)), ([0, 5, 3, 8], (1,)), ([0, 4, 6, 8], None), ([0, 0, 0, 0], None), ([2, 3, 3, 7], None)]


def rows_of(cu, T):
    """Rows that each sequence may own (its bounds clamped to the tensor)."""
    return [range(min(max(a, 0), T), min(max(b, 0), T)) for a, b in zip(cu, cu[1:])]


@pytest.mark.parametrize("cu,bad", BAD_BOUNDS)
def test_writing_names_a_bad_bound_and_stays_inside_the_sequences(cu, bad):
    """Sequences that own no row are looked at too; a position past a sequence's length is never written."""
    rng = np.random.default_rng(54)
    T, page, lens = 8, 16, [10, 9, 8]
    cd = ispa.kvq_desc(1, 64, page, 8, ispa.ISPA_KVQ_INT8)
    c = so.Cache("int8", 1, 64, page, 8, fill=0xAB)
    kvq, k = torch.as_tensor(c.buf.copy()).cuda(), rand16(rng, (T, 1, 64), torch.bfloat16).cuda()
    table = np.asarray([[3, 7], [5, 0], [6, 1]])
    assert reported() is None
    ispa.ispa_kvq_write(cd, k, k, ints(table), ints(lens), ints(cu), kvq)
    got = reported()
    assert got in bad if bad else got is None
    c.buf[:] = kvq.cpu().numpy()
    for b, n in enumerate(lens):
        for which in range(4):
            assert np.all(c.parts[which][table[b, 0], :, n:] == 0xAB) and np.all(c.parts[which][table[b, 1]] == 0xAB)
    if not bad:
        for b, rows in enumerate(rows_of(cu, T)):
            pos = np.arange(lens[b] - len(rows), lens[b])
            want = so.quantise("int8", f64(k[rows.start:rows.stop]))[0]
            assert np.array_equal(c.parts[0][table[b, 0], :, pos].reshape(-1, 64), want.reshape(-1, 64))


@pytest.mark.parametrize("cu,bad", BAD_BOUNDS)
def test_reading_names_a_bad_bound(cu, bad):
    rng = np.random.default_rng(55)
    T, page = 8, 16
    cd = ispa.kvq_desc(1, 64, page, 8, ispa.ISPA_KVQ_E4M3)
    c = so.Cache("e4m3", 1, 64, page, 8)
    table = np.asarray([[3, 7], [5, 0], [6, 1]])
    for b in range(3):
        c.put(table[b], np.arange(32), *(f64(rand16(rng, (32, 1, 64), torch.bfloat16)) for _ in range(2)))
    out = [torch.full((T, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert reported() is None
    ispa.ispa_kvq_read(cd, torch.as_tensor(c.buf).cuda(), ints(table), ints(cu), *out)
    got = reported()
    assert got in bad if bad else got is None
    if not bad:
        owned = np.zeros(T, bool)
        for b, rows in enumerate(rows_of(cu, T)):
            owned[rows.start:rows.stop] = True
            for x, want in zip(out, c.get(table[b], np.arange(len(rows)))):
                assert torch.equal(x[rows.start:rows.stop].cpu(), torch.from_numpy(want).to(torch.bfloat16))
        assert torch.all(out[0][torch.from_numpy(~owned).cuda()] == 7.0)


def test_reading_names_a_position_without_a_page():
    cd = ispa.kvq_desc(1, 64, 16, 4, ispa.ISPA_KVQ_INT4)
    kvq = torch.zeros(ispa.ispa_kvq_bytes(cd), dtype=torch.uint8, device="cuda")
    for begin, bad in (([0, 31, 0], 1), ([0, 0, -1], 2), ([30, 30, 30], None)):
        out = [torch.full((6, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        assert reported() is None
        ispa.ispa_kvq_read(cd, kvq, ints([[0, 1], [1, 2], [2, 3]]), ints([0, 2, 4, 6]), *out, seq_begin=ints(begin))
        assert reported() == bad
        assert torch.all(out[0] == 0) and torch.all(out[1] == 0)
