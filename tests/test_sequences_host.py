"""CPU tests of the sequence calls: layouts, refusals before any CUDA call, and pins of the 64-bit oracle."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

import kv_cache_compression_two_b200 as ispa
from oracle import seq_oracle as so

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
L = ispa.lib()
INVALID, UNSUPPORTED = ispa.ISPA_ERR_INVALID_ARG, ispa.ISPA_ERR_UNSUPPORTED


def cache(**kw):
    return ispa.KvqDesc(**(dict(H_kv=2, head_dim=128, page_tokens=16, n_pages=8, fmt=ispa.ISPA_KVQ_INT8) | kw))


def attn(**kw):
    return ispa.AttnSeqDesc(**(dict(B=2, H=8, H_kv=2, head_dim=128, in_dtype=ispa.ISPA_BF16, out_dtype=ispa.ISPA_BF16,
                                    causal=1, softmax_scale=0.0) | kw))


def last():
    return L.ispa_last_error().decode()


def write(d=None, **kw):
    a = dict(B=2, T=4, table=FAKE, max_pages=3, lens=FAKE, cu=FAKE, k=FAKE, ks=256, v=FAKE, vs=256, dt=ispa.ISPA_BF16,
             kvq=FAKE) | kw
    return L.ispa_kvq_write(ctypes.byref(d or cache()), *a.values(), None)


def read(d=None, **kw):
    a = dict(B=2, T=4, table=FAKE, max_pages=3, begin=None, cu=FAKE, kvq=FAKE, ko=FAKE, vo=FAKE, dt=ispa.ISPA_F16) | kw
    return L.ispa_kvq_read(ctypes.byref(d or cache()), *a.values(), None)


def attn_kvq(ad=None, cd=None, **kw):
    a = dict(T=4, cu=FAKE, table=FAKE, max_pages=3, lens=FAKE, q=FAKE, qs=1024, kvq=FAKE, o=FAKE, lse=FAKE, ws=FAKE,
             wb=1 << 40) | kw
    return L.ispa_attn_kvq(ctypes.byref(ad or attn()), ctypes.byref(cd or cache()), *a.values(), None)


def prompt(ad=None, **kw):
    a = dict(Tq=4, Tk=4, cq=FAKE, ck=FAKE, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, o=FAKE, lse=FAKE, ws=FAKE,
             wb=1 << 40) | kw
    return L.ispa_attn_prompt(ctypes.byref(ad or attn()), *a.values(), None)


def test_descriptors_match_the_header():
    text = open(os.path.join(ROOT, "include", "ispa.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, cls in (("ispa_kvq_desc", ispa.KvqDesc), ("ispa_attn_seq_desc", ispa.AttnSeqDesc)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
        fields = [f.strip() for line in body.split(";") if line.strip() for f in line.split(None, 1)[1].split(",")]
        assert fields == [f for f, _ in cls._fields_]


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("d", [64, 128])
def test_cache_bytes_match_the_oracle_layout(fmt, d):
    code = {"e4m3": ispa.ISPA_KVQ_E4M3, "int8": ispa.ISPA_KVQ_INT8, "int4": ispa.ISPA_KVQ_INT4}[fmt]
    for page, pages, H_kv in ((16, 1, 1), (32, 7, 3), (256, 5, 12)):
        want = so.Cache(fmt, H_kv, d, page, pages).buf.size
        assert L.ispa_kvq_bytes(ctypes.byref(cache(H_kv=H_kv, head_dim=d, page_tokens=page, n_pages=pages, fmt=code))) == want


@pytest.mark.parametrize("kw,frag", [
    (dict(H_kv=0), "H_kv"), (dict(n_pages=0), "n_pages"), (dict(head_dim=96), "head_dim"), (dict(page_tokens=8), "page_tokens"),
    (dict(page_tokens=48), "page_tokens"), (dict(page_tokens=512), "page_tokens"), (dict(fmt=3), "format"), (dict(fmt=-1), "format")])
def test_bad_caches_are_refused(kw, frag):
    d = cache(**kw)
    assert L.ispa_kvq_bytes(ctypes.byref(d)) == 0
    for call in (write, read):
        assert call(d) == INVALID and frag in last()
    assert attn_kvq(cd=d) == INVALID and frag in last()
    assert L.ispa_attn_kvq_workspace_bytes(ctypes.byref(attn()), ctypes.byref(d)) == 0


@pytest.mark.parametrize("kw,frag", [
    (dict(B=0), "B"), (dict(T=-1), "rows"), (dict(table=None), "block_table"), (dict(max_pages=0), "max_pages"),
    (dict(max_pages=1 << 30), "max_pages"), (dict(lens=None), "int32"), (dict(cu=FAKE + 2), "int32"), (dict(k=None), "aligned"),
    (dict(v=FAKE + 8), "aligned"), (dict(kvq=FAKE + 4), "aligned"), (dict(ks=255), "stride"), (dict(ks=128), "stride"),
    (dict(vs=260), "stride"), (dict(dt=ispa.ISPA_F32), "dtype"), (dict(dt=9), "dtype")])
def test_bad_writes_are_refused(kw, frag):
    assert write(**kw) == INVALID and frag in last()


@pytest.mark.parametrize("kw,frag", [
    (dict(B=0), "B"), (dict(T=-3), "rows"), (dict(table=None), "block_table"), (dict(begin=FAKE + 1), "int32"), (dict(cu=None), "int32"),
    (dict(ko=None), "aligned"), (dict(vo=FAKE + 2), "aligned"), (dict(kvq=None), "aligned"), (dict(dt=ispa.ISPA_F32), "dtype")])
def test_bad_reads_are_refused(kw, frag):
    assert read(**kw) == INVALID and frag in last()


@pytest.mark.parametrize("kw,frag", [
    (dict(B=0), "B"), (dict(H=7), "multiple"), (dict(H_kv=0), "H_kv"), (dict(H=258), "at most 128"), (dict(head_dim=32), "head_dim"),
    (dict(in_dtype=5), "in_dtype"), (dict(out_dtype=ispa.ISPA_F16), "out_dtype"), (dict(causal=2), "causal"),
    (dict(softmax_scale=math.inf), "softmax_scale")])
def test_bad_attentions_are_refused(kw, frag):
    d = attn(**kw)
    assert attn_kvq(d) == INVALID and frag in last()
    assert prompt(d) == INVALID and frag in last()
    assert L.ispa_attn_prompt_workspace_bytes(ctypes.byref(d)) == 0


def test_fp32_inputs_are_unsupported():
    d = attn(in_dtype=ispa.ISPA_F32, out_dtype=ispa.ISPA_F32)
    assert attn_kvq(d) == UNSUPPORTED and prompt(d) == UNSUPPORTED


@pytest.mark.parametrize("call,kw,frag", [
    (attn_kvq, dict(cd=cache(H_kv=4)), "heads"), (attn_kvq, dict(cd=cache(head_dim=64)), "heads"), (attn_kvq, dict(qs=1000), "stride"),
    (attn_kvq, dict(q=None), "aligned"), (attn_kvq, dict(o=FAKE + 8), "aligned"), (attn_kvq, dict(lse=FAKE + 2), "aligned"),
    (attn_kvq, dict(ws=None), "workspace"), (attn_kvq, dict(wb=64), "workspace"), (attn_kvq, dict(lens=None), "int32"),
    (prompt, dict(Tk=-1), "rows"), (prompt, dict(Tq=-1), "rows"), (prompt, dict(ks=128), "stride"), (prompt, dict(vs=257), "stride"),
    (prompt, dict(k=None), "aligned"), (prompt, dict(ck=None), "int32"), (prompt, dict(ws=FAKE + 8), "workspace"), (prompt, dict(wb=0), "workspace")])
def test_bad_attention_arguments_are_refused(call, kw, frag):
    assert call(**kw) == INVALID and frag in last()


def test_nothing_to_do_is_no_error():
    """T == 0 launches nothing (there is no GPU here)."""
    assert write(T=0, k=None, v=None) == ispa.ISPA_OK
    assert read(T=0, ko=None, vo=None) == ispa.ISPA_OK
    assert attn_kvq(T=0, q=None, o=None) == ispa.ISPA_OK
    assert prompt(Tq=0, q=None, o=None) == ispa.ISPA_OK


def test_other_calls_do_not_take_fp16():
    assert L.ispa_lse_merge(10, 2, 64, ispa.ISPA_F16, *([FAKE] * 6), None) == INVALID
    assert L.ispa_absorb_weight(64, 64, FAKE, ispa.ISPA_F16, FAKE, FAKE, ispa.ISPA_BF16, None) == INVALID


# ------------------------------------------------------------------ the oracle
def test_e4m3_codes_against_the_definition():
    import torch
    grid = so.e4m3_grid()
    for c in range(127):
        assert so.e4m3_codes(grid[c]) == c and so.e4m3_codes(-grid[c]) == c + 128
    x = np.concatenate([np.linspace(-460, 460, 20001), np.linspace(-0.03, 0.03, 4001),
                        (grid[:126] + grid[1:127]) / 2]).astype(np.float32)
    want = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(so.e4m3_codes(x), want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
def test_quantise_worked_values(fmt):
    x = np.zeros((1, 64))
    x[0, :4] = [2.0, -1.0, 0.5, 0.0]
    x[0, 32:34] = [0.25, 0.125]
    codes, rec = so.quantise(fmt, x)
    back = so.dequantise(fmt, codes, rec)[0]
    if fmt == "int8":
        assert codes.view(np.int8)[0, :4].tolist() == [127, -64, 32, 0]  # 63.5 and 31.75 to even / nearest
        assert np.allclose(back[:2], [2.0, -64 * 2 / 127])
    elif fmt == "e4m3":
        assert back[:4].tolist() == [2.0, -1.0, 0.5, 0.0] and back[32] == 0.25
    else:
        # group 0: g = 448, step 2/7; -3.5 -> -4, 1.75 -> 2; group 1: g = 56, step 0.25 / 7
        assert rec[0, 4:].tolist() == [126, int(so.e4m3_codes(56.0)), 0, 0, 0, 0][:4] and codes[0, 0] == (15 | (4 << 4))
        assert np.allclose(back[:4], [2.0, -8 / 7, 4 / 7, 0.0]) and np.isclose(back[32], 0.25) and np.isclose(back[33], 1 / 7)


@pytest.mark.parametrize("fmt,step", [("e4m3", 2.0 ** -4), ("int8", 0.5 / 127), ("int4", 0.5 / 7)])
def test_quantise_error_is_half_a_step(fmt, step):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 128)).astype(np.float16).astype(np.float64)
    back = so.dequantise(fmt, *so.quantise(fmt, x)).astype(np.float64)
    if fmt == "e4m3":  # relative to the value, or half the smallest step of the scale
        bound = step * np.abs(x) + np.abs(x).max(-1, keepdims=True) / 448 * 2.0 ** -10
    elif fmt == "int8":
        bound = step * np.abs(x).max(-1, keepdims=True)
    else:  # of the group's largest; its factor's rounding (2^-4) widens the step or clips the largest
        top = np.abs(x.reshape(200, 4, 32)).max(-1, keepdims=True)
        bound = np.broadcast_to(top * max(step * (1 + 2.0 ** -4), 2.0 ** -4), (200, 4, 32)).reshape(x.shape)
    # The scale and the product are rounded to fp32: 2 * 2^-24 of a value that is at most 254 half steps of int8
    # (fewer of the others), so a value halfway between two codes may be off by (1 + 254 * 2^-23) half steps.
    assert np.all(np.abs(back - x) <= bound * (1 + 254 * 2.0 ** -23))
    zero = so.dequantise(fmt, *so.quantise(fmt, np.full((3, 64), 2.0 ** -97)))
    assert np.all(zero == 0)


def test_attention_oracle_against_loops():
    rng = np.random.default_rng(1)
    n, length, H, H_kv, d = 3, 5, 4, 2, 8
    q, k, v = rng.standard_normal((n, H, d)), rng.standard_normal((length, H_kv, d)), rng.standard_normal((length, H_kv, d))
    for causal in (True, False):
        o, lse, absv, size = so.attention(q, k, v, causal)
        for i in range(n):
            for h in range(H):
                keys = range(length - n + i + 1) if causal else range(length)
                s = [sum(q[i, h, c] * k[j, h // 2, c] for c in range(d)) / math.sqrt(d) for j in keys]
                w = [math.exp(x) for x in s]
                assert math.isclose(lse[i, h], math.log(sum(w)), rel_tol=1e-12)
                for c in range(d):
                    assert math.isclose(o[i, h, c], sum(a * v[j, h // 2, c] for a, j in zip(w, keys)) / sum(w), rel_tol=1e-9, abs_tol=1e-12)
    o, lse, _, _ = so.attention(q, k[:1], v[:1], True)  # the first two queries see nothing
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.allclose(o[2, 0], v[0, 0])
    o, lse, _, _ = so.attention(q, k[:0], v[:0], False)
    assert np.all(o == 0) and np.all(np.isneginf(lse))


def test_binding_names_an_argument_that_is_no_tensor():
    torch = pytest.importorskip("torch")
    ispa._seq_init()
    d = cache()
    buf = torch.zeros(ispa.ispa_kvq_bytes(d), dtype=torch.uint8)
    table = torch.zeros(2, 3, dtype=torch.int32)
    assert ispa._cache(d, buf, table, 2, -1) == (buf.data_ptr(), table.data_ptr(), 3)
    for kvq, tab, name in ((None, table, "kvq"), (buf, [[0]], "block_table")):
        with pytest.raises(TypeError, match=name):
            ispa._cache(d, kvq, tab, 2, -1)
    with pytest.raises(ValueError, match="block_table"):
        ispa._cache(d, buf, table.view(-1), 2, -1)
    with pytest.raises(ValueError, match="block_table"):
        ispa._cache(d, buf, table, 3, -1)
    with pytest.raises(TypeError, match="workspace"):
        ispa._outputs(attn(), 1, torch.zeros(1, 8, 128, dtype=torch.bfloat16), None, 4096, -1)
