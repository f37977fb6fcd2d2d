"""A bound of the cached attention's outputs that follows each query, and a runner that uses it.

The weights of the second product are fp16 numbers in units in which the row's
largest p * s (softmax weight times the token's V scale) is at least 2^9, so that
one below fp16's normal numbers is off by at most 2^-25 / 2^9 = 2^-34 of that
largest, and its token's values are at most s * (largest code) = the row's amax
of V.  Over N keys that is N 2^-34 max_j(p_j amax_j): seq_helpers.check_attention
takes it as N 2^-25 times the array that smallest_step() returns.  (fp16 inputs
enter as two fp16 numbers, of which the second one has the same smallest step.)

The allowance of 2^-18 max|v| a key that seq_helpers names for the cached attention
(and that tests pass as max|v| * 2^7) has the wrong sign of exponent: it exceeds the
whole output of a long cache, so that those tests pin O by short caches and long ones
by the log-sum-exp alone.  The tests that use this file pin O at every length.
"""
import numpy as np
import torch

import kv_cache_compression_two_b200 as ispa
from oracle import seq_oracle as so
from seq_helpers import check_attention, f64, paged, rand16, starts

FMT = {"e4m3": ispa.ISPA_KVQ_E4M3, "int8": ispa.ISPA_KVQ_INT8, "int4": ispa.ISPA_KVQ_INT4}
CODE = {torch.bfloat16: ispa.ISPA_BF16, torch.float16: ispa.ISPA_F16, torch.float32: ispa.ISPA_F32}


def smallest_step(q, k, v, causal, scale=None):
    """2^-9 max_j(p_j amax(v_j)) of each query and head, [n, H, 1], for check_attention's vmax."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, H, d = q.shape
    length, H_kv = k.shape[:2]
    out = np.zeros((n, H, 1))
    if not n or not length:
        return out
    amax = np.abs(v).max(-1)
    seen = np.ones((n, length), bool)
    if causal:
        seen = np.arange(length)[None, :] <= np.arange(n)[:, None] + (length - n)
    for h in range(H):
        s = np.where(seen, (scale or 1.0 / np.sqrt(d)) * (q[:, h] @ k[:, h // (H // H_kv)].T), -np.inf)
        m = s.max(-1, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
        total = p.sum(-1, keepdims=True)
        w = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
        out[:, h, 0] = 2.0 ** -9 * (w * amax[:, h // (H // H_kv)]).max(-1)
    return out


def ints(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def run_cached(rng, fmt, q, k, v, lens, new, out=torch.float32, causal=True, page=32, scale=0.0):
    """Attention of packed q over caches of the packed k, v (16-bit tensors), every output within its query's bound."""
    B, (T, H, d), H_kv, dtype = len(lens), q.shape, k.shape[1], q.dtype
    table, pages = paged(rng, lens, page)
    c = so.Cache(fmt, H_kv, d, page, pages, fill=0x7F)  # unwritten bytes are NaN codes
    ck, cq = starts(lens), starts(new)
    for b, n in enumerate(lens):
        if n:
            c.put(table[b], np.arange(n), f64(k[ck[b]:ck[b + 1]]), f64(v[ck[b]:ck[b + 1]]))
    cd = ispa.kvq_desc(H_kv, d, page, pages, FMT[fmt])
    a = ispa.attn_seq_desc(B, H, H_kv, d, CODE[dtype], CODE[out], causal, scale)
    o, lse = torch.full((T, H, d), 7.0, dtype=out, device="cuda"), torch.full((T, H), 7.0, device="cuda")
    ws = torch.empty(ispa.ispa_attn_kvq_workspace_bytes(a, cd), dtype=torch.uint8, device="cuda")
    ispa.ispa_attn_kvq(a, cd, q.cuda(), torch.as_tensor(c.buf).cuda(), ints(table), ints(lens), ints(cq), o, lse,
                       workspace=ws)
    ispa.ispa_check_device_error()
    for b in range(B):
        if new[b]:
            rows = slice(cq[b], cq[b + 1])
            kk, vv = c.get(table[b], np.arange(lens[b]))
            ref = so.attention(f64(q[rows]), kk, vv, causal, scale or None)
            check_attention(o[rows], lse[rows], ref, 2.0 ** -11, d, lens[b],
                            smallest_step(f64(q[rows]), kk, vv, causal, scale), f"sequence {b}")
    return o, lse


def random_rows(rng, T, lens, H, H_kv, d, dtype, slope=0.0):
    """q, k, v; slope: V's mean runs from -slope to slope over each sequence, so that every stretch of it shows in O."""
    q, k, v = (rand16(rng, (n, h, d), dtype) for n, h in ((T, H), (sum(lens), H_kv), (sum(lens), H_kv)))
    if slope:
        v = (v.float() + torch.cat([torch.linspace(-slope, slope, n) for n in lens])[:, None, None]).to(dtype)
    return q, k, v
