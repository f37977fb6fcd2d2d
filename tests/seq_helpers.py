"""Builders and error bounds of the sequence calls' tests.

Bounds (relative half steps: bf16 2^-8, fp16 2^-11, fp32 2^-24).  With
A = the largest sum |q_i k_i| * scale of a query's keys, N its keys, W = sum of
weight * |v|:
  * a score is a sum of d products accumulated in fp32 (each addition off by at
    most 2^-23 of the sum of magnitudes: the tensor cores truncate) and scaled
    by a few fp32 products: off by at most (d + 8) 2^-23 A =: e;
  * exp2 of it adds 2^-21 (its error bound and the rounding of its argument,
    which is at most 2^-23 A / ln 2 <= e);
  * a weight is rounded once to the second product's type: r = 2^-11 in the
    cached attention, the input type's half step in the prompt attention.  The
    sum of weights is not rounded.  fp16 weights below 2^-14 of the reference
    are off by up to 2^-25 each, in units in which the normaliser is >= 1 (the
    cached attention's weights carry the V scale over 2^-6 of the largest: at
    most 2^-18 of the largest |v| a key);
  * so |o - exact| <= (r + 2 (e + 2^-21) + (N + 64) 2^-23) W + N 2^-25 max|v|
    plus the output's own rounding, and
    |lse - exact| <= e + (N + 64) 2^-23 + 2^-20 + 2^-22 |lse|.
"""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def starts(lens):
    return np.concatenate([[0], np.cumsum(np.asarray(lens, np.int64))]).astype(np.int32)


def rand16(rng, shape, dtype, wide=False):
    x = rng.standard_normal(shape).astype(np.float32)
    if wide and len(shape) == 3:  # large channels and rows of very different sizes
        x[..., 5::16] *= 8.0
        x *= np.exp2(rng.integers(-6, 5, shape[:2]))[..., None].astype(np.float32)
    return torch.from_numpy(x).to(dtype)


def paged(rng, lens, page, extra=3):
    """A shuffled block table (unused entries are junk) and the number of pages."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    order = rng.permutation(pages).astype(np.int32)
    table = rng.integers(-5, pages + 5, (len(lens), max(max(need), 1) + 1)).astype(np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def check_attention(got_o, got_lse, ref, weight_half, d, n_keys, vmax, what=""):
    o, lse, absv, size = ref
    e = (d + 8) * 2.0 ** -23 * size
    rel = weight_half + 2 * (e + 2.0 ** -21) + (n_keys + 64) * 2.0 ** -23
    out_half = HALF[got_o.dtype]
    g = f64(got_o)
    bound = rel[..., None] * absv + n_keys * 2.0 ** -25 * vmax
    bound = bound + out_half * (np.abs(o) + bound) + 2.0 ** -25
    err = np.abs(g - o)
    assert np.all(np.isfinite(g)), what
    worst = np.unravel_index(np.argmax(err - bound), err.shape) if err.size else None
    assert np.all(err <= bound), f"{what}: o off by {err[worst]:.3g} at {worst}, bound {bound[worst]:.3g}"
    if got_lse is not None:
        gl = f64(got_lse)
        assert np.array_equal(np.isneginf(gl), np.isneginf(lse)), what
        fin = np.isfinite(lse)
        bl = e + (n_keys + 64) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(fin, lse, 0))
        el = np.abs(np.where(fin, gl, 0) - np.where(fin, lse, 0))
        assert np.all(el <= bl), f"{what}: lse off by {(el - bl).max():.3g} over its bound"
