"""CPU tests of the bound that the cached attention's tests use: it tells a right output from wrong ones at every length."""
import numpy as np
import pytest
import torch

from oracle import seq_oracle as so
from seq_bounds import smallest_step
from seq_helpers import check_attention


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("n,d,G", [(60, 64, 2), (4097, 128, 1), (9001, 128, 4), (19001, 64, 1)])
def test_wrong_outputs_are_rejected(fmt, n, d, G):
    rng = np.random.default_rng([n, d])
    q = rng.standard_normal((1, G, d))
    slope = np.linspace(-4.0, 4.0, n)[:, None, None]
    k, v = (so.dequantise(fmt, *so.quantise(fmt, rng.standard_normal((n, 1, d)) + x)).astype(np.float64) for x in (0, slope))
    ref = so.attention(q, k, v, True)
    step = smallest_step(q, k, v, True)

    def check(o):
        check_attention(torch.from_numpy(np.asarray(o, np.float32)), None, ref, 2.0 ** -11, d, n, step)

    check(ref[0])
    part = slice(n // 8, n // 8 + max(n // 150, 2))  # what one of 150 parts holds
    last = max(n // 150, 2)
    wrong = {"zeros": 0 * ref[0], "negated": -ref[0], "half of the keys": so.attention(q, k[:n // 2], v[:n // 2], True)[0],
             "values in reverse": so.attention(q, k, v[::-1], True)[0],
             "a part left out": so.attention(q, np.delete(k, part, 0), np.delete(v, part, 0), True)[0],
             "a part twice": so.attention(q, np.concatenate([k, k[part]]), np.concatenate([v, v[part]]), True)[0],
             "the last part left out": so.attention(q, k[:-last], v[:-last], True)[0]}
    for what, o in wrong.items():
        with pytest.raises(AssertionError):
            check(o)
            pytest.fail(what)  # (reached when the check has let it pass)


def test_a_missed_rejection_is_seen():
    """pytest.fail's exception is not one that pytest.raises(AssertionError) takes."""
    assert not issubclass(pytest.fail.Exception, AssertionError)


def test_smallest_step_by_hand():
    q, k = np.ones((2, 1, 4)), np.zeros((3, 1, 4))
    v = np.array([1.0, -8.0, 64.0])[:, None, None] * np.array([0.5, -1.0, 0.25, 0.0])
    assert np.allclose(smallest_step(q, k, v, True)[:, 0, 0] * 2 ** 9, [8 / 2, 64 / 3])
    assert np.allclose(smallest_step(q, k, v, False)[:, 0, 0] * 2 ** 9, [64 / 3, 64 / 3])
    assert np.all(smallest_step(q, k[:1], v[:1], True)[0] == 0)  # sees no key
