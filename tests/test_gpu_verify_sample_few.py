"""Sampled verification of one to three requests, nothing left out: the data
are taken from the first seed all of whose decisions are clear of rounding (the
oracle's margins say so), and every number of every request is compared."""
import numpy as np
import pytest
import torch

from oracle import hs_oracle as O
from gpu_util import lib
from test_gpu_verify_sample import _case, _check, _run

pytestmark = pytest.mark.gpu

# A weight w = max(p - q, 0) is off by what p is, 2^-17 p at most: by 2^-13 of
# itself where w > p / 16, as the winners' are (checked). Decisions 2^-12 apart
# are then clear of rounding.
CLEAR = 2.0 ** -12


def _clear_case(B, d, V, dtype, probs, masked, greedy):
    for seed in range(60):
        c = _case(B * 131 + d * 17 + V + 1000003 * seed, B, d, V, dtype, probs, masked)
        if d > 4:
            c[4][:] *= 0.2                                 # some of many drafts are accepted
        if greedy:
            c[1][-1] = 0.0
        want = O.verify_sample(*c)
        if not (want[3] > CLEAR).all():
            continue
        for b in range(B):                                 # the winner's weight against its probability
            m, v = want[0][b], want[1][b]
            if probs and m < d and c[1][b] > 0 and np.exp(want[2][b, m]) - c[3][b, m, v] <= np.exp(want[2][b, m]) / 16:
                break
        else:
            return c, want
    raise AssertionError("no clear seed")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("B,d,V,masked,greedy", [
    (1, 0, 1, 0.0, False), (1, 0, 50257, 0.0, False), (1, 1, 2, 0.0, False), (1, 3, 1024, 0.0, False),
    (1, 7, 50257, 0.0, False), (1, 255, 64, 0.0, False), (1, 3, 40000, 0.0, False), (1, 3, 129280, 0.0, False),
    (1, 3, 129281, 0.3, False), (1, 5, 1001, 0.9, True), (2, 3, 1024, 0.0, True), (2, 40, 100, 0.0, False),
    (2, 3, 129280, 0.0, True), (3, 2, 50259, 0.0, True), (3, 15, 9999, 0.2, False)])
def test_few_requests_in_full(dtype, probs, B, d, V, masked, greedy):
    hs = lib()
    c, want = _clear_case(B, d, V, dtype, probs, masked, greedy)
    got = _run(hs, *c)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    _check(got, want)
