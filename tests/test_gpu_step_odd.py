"""Infinities and NaN in single tokens: what they reach is what they reach in a sequence of
one token, whatever the number of keys."""
import pytest
import torch

import selective_state_space_44_amd as ssm
from test_gpu_delta import BF16, F32, OPERANDS, problem, say

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def same_kind(a, b):
    """Infinities of the same sign and NaN at the same places."""
    return (torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a == INF, b == INF)
            and torch.equal(a == -INF, b == -INF))


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("K", [8, 40, 48, 64, 96, 120])
@pytest.mark.parametrize("n", [2, 60])
def test_delta_step(n, K, io):
    """Of few heads and of many, whose waves take one group of rows and four."""
    say("delta step, odd values", n, K, io)
    H, G, V = 12, 4, 40
    p = problem([1] * n, H, G, K, V, io, seed=K)
    for x in "qk":
        p[x] = p[x].abs().clamp(min=2.0 ** -10)
    p["v"][0, 1, 5], p["v"][1, 2, 39], p["v"][1, 0, 0] = INF, -INF, NAN
    p["h0"][0, 3, 7, 1] = INF
    h = p["h0"].clone()
    o = ssm.gated_delta_step(h, *(p[x] for x in OPERANDS), scale=0.3)
    ro, rh = ssm.gated_delta(*(p[x][:, None] for x in OPERANDS), p["h0"], scale=0.3,
                             return_last_state=True)
    ro = ro[:, 0]
    # a given state's infinity stays in its channel, in either call of no promised kind
    for x in (o[0, 3, 7], ro[0, 3, 7], h[0, 3, 7], rh[0, 3, 7]):
        assert not torch.isfinite(x).any()
    o[0, 3, 7] = ro[0, 3, 7] = 0.0
    h[0, 3, 7] = rh[0, 3, 7] = 0.0
    assert same_kind(o, ro) and same_kind(h, rh)
    # u = beta (inf - S k) = inf, S = inf k, o = inf (k . q), whose terms are all above 0
    assert o[0, 1, 5] == INF and o[1, 2, 39] == -INF and torch.isnan(o[1, 0, 0])
    assert torch.all(h[0, 1, 5] == INF) and torch.all(h[1, 2, 39] == -INF)
