"""States and adjoints of the gated delta rule carried over many chunks and spans of a
constant decay, with betas of 0: the given one times the decays' product."""
import pytest
import torch

from test_gpu_delta import BF16, DEV, F32, backward, forward, problem, say

pytestmark = pytest.mark.gpu

# Powers of two of a chunk's, or a span's, decay that lie differently between two fp32 numbers
DECAYS = [-4.9e-7, -9.9e-7, -1.65e-6, -1.74e-6, -3e-6]

# Every chunk, or every span and its own chunks after them, rounds a value once, at random:
# 512 at most.  sqrt(512) 2^-25 (a rounding's root mean square is under half of its largest,
# 2^-24), of up to 2^16 values the worst at four and a half times that: 2^-18.3.  A decay off
# by half a unit would drift by 256 2^-25 = 2^-17 over as many spans.
BOUND = 2.0 ** -18.3


def off(got, given, p):
    """Of every head's state, by the product of its own decays in 64 bits."""
    a = torch.exp(p["log_decay"].double().sum(0))
    ref = a[None, :, None, None] * given.double()
    return float(((got.double() - ref) / ref).abs().max())


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("decay", DECAYS)
@pytest.mark.parametrize("L,H,K,V", [(20000, 1, 64, 64), (32768, 1, 64, 64), (32768, 1, 128, 128),
                                     (16400, 2, 96, 40)])
def test_states_over_spans(L, H, K, V, decay, io):
    say("delta drift over spans", L, H, K, V, decay, io)
    p = problem([L], H, 1, K, V, io, seed=51, decay=decay)
    p["beta"][:] = 0.0
    _, h = forward(p, [L], False, 1.0)
    assert off(h, p["h0"], p) < BOUND


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("decay", DECAYS)
@pytest.mark.parametrize("L,H,K,V", [(20000, 1, 64, 64), (32768, 1, 128, 128)])
def test_adjoints_over_spans(L, H, K, V, decay, io):
    say("delta drift of adjoints", L, H, K, V, decay, io)
    p = problem([L], H, 1, K, V, io, seed=52, decay=decay)
    p["beta"][:] = 0.0
    p["dy"][:] = 0.0
    assert off(backward(p, [L], False, 1.0)["dh0"], p["dh_last"], p) < BOUND


@pytest.mark.parametrize("decay", DECAYS)
def test_packed_spans(decay):
    """A long sequence among two short ones."""
    say("delta drift over packed spans", decay)
    lens = [70, 25000, 5]
    p = problem(lens, 1, 1, 64, 64, BF16, seed=53, decay=decay)
    p["beta"][:] = 0.0
    _, h = forward(p, lens, True, 1.0)
    cut = {"log_decay": p["log_decay"][70:25070]}
    assert off(h[1:2], p["h0"][1:2], cut) < BOUND


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("decay", DECAYS)
def test_chunks_alone(decay, io):
    """So many heads that no sequence is cut into spans."""
    say("delta drift, no spans", decay, io)
    L, H = 20000, 256
    p = problem([1], H, 1, 64, 8, io, seed=54)
    at = dict(device=DEV)
    p = {"q": torch.zeros(L, 1, 64, dtype=io, **at), "k": p["k"].expand(L, 1, 64).contiguous(),
         "v": torch.ones(L, H, 8, dtype=io, **at), "log_decay": torch.full((L, H), decay, **at),
         "beta": torch.zeros(L, H, dtype=io, **at), "h0": p["h0"], "dy": torch.zeros(L, H, 8, dtype=io, **at),
         "dh_last": p["dh_last"]}
    _, h = forward(p, [L], False, 1.0)
    assert off(h, p["h0"], p) < BOUND
