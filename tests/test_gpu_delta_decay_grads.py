"""dlog_decay of the gated delta rule where little of it or nothing is left, against its
definition in float64, each value by its own terms.

A decay multiplies the state before its token: where there is none, or the decay is 0, its
gradient is 0.  Elsewhere value i is a_i (<D, S> - dr . e) (delta_ref.walk_bwd), of size
a_i (|D| |S| + |dr| |e|).  The kernel's terms are products of operands of 24 bits summed in
fp32 over up to 256 channels (sqrt(256) 2^-24 = 2^-20), by a decay between two tokens whose
exponent, up to 128 in powers of two, is rounded to 24 bits (ln 2 128 2^-24 = 2^-17.5 of it):
2^-15 of the size holds them, and 2^-118 what the exp2 of such an exponent leaves out."""
import pytest
import torch

import delta_ref as R
from test_gpu_delta import BF16, F32, backward, problem, say

pytestmark = pytest.mark.gpu
INF = float("inf")


def own_size(p, lens, scale):
    """dlog_decay in float64 and the size of its own terms, by token and head."""
    refs, sizes = [], []
    for n, s in R._cuts(lens):
        q, k, v, g, b, dy = (p[x][s] for x in ("q", "k", "v", "log_decay", "beta", "dy"))
        rep = v.shape[1] // q.shape[1]
        h0 = None if p["h0"] is None else p["h0"][n]
        _, last, states = R.walk(q, k, v, g, b, h0, scale)
        q, k, v, a, b, dy = (R._heads(q, rep), R._heads(k, rep), v.double(), torch.exp(g.double()),
                             b.double(), dy.double())
        d = torch.zeros_like(last) if p["dh_last"] is None else p["dh_last"][n].double()
        ref, size = torch.zeros_like(a), torch.zeros_like(a)
        norm = lambda x: x.flatten(1).norm(dim=1)
        for t in reversed(range(a.shape[0])):
            old = states[t]
            d = d + scale * dy[t][:, :, None] * q[t][:, None, :]
            e = (old * k[t][:, None, :]).sum(-1)
            dr = b[t][:, None] * (d * k[t][:, None, :]).sum(-1)
            ref[t] = a[t] * ((d * old).sum((1, 2)) - (dr * e).sum(-1))
            size[t] = a[t] * (norm(d) * norm(old) + norm(dr) * norm(e))
            d = a[t][:, None, None] * (d - dr[:, :, None] * k[t][:, None, :])
        refs.append(ref)
        sizes.append(size)
    return torch.cat(refs), torch.cat(sizes)


def check(got, p, lens, scale, what):
    ref, size = own_size(p, lens, scale)
    err = (got.double().reshape(ref.shape) - ref).abs()
    bad = err - 2.0 ** -15 * size - 2.0 ** -118
    if bad.numel() and float(bad.max()) > 0:
        i = int(bad.argmax())
        raise AssertionError(f"{what}: token and head {divmod(i, ref.shape[1])}: "
                             f"{float(got.flatten()[i])!r}, exactly {float(ref.flatten()[i])!r} of "
                             f"{float(size.flatten()[i])!r}")


def first_tokens(lens):
    at = 0
    for n in lens:
        if n:
            yield at
        at += n


SHAPES = [(4, 2, 64, 48), (2, 1, 128, 128), (3, 3, 40, 136)]


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("lens,packed", [([1], False), ([1] * 5, False), ([1, 1, 1], True), ([2, 2], False),
                                         ([5, 1, 70, 0, 64, 1, 130], True), ([200, 200], False)])
def test_first_tokens_without_states(lens, packed, io):
    """The decay of a first token multiplies nothing: 0.0, of either sign of zero."""
    say("dlog_decay first", lens, packed, io)
    for H, G, K, V in SHAPES:
        p = problem(lens, H, G, K, V, io, seed=sum(lens) + K, state=False)
        g = backward(p, lens, packed, 0.3)["dlog_decay"].reshape(-1, H)
        first = list(first_tokens(lens))
        assert torch.all(g[first] == 0.0), (K, V, g[first])
        check(g, p, lens, 0.3, f"{lens} {K}x{V}")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("decay", [-INF, -3e4, -1e4, -200.0])
def test_decays_of_zero(decay, io):
    """exp(log_decay) is 0 in fp32: so is its gradient, and what is left is no residue of
    the terms that it cut off."""
    say("dlog_decay zero", decay, io)
    lens = [100, 3, 37]
    for state in (False, True):
        p = problem(lens, 4, 2, 64, 64, io, seed=5, state=state, decay=decay)
        p["log_decay"][::7] = -0.01
        p["log_decay"][64:70] = -0.02
        g = backward(p, lens, True, 0.3)["dlog_decay"]
        assert torch.all(g[p["log_decay"] == decay] == 0.0)
        check(g, p, lens, 0.3, f"decay {decay}, {state}")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("decay", [-3.0, -8.0, -20.0, -60.0])
def test_decays_that_leave_little(decay, io):
    say("dlog_decay little", decay, io)
    lens = [100, 1, 37, 2]
    for H, G, K, V in SHAPES:
        for state in (False, True):
            p = problem(lens, H, G, K, V, io, seed=6, state=state, decay=decay)
            p["log_decay"][::7] = -0.01
            g = backward(p, lens, True, 0.3)["dlog_decay"]
            check(g, p, lens, 0.3, f"decay {decay}, {K}x{V}, {state}")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("decay", [None, -20.0, -3e4])
def test_over_spans(decay, io):
    """A long sequence of few heads, whose chunks' states come from spans."""
    say("dlog_decay spans", decay, io)
    p = problem([1100], 2, 1, 64, 64, io, seed=7, state=False, decay=decay)
    if decay is not None:
        p["log_decay"][::7] = -0.01
    g = backward(p, [1100], False, 0.3)["dlog_decay"][0]
    assert torch.all(g[0] == 0.0)
    if decay == -3e4:
        assert torch.all(g[p["log_decay"] == decay] == 0.0)
    check(g, p, [1100], 0.3, f"spans, decay {decay}")
