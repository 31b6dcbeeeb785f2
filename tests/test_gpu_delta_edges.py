"""The gated delta rule on the GPU at the edge of what its calls take: values that are
no numbers, streams and graphs, workspaces, autograd, refusals."""
import pytest
import torch

import delta_ref as R
import selective_state_space_44_amd as ssm
from test_gpu_delta import (BF16, DEV, F32, OPERANDS, backward, cu_of, forward, gen, problem, say,
                            shaped)

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay", "beta"])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_what_odd_values_reach_forward(where, value, io):
    """A NaN or an infinity at one token: earlier tokens, other sequences and other heads
    are as they are without it; q's reaches its own token alone, v's its own channel."""
    say("delta odd", where, value, io)
    if where == "log_decay" and value == -INF:
        return  # a decay like any other
    lens, H, G = [100, 80], 4, 2
    p = problem(lens, H, G, 64, 64, io, seed=1)
    s, head = 70, 1                     # of the first sequence, in its second chunk
    bad = {**p, where: p[where].clone()}
    if where in "qkv":
        bad[where][s, head // (1 if where == "v" else 2), 5] = value
    else:
        bad[where][s, head] = value
    heads = [head] if where in ("v", "log_decay", "beta") else [0, 1]
    others = [h for h in range(H) if h not in heads]
    (o, h), (o0, h0) = forward(bad, lens, True, 0.3), forward(p, lens, True, 0.3)
    torch.cuda.synchronize()
    assert torch.equal(o[:, others], o0[:, others]) and torch.equal(h[:, others], h0[:, others])
    assert torch.equal(o[100:], o0[100:]) and torch.equal(h[1], h0[1])
    ro, _ = R.prompt(p, lens, 0.3)
    for at in heads:
        R.check(o[:s, at], ro[:s, at], f"{where} before", io is BF16)
        if where == "q":
            R.check(o[s + 1:100, at], ro[s + 1:100, at], "q after", io is BF16)
        if where == "v":
            rest = [c for c in range(64) if c != 5]
            R.check(o[s:100, at][:, rest], ro[s:100, at][:, rest], "other channels", io is BF16)
            assert not torch.isfinite(o[s:100, at, 5]).any()
            assert torch.isfinite(h[0, at][rest]).all()


@pytest.mark.parametrize("io", [BF16, F32])
def test_odd_given_states(io):
    """Of a given state: its own value channel alone."""
    say("delta odd state", io)
    lens = [100, 80]
    p = problem(lens, 2, 1, 64, 64, io, seed=2)
    h0 = p["h0"].clone()
    h0[0, 1, 7, 3] = NAN
    o, h = forward({**p, "h0": h0}, lens, True, 0.3)
    ro, rh = R.prompt(p, lens, 0.3)
    rest = [c for c in range(64) if c != 7]
    R.check(o[:, :, rest], ro[:, :, rest], "o", io is BF16)
    R.check(h[:, :, rest], rh[:, :, rest], "h", io is BF16)
    assert torch.isfinite(o[100:]).all() and torch.isnan(h[0, 1, 7]).all()


@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay", "beta", "dy", "h0", "dh_last"])
def test_what_odd_values_reach_backward(where):
    """Their sequence, and the value heads that share their key head."""
    say("delta odd backward", where)
    lens = [100, 80]
    p = problem(lens, 4, 2, 64, 64, BF16, seed=3)
    bad = {**p, where: p[where].clone()}
    bad[where].view(-1)[bad[where][0].numel() // 100] = NAN    # token 0 or sequence 0, head 0
    g, g0 = backward(bad, lens, True, 0.3), backward(p, lens, True, 0.3)
    torch.cuda.synchronize()
    for n in R.GRADS:
        at = slice(1, None) if n == "dh0" else slice(100, None)
        assert torch.equal(g[n][at], g0[n][at]), n
        hs = slice(1, None) if n in ("dq", "dk") else slice(2, None)
        assert torch.equal(g[n][:, hs], g0[n][:, hs]), n


@pytest.mark.parametrize("io", [BF16, F32])
def test_another_stream_and_given_outputs(io):
    say("delta stream", io)
    lens = [130, 130]
    p = problem(lens, 4, 2, 64, 64, io, seed=4)
    plain = forward(p, lens, False, 0.3)
    grads = backward(p, lens, False, 0.3)
    x, _ = shaped(p, lens, False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = torch.empty_like(x["v"])
        ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
        got = ssm.gated_delta(*(x[n] for n in OPERANDS), x["h0"], scale=0.3, out=out, workspace=ws,
                              return_last_state=True)
        ws.fill_(255)
        back = ssm.gated_delta_bwd(*(x[n] for n in OPERANDS), x["h0"], dy=x["dy"],
                                   dh_last=x["dh_last"], scale=0.3, workspace=ws)
    side.synchronize()
    assert got[0] is out
    assert all(torch.equal(a, b) for a, b in zip(plain, got))
    assert all(torch.equal(grads[n], back[n]) for n in R.GRADS)


@pytest.mark.parametrize("io", [BF16, F32])
def test_captured(io):
    """Two graphs of a pass each, replayed in turn with new values and eager work between,
    give what the eager calls give."""
    say("delta captured", io)
    lens = [90, 33]
    cu = cu_of(lens)
    p = problem(lens, 4, 2, 64, 64, io, seed=5)
    pool = torch.randn((4, 4, 64, 64), generator=gen(6), device=DEV)

    def calls(h):
        o, last = ssm.gated_delta(*(p[n] for n in OPERANDS), p["h0"], scale=0.3, cu_seqlens=cu,
                                  return_last_state=True)
        g = ssm.gated_delta_bwd(*(p[n] for n in OPERANDS), p["h0"], dy=p["dy"],
                                dh_last=p["dh_last"], scale=0.3, cu_seqlens=cu)
        s = ssm.gated_delta_step(h, *(p[n][:4] for n in OPERANDS), scale=0.3)
        return [o, last, *g.values(), s, h]
    graphs = []
    for _ in range(2):
        h = pool.clone()
        calls(h.clone())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = calls(h)
        graphs.append((graph, outs, h))
    for i in range(4):
        p["v"].copy_(torch.randn(p["v"].shape, generator=gen(10 + i), device=DEV))
        for graph, outs, h in graphs:
            h.copy_(pool)
            graph.replay()
            torch.cuda.synchronize()
            eager = calls(pool.clone())
            assert all(torch.equal(a, b) for a, b in zip(outs, eager)), i


def test_two_calls_at_once():
    """On two streams, each with its own workspace."""
    say("delta at once")
    lens = [500]
    ps = [problem(lens, 8, 4, 128, 128, BF16, seed=20 + i) for i in range(2)]
    plain = [(forward(p, lens, False, 0.3), backward(p, lens, False, 0.3)) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [None, None]
    for i, (p, s) in enumerate(zip(ps, streams)):
        with torch.cuda.stream(s):
            got[i] = (forward(p, lens, False, 0.3), backward(p, lens, False, 0.3))
    torch.cuda.synchronize()
    for (f, b), (f2, b2) in zip(plain, got):
        assert all(torch.equal(x, y) for x, y in zip(f, f2))
        assert all(torch.equal(b[n], b2[n]) for n in R.GRADS)


def test_nothing_to_do():
    """No sequences, no heads, no tokens: the state is the given one, gradients pass."""
    say("delta empty")
    f = lambda *s, dtype=BF16: torch.randn(s, generator=gen(1), device=DEV).to(dtype)
    h0 = f(2, 4, 16, 8, dtype=F32)
    q, v, b = f(2, 0, 2, 8), f(2, 0, 4, 16), f(2, 0, 4)
    ld = b.float()
    o, h = ssm.gated_delta(q, q, v, ld, b, h0, return_last_state=True)
    assert o.shape == v.shape and torch.equal(h, h0)
    _, h = ssm.gated_delta(q, q, v, ld, b, return_last_state=True)
    assert torch.all(h == 0)
    g = ssm.gated_delta_bwd(q, q, v, ld, b, h0, dy=v, dh_last=h0)
    assert torch.equal(g["dh0"], h0) and g["dq"].shape == q.shape
    g = ssm.gated_delta_bwd(q, q, v, ld, b, h0, dy=v)
    assert torch.all(g["dh0"] == 0)
    e = torch.zeros(1, dtype=torch.int32, device=DEV)
    q0, v0, b0 = q[0], v[0], b[0]
    assert ssm.gated_delta(q0, q0, v0, b0.float(), b0, cu_seqlens=e).shape == v0.shape
    q0, v0, b0 = f(0, 5, 2, 8), f(0, 5, 4, 16), f(0, 5, 4)
    assert ssm.gated_delta(q0, q0, v0, b0.float(), b0).shape == v0.shape
    v0, b0 = f(2, 5, 0, 16), f(2, 5, 0)
    q0 = f(2, 5, 1, 8)
    assert ssm.gated_delta(q0, q0, v0, b0.float(), b0).shape == v0.shape
    h = f(3, 4, 16, 8, dtype=F32)
    keep = h.clone()
    out = ssm.gated_delta_step(h, f(0, 2, 8), f(0, 2, 8), f(0, 4, 16), f(0, 4, dtype=F32), f(0, 4))
    assert out.shape == (0, 4, 16) and torch.equal(h, keep)


def test_refusals():
    say("delta refusals")
    p = problem([20, 20], 4, 2, 64, 64, BF16, seed=6)
    x, _ = shaped(p, [20, 20], False)
    ops = {n: x[n] for n in OPERANDS}

    def call(**kw):
        a = {**ops, "h0": None, **kw}
        opts = {n: a.pop(n) for n in list(a) if n not in OPERANDS + ("h0",)}
        return ssm.gated_delta(*(a[n] for n in OPERANDS), a["h0"], **opts)
    bad = [dict(q=x["q"][0]), dict(k=x["k"].float()), dict(v=x["v"][:, :10]),
           dict(log_decay=x["log_decay"].to(BF16)), dict(beta=x["beta"].float()),
           dict(beta=x["beta"][..., :2]), dict(log_decay=x["log_decay"].transpose(0, 1)),
           dict(h0=p["h0"][:1]), dict(h0=p["h0"].to(BF16)), dict(q=x["q"].cpu()),
           dict(v=x["v"][:, :, :3]), dict(out=torch.empty_like(x["v"]).float()),
           dict(q=x["q"][..., ::2], k=x["k"][..., ::2]), dict(workspace=torch.empty(8)),
           dict(cu_seqlens=cu_of([20, 20])), dict(beta=None), dict(v=None)]
    for kw in bad:
        with pytest.raises((ValueError, ssm.SsmError)):
            call(**kw)
    with pytest.raises((ValueError, ssm.SsmError)):            # 136 keys
        q = torch.zeros(2, 20, 2, 136, dtype=BF16, device=DEV)
        call(q=q, k=q)
    with pytest.raises((ValueError, ssm.SsmError)):
        call(q=x["q"][..., :20].contiguous(), k=x["k"][..., :20].contiguous())
    with pytest.raises(ssm.SsmError):                          # written where it is read
        call(out=x["v"])
    with pytest.raises(ValueError):
        ssm.gated_delta_bwd(*ops.values(), dy=x["dy"][:1])
    with pytest.raises(ValueError):
        ssm.gated_delta_bwd(*ops.values(), dy=x["dy"], dh_last=p["h0"][:1])
    h = torch.zeros(1, 4, 64, 64, device=DEV)
    row = {n: p[n][:2] for n in OPERANDS}
    with pytest.raises(ValueError):                            # two rows, one state
        ssm.gated_delta_step(h, *row.values())
    with pytest.raises(ValueError):
        ssm.gated_delta_step(h.to(BF16), *(t[:1] for t in row.values()))
    torch.cuda.synchronize()
    assert torch.isfinite(call()).all()                        # and still works


class _Off:
    """A module of native calls that leaves every call to Python."""

    def __getattr__(self, name):
        return lambda *a: None


@pytest.mark.parametrize("io", [BF16, F32])
def test_native_calls_agree(io, monkeypatch):
    lens = [40, 0, 33]
    p = problem(lens, 4, 2, 64, 48, io, seed=7)
    x = torch.randn(5, 3, 70, generator=gen(8), device=DEV).to(io)[:, :, :65]
    w, b = (torch.randn(65, generator=gen(i), device=DEV) for i in (1, 2))
    dy = torch.randn(5, 3, 65, generator=gen(9), device=DEV).to(io)

    def calls():
        yield forward(p, lens, True, 0.3)
        yield tuple(backward(p, lens, True, 0.3)[n] for n in R.GRADS)
        h = p["h0"].clone()
        yield ssm.gated_delta_step(h, *(p[n][:3] for n in OPERANDS), scale=0.3), h
        yield ssm.layer_norm(x, w, b), ssm.layer_norm(x)
        g = ssm.layer_norm_bwd(x, w, dy=dy)
        yield tuple(g.values())
        g = ssm.layer_norm_bwd(x, dy=dy, need_dweight=False, need_dbias=False)
        assert g["dweight"] is None and g["dbias"] is None
        yield (g["dx"],)
    native = list(calls())
    monkeypatch.setattr(ssm, "_native", lambda: _Off())
    for a, c in zip(native, calls()):
        assert all(torch.equal(s, t) for s, t in zip(a, c))


def _leaves(seed=0):
    p = problem([60], 4, 2, 32, 48, F32, seed=seed)
    x, _ = shaped(p, [60], False)
    return [x[n].clone().requires_grad_() for n in OPERANDS] + [p["h0"].clone().requires_grad_()], p


def test_autograd():
    """The wrapper's gradients are those of the call; of an output that is not used, none."""
    say("delta autograd")
    leaves, p = _leaves()
    o, h = ssm.GatedDelta.apply(*leaves, 0.3)
    grads = torch.autograd.grad((o * p["dy"].view(o.shape)).sum() + (h * p["dh_last"]).sum(), leaves)
    got = backward(p, [60], False, 0.3)
    for n, g in zip(R.GRADS, grads):
        assert torch.equal(g, got[n].view(g.shape)), n
    o, h = ssm.GatedDelta.apply(*leaves, 0.3)
    alone = torch.autograd.grad(h.sum(), leaves)
    ref, _ = R.prompt_bwd({**p, "dy": torch.zeros_like(p["dy"]),
                           "dh_last": torch.ones_like(p["dh_last"])}, [60], 0.3)
    for n, g in zip(R.GRADS[1:4], alone[1:4]):
        R.check(g[0], ref[n], n, False)


def test_autograd_refuses():
    leaves, _ = _leaves()
    o, _ = ssm.GatedDelta.apply(*leaves, torch.tensor(0.5, device=DEV, requires_grad=True))
    with pytest.raises(ValueError, match="gradient"):
        o.sum().backward()
    o, _ = ssm.GatedDelta.apply(*leaves, 0.3)
    g = torch.autograd.grad(o.square().sum(), leaves, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        sum(t.square().sum() for t in g).backward()
    kept = leaves[-1].detach().clone()
    o, _ = ssm.GatedDelta.apply(*leaves[:5], kept, 0.3)
    ssm.gated_delta_step(kept, *(t.detach()[:, 0].contiguous() for t in leaves[:5]))
    with pytest.raises(RuntimeError, match="inplace"):
        o.sum().backward()


def test_gradients_from_odd_addresses():
    """Outputs joined behind a single number: their gradients begin off the 16-byte
    boundary."""
    leaves, _ = _leaves()
    f = lambda: ssm.GatedDelta.apply(*leaves, 0.3)
    plain = torch.autograd.grad(sum(t.square().sum() for t in f()), leaves)
    joined = torch.cat([leaves[0].flatten()[:1].detach(), *(t.flatten() for t in f())])
    got = torch.autograd.grad(joined[1:].square().sum(), leaves)
    assert all(torch.equal(a, b) for a, b in zip(plain, got))
