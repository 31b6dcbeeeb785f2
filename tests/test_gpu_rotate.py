"""Head norm with rotation on the GPU (``qk_norm_rotate`` and its backward)
against the definition in float64 (linattn_ref.rotate).

Bounds.  Forward: a channel is a pair's two products, each with the row's
1 / sqrt (its sum of d fp32 squares is off by at most d 2^-24, halved by the
root; d <= 256: 2^-17) and a few fp32 roundings: 2^-15 of the pair's length
(the norm of u times the weights).  Backward: the same on dx's mass r (|w g| +
|x r| mean |w g x r|), and for the weights' gradients n fp32 terms, added in
runs below 1024 and then in order over at most 1024 blocks: 2^-13 of their mass
would be the worst case and 2^-15 covers the runs used here.  Storing bf16 adds
2^-8 of the value."""
import pytest
import torch

import linattn_ref as R
import selective_state_space_44_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def _problem(T, hq, hk, dim, rot, io, seed=0, weights=True, npos=500):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)
    w = rand(T, (hq + 2 * hk) * dim).to(io)     # a fused projection's output
    q = w[:, :hq * dim].unflatten(1, (hq, dim))
    k = w[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim))
    cos, sin = R.angles(npos, rot, DEV) if rot else (None, None)
    pos = torch.randint(0, npos, (T,), generator=g, device=DEV)
    return {"q": q, "k": k, "cos": cos, "sin": sin, "positions": pos,
            "q_weight": 1 + 0.2 * rand(dim) if weights else None,
            "k_weight": 1 + 0.2 * rand(dim) if weights else None}, \
        {"dq_out": rand(T, hq, dim).to(io), "dk_out": rand(T, hk, dim).to(io)}


def _partner(x, n, interleaved):
    """|x| plus the pair's other member's, the pair's length at most."""
    y = x.abs().clone()
    i = torch.arange(n, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    s = y[..., ia] + y[..., ib]
    y[..., ia], y[..., ib] = s, s
    return y


def _check_fwd(p, interleaved, what):
    q, k = ssm.qk_norm_rotate(**p, eps=EPS, interleaved=interleaved)
    torch.cuda.synchronize()
    n = 0 if p["cos"] is None else p["cos"].shape[1]
    for got, x, w in ((q, p["q"], p["q_weight"]), (k, p["k"], p["k_weight"])):
        ref = R.rotate(x, w, p["cos"], p["sin"], p["positions"], EPS, interleaved)
        u = R.rotate(x, w, None, None, None, EPS, interleaved)
        R.check(got, ref, _partner(u, n, interleaved), what, parts=False)


def _grads(x, w, cos, sin, pos, dy, interleaved):
    """dx, dw and their masses in float64."""
    x, dy = x.to(R.F64), dy.to(R.F64)
    n = 0 if cos is None else cos.shape[1]
    g, gm = dy.clone(), _partner(dy, n, interleaved)
    if n:
        i = torch.arange(n, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        z = torch.complex(dy[..., ia], dy[..., ib]) * torch.complex(
            cos.to(R.F64), -sin.to(R.F64))[pos][:, None]
        g[..., ia], g[..., ib] = z.real, z.imag
    m = torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    w = torch.ones(x.shape[-1], dtype=R.F64, device=x.device) if w is None else w.to(R.F64)
    dx = (w * g - x / m * (w * g * x / m).mean(-1, keepdim=True)) / m
    wa = w.abs()
    dxm = (wa * gm + (x / m).abs() * (wa * gm * (x / m).abs()).mean(-1, keepdim=True)) / m
    return dx, (g * x / m).sum((0, 1)), dxm, (gm * (x / m).abs()).sum((0, 1))


def _check_bwd(p, b, interleaved, what):
    r = ssm.qk_norm_rotate_bwd(**p, **b, eps=EPS, interleaved=interleaved)
    torch.cuda.synchronize()
    for n in "qk":
        dx, dw, dxm, dwm = _grads(p[n], p[n + "_weight"], p["cos"], p["sin"], p["positions"],
                                  b[f"d{n}_out"], interleaved)
        R.check(r["d" + n], dx, dxm, f"d{n} {what}", parts=False)
        if p[n + "_weight"] is not None:
            R.check(r[f"d{n}_weight"], dw, dwm, f"d{n}_weight {what}")
        else:
            assert r[f"d{n}_weight"] is None


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 32), (64, 0), (80, 80), (80, 40), (96, 48),
                                     (256, 256), (256, 4), (8, 8), (8, 4), (24, 12), (136, 100)])
def test_dims(dim, rot, interleaved, io):
    print(f"rotate dim={dim} rot={rot} {interleaved} {io}", flush=True)
    p, b = _problem(7, 5, 3, dim, rot, io, seed=dim + rot)
    _check_fwd(p, interleaved, f"{dim}/{rot}")
    _check_bwd(p, b, interleaved, f"{dim}/{rot}")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (1, 40, 8), (3, 1, 0), (3, 0, 2), (131, 7, 7),
                                     (1500, 5, 1)])
def test_tokens_and_heads(T, hq, hk, io):
    print(f"rotate T={T} heads {hq}/{hk} {io}", flush=True)
    p, b = _problem(T, hq, hk, 64, 64, io, seed=T, weights=T != 131)
    if hk == 0:
        p["k_weight"] = None
    if hq == 0:
        p["q_weight"] = None
    _check_fwd(p, False, "fwd")
    _check_bwd(p, b, False, "bwd")


def test_positions_default_and_batch():
    """[batch, seqlen, ...] without positions: every sequence starts at 0."""
    p, b = _problem(3 * 50, 4, 2, 64, 64, BF16, seed=4)
    p["positions"] = torch.arange(50, device=DEV).repeat(3)
    flat = ssm.qk_norm_rotate(**p)
    gflat = ssm.qk_norm_rotate_bwd(**p, **b)
    shape = lambda t: t.unflatten(0, (3, 50))
    p4 = {**p, "q": shape(p["q"]), "k": shape(p["k"]), "positions": None}
    got = ssm.qk_norm_rotate(**p4)
    g4 = ssm.qk_norm_rotate_bwd(**p4, **{n: shape(t) for n, t in b.items()})
    for x, y in zip(got, flat):
        assert x.shape[:2] == (3, 50) and torch.equal(x.flatten(0, 1), y)
    for n in ("dq", "dk"):
        assert torch.equal(g4[n].flatten(0, 1), gflat[n])
    assert torch.equal(g4["dq_weight"], gflat["dq_weight"])


@pytest.mark.parametrize("io", [BF16, F32])
def test_positions_outside_the_table_are_nan(io):
    p, _ = _problem(5, 2, 2, 64, 32, io, seed=6, npos=10)
    p["positions"] = torch.tensor([0, 10, -1, 9, 1 << 40], device=DEV)
    q, k = ssm.qk_norm_rotate(**p)
    torch.cuda.synchronize()
    for x in (q.float(), k.float()):
        assert torch.isnan(x[[1, 2, 4]][..., :32]).all()
        assert torch.isfinite(x[[0, 3]]).all() and torch.isfinite(x[..., 32:]).all()


@pytest.mark.parametrize("io", [BF16, F32])
def test_rows_of_zeros_and_infinities(io):
    p, b = _problem(4, 2, 2, 64, 64, io, seed=8)
    clean, _ = ssm.qk_norm_rotate(**p)
    clean = clean.clone()
    p["q"][1, 0] = 0.0
    p["q"][2, 1, 3] = float("nan")
    q, _ = ssm.qk_norm_rotate(**p)
    g = ssm.qk_norm_rotate_bwd(**p, **b)
    torch.cuda.synchronize()
    assert torch.count_nonzero(q[1, 0]) == 0 and torch.isfinite(g["dq"][1].float()).all()
    assert torch.isnan(q[2, 1].float()).all()
    same = torch.ones(4, 2, dtype=torch.bool, device=DEV)
    same[1, 0] = same[2, 1] = False
    assert torch.equal(q[same], clean[same])


def test_empty():
    p, b = _problem(0, 2, 2, 64, 64, BF16)
    q, k = ssm.qk_norm_rotate(**p)
    g = ssm.qk_norm_rotate_bwd(**p, **b)
    assert q.shape == (0, 2, 64)
    assert torch.count_nonzero(g["dq_weight"]) == 0 and torch.count_nonzero(g["dk_weight"]) == 0


def test_gradients_against_differences():
    """Central differences of the float64 definition along random directions;
    third derivatives at step 1e-5 leave about 1e-9 of the scale."""
    p, b = _problem(6, 3, 2, 32, 16, F32, seed=9)
    g = ssm.qk_norm_rotate_bwd(**p, **b)

    def loss(x):
        return sum(float((R.rotate(x[n], x[n + "_weight"], p["cos"], p["sin"], p["positions"],
                                   1e-6, False) * b[f"d{n}_out"]).sum()) for n in "qk")
    x = {n: p[n].double() for n in ("q", "k", "q_weight", "k_weight")}
    for name in x:
        d = torch.randn(x[name].shape, generator=torch.Generator(device=DEV).manual_seed(3),
                        device=DEV, dtype=torch.float64)
        e = 1e-5
        up, down = dict(x), dict(x)
        up[name], down[name] = x[name] + e * d, x[name] - e * d
        fd = (loss(up) - loss(down)) / (2 * e)
        got = g["d" + name].double()
        assert abs(float((got * d).sum()) - fd) <= 2.0 ** -15 * float((got * d).abs().sum()), name


def test_autograd_and_determinism():
    p, b = _problem(300, 6, 2, 128, 128, BF16, seed=10)
    x = {n: p[n].clone().requires_grad_() for n in ("q", "k", "q_weight", "k_weight")}
    q, k = ssm.QkNormRotate.apply(x["q"], x["k"], p["cos"], p["sin"], p["positions"],
                                  x["q_weight"], x["k_weight"], 1e-6, False)
    torch.autograd.backward([q, k], [b["dq_out"], b["dk_out"]])
    g = ssm.qk_norm_rotate_bwd(**p, **b)
    for n in x:
        assert torch.equal(x[n].grad, g["d" + n]), n


def test_large_offsets():
    """Tokens past 2^31 elements of a strided operand."""
    T, stride = 66000, 1 << 15
    wide = torch.zeros(T, stride, dtype=BF16, device=DEV)
    tail = torch.randn(T, 128, device=DEV).to(BF16)
    wide[:, :128] = tail
    cos, sin = R.angles(64, 64, DEV)
    pos = torch.arange(T, device=DEV) % 64
    cut = lambda m: (m[:, :64].unflatten(1, (1, 64)), m[:, 64:128].unflatten(1, (1, 64)))
    a = ssm.qk_norm_rotate(*cut(wide), cos, sin, pos)
    c = ssm.qk_norm_rotate(*cut(tail), cos, sin, pos)
    torch.cuda.synchronize()
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
