"""Linear attention with one decay per head on the GPU (``linear_attn``,
``linear_attn_bwd``, ``linear_attn_step``) against its definition in float64
(linattn_ref.py, which also derives the bounds)."""
import pytest
import torch

import linattn_ref as R
import selective_state_space_44_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rand(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _decays(H, lo=-1.0, hi=-9.0):
    return -torch.exp2(torch.linspace(lo, hi, H, device=DEV)) if H > 1 else \
        torch.full((1,), -0.05, device=DEV)


def _cu(lens):
    return torch.tensor([0] + list(lens), dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def _problem(lens, H, G, K, V, io, seed=0, h0=True, strided=False):
    g = _gen(seed)
    T = sum(lens)
    if strided:                        # slices of one fused projection
        w = _rand(g, T, (H + G) * K + G * V + 8, dtype=io)
        q = w[:, :H * K].unflatten(1, (H, K))
        k = w[:, H * K:(H + G) * K].unflatten(1, (G, K))
        v = w[:, (H + G) * K:(H + G) * K + G * V].unflatten(1, (G, V))
    else:
        q, k, v = (_rand(g, T, h, d, dtype=io) for h, d in ((H, K), (G, K), (G, V)))
    p = {"q": q, "k": k, "v": v, "log_decay": _decays(H),
         "h0": _rand(g, len(lens), H, V, K) if h0 else None}
    back = {"dy": _rand(g, T, H, V, dtype=io), "dh_last": _rand(g, len(lens), H, V, K)}
    return p, back


def _say(*a):
    print(*a, flush=True)


def _check_fwd(p, lens, scale=0.3, packed=True, nsplit=0, what=""):
    q, k, v, gd, h0 = (p[n] for n in ("q", "k", "v", "log_decay", "h0"))
    (o_ref, h_ref), (o_mass, h_mass) = R.prompt(q, k, v, gd, h0, scale, lens)
    if packed:
        o, h = ssm.linear_attn(q, k, v, gd, h0, scale=scale, cu_seqlens=_cu(lens),
                               return_last_state=True, nsplit=nsplit)
    else:
        q, k, v = (t.unflatten(0, (len(lens), lens[0])) for t in (q, k, v))
        o, h = ssm.linear_attn(q, k, v, gd, h0, scale=scale, return_last_state=True,
                               nsplit=nsplit)
    torch.cuda.synchronize()
    R.check(o, o_ref, o_mass, f"o {what}")
    R.check(h, h_ref, h_mass, f"h {what}")
    return o, h


GRADS = ("dq", "dk", "dv", "dlog_decay", "dh0")


def _check_bwd(p, b, lens, scale=0.3, packed=True, nsplit=0, what=""):
    q, k, v, gd, h0 = (p[n] for n in ("q", "k", "v", "log_decay", "h0"))
    dy, dh = b["dy"], b["dh_last"]
    ref, mass = R.prompt_bwd(q, k, v, gd, h0, scale, lens, dy, dh)
    if packed:
        cu = _cu(lens)
    else:
        cu = None
        q, k, v, dy = (t.unflatten(0, (len(lens), lens[0])) for t in (q, k, v, dy))
    g = ssm.linear_attn_bwd(q, k, v, gd, h0, dy=dy, dh_last=dh, scale=scale, cu_seqlens=cu,
                            need_dlog_decay=True, nsplit=nsplit)
    torch.cuda.synchronize()
    for n in GRADS:
        R.check(g[n], ref[n], mass[n], f"{n} {what}")
    return g


DIMS = [(64, 64), (128, 128), (128, 64), (64, 128), (96, 40), (8, 8), (256, 256), (24, 200)]


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("K,V", DIMS)
def test_dims(K, V, io):
    """Ragged packed sequences, some empty, some of one token, with states and
    grouped heads, from strided slices."""
    lens = [0, 1, 65, 130, 0, 17]
    _say(f"linattn dims K={K} V={V} {io}")
    p, b = _problem(lens, 4, 2, K, V, io, seed=K + V, strided=True)
    _check_fwd(p, lens, what=f"{K}x{V}")
    _check_bwd(p, b, lens, what=f"{K}x{V}")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
def test_lengths(L, io):
    _say(f"linattn L={L} {io}")
    lens = [L, L]
    p, b = _problem(lens, 2, 2, 64, 64, io, seed=L)
    _check_fwd(p, lens, packed=False, what=f"L={L}")
    _check_bwd(p, b, lens, packed=False, what=f"L={L}")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("nsplit", [1, 2, 3, 7])
def test_segments(nsplit, io):
    """Sequences cut into segments, also more of them than the sequence has
    chunks, and ragged ends."""
    _say(f"linattn nsplit={nsplit} {io}")
    lens = [449, 1, 0, 300, 64]
    p, b = _problem(lens, 3, 1, 64, 128, io, seed=nsplit)
    _check_fwd(p, lens, nsplit=nsplit, what=f"nsplit={nsplit}")
    _check_bwd(p, b, lens, nsplit=nsplit, what=f"nsplit={nsplit}")
    p, b = _problem([333, 333], 2, 2, 128, 64, io, seed=nsplit, h0=False)
    _check_fwd(p, [333, 333], packed=False, nsplit=nsplit, what="batch")
    b["dh_last"] = None
    _check_bwd(p, b, [333, 333], packed=False, nsplit=nsplit, what="batch")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("K,V", [(64, 128), (128, 64), (48, 64), (128, 128), (200, 40), (24, 256)])
def test_segments_of_other_heads(K, V, io):
    """Segments with every width of block, the decay's gradient among the
    results; grouped heads."""
    _say(f"linattn segments {K}x{V} {io}")
    lens = [200, 1, 0, 330]
    p, b = _problem(lens, 4, 2, K, V, io, seed=K + V)
    _check_fwd(p, lens, nsplit=3, what=f"segments {K}x{V}")
    _check_bwd(p, b, lens, nsplit=3, what=f"segments {K}x{V}")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("H,G", [(1, 1), (5, 1), (6, 2), (40, 8)])
def test_heads(H, G, io):
    _say(f"linattn heads {H}/{G} {io}")
    lens = [70, 3]
    p, b = _problem(lens, H, G, 32, 48, io, seed=H)
    _check_fwd(p, lens, what=f"{H}/{G}")
    _check_bwd(p, b, lens, what=f"{H}/{G}")


@pytest.mark.parametrize("io", [BF16, F32])
def test_decays(io):
    """No decay, decays that leave nothing of the previous token, -inf (only
    the token itself), and one that grows."""
    lens = [150, 1]
    p, b = _problem(lens, 6, 6, 64, 64, io, seed=3)
    p["log_decay"] = torch.tensor([0.0, -30.0, -200.0, -3.4e38, -1e-4, 0.01], device=DEV)
    _say(f"linattn decays {io}")
    _check_fwd(p, lens, what="decays")
    _check_bwd(p, b, lens, what="decays")
    q, k, v = p["q"][:150], p["k"][:150], p["v"][:150]
    inf = torch.full((6,), float("-inf"), device=DEV)
    o, h = ssm.linear_attn(q[None], k[None], v[None], inf, p["h0"][:1], return_last_state=True)
    o_ref = (q.double() * k.double()).sum(-1, keepdim=True) * v.double()
    mass = (q.double() * k.double()).abs().sum(-1, keepdim=True) * v.double().abs()
    R.check(o, o_ref, mass, "o, -inf")
    last = v[-1].double()[:, :, None] * k[-1].double()[:, None, :]
    R.check(h, last[None], last[None].abs(), "h, -inf")


def test_nan_and_inf_stay_where_they_belong():
    """A NaN or an infinity of one head and sequence reaches later outputs of
    that head and sequence only, and none before it."""
    lens = [100, 90]
    for bad in (float("nan"), float("inf")):
        p, _ = _problem(lens, 4, 4, 64, 64, BF16, seed=9)
        clean = ssm.linear_attn(p["q"], p["k"], p["v"], p["log_decay"], p["h0"],
                                cu_seqlens=_cu(lens))
        p["v"][40, 1, 5] = bad
        o, h = ssm.linear_attn(p["q"], p["k"], p["v"], p["log_decay"], p["h0"],
                               cu_seqlens=_cu(lens), return_last_state=True)
        same = torch.ones(190, 4, dtype=torch.bool, device=DEV)
        same[40:100, 1] = False
        assert torch.equal(o[same], clean[same])
        assert not torch.isfinite(o[40:100, 1, 5].float()).any()
        assert not torch.isfinite(h[0, 1, 5]).any() and torch.isfinite(h[1]).all()
        others = torch.arange(64, device=DEV) != 5
        assert torch.isfinite(o[:, :, others].float()).all()


@pytest.mark.parametrize("io", [BF16, F32])
def test_empty(io):
    h0 = _rand(_gen(1), 3, 2, 16, 24)
    z = lambda *s: torch.empty(s, dtype=io, device=DEV)
    gd = _decays(2)
    o, h = ssm.linear_attn(z(3, 0, 2, 24), z(3, 0, 2, 24), z(3, 0, 2, 16), gd, h0,
                           return_last_state=True)
    assert o.shape == (3, 0, 2, 16) and torch.equal(h, h0)
    o, h = ssm.linear_attn(z(0, 2, 24), z(0, 2, 24), z(0, 2, 16), gd, h0,
                           cu_seqlens=_cu([0, 0, 0]), return_last_state=True)
    assert torch.equal(h, h0)
    g = ssm.linear_attn_bwd(z(3, 0, 2, 24), z(3, 0, 2, 24), z(3, 0, 2, 16), gd, h0,
                            dy=z(3, 0, 2, 16), dh_last=h0, need_dlog_decay=True)
    assert torch.equal(g["dh0"], h0) and torch.count_nonzero(g["dlog_decay"]) == 0
    o = ssm.linear_attn(z(0, 5, 2, 24), z(0, 5, 2, 24), z(0, 5, 2, 16), gd)
    assert o.shape == (0, 5, 2, 16)


@pytest.mark.parametrize("io", [BF16, F32])
def test_cut_ranges(io):
    """cu_seqlens that leave the tokens are cut to them: nothing outside is
    read or written, and what lies inside is computed."""
    p, _ = _problem([50], 2, 2, 64, 64, io, seed=5, h0=False)
    out = torch.full((50, 2, 64), 7.0, dtype=io, device=DEV)
    cu = torch.tensor([-5, 20, 10, 90], dtype=torch.int32, device=DEV)
    o, h = ssm.linear_attn(p["q"], p["k"], p["v"], p["log_decay"], cu_seqlens=cu, out=out,
                           return_last_state=True)
    (r0, s0), (m0, sm0) = R.prompt(p["q"], p["k"], p["v"], p["log_decay"], None, 1.0, [20])
    (r2, s2), (m2, sm2) = R.prompt(p["q"][10:], p["k"][10:], p["v"][10:], p["log_decay"], None,
                                   1.0, [40])
    R.check(h[0], s0[0], sm0[0], "first state")
    assert torch.count_nonzero(h[1]) == 0
    R.check(h[2], s2[0], sm2[0], "last state")
    R.check(o[:10], r0[:10], m0[:10], "o")
    R.check(o[20:], r2[10:], m2[10:], "o")


@pytest.mark.parametrize("io", [BF16, F32])
def test_step_continues_the_prompt(io):
    """A prompt, then single tokens on its final state: the states and outputs
    of the whole sequence."""
    H, G, K, V, B, n, m = 6, 3, 96, 72, 5, 37, 4
    p, _ = _problem([n + m] * B, H, G, K, V, io, seed=11)
    q, k, v = (p[x].unflatten(0, (B, n + m)) for x in "qkv")
    (o_ref, h_ref), (o_mass, h_mass) = R.prompt(p["q"], p["k"], p["v"], p["log_decay"], p["h0"],
                                                0.2, [n + m] * B)
    _, h = ssm.linear_attn(*(t[:, :n].contiguous() for t in (q, k, v)), p["log_decay"], p["h0"],
                           scale=0.2, return_last_state=True)
    slots = torch.tensor([4, 0, 6, 2, 1], dtype=torch.int32, device=DEV)
    pool = torch.full((7, H, V, K), 3.0, device=DEV)
    pool[slots.long()] = h
    o_ref, o_mass = (t.view(B, n + m, H, V) for t in (o_ref, o_mass))
    for t in range(n, n + m):
        o = ssm.linear_attn_step(pool, q[:, t], k[:, t], v[:, t], p["log_decay"], scale=0.2,
                                 slots=slots)
        R.check(o, o_ref[:, t], o_mass[:, t], f"o at {t}")
    R.check(pool[slots.long()], h_ref, h_mass, "state")
    assert torch.all(pool[[3, 5]] == 3.0)


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("K,V", [(8, 8), (64, 64), (128, 128), (96, 40), (160, 24), (256, 256)])
def test_step(K, V, io):
    B, H, G = 3, 4, 2
    g = _gen(K)
    q, k, v = (_rand(g, B, h, d, dtype=io) for h, d in ((H, K), (G, K), (G, V)))
    h = _rand(g, B, H, V, K)
    gd = torch.tensor([0.0, -0.1, -50.0, float("-inf")], device=DEV)
    h_in = h.clone()
    o = ssm.linear_attn_step(h, q, k, v, gd, scale=1.5)
    finite = gd.clamp(min=-3e38)
    h_in[:, 3] = 0.0                    # -inf forgets the state
    for b in range(B):
        r, s = R.walk(q[b:b + 1], k[b:b + 1], v[b:b + 1], finite, h_in[b], 1.5)
        rm, sm = R.walk(q[b:b + 1].abs(), k[b:b + 1].abs(), v[b:b + 1].abs(), finite,
                        h_in[b].abs(), 1.5)
        R.check(o[b], r[0], rm[0], "o")
        R.check(h[b], s, sm, "h")


def test_step_slots_outside_are_left_alone():
    g = _gen(2)
    q, k, v = (_rand(g, 4, 2, 32, dtype=BF16) for _ in range(3))
    h = _rand(g, 3, 2, 32, 32)
    before = h.clone()
    slots = torch.tensor([-1, 3, 1, 1 << 30], dtype=torch.int32, device=DEV)
    out = torch.full((4, 2, 32), 5.0, dtype=BF16, device=DEV)
    ssm.linear_attn_step(h, q, k, v, _decays(2), slots=slots, out=out)
    torch.cuda.synchronize()
    assert torch.count_nonzero(out[[0, 1, 3]]) == 0 and torch.count_nonzero(out[2]) > 0
    assert torch.equal(h[[0, 2]], before[[0, 2]]) and not torch.equal(h[1], before[1])


def test_gradients_against_differences():
    """Directional derivatives of a loss on the float64 definition, by central
    differences, against the fp32 kernels' gradients.  The loss is a
    polynomial in all but the decay; step 1e-4 leaves an error of about 1e-7 of
    its scale, the fp32 gradients 2^-15 of their mass."""
    lens = [70, 5]
    scale = 0.25
    p, b = _problem(lens, 4, 2, 32, 24, F32, seed=21)
    g = ssm.linear_attn_bwd(*(p[n] for n in ("q", "k", "v", "log_decay", "h0")), dy=b["dy"],
                            dh_last=b["dh_last"], scale=scale, cu_seqlens=_cu(lens),
                            need_dlog_decay=True)
    _, mass = R.prompt_bwd(p["q"], p["k"], p["v"], p["log_decay"], p["h0"], scale, lens, b["dy"],
                           b["dh_last"])

    def loss(x):
        tot, at = 0.0, 0
        for n, L in enumerate(lens):
            s = slice(at, at + L)
            o, h = R.walk(x["q"][s], x["k"][s], x["v"][s], x["log_decay"], x["h0"][n], scale)
            tot = tot + (o * b["dy"][s]).sum() + (h * b["dh_last"][n]).sum()
            at += L
        return float(tot)
    for name in ("q", "k", "v", "log_decay", "h0"):
        d = _rand(_gen(5), *p[name].shape).double()
        x = {n: t.double() for n, t in p.items()}
        e = 1e-4
        up, down = dict(x), dict(x)
        up[name], down[name] = x[name] + e * d, x[name] - e * d
        fd = (loss(up) - loss(down)) / (2 * e)
        got = float((g["d" + name].double() * d).sum())
        m = float((mass["d" + name] * d.abs()).sum())
        assert abs(got - fd) <= (2.0 ** -15 + 1e-6) * m, (name, got, fd, m)


def test_autograd():
    lens = [30, 41]
    p, b = _problem(lens, 4, 2, 64, 64, BF16, seed=31)
    x = {n: t.clone().requires_grad_() for n, t in p.items()}
    o, h = ssm.LinearAttention.apply(x["q"], x["k"], x["v"], x["log_decay"], x["h0"], 0.5,
                                     _cu(lens))
    torch.autograd.backward([o, h], [b["dy"], b["dh_last"]])
    g = ssm.linear_attn_bwd(*(p[n] for n in ("q", "k", "v", "log_decay", "h0")), dy=b["dy"],
                            dh_last=b["dh_last"], scale=0.5, cu_seqlens=_cu(lens),
                            need_dlog_decay=True)
    for n in x:
        assert torch.equal(x[n].grad, g["d" + n]), n
    # the state unused, no state given: the same as without them
    x = {n: p[n].clone().requires_grad_() for n in ("q", "k", "v")}
    o, _ = ssm.LinearAttention.apply(x["q"], x["k"], x["v"], p["log_decay"], None, 0.5, _cu(lens))
    o.backward(b["dy"])
    g = ssm.linear_attn_bwd(p["q"], p["k"], p["v"], p["log_decay"], dy=b["dy"], scale=0.5,
                            cu_seqlens=_cu(lens))
    for n in x:
        assert torch.equal(x[n].grad, g["d" + n]), n


@pytest.mark.parametrize("io", [BF16, F32])
def test_deterministic_and_on_another_stream(io):
    lens = [300, 77, 500]
    p, b = _problem(lens, 5, 1, 128, 128, io, seed=41)
    args = [p[n] for n in ("q", "k", "v", "log_decay", "h0")]

    def both():
        f = ssm.linear_attn(*args, cu_seqlens=_cu(lens), return_last_state=True)
        g = ssm.linear_attn_bwd(*args, dy=b["dy"], dh_last=b["dh_last"], cu_seqlens=_cu(lens),
                                need_dlog_decay=True)
        return [*f, *(g[n] for n in GRADS)]
    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = both()
    side.synchronize()
    for x, y in zip(first, again):
        assert torch.equal(x, y)


def test_deterministic_with_equal_lengths():
    """Sequences of one length tie in the order of work; the decay's gradient,
    summed over them, still repeats bit for bit.  More sequences than one round
    of the sort holds, so that every round's are placed."""
    lens = [70] * 300 + [1] * 800 + [0, 65]
    p, b = _problem(lens, 2, 1, 32, 32, BF16, seed=43)
    args = [p[n] for n in ("q", "k", "v", "log_decay", "h0")]
    cu = _cu(lens)

    def once():
        return ssm.linear_attn_bwd(*args, cu_seqlens=cu, dy=b["dy"], dh_last=b["dh_last"],
                                   need_dlog_decay=True)
    first = once()
    for _ in range(3):
        again = once()
        for n in GRADS:
            assert torch.equal(first[n], again[n]), n
    keep = [0, 299, 1023, 1024, 1101]
    ends = torch.tensor(lens).cumsum(0).tolist()
    for i in keep:
        lo, n = ends[i] - lens[i], lens[i]
        if n == 0:
            continue
        one = {k: v[lo:lo + n] for k, v in p.items() if k in "qkv"}
        o = ssm.linear_attn(one["q"], one["k"], one["v"], p["log_decay"], p["h0"][i:i + 1],
                            cu_seqlens=_cu([n]))
        o_all = ssm.linear_attn(*args, cu_seqlens=cu)[lo:lo + n]
        assert torch.equal(o, o_all), i


def test_long_sequence_with_segments():
    """One sequence of 20,000 tokens in the automatic plan, two heads, against
    the definition; a slow decay reaches over many segments."""
    L = 20000
    p, _ = _problem([L], 2, 1, 64, 64, BF16, seed=51)
    p["log_decay"] = torch.tensor([-1e-4, -0.02], device=DEV)
    _say("linattn long")
    _check_fwd(p, [L], packed=False, what="long")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("K,V,H", [(64, 64, 4), (64, 64, 36), (128, 128, 4), (96, 64, 4)])
def test_plans_of_few_heads(K, V, H, io):
    """The automatic plan of few heads and some hundred tokens, which cuts: one
    sequence, and packed ones longer and shorter than the mean the plan goes by."""
    _say(f"linattn plan {K}x{V} {H} heads {io}")
    for lens, packed in (([550], False), ([550], True), ([900, 0, 197, 3], True), ([1], True)):
        p, b = _problem(lens, H, 2, K, V, io, seed=K + H)
        _check_fwd(p, lens, packed=packed, what=f"{lens}")
        _check_bwd(p, b, lens, packed=packed, what=f"{lens}")
        # without the decay's gradient the plan may be another
        q, k, v, gd, h0 = (p[n] for n in ("q", "k", "v", "log_decay", "h0"))
        ref, mass = R.prompt_bwd(q, k, v, gd, h0, 0.3, lens, b["dy"], b["dh_last"])
        g = ssm.linear_attn_bwd(q, k, v, gd, h0, dy=b["dy"], dh_last=b["dh_last"], scale=0.3,
                                cu_seqlens=_cu(lens))
        for n in ("dq", "dk", "dv", "dh0"):
            R.check(g[n], ref[n], mass[n], f"{lens} {n}")


@pytest.mark.parametrize("io", [BF16, F32])
def test_many_packed_segments(io):
    """More blocks than the chip holds, the last of them without a unit: what
    they leave where the decay's gradient is summed must not reach the states
    that other blocks have stored by then."""
    lens = [130 + 7 * (i % 9) for i in range(30)]
    p, b = _problem(lens, 16, 4, 128, 128, io, seed=71)
    # the first head's decay reaches furthest, and no two terms cancel
    for t in (p, b):
        t.update({n: x.abs() for n, x in t.items()})
    p["log_decay"] = _decays(16).flip(0).contiguous()
    _say(f"linattn many packed segments {io}")
    _check_bwd(p, b, lens, nsplit=3, what="many segments")


def test_large_offsets():
    """Tokens past 2^31 elements: the last tokens of a strided operand equal
    those of a packed copy."""
    T, stride = 66000, 1 << 15
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 5 GB")
    buf = torch.zeros(T * stride, dtype=BF16, device=DEV)
    wide = buf.view(T, stride)
    lens = [65000, 1000]
    small = _rand(_gen(61), T, 3 * 64, dtype=BF16)
    wide[:, :192] = small
    cut = lambda m: [m[:, i * 64:(i + 1) * 64].unflatten(1, (1, 64)) for i in range(3)]
    gd = torch.full((1,), -0.01, device=DEV)
    o1 = ssm.linear_attn(*cut(wide), gd, cu_seqlens=_cu(lens))
    o2 = ssm.linear_attn(*cut(small), gd, cu_seqlens=_cu(lens))
    torch.cuda.synchronize()
    assert torch.equal(o1, o2)
    (ref, _), (mass, _) = R.prompt(*(t[65000:] for t in cut(small)), gd, None, 1.0, [1000])
    R.check(o1[65000:], ref, mass, "last tokens")


def test_in_a_graph():
    """Captured once, replayed on new inputs with eager work between."""
    lens = [200, 33]
    p, _ = _problem(lens, 4, 2, 64, 64, BF16, seed=71)
    cu = _cu(lens)
    out = torch.empty(233, 4, 64, dtype=BF16, device=DEV)
    args = [p[n] for n in ("q", "k", "v", "log_decay", "h0")]
    ssm.linear_attn(*args, cu_seqlens=cu, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssm.linear_attn(*args, cu_seqlens=cu, out=out)
    for i in range(3):
        for n in ("q", "k", "v"):
            p[n].copy_(_rand(_gen(80 + i), *p[n].shape))
        eager = ssm.linear_attn(*args, cu_seqlens=cu)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i
