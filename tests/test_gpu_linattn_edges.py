"""Linear attention with one decay per head on the GPU: calls at the edge of
what the entry points take, against the definition in float64 (linattn_ref.py,
which also derives the bounds)."""
import ctypes

import pytest
import torch

import linattn_ref as R
import selective_state_space_44_amd as ssm
import test_gpu_linattn as base

pytestmark = pytest.mark.gpu
DEV = base.DEV
BF16, F32 = torch.bfloat16, torch.float32


def _at(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _bwd_abi(p, b, cu, nsplit, fill, scale=0.3):
    """``ssm_linattn_bwd`` on packed tokens into outputs that hold ``fill``, with
    a workspace of NaN: its outputs by name."""
    lib = ssm.load_library()
    q, k, v = p["q"], p["k"], p["v"]
    (T, H, K), (_, G, V), n = q.shape, v.shape, cu.numel() - 1
    code = ssm.SSM_DTYPE_BF16 if q.dtype is BF16 else ssm.SSM_DTYPE_F32
    out = {"d" + x: torch.full(p[x].shape, fill, dtype=p[x].dtype, device=DEV)
           for x in ("q", "k", "v", "log_decay")}
    out["dh0"] = torch.full((n, H, V, K), fill, device=DEV)
    need = lib.ssm_linattn_bwd_workspace_bytes(n, T, 1, H, G, K, V, code, 1, nsplit)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    st = lib.ssm_linattn_bwd(
        n, T, _at(cu), H, G, K, V, code, _at(q), q.stride(0), _at(k), k.stride(0), _at(v),
        v.stride(0), _at(p["log_decay"]), scale, _at(p["h0"]), _at(b["dy"]), b["dy"].stride(0),
        _at(b["dh_last"]), *(_at(out[x]) for x in base.GRADS), nsplit, _at(ws), need,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == ssm.SSM_OK
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("nsplit", [1, 3])
@pytest.mark.parametrize("H,G", [(4, 2), (3, 3)])
def test_backward_leaves_tokens_of_no_sequence_alone(H, G, nsplit, io):
    """cu_seqlens that start past the first token and end before the last (a
    buffer padded to a fixed size): dq, dk and dv keep there what they held."""
    base._say(f"linattn bwd, uncovered tokens, {H}/{G} nsplit={nsplit} {io}")
    lens, first, T = [150, 0, 50], 3, 220
    end = first + sum(lens)
    p, b = base._problem([T, 0, 0], H, G, 64, 64, io, seed=91)
    cu = base._cu(lens) + first
    got = _bwd_abi(p, b, cu, nsplit, 7.0)
    cut = lambda d: {n: t[first:end] if n in ("q", "k", "v", "dy") else t for n, t in d.items()}
    pc, bc = cut(p), cut(b)
    ref, mass = R.prompt_bwd(pc["q"], pc["k"], pc["v"], p["log_decay"], p["h0"], 0.3, lens,
                             bc["dy"], b["dh_last"])
    for n in ("dq", "dk", "dv"):
        assert torch.all(got[n][:first] == 7.0) and torch.all(got[n][end:] == 7.0), n
        R.check(got[n][first:end], ref[n], mass[n], n)
    for n in ("dlog_decay", "dh0"):
        R.check(got[n], ref[n], mass[n], n)


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("nsplit", [1, 2])
def test_states_carry_24_bits(nsplit, io):
    """Given states that cancel, to fp32 rounding, what one token 64 steps away
    leaves: what the other tokens read of it is the rounding alone.  Either
    side is rounded in a power (its exponent, about 1, twice and the
    exponential: 3 2^-24) and in two products: together 10 2^-24 of the token's
    term, 2^-21 of the mass, which counts both sides.  An operand in two bf16
    parts is off by up to 2^-18 of its side."""
    base._say(f"linattn 24 bits nsplit={nsplit} {io}")
    L, H, K, V, scale = 70, 2, 64, 48, 0.37
    g = base._gen(17)
    some = lambda *s: (torch.rand(s, generator=g, device=DEV) + 0.5).to(io)
    decay = torch.tensor([-0.011, -0.007], device=DEV)
    a = torch.exp(decay.double())
    # forward: the first token alone writes, the last six read
    q, k, v, dy = some(L, H, K), some(L, H, K), some(L, H, V), some(L, H, V)
    k1, v1 = k.clone(), v.clone()
    k1[1:], v1[1:] = 0, 0
    outer = lambda x, y: x.double()[:, :, None] * y.double()[:, None, :]
    h0 = (-outer(v[0], k[0]) / a[:, None, None]).float()[None]
    o, h = ssm.linear_attn(q[None], k1[None], v1[None], decay, h0, scale=scale,
                           return_last_state=True, nsplit=nsplit)
    back = ssm.linear_attn_bwd(q[None], k1[None], v1[None], decay, h0, dy=dy[None], scale=scale,
                               nsplit=nsplit)
    (o_ref, h_ref), (o_mass, h_mass) = R.prompt(q, k1, v1, decay, h0, scale, [L])
    ref, mass = R.prompt_bwd(q, k1, v1, decay, h0, scale, [L], dy, None)
    # back in time: the last token alone asks of the states, the first six read
    q1, dy1 = q.clone(), dy.clone()
    q1[:-1], dy1[:-1] = 0, 0
    dh = (-scale * outer(dy[-1], q[-1])).float()[None]
    rev = ssm.linear_attn_bwd(q1[None], k[None], v[None], decay, dy=dy1[None], dh_last=dh,
                              scale=scale, nsplit=nsplit)
    rref, rmass = R.prompt_bwd(q1, k, v, decay, None, scale, [L], dy1, dh)
    torch.cuda.synchronize()
    for got, r, m, what in ((o[0, 64:], o_ref[64:], o_mass[64:], "o"), (h, h_ref, h_mass, "h"),
                            (back["dq"][0, 64:], ref["dq"][64:], mass["dq"][64:], "dq"),
                            (rev["dk"][0, :6], rref["dk"][:6], rmass["dk"][:6], "dk"),
                            (rev["dv"][0, :6], rref["dv"][:6], rmass["dv"][:6], "dv"),
                            (rev["dh0"], rref["dh0"], rmass["dh0"], "dh0")):
        off = (got.double() - r).abs() - 2.0 ** -8 * 1.01 * r.abs() * (got.dtype is BF16)
        assert float((off / m).max()) <= 2.0 ** -21, (what, float((off / m).max()) * 2 ** 21)


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("packed", [True, False])
def test_short_sequences_of_growing_states(packed, io):
    """Decays that grow so fast that 63 steps overflow (or 31), over so few tokens that
    nothing does."""
    base._say(f"linattn growing packed={packed} {io}")
    for lens in ([1, 5, 20, 0],) if packed else ([1, 1], [5, 5], [20, 20]):
        p, b = base._problem(lens, 4, 2, 32, 48, io, seed=sum(lens))
        p["log_decay"] = torch.tensor([1.5, 3.0, -0.1, 2.0], device=DEV)
        base._check_fwd(p, lens, packed=packed, what=f"growing {lens}")
        base._check_bwd(p, b, lens, packed=packed, what=f"growing {lens}")


@pytest.mark.parametrize("io", [BF16, F32])
def test_segments_of_one_long_sequence_among_short_ones(io):
    """Packed, the mean below a chunk, segments asked for."""
    base._say(f"linattn one long {io}")
    lens = [1, 3] * 20 + [700] + [2, 0] * 10
    p, b = base._problem(lens, 4, 2, 64, 64, io, seed=93)
    base._check_fwd(p, lens, nsplit=4, what="one long")
    base._check_bwd(p, b, lens, nsplit=4, what="one long")


@pytest.mark.parametrize("io", [BF16, F32])
def test_spare_blocks_of_given_segments(io):
    """Segments asked for of long and short sequences, more blocks than the chip
    holds, the last of them without a unit."""
    base._say(f"linattn spare blocks {io}")
    lens = [130 + 7 * (i // 2 % 9) if i % 2 else 20 for i in range(60)]
    p, b = base._problem(lens, 16, 4, 128, 128, io, seed=97)
    for t in (p, b):                    # no two terms cancel
        t.update({n: x.abs() for n, x in t.items()})
    p["log_decay"] = base._decays(16).flip(0).contiguous()
    base._check_bwd(p, b, lens, nsplit=3, what="spare blocks")


def test_overlapping_sequences_of_more_units_than_32_bits_count():
    """cu_seqlens that run up and down: 32,768 sequences over the same tokens, in
    131,072 segments each.  The table of segments holds the first of them."""
    T, n = 1 << 23, 1 << 16
    base._say("linattn overlapping sequences")
    g = base._gen(3)
    q, k, v = (torch.randn(T, 1, 8, generator=g, device=DEV, dtype=BF16) for _ in range(3))
    decay = torch.full((1,), -0.01, device=DEV)
    cu = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    cu[1::2] = T
    whole = ssm.linear_attn(q, k, v, decay, cu_seqlens=cu[:2].contiguous(), nsplit=T // 64)
    torch.cuda.synchronize()
    o = ssm.linear_attn(q, k, v, decay, cu_seqlens=cu, nsplit=T // 64)
    torch.cuda.synchronize()
    assert torch.equal(o, whole)


def _halves(f, n):
    """f over the first half of n rows, then over the rest, joined."""
    parts = [f(slice(0, n // 2)), f(slice(n // 2, n))]
    return [torch.cat(p) for p in zip(*parts)]


@pytest.mark.parametrize("io", [BF16, F32])
def test_more_threads_than_a_grid_holds(io):
    """65,664 sequences of a token, 128 heads: more than 2^32 threads, which a
    launch does not take.  The same as two calls on half of them."""
    base._say(f"linattn large grids {io}")
    B, H, K, V = 65664, 128, 8, 72
    g = base._gen(5)
    r = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=io)
    q, k, v, dy = r(B, 1, H, K), r(B, 1, 1, K), r(B, 1, 1, V), r(B, 1, H, V)
    decay = base._decays(H)
    o = ssm.linear_attn(q, k, v, decay)
    half, = _halves(lambda s: (ssm.linear_attn(q[s], k[s], v[s], decay),), B)
    assert torch.equal(o, half)
    del o, half
    grads = lambda s: ssm.linear_attn_bwd(q[s], k[s], v[s], decay, dy=dy[s], need_dh0=False,
                                          need_dlog_decay=True)
    whole = grads(slice(None))
    parts = _halves(lambda s: tuple(grads(s)[n] for n in ("dq", "dk", "dv")), B)
    for n, p in zip(("dq", "dk", "dv"), parts):
        assert torch.equal(whole[n], p), n
    # one token on no state: nothing depends on the decay
    assert torch.count_nonzero(whole["dlog_decay"]) == 0
    del whole, parts
    torch.cuda.empty_cache()


def test_more_threads_than_a_grid_holds_step():
    B, H, D = (1 << 19) + 3, 128, 8
    base._say("linattn large grids, step")
    if torch.cuda.get_device_properties(0).total_memory < 128 << 30:
        pytest.skip("needs 40 GB")
    g = base._gen(6)
    q, k, v = (torch.randn((B, n, D), generator=g, device=DEV, dtype=BF16) for n in (H, 1, 1))
    h = torch.full((B, H, D, D), 0.5, device=DEV)
    again = h.clone()
    decay = base._decays(H)
    o = ssm.linear_attn_step(h, q, k, v, decay)
    half, = _halves(lambda s: (ssm.linear_attn_step(again[s], q[s], k[s], v[s], decay),), B)
    assert torch.equal(o, half) and torch.equal(h, again)
    del h, again, o, half, q
    torch.cuda.empty_cache()


def test_more_threads_than_a_grid_holds_rotate():
    B, L, D = 16500, 2048, 136
    base._say("rotate large grids")
    if torch.cuda.get_device_properties(0).total_memory < 128 << 30:
        pytest.skip("needs 60 GB")
    g = base._gen(7)
    q, k = (torch.randn((B, L, 1, D), generator=g, device=DEV, dtype=BF16) for _ in "qk")
    cos, sin = R.angles(L, 4, DEV)
    whole = ssm.qk_norm_rotate(q, k, cos, sin)
    for s in (slice(0, 100), slice(B // 2, B // 2 + 100), slice(B - 200, B)):
        for x, y in zip(whole, ssm.qk_norm_rotate(q[s], k[s], cos, sin)):
            assert torch.equal(x[s], y)
    del whole, q, k
    torch.cuda.empty_cache()


def test_more_states_than_a_grid_holds_threads():
    """No tokens: the final states are the given ones, all of them."""
    B, H, D = (1 << 19) + 3, 128, 8
    base._say("linattn large states, no tokens")
    if torch.cuda.get_device_properties(0).total_memory < 128 << 30:
        pytest.skip("needs 40 GB")
    h0 = torch.rand((B, H, D, D), generator=base._gen(8), device=DEV)
    z = torch.empty((B, 0, H, D), dtype=BF16, device=DEV)
    _, h = ssm.linear_attn(z, z, z, base._decays(H), h0, return_last_state=True)
    assert torch.equal(h, h0)
    g = ssm.linear_attn_bwd(z, z, z, base._decays(H), h0, dy=z, dh_last=h0)
    assert torch.equal(g["dh0"], h0)
    del h, h0, g
    torch.cuda.empty_cache()


def _long_sums(q, k, v, decay, dy):
    """Final state, dh0 and dlog_decay of one sequence from no state, in float64
    by chunks of 256 tokens: q, dy [L, H, d], one key head; scale 1."""
    C, (L, H, K), V = 256, q.shape, v.shape[1]
    a = decay.double()
    S = torch.zeros(H, V, K, dtype=R.F64, device=DEV)
    T, adj, dg = S.clone(), S.clone(), torch.zeros(H, dtype=R.F64, device=DEV)
    i = torch.arange(C, device=DEV, dtype=R.F64)
    power = lambda n: torch.exp(a[:, None] * n)[..., None]
    d = i[:, None] - i[None]
    D = torch.exp(a[:, None, None] * d.clamp(min=0)) * d.clamp(min=0)
    e = torch.exp(a * C)[:, None, None]
    for c in range(0, L, C):
        s = slice(c, c + C)
        qc, yc = (x[s].double().transpose(0, 1).contiguous() for x in (q, dy))
        kc, vc = k[s].double(), v[s].double()
        o = ((qc @ kc.T.contiguous()) * D) @ vc
        st, tt = (x.transpose(1, 2).contiguous() for x in (S, T))
        o = o + power(i + 1) * ((i + 1)[:, None] * (qc @ st) + qc @ tt)
        dg = dg + (o * yc).sum((1, 2))
        w = (power(C - 1 - i) * vc).transpose(1, 2).contiguous()
        wt = (power(C - 1 - i) * (C - 1 - i)[:, None] * vc).transpose(1, 2).contiguous()
        T = e * (T + C * S) + wt @ kc
        S = e * S + w @ kc
        adj = adj + (power(c + 1 + i) * yc).transpose(1, 2).contiguous() @ qc
    return S, adj, dg


@pytest.mark.parametrize("io,nsplit", [(BF16, 1), (BF16, 512), (F32, 1), (F32, 512)])
def test_slow_decays_do_not_drift(io, nsplit):
    """65,536 tokens of one sign, uncut or in 512 segments, at decays that keep
    nearly all of them.  A state takes in n pieces in r roundings each, at most
    2^-24 of it: r sqrt(n) is below 9 sqrt(2048), which leaves 2^-18 in rms of
    independent ones.  What all elements share (the mean over 256) is the
    powers' error, 4 2^-24, and 4 standard deviations of the mean of the rest:
    2^-19.  The same for the decay's gradient, a sum of such states."""
    base._say(f"linattn drift {io} nsplit={nsplit}")
    L, H, D = 65536, 8, 16
    g = base._gen(1)
    some = lambda *s: (torch.rand(s, generator=g, device=DEV) + 0.5).to(io)
    q, k, v, dy = some(L, H, D), some(L, 1, D), some(L, 1, D), some(L, H, D)
    decay = -torch.tensor([1e-6, 3e-6, 1e-5, 2e-5, 3e-5, 5e-5, 7e-5, 1e-4], device=DEV)
    x = [t[None] for t in (q, k, v)]
    _, h = ssm.linear_attn(*x, decay, return_last_state=True, nsplit=nsplit)
    grads = ssm.linear_attn_bwd(*x, decay, dy=dy[None], nsplit=nsplit)
    S, adj, _ = _long_sums(q, k[:, 0], v[:, 0], decay, dy)
    torch.cuda.synchronize()
    for got, ref, what in ((h[0], S, "h"), (grads["dh0"][0], adj, "dh0")):
        off = (got.double() - ref) / ref
        print(what, off.mean((1, 2)).tolist(), float(off.square().mean().sqrt()), flush=True)
        assert float(off.mean((1, 2)).abs().max()) <= 2.0 ** -19, what
        assert float(off.square().mean((1, 2)).sqrt().max()) <= 2.0 ** -18, what


@pytest.mark.parametrize("io", [BF16, F32])
def test_decay_gradient_of_a_long_sequence(io):
    """65,536 tokens uncut, terms of one sign: the sum over the chunks is not
    kept in fp32.  The states' error of the test above and the powers of the
    outputs, 2^-19 each."""
    base._say(f"linattn long decay gradient {io}")
    L, H, D = 65536, 8, 16
    g = base._gen(2)
    some = lambda *s: (torch.rand(s, generator=g, device=DEV) + 0.5).to(io)
    q, k, v, dy = some(L, H, D), some(L, 1, D), some(L, 1, D), some(L, H, D)
    decay = -torch.tensor([1e-6, 3e-6, 1e-5, 1e-4, 1e-3, 1e-2, 0.1, 1.0], device=DEV)
    grads = ssm.linear_attn_bwd(*(t[None] for t in (q, k, v)), decay, dy=dy[None], nsplit=1,
                                need_dlog_decay=True, need_dh0=False)
    _, _, dg = _long_sums(q, k[:, 0], v[:, 0], decay, dy)
    off = (grads["dlog_decay"].double() - dg) / dg
    print(off.tolist(), flush=True)
    assert float(off.abs().max()) <= 2.0 ** -18


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("t", [40, 66, 130])
def test_decay_gradient_of_single_terms(t, io):
    """One token writes, one reads, through one channel each: dlog_decay is one
    product t a^t v k q dy, from the pair product (40), the state (66) and the
    state after another chunk (130).  Its powers have exponents of at most 1.5
    (two of them, 4 2^-24 each with the exponential) and it is rounded in eight
    products: 2^-20.  A state or a pair in two bf16 parts is off by 2^-18."""
    base._say(f"linattn single terms t={t} {io}")
    H, D, L = 64, 32, 140
    g = base._gen(t)
    q, k, v, dy = (torch.zeros(1, L, H, D, dtype=io, device=DEV) for _ in range(4))
    x = (torch.rand((4, H), generator=g, device=DEV) + 0.5).to(io)
    k[0, 0, :, 7], v[0, 0, :, 9], q[0, t, :, 7], dy[0, t, :, 9] = x
    decay = -torch.rand(H, generator=g, device=DEV) / t
    got = ssm.linear_attn_bwd(q, k, v, decay, dy=dy, need_dlog_decay=True, nsplit=1)["dlog_decay"]
    ref = t * torch.exp(decay.double() * t) * x.double().prod(0)
    off = float(((got.double() - ref) / ref).abs().max())
    assert off <= 2.0 ** -20, off * 2 ** 20


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("nsplit", [1, 2])
@pytest.mark.parametrize("K,V", [(64, 64), (40, 128)])
@pytest.mark.parametrize("what", ["q", "k", "v", "dy"])
def test_nan_and_inf_reach_what_they_enter_only(what, K, V, nsplit, io):
    """One bad value of token 40 in the first of two sequences: what it enters
    is not finite, and everything else is the same bits as without it."""
    base._say(f"linattn bad {what} {K}x{V} nsplit={nsplit} {io}")
    lens, t, c = [150, 90], 40, 5
    n = lens[0]

    def run(p, b):
        args = [p[x] for x in ("q", "k", "v", "log_decay", "h0")]
        cu = base._cu(lens)
        o, h = ssm.linear_attn(*args, cu_seqlens=cu, return_last_state=True, nsplit=nsplit)
        grads = ssm.linear_attn_bwd(*args, dy=b["dy"], dh_last=b["dh_last"], cu_seqlens=cu,
                                    need_dlog_decay=True, nsplit=nsplit)
        return {"o": o, "h": h, **grads}
    p, b = base._problem(lens, 4, 2, K, V, io, seed=101)
    clean = run(p, b)
    all_ = slice(None)
    # heads 2 and 3 read key head 1; head 1 reads key head 0
    after, upto, here = slice(t, n), slice(0, t + 1), t
    enters = {"q": {"o": (here, 1), "dk": (upto, 0, c), "dv": (upto, 0), "dh0": (0, 1, all_, c),
                    "dlog_decay": (1,)},
              "k": {"o": (after, slice(2, 4)), "h": (0, slice(2, 4), all_, c),
                    "dq": (after, slice(2, 4), c), "dv": (here, 1), "dlog_decay": (slice(2, 4),)},
              "v": {"o": (after, slice(2, 4), c), "h": (0, slice(2, 4), c),
                    "dq": (after, slice(2, 4)), "dk": (here, 1), "dlog_decay": (slice(2, 4),)},
              "dy": {"dq": (here, 1), "dk": (upto, 0), "dv": (upto, 0, c), "dh0": (0, 1, c),
                     "dlog_decay": (1,)}}[what]
    for value in (float("nan"), float("inf"), float("-inf")):
        x = b if what == "dy" else p
        good = x[what]
        x[what] = good.clone()
        x[what][t, 1, c] = value
        got = run(p, b)
        x[what] = good
        torch.cuda.synchronize()
        for name, y in got.items():
            bad = torch.zeros(y.shape, dtype=torch.bool, device=DEV)
            if name in enters:
                bad[enters[name]] = True
            assert not torch.isfinite(y[bad]).any(), (name, value)
            assert torch.equal(y[~bad], clean[name][~bad]), (name, value)


@pytest.mark.parametrize("io", [BF16, F32])
def test_single_tokens_of_long_sequences(io):
    """Rows that are one token of each of many sequences, millions of elements
    apart: the same as from copies."""
    B, L, H, G, D, t = 3, 1100, 40, 8, 128, 1000
    base._say(f"linattn far rows {io}")
    g = base._gen(12)
    w = torch.randn((B, L, H + 2 * G, D), generator=g, device=DEV).to(io)
    rows = [w[:, t, :H], w[:, t, H:H + G], w[:, t, H + G:]]
    copies = [x.contiguous() for x in rows]
    cos, sin = R.angles(64, D, DEV)
    pos = torch.tensor([5, 0, 63], device=DEV)
    for x, y in zip(ssm.qk_norm_rotate(*rows[:2], cos, sin, pos),
                    ssm.qk_norm_rotate(*copies[:2], cos, sin, pos)):
        assert torch.equal(x, y)
    back = [ssm.qk_norm_rotate_bwd(*x[:2], cos, sin, pos, dq_out=x[0], dk_out=x[1])
            for x in (rows, copies)]
    assert torch.equal(back[0]["dq"], back[1]["dq"]) and torch.equal(back[0]["dk"], back[1]["dk"])
    h = torch.randn((B, H, D, D), generator=g, device=DEV)
    again = h.clone()
    o = ssm.linear_attn_step(h, *rows, base._decays(H))
    assert torch.equal(o, ssm.linear_attn_step(again, *copies, base._decays(H)))
    assert torch.equal(h, again)


def test_native_calls_in_a_graph():
    """Rotation, prompt and single token by the native calls, captured once and
    replayed on new inputs with eager work between."""
    base._say("native calls in a graph")
    p, _ = base._problem([70], 4, 2, 64, 64, BF16, seed=71)
    x = [p[n][None] for n in ("q", "k", "v")]
    cos, sin = R.angles(70, 64, DEV)
    state = torch.zeros(1, 4, 64, 64, device=DEV)

    def calls():
        q, k = ssm.qk_norm_rotate(*x[:2], cos, sin)
        o, h = ssm.linear_attn(q, k, x[2], p["log_decay"], return_last_state=True, nsplit=2)
        state.copy_(h)
        o1 = ssm.linear_attn_step(state, q[:, -1], k[:, -1], x[2][:, -1], p["log_decay"])
        return o, o1
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls()
    for i in range(3):
        for n in ("q", "k", "v"):
            p[n].copy_(base._rand(base._gen(80 + i), *p[n].shape))
        eager = [t.clone() for t in calls()]
        after = state.clone()
        state.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager)), i
        assert torch.equal(state, after), i
