"""The gated delta rule on the GPU against its definition in float64
(delta_ref.py, which also derives the bounds)."""
import pytest
import torch

import delta_ref as R
import selective_state_space_44_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def problem(lens, H, G, K, V, io, seed=0, state=True, decay=None):
    """Operands of flat tokens: keys and queries of norm 1, decays from 0.9 to nearly 1
    (or the given one), betas of (0, 1)."""
    g, T, n = gen(seed), sum(lens), len(lens)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    ld = -0.1 * torch.rand((T, H), generator=g, device=DEV) ** 2
    return {"q": unit(r(T, G, K)).to(io), "k": unit(r(T, G, K)).to(io), "v": r(T, H, V).to(io),
            "log_decay": ld if decay is None else torch.full_like(ld, decay),
            "beta": torch.sigmoid(r(T, H)).to(io), "h0": r(n, H, V, K) if state else None,
            "dy": r(T, H, V).to(io), "dh_last": r(n, H, V, K) if state else None}


def cu_of(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).to(DEV)


OPERANDS = ("q", "k", "v", "log_decay", "beta")


def shaped(p, lens, packed):
    if packed:
        return p, cu_of(lens)
    at = {n: p[n].unflatten(0, (len(lens), lens[0])) for n in OPERANDS + ("dy",)}
    return {**p, **at}, None


def forward(p, lens, packed, scale):
    x, cu = shaped(p, lens, packed)
    return ssm.gated_delta(*(x[n] for n in OPERANDS), x["h0"], scale=scale, cu_seqlens=cu,
                           return_last_state=True)


def backward(p, lens, packed, scale):
    x, cu = shaped(p, lens, packed)
    return ssm.gated_delta_bwd(*(x[n] for n in OPERANDS), x["h0"], dy=x["dy"],
                               dh_last=x["dh_last"], scale=scale, cu_seqlens=cu,
                               need_dh0=True)


def check_forward(p, lens, packed, scale=0.3, what=""):
    o, h = forward(p, lens, packed, scale)
    torch.cuda.synchronize()
    ro, rh = R.prompt(p, lens, scale)
    bf = p["q"].dtype is BF16
    R.check(o, ro, what + " o", bf)
    R.check(h, rh, what + " h", bf)


def check_backward(p, lens, packed, scale=0.3, what=""):
    g = backward(p, lens, packed, scale)
    torch.cuda.synchronize()
    ref, mass = R.prompt_bwd(p, lens, scale)
    for n in R.GRADS:
        R.check(g[n], ref[n], f"{what} {n}", p["q"].dtype is BF16,
                mass if n == "dlog_decay" else None)


LENGTHS = [([1], False), ([2, 2], False), ([63], False), ([64], False), ([65], False),
           ([128], False), ([129, 129, 129], False), ([200], False),
           ([1, 0, 70, 64, 3, 130], True), ([0, 0, 5], True)]
SHAPES = [(1, 1, 8, 8), (4, 2, 64, 64), (3, 3, 128, 128), (5, 1, 96, 40), (6, 2, 48, 80),
          (2, 1, 120, 136), (2, 2, 16, 256), (4, 4, 128, 16)]


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("lens,packed", LENGTHS)
def test_lengths(lens, packed, io):
    say("delta lengths", lens, packed, io)
    for H, G, K, V in ((4, 2, 64, 48), (2, 1, 128, 128)):
        p = problem(lens, H, G, K, V, io, seed=sum(lens))
        check_forward(p, lens, packed, what=f"{lens} {K}x{V}")
        check_backward(p, lens, packed, what=f"{lens} {K}x{V}")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("H,G,K,V", SHAPES)
def test_head_layouts(H, G, K, V, io):
    say("delta heads", H, G, K, V, io)
    for state in (False, True):
        p = problem([130, 130], H, G, K, V, io, seed=K + V, state=state)
        check_forward(p, [130, 130], False, what=f"{H}/{G} {K}x{V}")
        check_backward(p, [130, 130], False, what=f"{H}/{G} {K}x{V}")


@pytest.mark.parametrize("io", [BF16, F32])
def test_many_heads_take_the_wide_blocks(io):
    """More than 128 blocks of 128 value channels: the forward in blocks of eight waves."""
    say("delta wide", io)
    p = problem([140, 140, 140], 48, 12, 128, 128, io, seed=3)
    check_forward(p, [140, 140, 140], False, what="wide")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("decay", [0.0, -1e-6, -3.0, -60.0, -3e4, float("-inf")])
def test_decays(decay, io):
    say("delta decay", decay, io)
    p = problem([100, 37], 4, 2, 64, 64, io, seed=5, decay=decay)
    # some tokens keep theirs
    p["log_decay"][::7] = -0.01
    check_forward(p, [100, 37], True, what=f"decay {decay}")
    check_backward(p, [100, 37], True, what=f"decay {decay}")


@pytest.mark.parametrize("io", [BF16, F32])
def test_growing_decays(io):
    """Decays above 0 over so few tokens that nothing overflows: what a longer sequence
    would reach weighs nothing.  Errors grow with the state, whose last values the
    bounds go by."""
    say("delta growing", io)
    for lens in ([1, 5, 20, 0],):
        p = problem(lens, 4, 2, 32, 48, io, seed=11, decay=1.5)
        p["log_decay"][:, 1] = 3.0
        check_forward(p, lens, True, what="growing")


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_betas(beta, io):
    """beta 0 writes nothing and has a gradient all the same; 1 replaces what a key
    holds."""
    say("delta beta", beta, io)
    p = problem([150], 4, 2, 64, 64, io, seed=7)
    p["beta"][:] = beta
    p["beta"][::5] = 0.5
    check_forward(p, [150], False, what=f"beta {beta}")
    check_backward(p, [150], False, what=f"beta {beta}")


@pytest.mark.parametrize("io", [BF16, F32])
def test_like_keys(io):
    """Keys all alike, betas 1 and no decay: the triangle's inverse is bounded, the
    powers that a series of it would sum are not.  (A bf16 key's norm is off 1 by up to
    2^-9: 64 tokens that each keep up to 2^-8 of what they replace.)"""
    say("delta like keys", io)
    p = problem([192], 2, 1, 64, 64, io, seed=9, decay=0.0)
    p["k"][:] = p["k"][:1]
    p["beta"][:] = 1.0
    check_forward(p, [192], False, what="like keys")
    check_backward(p, [192], False, what="like keys")


@pytest.mark.parametrize("io", [BF16, F32])
def test_operands_of_other_sizes(io):
    """Keys and queries of norms far from 1 with betas to match, and values of any size."""
    say("delta sizes", io)
    for size, beta in ((30.0, 1e-3), (1e-3, 1.0), (2.0 ** -40, 1.0)):
        p = problem([130], 2, 2, 64, 64, io, seed=13)
        p["k"] = (p["k"].float() * size).to(io)
        p["q"] = (p["q"].float() * 100.0).to(io)
        p["v"] = (p["v"].float() * 1e6).to(io)
        p["beta"] = (p["beta"].float() * beta).to(io)
        check_forward(p, [130], False, what=f"keys of {size}")
        check_backward(p, [130], False, what=f"keys of {size}")


def test_strided_operands():
    """Slices of one projection, other strides for each, a sliced gradient."""
    say("delta strided")
    lens, H, G, K, V = [70, 70], 4, 2, 64, 48
    p = problem(lens, H, G, K, V, BF16, seed=21)
    wide = torch.full((140, H * V + 2 * G * K + 24), float("nan"), dtype=BF16, device=DEV)
    q = wide[:, :G * K].unflatten(-1, (G, K))
    v = wide[:, G * K + 8:G * K + 8 + H * V].unflatten(-1, (H, V))
    k = wide[:, -G * K:].unflatten(-1, (G, K))
    dy = torch.full((140, H * V + 16), float("nan"), dtype=BF16, device=DEV)[:, 8:-8].unflatten(
        -1, (H, V))
    for t, n in ((q, "q"), (v, "v"), (k, "k"), (dy, "dy")):
        t.copy_(p[n])
    s = {**p, "q": q, "v": v, "k": k, "dy": dy}
    for packed in (False, True):
        plain, got = forward(p, lens, packed, 0.3), forward(s, lens, packed, 0.3)
        assert all(torch.equal(a, b) for a, b in zip(plain, got))
        plain, got = backward(p, lens, packed, 0.3), backward(s, lens, packed, 0.3)
        assert all(torch.equal(plain[n], got[n]) for n in R.GRADS)


@pytest.mark.parametrize("io", [BF16, F32])
def test_tokens_of_no_sequence(io):
    """cu_seqlens that start past the first token and end before the last: outputs there
    stay what they were."""
    say("delta uncovered", io)
    lens, first, T = [90, 0, 40], 5, 150
    end = first + sum(lens)
    p = problem([T], 4, 2, 64, 64, io, seed=31, state=False)
    p["h0"] = torch.randn((3, 4, 64, 64), generator=gen(1), device=DEV)
    p["dh_last"] = torch.randn((3, 4, 64, 64), generator=gen(2), device=DEV)
    cu = cu_of(lens) + first
    out = torch.full_like(p["v"], 7.0)
    ssm.gated_delta(*(p[n] for n in OPERANDS), p["h0"], scale=0.3, cu_seqlens=cu, out=out)
    assert torch.all(out[:first] == 7.0) and torch.all(out[end:] == 7.0)
    cut = {n: t[first:end] if n in OPERANDS + ("dy",) else t for n, t in p.items()}
    R.check(out[first:end], R.prompt(cut, lens, 0.3)[0], "o", io is BF16)
    g = ssm.gated_delta_bwd(*(p[n] for n in OPERANDS), p["h0"], dy=p["dy"], dh_last=p["dh_last"],
                            scale=0.3, cu_seqlens=cu)
    ref, mass = R.prompt_bwd(cut, lens, 0.3)
    for n in R.GRADS:
        got = g[n] if n == "dh0" else g[n][first:end]
        R.check(got, ref[n], n, io is BF16, mass if n == "dlog_decay" else None)


@pytest.mark.parametrize("n", [1500, 4500])
def test_many_sequences(n):
    """More sequences than one strip of the table, and than are put in order."""
    say("delta many sequences", n)
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 4, (n,), generator=g).tolist()
    lens[n // 2] = 150
    p = problem(lens, 2, 1, 16, 16, BF16, seed=n)
    o, h = forward(p, lens, True, 0.3)
    g_ = backward(p, lens, True, 0.3)
    torch.cuda.synchronize()
    pick = [0, 1, n // 2 - 1, n // 2, n // 2 + 1, n - 1]
    at = [0] + torch.tensor(lens).cumsum(0).tolist()
    for i in pick:
        s = slice(at[i], at[i + 1])
        one = {x: (t[s] if x in OPERANDS + ("dy",) else t[i:i + 1]) for x, t in p.items()}
        ro, rh = R.prompt(one, [lens[i]], 0.3)
        R.check(o[s], ro, f"o of {i}", True)
        R.check(h[i:i + 1], rh, f"h of {i}", True)
        ref, mass = R.prompt_bwd(one, [lens[i]], 0.3)
        for x in R.GRADS:
            R.check(g_[x][i:i + 1] if x == "dh0" else g_[x][s], ref[x], f"{x} of {i}", True,
                    mass if x == "dlog_decay" else None)


def test_overlapping_cuts_stay_in_bounds():
    """cu_seqlens that run up and down (its values are not checked): more chunks than the
    workspace holds are left out, and the sequences before them are as they should be."""
    say("delta overlapping")
    p = problem([200], 2, 1, 64, 64, BF16, seed=41, state=False)
    cu = torch.tensor([0, 200, 0, 200, -5, 300], dtype=torch.int32, device=DEV)
    o, h = ssm.gated_delta(*(p[n] for n in OPERANDS), scale=0.3, cu_seqlens=cu,
                           return_last_state=True)
    ssm.gated_delta_bwd(*(p[n] for n in OPERANDS), dy=p["dy"], scale=0.3, cu_seqlens=cu)
    torch.cuda.synchronize()
    ro, rh = R.prompt(p, [200], 0.3)
    R.check(h[:1], rh, "h", True)


@pytest.mark.parametrize("io", [BF16, F32])
def test_long_undecayed_states_do_not_drift(io):
    """Betas of 0: the state is the given one times the decays' product, through 313
    chunks whose decays are rounded alike."""
    say("delta drift", io)
    L = 20000
    p = problem([L], 1, 1, 64, 64, io, seed=51, decay=-3e-6)
    p["beta"][:] = 0.0
    _, h = forward(p, [L], False, 1.0)
    ref = torch.exp(p["log_decay"][:, 0].double().sum()) * p["h0"].double()
    # every chunk rounds the state once, at random: sqrt(313) 2^-25 of a value, 2^-20 six
    # times over; a decay off by half a unit would be 313 2^-25 = 2^-16.7
    assert float(((h.double() - ref) / ref).abs().max()) < 2.0 ** -18.5


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("K,V,H,G", [(64, 64, 4, 2), (128, 128, 3, 1), (48, 136, 2, 2), (8, 8, 1, 1)])
def test_steps(K, V, H, G, io):
    """Single tokens on a pool of states, against the definition; slots in any order,
    padding rows, and rows far apart."""
    say("delta step", K, V, H, G, io)
    n, pool = 5, 9
    p = problem([1] * n, H, G, K, V, io, seed=K)
    states = torch.randn((pool, H, V, K), generator=gen(3), device=DEV)
    slots = torch.tensor([4, -1, 0, 8, 9], dtype=torch.int32, device=DEV)
    h = states.clone()
    o = ssm.gated_delta_step(h, *(p[x] for x in OPERANDS), scale=0.3, slots=slots)
    torch.cuda.synchronize()
    on = [i for i, s in enumerate(slots.tolist()) if 0 <= s < pool]
    at = [slots[i].item() for i in on]
    ref = {**{x: p[x][on] for x in OPERANDS}, "h0": states[at]}
    ro, rh = R.prompt(ref, [1] * len(on), 0.3)
    R.check(o[on], ro, "o", io is BF16)
    R.check(h[at], rh, "h", io is BF16)
    off = [i for i in range(n) if i not in on]
    assert torch.all(o[off] == 0)
    rest = [i for i in range(pool) if i not in at]
    assert torch.equal(h[rest], states[rest])
    # one token of each of long sequences
    far = {x: torch.zeros((n, 3, *p[x].shape[1:]), dtype=p[x].dtype, device=DEV) for x in "qkv"}
    for x in "qkv":
        far[x][:, 1] = p[x]
    again = states.clone()
    o2 = ssm.gated_delta_step(again, *(far[x][:, 1] for x in "qkv"), p["log_decay"], p["beta"],
                              scale=0.3, slots=slots)
    assert torch.equal(o, o2) and torch.equal(h, again)


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("K,V", [(8, 8), (64, 64), (96, 40), (128, 136)])
def test_steps_of_many_heads(K, V, io):
    """Enough heads that a wave takes four groups of eight rows: against the definition, and
    bit for bit what the sequences give one by one, whose waves take a single group."""
    say("delta step, many heads", K, V, io)
    n, H, G = 45, 12, 4
    p = problem([1] * n, H, G, K, V, io, seed=K + 1)
    states = torch.randn((n, H, V, K), generator=gen(4), device=DEV)
    slots = torch.arange(n - 1, -1, -1, dtype=torch.int32, device=DEV)
    slots[7] = -1
    h, each = states.clone(), states.clone()
    o = ssm.gated_delta_step(h, *(p[x] for x in OPERANDS), scale=0.3, slots=slots)
    rows = [ssm.gated_delta_step(each, *(p[x][i:i + 1] for x in OPERANDS), scale=0.3,
                                 slots=slots[i:i + 1]) for i in range(n)]
    torch.cuda.synchronize()
    assert torch.equal(o, torch.cat(rows)) and torch.equal(h, each)
    on = [i for i in range(n) if i != 7]
    at = [n - 1 - i for i in on]
    ref = {**{x: p[x][on] for x in OPERANDS}, "h0": states[at]}
    ro, rh = R.prompt(ref, [1] * len(on), 0.3)
    R.check(o[on], ro, "o", io is BF16)
    R.check(h[at], rh, "h", io is BF16)
    assert torch.all(o[7] == 0) and torch.equal(h[n - 8], states[n - 8])


@pytest.mark.parametrize("io", [BF16, F32])
def test_prompt_and_steps_agree(io):
    """A prompt, then tokens one by one, is the whole sequence in one call."""
    say("delta prompt and steps", io)
    p = problem([75], 4, 2, 64, 64, io, seed=61)
    cut = {n: (t[:70] if n in OPERANDS + ("dy",) else t) for n, t in p.items()}
    o, h = forward(cut, [70], False, 0.3)
    rows = [ssm.gated_delta_step(h, *(p[x][t:t + 1] for x in OPERANDS), scale=0.3)
            for t in range(70, 75)]
    torch.cuda.synchronize()
    ro, rh = R.prompt(p, [75], 0.3)
    R.check(torch.cat([o[0], *rows]), ro, "o", io is BF16)
    R.check(h, rh, "h", io is BF16)


@pytest.mark.parametrize("io", [BF16, F32])
def test_repeats_bit_for_bit(io):
    say("delta repeats", io)
    lens = [300, 17, 64]
    p = problem(lens, 6, 2, 128, 128, io, seed=71)
    a, b = forward(p, lens, True, 0.3), forward(p, lens, True, 0.3)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = backward(p, lens, True, 0.3), backward(p, lens, True, 0.3)
    assert all(torch.equal(a[n], b[n]) for n in R.GRADS)


@pytest.mark.parametrize("io", [BF16, F32])
def test_gradients_against_differences(io):
    """Along a direction of each operand, against central differences of the definition:
    the step's third derivative leaves 2^-20 or so, the bound is the gradients' own.  The
    gradients of bf16 operands are rounded, 2^-8 of each term at most: 2^-8 of the product
    of the norms holds them."""
    say("delta differences", io)
    lens, scale = [40, 33], 0.3
    p = problem(lens, 4, 2, 32, 24, io, seed=81)
    got = backward(p, lens, True, scale)
    p64 = {n: t.double() for n, t in p.items()}

    def loss(x):
        o, h = R.prompt(x, lens, scale)
        return (o * p64["dy"]).sum() + (h * p64["dh_last"]).sum()
    for n in OPERANDS + ("h0",):
        d = torch.randn(p64[n].shape, generator=gen(5), device=DEV, dtype=torch.float64)
        step = 2.0 ** -12
        diff = (loss({**p64, n: p64[n] + step * d}) - loss({**p64, n: p64[n] - step * d})) / (2 * step)
        g = got["d" + n].double().reshape(d.shape)
        size = float(g.norm() * d.norm())
        eps = 2.0 ** -8 if got["d" + n].dtype is BF16 else 2.0 ** -16
        assert abs(float((g * d).sum() - diff)) <= eps * size, n
