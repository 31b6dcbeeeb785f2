"""The gated delta rule and layer norm from their definitions in float64, the
delta rule token by token with its adjoint.  Shared by the tests; nothing here is
used by the package.

Bounds.  Sums are fp32 (24 bits), what enters a state or its adjoint keeps 24 bits,
and what is only rounded to bf16 next keeps 16 (2^-17 of every operand).  A result
is a few hundred such roundings of random sign deep, each about 2^-24 of the
result's size (sqrt(512) 2^-24 < 2^-19), and passes a handful of chunks before it is
forgotten: 2^-18 of its 2-norm, and 2^-15 more where two-part operands enter
(bf16).  Rounded to bf16, whose steps are 2^-7 of a power of two, it is off by at most
half a step, 2^-8 of itself.  A single value may be
six times the root mean square off, of up to 2^20 values: 2^-14 of the largest of
its sequence and head.  (The recurrence does not amplify what it carries on: beta
|k|^2 <= 2 and no decay above 0, where a test does not say otherwise.)"""
import torch

F64 = torch.float64
GRADS = ("dq", "dk", "dv", "dlog_decay", "dbeta", "dh0")


def _heads(t, rep):
    return t.to(F64).repeat_interleave(rep, 1)


def walk(q, k, v, g, b, h0, scale):
    """One sequence: q, k [L, G, K], v [L, H, V], g, b [L, H] -> o, h_last, states."""
    H, rep = v.shape[1], v.shape[1] // q.shape[1]
    q, k, v, a, b = _heads(q, rep), _heads(k, rep), v.to(F64), torch.exp(g.to(F64)), b.to(F64)
    s = (torch.zeros(H, v.shape[2], q.shape[2], dtype=F64, device=q.device) if h0 is None
         else h0.to(F64))
    o, states = torch.zeros_like(v), [s]
    for t in range(q.shape[0]):
        s = a[t][:, None, None] * s
        u = b[t][:, None] * (v[t] - (s * k[t][:, None, :]).sum(-1))
        s = s + u[:, :, None] * k[t][:, None, :]
        o[t] = scale * (s * q[t][:, None, :]).sum(-1)
        states.append(s)
    return o, s, states


def walk_bwd(q, k, v, g, b, h0, scale, dy, dh):
    """Adjoint of ``walk``: gradients by name, and the sizes of dlog_decay's terms."""
    L, G, K = q.shape
    H, V = v.shape[1:]
    rep = H // G
    _, last, states = walk(q, k, v, g, b, h0, scale)
    q, k, v, a, b, dy = (_heads(q, rep), _heads(k, rep), v.to(F64), torch.exp(g.to(F64)), b.to(F64),
                         dy.to(F64))
    d = torch.zeros_like(last) if dh is None else dh.to(F64)
    dq, dk = (torch.zeros(L, H, K, dtype=F64, device=q.device) for _ in "12")
    dv, dg, db = torch.zeros_like(v), torch.zeros_like(b), torch.zeros_like(b)
    mass = torch.zeros_like(b)
    for t in reversed(range(L)):
        old, new, at = states[t], states[t + 1], a[t][:, None, None]
        if t % 64 == 63 or t == L - 1:
            mass[t] = (d * new).flatten(1).norm(dim=1) + d.flatten(1).norm(dim=1) * new.flatten(
                1).norm(dim=1) * 2.0 ** -4
        d = d + scale * dy[t][:, :, None] * q[t][:, None, :]
        dq[t] = scale * (new * dy[t][:, :, None]).sum(1)
        e = (old * k[t][:, None, :]).sum(-1)
        r = v[t] - a[t][:, None] * e
        du = (d * k[t][:, None, :]).sum(-1)
        dr = b[t][:, None] * du
        db[t], dv[t] = (du * r).sum(-1), dr
        dk[t] = (d * (b[t][:, None] * r)[:, :, None]).sum(1) - at[..., 0] * (
            old * dr[:, :, None]).sum(1)
        dg[t] = a[t] * ((d * old).sum((1, 2)) - (dr * e).sum(-1))
        d = at * (d - dr[:, :, None] * k[t][:, None, :])
    mass += q.norm(dim=-1) * dq.norm(dim=-1) + v.norm(dim=-1) * dv.norm(dim=-1)
    for t in reversed(range(L - 1)):       # the chunk's sums run from its end
        if t % 64 != 63:
            mass[t] += mass[t + 1]
    return {"dq": dq.view(L, G, rep, K).sum(2), "dk": dk.view(L, G, rep, K).sum(2), "dv": dv,
            "dlog_decay": dg, "dbeta": db, "dh0": d}, mass


def _cuts(lens):
    at = 0
    for n, L in enumerate(lens):
        yield n, slice(at, at + L)
        at += L


def prompt(p, lens, scale):
    """Flat tokens cut by ``lens``: o, h_last."""
    os_, hs = [], []
    for n, s in _cuts(lens):
        o, h, _ = walk(*(p[x][s] for x in ("q", "k", "v", "log_decay", "beta")),
                       None if p["h0"] is None else p["h0"][n], scale)
        os_.append(o)
        hs.append(h)
    return torch.cat(os_), torch.stack(hs)


def prompt_bwd(p, lens, scale):
    """Gradients by name, and the sizes of dlog_decay's terms."""
    parts, mass = [], []
    for n, s in _cuts(lens):
        r, m = walk_bwd(*(p[x][s] for x in ("q", "k", "v", "log_decay", "beta")),
                        None if p["h0"] is None else p["h0"][n], scale, p["dy"][s],
                        None if p["dh_last"] is None else p["dh_last"][n])
        parts.append(r)
        mass.append(m)
    r = {n: torch.cat([x[n] for x in parts]) for n in GRADS[:-1]}
    r["dh0"] = torch.stack([x["dh0"] for x in parts])
    return r, torch.cat(mass)


def check(got, ref, what, bf16, mass=None):
    """``bf16``: the operands are.  ``mass``: sizes that the bounds go by, of every
    value, in place of the values' own."""
    got64 = got.to(F64).reshape(ref.shape)
    assert torch.isfinite(got64).all(), f"{what}: not finite"
    if ref.numel() == 0:
        return
    err = (got64 - ref).abs()
    half = 2.0 ** -8 * 1.01 * ref.abs() if got.dtype is torch.bfloat16 else torch.zeros_like(ref)
    eps = 2.0 ** -18 + (2.0 ** -15 if bf16 and got.dtype is torch.bfloat16 else 0.0)
    size = ref if mass is None else mass
    over = (err - half).clamp(min=0.0)
    assert float(over.norm()) <= eps * float(size.norm()) + 1e-37, (
        what, "2-norm", float(over.norm() / size.norm().clamp(min=1e-300)), "of", eps)
    top = float(size.abs().max())
    bad = over - 2.0 ** -14 * top - 1e-37
    if float(bad.max()) > 0:
        i = int(bad.argmax())
        raise AssertionError(f"{what}: worst at flat {i}: got {float(got64.flatten()[i])!r} ref "
                             f"{float(ref.flatten()[i])!r}, largest {top!r}")


def norm(x, w, b, eps):
    x = x.to(F64)
    x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    y = y if w is None else y * w.to(F64)
    return y if b is None else y + b.to(F64)


def norm_bwd(x, w, dy, eps):
    """dx, dweight, dbias of rows [n, dim]."""
    x, dy = x.to(F64), dy.to(F64)
    x = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    h, g = x * r, dy if w is None else dy * w.to(F64)
    dx = r * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)
