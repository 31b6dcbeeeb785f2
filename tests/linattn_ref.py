"""Linear attention with one decay per head, and the head norm with rotation,
from their definitions in float64: token-by-token recurrences and their
adjoints.  Shared by the GPU tests; nothing here is used by the package.

Error bounds.  Every result is a sum of products, so its size before
cancellation is the same sum over absolute values ("mass").  Operands that are
bf16 enter exactly; a weighted product or a state that enters a product as two
bf16 parts (8 significant bits each) is off by at most 2^-16 of itself, and a
result passes through two such places (2^-15); sums of n fp32 terms add at most
n 2^-24 of the mass, n below 512 here for the terms that share an accumulator
between decays (2^-15).  A computed value is therefore within 2^-14 of its
mass; fp32 operands and fp32 states have no two-part places and stay within
2^-15.  Storing bf16 adds half a unit of its last place, 2^-8 of the value."""
import torch

F64 = torch.float64


def walk(q, k, v, g, h0, scale):
    """One sequence: q [L, H, K], k [L, G, K], v [L, G, V] -> o, h_last."""
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    H, rep = q.shape[1], q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    a = torch.exp(g.to(F64))[:, None, None]
    s = (torch.zeros(H, v.shape[2], q.shape[2], dtype=F64, device=q.device) if h0 is None
         else h0.to(F64))
    o = torch.zeros(q.shape[0], H, v.shape[2], dtype=F64, device=q.device)
    for t in range(q.shape[0]):
        s = a * s + v[t][:, :, None] * k[t][:, None, :]
        o[t] = scale * (s * q[t][:, None, :]).sum(-1)
    return o, s


def walk_bwd(q, k, v, g, h0, scale, dy, dh):
    """Adjoint of ``walk``: dq, dk, dv, dg, dh0."""
    q, k, v, dy = q.to(F64), k.to(F64), v.to(F64), dy.to(F64)
    H, G = q.shape[1], k.shape[1]
    rep = H // G
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    a = torch.exp(g.to(F64))[:, None, None]
    L, K, V, dev = q.shape[0], q.shape[2], v.shape[2], q.device
    zero = torch.zeros(H, V, K, dtype=F64, device=dev)
    s = zero if h0 is None else h0.to(F64)
    tan = zero
    dq, dk, dv = (torch.zeros(L, H, d, dtype=F64, device=dev) for d in (K, K, V))
    dg = torch.zeros(H, dtype=F64, device=dev)
    for t in range(L):
        tan = a * (tan + s)
        s = a * s + v[t][:, :, None] * k[t][:, None, :]
        dq[t] = scale * (s * dy[t][:, :, None]).sum(1)
        dg += scale * (tan * dy[t][:, :, None] * q[t][:, None, :]).sum((1, 2))
    adj = zero if dh is None else dh.to(F64)
    dg += (tan * adj).sum((1, 2))
    for t in reversed(range(L)):
        adj = adj + scale * dy[t][:, :, None] * q[t][:, None, :]
        dv[t] = (adj * k[t][:, None, :]).sum(-1)
        dk[t] = (adj * v[t][:, :, None]).sum(1)
        adj = a * adj
    return {"dq": dq, "dk": dk.view(L, G, rep, K).sum(2), "dv": dv.view(L, G, rep, V).sum(2),
            "dlog_decay": dg, "dh0": adj}


def _abs(t):
    return None if t is None else t.abs()


def prompt(q, k, v, g, h0, scale, lens):
    """Flat tokens [T, ...] cut by ``lens``: (o, h_last) and their masses."""
    outs = []
    for f in (lambda t: t, _abs):
        os_, hs, at = [], [], 0
        for n, L in enumerate(lens):
            sl = slice(at, at + L)
            o, h = walk(f(q[sl]), f(k[sl]), f(v[sl]), g, None if h0 is None else f(h0[n]),
                        abs(scale) if f is _abs else scale)
            os_.append(o)
            hs.append(h)
            at += L
        outs.append((torch.cat(os_), torch.stack(hs)))
    return outs


def prompt_bwd(q, k, v, g, h0, scale, lens, dy, dh):
    """Gradients by name and their masses; dlog_decay summed over sequences."""
    outs = []
    for f in (lambda t: t, _abs):
        parts, at = [], 0
        for n, L in enumerate(lens):
            sl = slice(at, at + L)
            parts.append(walk_bwd(f(q[sl]), f(k[sl]), f(v[sl]), g,
                                  None if h0 is None else f(h0[n]),
                                  abs(scale) if f is _abs else scale, f(dy[sl]),
                                  None if dh is None else f(dh[n])))
            at += L
        r = {n: torch.cat([p[n] for p in parts]) for n in ("dq", "dk", "dv")}
        r["dh0"] = torch.stack([p["dh0"] for p in parts])
        r["dlog_decay"] = sum(p["dlog_decay"] for p in parts)
        outs.append(r)
    return outs


def check(got, ref, mass, what, parts=None):
    """``parts``: the operands are bf16 (products in two parts); default: by got's type."""
    got64 = got.to(F64).reshape(ref.shape)
    assert torch.isfinite(got64).all(), f"{what}: not finite"
    bf16 = got.dtype == torch.bfloat16
    eps = 2.0 ** -14 if bf16 and parts is None else 2.0 ** -15
    bound = eps * mass + (2.0 ** -8 * 1.01 * ref.abs() if bf16 else 0.0) + 1e-37
    bad = (got64 - ref).abs() - bound
    if bad.numel() and float(bad.max()) > 0:
        i = int(bad.argmax())
        raise AssertionError(f"{what}: {int((bad > 0).sum())} of {bad.numel()} off, worst at flat "
                             f"{i}: got {float(got64.flatten()[i])!r} ref "
                             f"{float(ref.flatten()[i])!r} bound {float(bound.flatten()[i])!r}")


def rotate(x, w, cos, sin, pos, eps, interleaved):
    """[T, h, d] by complex numbers."""
    x = x.to(F64)
    u = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    u = u if w is None else u * w.to(F64)
    n = 0 if cos is None else cos.shape[1]
    if n == 0:
        return u
    i = torch.arange(n, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    z = torch.complex(u[..., ia], u[..., ib]) * torch.complex(
        cos.to(F64), sin.to(F64))[pos][:, None]
    out = u.clone()
    out[..., ia], out[..., ib] = z.real, z.imag
    return out


def angles(npos, rot, device):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=F64, device=device) / max(rot, 1))
    t = torch.arange(npos, dtype=F64, device=device)[:, None] * f
    return t.cos().float(), t.sin().float()
