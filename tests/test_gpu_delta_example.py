"""The example layer on layer norm, head norm with rotation and the gated delta rule: it
trains and serves, and its gradients are those of the formulas in float64."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "gated_delta_layer.py")


def _example():
    spec = importlib.util.spec_from_file_location("gated_delta_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _plain(p, layer, x, h):
    """The layer's output and final states in float64 on the CPU, token by token, from the
    parameters p."""
    G, H, K, V = layer.key_heads, layer.heads, layer.kdim, layer.vdim

    def norm(t, w, b):
        t = t - t.mean(-1, keepdim=True)
        return t / (t.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    def turned(t):  # [batch, seqlen, G, K]
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * K ** -0.5
        c, s = (layer.cos.double().cpu()[:x.shape[1], None], layer.sin.double().cpu()[:x.shape[1], None])
        a, b = t[..., :K // 2], t[..., K // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1).repeat_interleave(H // G, 2)

    q, k, v, a, b = (norm(x, p["norm_w"], p["norm_b"]) @ p["w_in"].T).split([G * K, G * K, H * V, H, H], -1)
    q, k, v = turned(q.unflatten(-1, (G, K))), turned(k.unflatten(-1, (G, K))), v.unflatten(-1, (H, V))
    decay = torch.exp(-p["rate"] * torch.nn.functional.softplus(a + p["decay_bias"]))
    beta, outs = torch.sigmoid(b), []
    for t in range(x.shape[1]):
        h = decay[:, t, :, None, None] * h
        r = v[:, t] - (h @ k[:, t, :, :, None])[..., 0]
        h = h + (beta[:, t, :, None] * r)[..., None] * k[:, t, :, None]
        outs.append((h @ q[:, t, :, :, None])[..., 0])
    o = norm(torch.stack(outs, 1), p["out_w"], p["out_b"])
    return x + o.flatten(-2) @ p["w_out"].T, h


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_trains_and_serves(dtype):
    """What is served token by token is what the whole sequences give.  Served and whole,
    every token goes through the same roundings: in bf16 those of the normed x, of q, k, v
    and beta, of o, normed o and y (which the projections' different summation order may
    flip), so 8 half-steps, 8 * 2^-8 of the largest value; in fp32 sums of up to 128 terms
    four deep, 4 * 128 * 2^-24 for both sides.  The recurrence mixes up to 100 tokens of
    random sign whose flips are independent; twice the bounds cover them."""
    m = _example()
    torch.manual_seed(0)
    layer = m.GatedDeltaLayer(128, 4, 2, 32, 48, 512, "cuda:0", dtype)
    losses = m.train(layer, 4, 2, 100)
    print(losses, flush=True)
    assert all(math.isfinite(x) for x in losses)
    worst, size = m.serve(layer, [70, 1, 33], 5)
    bound = 16 * 2.0 ** -8 if dtype is torch.bfloat16 else 16 * 128 * 2.0 ** -24
    print(worst, size, flush=True)
    assert worst <= bound * size


def test_layer_gradients():
    """In fp32: a gradient is a few products of up to 512 terms deep, each off by at most
    sqrt(512) 2^-24 < 2^-19 of its 2-norm, about sixteen of them from the loss to a
    parameter: 2^-15.  (The parameters that every token's layer norm meets sum terms of
    both signs, sqrt(tokens) of a term's size of 200 such: within the same.)"""
    m = _example()
    torch.manual_seed(1)
    layer = m.GatedDeltaLayer(64, 4, 2, 32, 48, 512, "cuda:0", torch.float32)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(2, 100, 64, generator=g)
    h0 = torch.randn(2, 4, 48, 32, generator=g)
    dy, dh = torch.randn(2, 100, 64, generator=g), torch.randn(2, 4, 48, 32, generator=g)
    xg, hg = x.cuda().requires_grad_(), h0.cuda().requires_grad_()
    y, h = layer(xg, h0=hg)
    ((y * dy.cuda()).sum() + (h * dh.cuda()).sum()).backward()
    p = {n: t.detach().double().cpu().requires_grad_() for n, t in layer.named_parameters()}
    xr, hr = x.double().requires_grad_(), h0.double().requires_grad_()
    yr, hl = _plain(p, layer, xr, hr)
    ((yr * dy.double()).sum() + (hl * dh.double()).sum()).backward()
    pairs = [("y", y, yr), ("h", h, hl), ("x", xg.grad, xr.grad), ("h0", hg.grad, hr.grad)]
    pairs += [(n, t.grad, p[n].grad) for n, t in layer.named_parameters()]
    for n, got, ref in pairs:
        ref = ref.detach()
        err = (got.detach().double().cpu() - ref).norm() / ref.norm()
        print(n, float(err), flush=True)
        assert float(err) <= 2.0 ** -15, n
