"""The gated delta rule and rotary positions in 64 bits on the CPU, straight
from their definitions (include/ssm_delta.h, include/ssm_rotary.h), and the
tolerances the kernels are held to.

Errors are 2-norms of the difference over the 2-norm of the reference.

Tolerances.  bf16 outputs are rounded once, by at most half a step, 2^-8 of the
value; what is rounded is formed from 16-bit planes (2^-16 for each of a handful of
factors), so 1.25 * 2^-8 bounds the sum.  fp32 results come from at most five
products in a row, each a sum of at most 256 terms: independent roundings of
2^-24 grow with the root of the count, 16 of them a product and 80 in all;
128 * 2^-24 leaves room for the plane products' own 2^-24 terms.  dg is the
difference of sums of that kind over the whole chunk: 512 * 2^-24 in fp32, and
in bf16 (16-bit planes, a cancellation of at most 16) 1.5 * 2^-8.
"""
import math

import torch

TOL = {torch.bfloat16: 1.25 * 2.0 ** -8, torch.float32: 128 * 2.0 ** -24}
TOL_DG = {torch.bfloat16: 1.5 * 2.0 ** -8, torch.float32: 512 * 2.0 ** -24}


def err(a, ref):
    a, ref = a.detach().double().cpu(), ref.detach().double().cpu()
    assert a.shape == ref.shape, (a.shape, ref.shape)
    if not torch.isfinite(a).all():
        return math.inf
    d, n = float((a - ref).norm()), float(ref.norm())
    return d / n if n else d


def make(B, L, Hk, Hv, K, V, dtype, seed, h0=True, device="cpu"):
    """Inputs as a model leaves them: unit queries and keys, decays between about 0.2 and 1."""
    g = torch.Generator().manual_seed(seed)

    def n(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    q, k = [x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt() for x in
            (torch.nn.functional.silu(n(B, L, Hk, K)), torch.nn.functional.silu(n(B, L, Hk, K)))]
    rate = torch.rand(Hv, generator=g, dtype=torch.float64) * 2
    out = dict(q=q, k=k, v=n(B, L, Hv, V), g=-rate.exp() * torch.nn.functional.softplus(n(B, L, Hv) - 3),
               beta=torch.sigmoid(n(B, L, Hv)))
    out = {a: x.to(dtype).to(device) for a, x in out.items()}
    out["h0"] = (0.3 * n(B, Hv, V, K)).float().to(device) if h0 else None
    return out


def reference(q, k, v, g, beta, h0, scale=None, lengths=None):
    """(y, h_last), one step at a time; differentiable.  Rows behind a length are zeros of y."""
    B, L, Hk, K = q.shape
    Hv, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    own = torch.arange(Hv) // (Hv // Hk)
    S = torch.zeros(B, Hv, V, K, dtype=torch.float64) if h0 is None else h0
    lens = torch.full((B,), L) if lengths is None else lengths.clamp(0, L)
    ys = []
    for t in range(L):
        live = (t < lens).view(B, 1, 1, 1)
        kt, qt = k[:, t, own], q[:, t, own]
        d = S * g[:, t].exp()[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - (d * kt[:, :, None]).sum(-1))
        new = d + u[..., None] * kt[:, :, None]
        S = torch.where(live, new, S)
        ys.append(torch.where(live[..., 0], scale * (S * qt[:, :, None]).sum(-1), 0.0))
    return torch.stack(ys, 1), S


NAMES = ("q", "k", "v", "g", "beta", "h0")


def wide(inputs):
    return {n: None if inputs[n] is None else inputs[n].detach().cpu().double() for n in NAMES}


def reference_grads(inputs, dy, dh, scale=None, lengths=None):
    w = {n: None if x is None else x.requires_grad_() for n, x in wide(inputs).items()}
    y, h = reference(**w, scale=scale, lengths=lengths)
    loss = (y * dy.cpu().double()).sum()
    if dh is not None:
        loss = loss + (h * dh.cpu().double()).sum()
    loss.backward()
    return {"d" + n: x.grad for n, x in w.items() if x is not None}


def rotary_reference(x, inv_freq, positions, interleaved=False, amplitude=1.0, inverse=False):
    x = x.detach().cpu().double().clone()
    R = 2 * inv_freq.numel()
    t = positions.cpu().double()[:, :, None, None] * inv_freq.cpu().double()
    c, s = amplitude * t.cos(), amplitude * t.sin() * (-1 if inverse else 1)
    ia, ib = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = x[..., ia].clone(), x[..., ib].clone()
    x[..., ia], x[..., ib] = a * c - b * s, a * s + b * c
    return x
