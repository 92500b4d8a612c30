"""64-bit references of the operators around linear layers, from their definitions (torch on any device; nothing of the
library)."""
import math

import torch

U32 = 2.0 ** -24  # half a step of fp32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(v, dtype):
    """The most by which rounding to the type moves v: half a step of its size, and below the smallest normal number,
    where steps no longer shrink, half of the step there."""
    return v.abs().clamp_min(torch.finfo(dtype).smallest_normal) * half_step(dtype)


def random_bits(seed, offset, M, N, device="cpu"):
    """16 bits for each element: Philox4x32-10, by products of 16-bit halves."""
    mask, low = 0xFFFF, 0xFFFFFFFF
    seed, offset = seed % 2 ** 64, offset % 2 ** 64

    def halves(a, b):
        ll, lh, hl, hh = (a & mask) * (b & mask), (a & mask) * (b >> 16), (a >> 16) * (b & mask), (a >> 16) * (b >> 16)
        mid = (ll >> 16) + (lh & mask) + (hl & mask)
        return hh + (lh >> 16) + (hl >> 16) + (mid >> 16), (mid & mask) << 16 | ll & mask

    groups = -(-N // 8)
    c = [torch.arange(groups, device=device).expand(M, groups), torch.arange(M, device=device)[:, None].expand(M, groups),
         torch.full((M, groups), offset & low, device=device), torch.full((M, groups), offset >> 32, device=device)]
    k = [seed & low, seed >> 32]
    for _ in range(10):
        (h0, l0), (h1, l1) = halves(c[0], 0xD2511F53), halves(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k[0], l1, h0 ^ c[3] ^ k[1], l0]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return torch.stack([v for w in c for v in (w & mask, w >> 16)], 2).reshape(M, groups * 8)[:, :N]


def drop(v, p, rng):
    """dropout(v) in 64 bits; rng is (seed, offset)."""
    least = round(65536 * p)
    if least == 0:
        return v
    kept = random_bits(*rng, *v.shape, device=v.device) >= least
    return torch.where(kept, v / (1 - least / 65536) if least < 65536 else v, torch.zeros_like(v))


def act(z, kind):
    if kind == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if kind == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z


def act_grad(z, kind):
    if kind == "relu":
        return torch.where(z > 0, 1.0, torch.where(torch.isnan(z), z, torch.zeros_like(z)))
    if kind == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-k * (z + 0.044715 * z ** 3)))
        return s + z * s * (1 - s) * k * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def norm(v, kind, weight, bias, eps):
    """(output, normalised, factor)"""
    if kind is None:
        return v, v, None
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + eps)
    hat = v * r
    out = hat if weight is None else hat * weight
    return (out if bias is None else out + bias), hat, r


def norm_grad(d, kind, weight, hat, r):
    g = d if weight is None else d * weight
    v = g - hat * (g * hat).mean(1, keepdim=True)
    return r * (v - g.mean(1, keepdim=True) if kind == "layer" else v)


def norm_join(y, x=None, gate=None, scale=1.0, post=None, post_weight=None, post_bias=None, pre=None, weight=None, bias=None,
              eps=1e-6):
    """All of the forward pass in 64 bits, as a dict, and as "|name|" the sizes of what each value is the sum of: what its
    rounding errors are relative to, where the terms cancel."""
    y, x, gate, post_weight, post_bias, weight, bias = (
        None if t is None else t.detach().double() for t in (y, x, gate, post_weight, post_bias, weight, bias))
    one = lambda t, none: none if t is None else t.abs()

    def hat_size(hat, r, size, kind):
        # a centred value is a difference; the factor's relative error is that of the mean square of such values
        if kind is None:
            return size, 0.0
        s = r * (size + (size.mean(1, keepdim=True) if kind == "layer" else 0))
        of_r = (hat.abs() * s).mean(1, keepdim=True)
        return s + hat.abs() * of_r, of_r

    u, yhat, yr = norm(y, post, post_weight, post_bias, eps)
    ysize, y_of_r = hat_size(yhat, yr, y.abs(), post)
    usize = ysize * one(post_weight, 1.0) + one(post_bias, 0.0)
    wide = torch.ones_like(y) if gate is None else gate.repeat_interleave(y.shape[0] // gate.shape[0], 0)
    h = scale * wide * u + (0 if x is None else x)
    hsize = scale * wide.abs() * usize + one(x, 0.0)
    n, hhat, hr = norm(h, pre, weight, bias, eps)
    hhsize, h_of_r = hat_size(hhat, hr, hsize, pre)
    return {"u": u, "yhat": yhat, "yr": yr, "gate": wide, "h": h, "n": n, "hhat": hhat, "hr": hr, "|u|": usize, "|yhat|": ysize,
            "|hhat|": hhsize, "y of r": y_of_r, "h of r": h_of_r}


def norm_join_grad(f, dh, dn, gate_rows, scale, post, post_weight, pre, weight):
    """Gradients from norm_join's dict, and as "|name|" the sizes of their terms."""
    post_weight, weight = (None if t is None else t.detach().double() for t in (post_weight, weight))
    o = {}

    def size(g, kind, w, hat, r, of_r):
        g = g if w is None else g * w.abs()
        s = g + hat * (g * hat).mean(1, keepdim=True) + (g.mean(1, keepdim=True) if kind == "layer" else 0)
        return r * s * (1 + of_r)

    dH = torch.zeros_like(f["h"]) if dh is None else dh.double()
    s = dH.abs()
    if dn is not None:
        dn = dn.double()
        dH = dH + norm_grad(dn, pre, weight, f["hhat"], f["hr"])
        s = s + size(dn.abs(), pre, weight, f["|hhat|"], f["hr"], f["h of r"])
        o["dweight"], o["|dweight|"] = (dn * f["hhat"]).sum(0), (dn.abs() * f["|hhat|"]).sum(0)
        o["dbias"], o["|dbias|"] = dn.sum(0), dn.abs().sum(0)
    o["dx"], o["|dx|"] = dH, s
    du, s = dH * scale, s * scale
    if gate_rows:
        D = du.shape[1]
        o["dgate"], o["|dgate|"] = (du * f["u"]).view(gate_rows, -1, D).sum(1), (s * f["|u|"]).view(gate_rows, -1, D).sum(1)
    du, s = du * f["gate"], s * f["gate"].abs()
    o["dy"], o["|dy|"] = du, s
    if post:
        o["dpost_weight"], o["|dpost_weight|"] = (du * f["yhat"]).sum(0), (s * f["|yhat|"]).sum(0)
        o["dpost_bias"], o["|dpost_bias|"] = du.sum(0), s.sum(0)
        o["dy"] = norm_grad(du, post, post_weight, f["yhat"], f["yr"])
        o["|dy|"] = size(s, post, post_weight, f["|yhat|"], f["yr"], f["y of r"])
    return o
