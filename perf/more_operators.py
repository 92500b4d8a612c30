"""Cases for the operators at the sides of a block's linear layers: a matrix product with its epilogue, the norms around
a block's end, dropout.

Definitions:

* dropout: r(i, j) is the 16-bit lane j % 8 of Philox4x32-10 (Salmon and others, 2011) with the seed's two words as key
  and (j / 8, i, the offset's two words) as counter; lane 2 w + 1 is the upper half of output word w.  With
  T = round(65536 p), an element v of row i, column j becomes v / (1 - T / 65536) where r >= T, else 0.
* linear: z = x @ w + bias, out = residual + dropout(act(z)).  Training: also the gradients of x, w, bias and residual.
* norm: u = post-norm of y (or y), h = x + scale * gate * u, n = pre-norm of h.  A norm is v / sqrt(mean(v^2) + eps)
  ("rms") or (v - mean) / sqrt(var + eps) ("layer"), times a weight, plus a bias.  A gate row serves M / G rows of y.
  Training: also the gradients of y, x, gate, weights and biases.
"""
import math

import torch

#: Set by the program that runs the cases: False for the plain forms, True for the framework's operators.
own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_EPS = 1e-6


def listed():
    return [
        # one token through an up projection: the weights are read once
        {"name": "linear_token", "op": "linear", "train": False, "M": 1, "K": 4096, "N": 14336, "src": "bf16",
         "trans": False, "bias": True, "act": "gelu_tanh", "residual": False, "p": 0.0},
        # a decoding batch through a down projection whose weights are stored (N, K), added to the residual stream
        {"name": "linear_batch", "op": "linear", "train": False, "M": 48, "K": 14336, "N": 4096, "src": "bf16",
         "trans": True, "bias": False, "act": "none", "residual": True, "p": 0.0},
        # a short prompt, nothing a multiple of anything
        {"name": "linear_odd", "op": "linear", "train": False, "M": 333, "K": 1000, "N": 1111, "src": "f16",
         "trans": False, "bias": True, "act": "silu", "residual": True, "p": 0.0},
        # a prompt through an up projection
        {"name": "linear_prompt", "op": "linear", "train": False, "M": 4096, "K": 4096, "N": 14336, "src": "bf16",
         "trans": False, "bias": True, "act": "gelu", "residual": False, "p": 0.0},
        # a training step of an up projection: activation, bias, all gradients
        {"name": "linear_train", "op": "linear", "train": True, "M": 4096, "K": 4096, "N": 14336, "src": "bf16",
         "trans": False, "bias": True, "act": "gelu_tanh", "residual": False, "p": 0.0},
        # a training step of a narrow model's down projection: dropout before the residual, all gradients
        {"name": "linear_train_drop", "op": "linear", "train": True, "M": 2048, "K": 4096, "N": 1024, "src": "f16",
         "trans": False, "bias": True, "act": "none", "residual": True, "p": 0.1},
        # the end of a block while decoding one token: latency only
        {"name": "norm_token", "op": "norm", "train": False, "M": 1, "D": 4096, "src": "bf16", "res": "bf16", "x": True,
         "gate": "none", "groups": 1, "post": "none", "pre": "rms", "affine": True},
        # a long prompt: post-norm, a learned scale for each channel, a 32-bit residual stream, the next block's pre-norm
        {"name": "norm_prompt", "op": "norm", "train": False, "M": 16384, "D": 4096, "src": "bf16", "res": "f32", "x": True,
         "gate": "channel", "groups": 1, "post": "rms", "pre": "rms", "affine": True},
        # a training step of conditioned blocks: a gate for each of 8 sequences, layer norm before the next block
        {"name": "norm_train", "op": "norm", "train": True, "M": 16384, "D": 4096, "src": "bf16", "res": "bf16", "x": True,
         "gate": "sequence", "groups": 8, "post": "none", "pre": "layer", "affine": True},
        # a training step of odd sizes, rows that do not start on 16 bytes, both norms
        {"name": "norm_train_odd", "op": "norm", "train": True, "M": 1537, "D": 5003, "src": "f16", "res": "f16", "x": True,
         "gate": "channel", "groups": 1, "post": "rms", "pre": "rms", "affine": True},
        # a block's output on its way to the residual stream of a training batch
        {"name": "dropout_residual", "op": "dropout", "train": False, "M": 16384, "N": 4096, "src": "bf16", "residual": True, "p": 0.1},
        # embeddings in 32 bits, odd sizes, forward and gradient
        {"name": "dropout_train_odd", "op": "dropout", "train": True, "M": 1537, "N": 5003, "src": "f32", "residual": False, "p": 0.25},
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["linear", "linear", "norm", "norm", "dropout"])
        c = {"op": op, "train": rng.random() < 0.5, "src": rng.choice(["bf16", "bf16", "f16"])}
        if op == "linear":
            c["M"], c["K"], c["N"] = _log(rng, 1, 16384), _log(rng, 100, 16384), _log(rng, 100, 16384)
            if rng.random() < 0.5:  # half of all layers have widths of whole cache lines
                c["K"], c["N"] = (c["K"] + 63) // 64 * 64, (c["N"] + 63) // 64 * 64
            c["trans"], c["bias"], c["residual"] = rng.random() < 0.5, rng.random() < 0.7, rng.random() < 0.5
            # no relu in training: where a sum is next to its step, one rounding changes a whole row of gradients
            c["act"] = rng.choice(["none", "gelu", "gelu_tanh", "silu"] + ([] if c["train"] else ["relu"]))
            c["p"] = round(rng.uniform(0.05, 0.5), 3) if c["train"] and rng.random() < 0.5 else 0.0
            if c["M"] * c["K"] * c["N"] * (3 if c["train"] else 1) > 3 * 4096 * 4096 * 14336:
                continue
            return c
        if op == "dropout":
            c["M"], c["N"] = _log(rng, 1, 65536), _log(rng, 64, 16384)
            c["src"] = rng.choice(["bf16", "f16", "f32"])
            c["residual"], c["p"] = rng.random() < 0.5, round(rng.uniform(0.02, 0.6), 3)
            if c["M"] * c["N"] > 16384 * 4096:
                continue
            return c
        c["gate"] = rng.choice(["none", "channel", "sequence", "token"])
        rows = _log(rng, 1, 16384)
        c["groups"] = _log(rng, 1, 64) if c["gate"] == "sequence" else 1
        c["M"], c["D"] = rows * c["groups"], _log(rng, 64, 16384)
        if rng.random() < 0.5:
            c["D"] = (c["D"] + 63) // 64 * 64
        c["src"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        c["res"] = rng.choice([c["src"], c["src"], "f32"])
        c["x"], c["affine"] = rng.random() < 0.8, rng.random() < 0.8
        c["post"], c["pre"] = rng.choice(["none", "rms", "layer"]), rng.choice(["rms", "rms", "layer", "none"])
        if c["post"] == "none" and c["pre"] == "none":
            continue
        if not c["x"]:
            c["res"] = c["src"]
        if c["M"] * c["D"] > 16384 * 4096:
            continue
        return c


def _values(g, M, K, spread):
    """Normal values whose rows and columns differ in size, as activations, weights and gradients have them."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x *= torch.exp(spread * torch.randn(M, 1, generator=g, device="cuda"))
    x *= torch.exp(0.5 * torch.randn(1, K, generator=g, device="cuda"))
    return x


def _unit(x):
    return x / x.square().mean().sqrt()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = dict(case), {"case": dict(case)}
    src, M, train = _T[c["src"]], c["M"], c["train"]
    if c.get("p", 0.0) > 0:
        s["rng"] = torch.tensor([(seed * 0x9E3779B1 + 12345) % 2 ** 62, 3 + seed], dtype=torch.int64, device="cuda")
    if c["op"] == "linear":
        K, N = c["K"], c["N"]
        s["x"] = _unit(_values(g, M, K, 0.5)).to(src)
        w = _values(g, N, K, 0.2).t() if c["trans"] else _values(g, K, N, 0.2)
        s["w"] = (_unit(w) / math.sqrt(K)).to(src)  # keeps the strides: (N, K) in memory where transposed
        s["bias"] = (0.1 * torch.randn(N, generator=g, device="cuda")).to(src) if c["bias"] else None
        s["residual"] = torch.randn(M, N, generator=g, device="cuda").to(src) if c["residual"] else None
        leaves = ("x", "w", "bias", "residual")
        if train:
            s["dy"] = _unit(_values(g, M, N, 0.5)).to(src)
        else:
            s["out"] = torch.empty(M, N, dtype=src, device="cuda")
    elif c["op"] == "norm":
        D, res = c["D"], _T[c["res"]]
        s["y"] = _unit(_values(g, M, D, 0.5)).to(src)
        s["x"] = (4 * _unit(_values(g, M, D, 0.3)) + 0.2).to(res) if c["x"] else None
        rows = {"none": 0, "channel": 1, "sequence": c["groups"], "token": M}[c["gate"]]
        s["gate"] = (0.5 + 0.3 * torch.randn(rows, D, generator=g, device="cuda")).to(src) if rows else None
        for name in ("post", "pre"):
            has = c[name] != "none" and c["affine"]
            s[name + "_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(src) if has else None
            has = has and c[name] == "layer"
            s[name + "_bias"] = (0.1 * torch.randn(D, generator=g, device="cuda")).to(src) if has else None
        leaves = ("y", "x", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")
        joins = _joins(c)
        if train:
            s["dh"] = _unit(_values(g, M, D, 0.5)).to(res) if joins else None
            s["dn"] = _unit(_values(g, M, D, 0.5)).to(src) if c["pre"] != "none" else None
        else:
            s["h"] = torch.empty(M, D, dtype=res, device="cuda") if joins else None
            s["n"] = torch.empty(M, D, dtype=src, device="cuda") if c["pre"] != "none" else None
    else:
        N = c["N"]
        s["x"] = _values(g, M, N, 0.5).to(src)
        s["residual"] = torch.randn(M, N, generator=g, device="cuda").to(src) if c["residual"] else None
        leaves = ("x", "residual")
        if train:
            s["dy"] = _values(g, M, N, 0.5).to(src)
        else:
            s["out"] = torch.empty(M, N, dtype=src, device="cuda")
    if train:
        s["leaves"] = [k for k in leaves if s[k] is not None]
        for k in s["leaves"]:
            s[k].requires_grad_()
    return s


def _joins(c):
    """Whether h is anything but y."""
    return c["x"] or c["gate"] != "none" or c["post"] != "none"


_SCALE = 0.75  # the norm cases' residual scale


# ------------------------------------------------------------------ plain forms

def _words(rng):
    """The generator's key and offset as four 32-bit words, (1, 1) tensors."""
    v = torch.stack((rng & 0xFFFFFFFF, rng >> 32 & 0xFFFFFFFF))  # (low, high) x (seed, offset)
    return v[0, 0].view(1, 1), v[1, 0].view(1, 1), v[0, 1].view(1, 1), v[1, 1].view(1, 1)


def _philox(rng, M, N):
    """16-bit random numbers (M, N), by 64-bit products of which the two halves are taken."""
    low, mask = 0xFFFFFFFF, 0xFFFF
    k0, k1, o0, o1 = _words(rng)
    groups = (N + 7) // 8
    c0 = torch.arange(groups, device=rng.device).view(1, -1).expand(M, -1)
    c1 = torch.arange(M, device=rng.device).view(-1, 1).expand(-1, groups)
    c2, c3 = o0.expand(M, groups), o1.expand(M, groups)
    for i in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # wrap around at 64 bits
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    lanes = [v for c in (c0, c1, c2, c3) for v in (c & mask, c >> 16)]
    return torch.stack(lanes, 2).view(M, groups * 8)[:, :N]


def _drop(v, rng, p):
    t = round(p * 65536)
    return torch.where(_philox(rng, *v.shape) >= t, v * (65536.0 / (65536 - t)), 0.0)


_ROOT = math.sqrt(2 / math.pi)


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_ROOT * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_ROOT * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _ROOT * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        e = 1 / (1 + torch.exp(-z))
        return e * (1 + z * (1 - e))
    return torch.ones_like(z)


def _norm(v, kind, weight, bias):
    """The norm of v, the normalised v and the factor that normalised it."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + _EPS)
    hat = v * r
    out = hat if weight is None else hat * weight.float()
    return (out if bias is None else out + bias.float()), hat, r


def _norm_grad(d, kind, weight, hat, r):
    """Gradients of a norm's input and weight from that of its output."""
    g = d if weight is None else d * weight.float()
    dv = g - hat * (g * hat).mean(1, keepdim=True)
    if kind == "layer":
        dv = dv - g.mean(1, keepdim=True)
    return dv * r, (d * hat).sum(0)


def _plain_norm(s):
    c = s["case"]
    y = s["y"].float()
    u, yhat, yr = _norm(y, c["post"], s["post_weight"], s["post_bias"]) if c["post"] != "none" else (y, None, None)
    gate, h = None, u
    if s["gate"] is not None:
        gate = s["gate"].float().repeat_interleave(c["M"] // s["gate"].shape[0], 0)
        h = gate * h
    joins = _joins(c)
    if joins:
        h = _SCALE * h
    if s["x"] is not None:
        h = s["x"].float() + h
    o = {}
    if joins:
        o["h"] = h.to(_T[c["res"]])
    if c["pre"] != "none":
        n, hhat, hr = _norm(h, c["pre"], s["pre_weight"], s["pre_bias"])
        o["n"] = n.to(_T[c["src"]])
    if not c["train"]:
        return o
    dH = 0
    if joins:
        dH = s["dh"].float()
    if c["pre"] != "none":
        dn = s["dn"].float()
        dv, dw = _norm_grad(dn, c["pre"], s["pre_weight"], hhat, hr)
        dH = dH + dv
        o["pre_weight"], o["pre_bias"] = dw, dn.sum(0)
    o["x"] = dH
    du = dH * _SCALE if joins else dH
    if gate is not None:
        o["gate"] = (du * u).view(s["gate"].shape[0], -1, c["D"]).sum(1)
        du = du * gate
    o["y"] = du
    if c["post"] != "none":
        o["y"], o["post_weight"] = _norm_grad(du, c["post"], s["post_weight"], yhat, yr)
        o["post_bias"] = du.sum(0)
    return {k: o[k] for k in ("h", "n") if k in o} | {"d" + k: o[k].to(s[k].dtype) for k in s["leaves"]}


def _plain_linear(s):
    c = s["case"]
    x, w, src = s["x"].float(), s["w"].float(), _T[c["src"]]
    z = x @ w
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if c["p"] > 0:
        y = _drop(y, s["rng"], c["p"])
    if s["residual"] is not None:
        y = s["residual"].float() + y
    if not c["train"]:
        return {"out": y.to(src)}
    dz = s["dy"].float()
    if c["p"] > 0:
        dz = _drop(dz, s["rng"], c["p"])
    dz = dz * _act_grad(z, c["act"])
    o = {"out": y.to(src), "dx": (dz @ w.t()).to(src), "dw": (x.t() @ dz).to(src)}
    if s["bias"] is not None:
        o["dbias"] = dz.sum(0).to(src)
    if s["residual"] is not None:
        o["dresidual"] = s["dy"]
    return o


def _plain_dropout(s):
    c = s["case"]
    y = _drop(s["x"].float(), s["rng"], c["p"])
    if s["residual"] is not None:
        y = s["residual"].float() + y
    o = {"out": y.to(s["x"].dtype)}
    if c["train"]:
        o["dx"] = _drop(s["dy"].float(), s["rng"], c["p"]).to(s["x"].dtype)
        if s["residual"] is not None:
            o["dresidual"] = s["dy"]
    return o


def _grads(s, outs, douts):
    leaves = [s[k] for k in s["leaves"]]
    return dict(zip(("d" + k for k in s["leaves"]), torch.autograd.grad(outs, leaves, douts)))


def run(s):
    c = s["case"]
    if not own:
        with torch.no_grad():
            return {"linear": _plain_linear, "norm": _plain_norm, "dropout": _plain_dropout}[c["op"]](s)
    import gemm_collective_tiles_gb300 as gct
    if c["op"] == "linear":
        act = None if c["act"] == "none" else c["act"]
        if not c["train"]:
            s["ws"] = gct.matmul_act(s["x"], s["w"], s["out"], bias=s["bias"], act=act, residual=s["residual"], workspace=s.get("ws"))
            return {"out": s["out"]}
        y = gct.linear_act(s["x"], s["w"], bias=s["bias"], act=act, residual=s["residual"], p=c["p"], rng=s.get("rng"))
        return {"out": y.detach()} | _grads(s, [y], [s["dy"]])
    if c["op"] == "dropout":
        if not c["train"]:
            gct.dropout_add(s["x"], s["out"], c["p"], s["rng"], residual=s["residual"])
            return {"out": s["out"]}
        y = gct.dropout(s["x"], c["p"], s["rng"], residual=s["residual"])
        return {"out": y.detach()} | _grads(s, [y], [s["dy"]])
    kinds = {k: None if c[k] == "none" else c[k] for k in ("post", "pre")}
    norms = dict(kinds, post_weight=s["post_weight"], post_bias=s["post_bias"], weight=s["pre_weight"], bias=s["pre_bias"],
                 eps=_EPS, x=s["x"], gate=s["gate"], scale=_SCALE if _joins(c) else 1.0)
    if not c["train"]:
        gct.norm_join(s["y"], s["h"], s["n"], **norms)
        return {k: s[k] for k in ("h", "n") if s[k] is not None}
    h, n = gct.block_norm(s["y"], **norms)
    o, d = {}, {}
    if s["dh"] is not None:
        o["h"], d["h"] = h, s["dh"]
    if s["dn"] is not None:
        o["n"], d["n"] = n, s["dn"]
    return {k: v.detach() for k, v in o.items()} | _grads(s, list(o.values()), list(d.values()))


def work(case):
    c = case
    M, e = c["M"], _SIZE[c["src"]]
    if c["op"] == "linear":
        K, N = c["K"], c["N"]
        b = (M * K + K * N + M * N) * e + (N * e if c["bias"] else 0) + (M * N * e if c["residual"] else 0)
        if c["train"]:  # dy comes in, the gradients of x, w and bias go out
            b += (M * N + M * K + K * N) * e + (N * e if c["bias"] else 0)
        return {"bytes": b, "flops": (6 if c["train"] else 2) * M * N * K}
    if c["op"] == "dropout":
        n = M * c["N"]
        return {"bytes": n * e * (2 + c["residual"] + 2 * c["train"]), "flops": n * (2 if c["train"] else 1)}
    n, res = M * c["D"], _SIZE[c["res"]]
    h, pre = _joins(c), c["pre"] != "none"
    rows = {"none": 0, "channel": 1, "sequence": c["groups"], "token": M}[c["gate"]]
    vectors = 0
    for k in ("post", "pre"):
        if c["affine"] and c[k] != "none":
            vectors += 2 if c[k] == "layer" else 1
    weights = (rows + vectors) * c["D"] * e
    b = n * (e + res * c["x"] + res * h + e * pre) + weights
    f = 4 + 4 * (c["post"] != "none") + 4 * pre
    if c["train"]:  # dh and dn come in, the gradients of y, x, gate and weights go out
        b += n * (res * h + e * pre + e + res * c["x"]) + weights
        f *= 3
    return {"bytes": b, "flops": f * n}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _halves(a, b):
    """Upper and lower 32 bits of the product of a (below 2^32) and the constant b, without a 64-bit overflow."""
    lo, hi = a * (b & 0xFFFF), a * (b >> 16)
    mid = (lo >> 16) + (hi & 0xFFFF) + ((hi >> 16 & 0xFFFFFFFF) << 16)
    return mid >> 16, (mid & 0xFFFF) << 16 | lo & 0xFFFF


def _kept(rng, p, M, N):
    """The factor of each element: 0 where it is dropped."""
    seed, offset = (int(v) % 2 ** 64 for v in rng.tolist())
    i = torch.arange(M, device="cuda")[:, None]
    j = torch.arange(-(-N // 8), device="cuda")[None, :]
    x = [j + 0 * i, i + 0 * j, 0 * (i + j) + offset % 2 ** 32, 0 * (i + j) + offset // 2 ** 32]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        h0, l0 = _halves(x[0], 0xD2511F53)
        h1, l1 = _halves(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    column = torch.arange(N, device="cuda")
    least = round(65536 * p)
    factor = torch.empty(M, N, dtype=torch.float64, device="cuda")
    for lane in range(8):
        r = x[lane // 2] // 65536 if lane % 2 else x[lane // 2] % 65536
        at = column[lane::8]
        factor[:, at] = (r[:, :at.numel()] >= least).double() / (1 - least / 65536)
    return factor


def _act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return z * torch.erfc(-z / 2 ** 0.5) / 2
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _norm64(v, kind, weight, bias):
    if kind == "none":
        return v
    centred = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    out = centred * (centred.pow(2).mean(-1, keepdim=True) + _EPS).rsqrt()
    if weight is not None:
        out = out * weight
    return out if bias is None else out + bias


def exact(case, seed):
    s = prepare(case, seed)
    c, M = case, case["M"]
    wide = {k: v.detach().double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    for k in s.get("leaves", ()):
        wide[k].requires_grad_()
    if c["op"] == "norm":
        h = _norm64(wide["y"], c["post"], wide["post_weight"], wide["post_bias"])
        if wide["gate"] is not None:
            G = wide["gate"].shape[0]
            h = (h.view(G, M // G, -1) * wide["gate"][:, None, :]).view(M, -1)
        outs, douts = {}, {}
        if _joins(c):
            h = h * _SCALE + (0 if wide["x"] is None else wide["x"])
            outs["h"], douts["h"] = h, wide.get("dh")
        if c["pre"] != "none":
            outs["n"], douts["n"] = _norm64(h, c["pre"], wide["pre_weight"], wide["pre_bias"]), wide.get("dn")
    else:
        y = wide["x"]
        if c["op"] == "linear":
            y = wide["x"] @ wide["w"]
            if wide["bias"] is not None:
                y = y + wide["bias"]
            y = _act64(y, c["act"])
        if c["p"] > 0:
            y = y * _kept(s["rng"], c["p"], *y.shape)
        if wide["residual"] is not None:
            y = y + wide["residual"]
        outs, douts = {"out": y}, {"out": wide.get("dy")}
    o = {k: v.detach() for k, v in outs.items()}
    if c["train"]:
        grads = torch.autograd.grad(list(outs.values()), [wide[k] for k in s["leaves"]], list(douts.values()))
        o |= dict(zip(("d" + k for k in s["leaves"]), grads))
    return o
