"""Cases for the block-scaled 8-bit float operators: quantisation, matrix product, weight gradient.

Definitions (all of them over blocks of 128):

* quantize: x (M, K) is cut into blocks, 1 x 128 ("rows": activations and
  gradients) or 128 x 128 ("tiles": weights).  amax is the largest finite |x|
  of a block, raised to at least FMAX * 2^PMIN.  With ``pow2`` the scale is
  the smallest power of two with amax <= scale * FMAX and the codes are
  rne8(x / scale); without it the scale is amax / FMAX and the codes are
  rne8(x * (FMAX / amax)), each step rounded to 32 bits.
* matmul: out = (codes of A * scale of A) @ (codes of B * scale of B) + bias,
  A (M, K) with 1 x 128 scales, B (K, N) with 128 x 128 scales.
* weight_grad: out (K, N) = (codes of X * scale of X)^T @ dY: the backward
  pass of a linear layer that kept its input X (M, K) as an 8-bit checkpoint.
"""
import math

import torch

#: Set by the program that runs the cases: False for the plain forms, True for the framework's operators.
own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
      "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one token's activation before a single-token product: latency only
        {"name": "quant_token", "op": "quantize", "M": 1, "K": 4096, "src": "bf16", "fp8": "e4m3", "block": "rows", "pow2": True},
        # the input of a linear layer, kept as an 8-bit checkpoint of a 16384-token training batch
        {"name": "quant_train", "op": "quantize", "M": 16384, "K": 4096, "src": "bf16", "fp8": "e4m3", "block": "rows", "pow2": True},
        # 32-bit gradients of odd sizes, rows that do not start on 16 bytes, the wider-range code type
        {"name": "quant_odd", "op": "quantize", "M": 1537, "K": 5003, "src": "f32", "fp8": "e5m2", "block": "rows", "pow2": False},
        # a weight matrix after an optimizer step
        {"name": "quant_weight", "op": "quantize", "M": 4096, "K": 14336, "src": "bf16", "fp8": "e4m3", "block": "tiles", "pow2": False},
        # a single token through an up projection: the weights are read once
        {"name": "mm_token", "op": "matmul", "M": 1, "K": 4096, "N": 14336, "fp8": "e4m3", "trans": False, "bias": False, "out": "bf16"},
        # a decoding batch through a down projection whose weights are stored (N, K)
        {"name": "mm_batch", "op": "matmul", "M": 48, "K": 14336, "N": 4096, "fp8": "e4m3", "trans": True, "bias": False, "out": "bf16"},
        # a short prompt, nothing a multiple of anything
        {"name": "mm_odd", "op": "matmul", "M": 333, "K": 1000, "N": 1111, "fp8": "e4m3", "trans": False, "bias": True, "out": "f16"},
        # forward pass of a training batch
        {"name": "mm_forward", "op": "matmul", "M": 4096, "K": 4096, "N": 14336, "fp8": "e4m3", "trans": False, "bias": True, "out": "bf16"},
        # input gradient: dY in the wider-range codes times the transposed weights
        {"name": "mm_dgrad", "op": "matmul", "M": 8192, "K": 8192, "N": 8192, "fp8": "e5m2", "trans": True, "bias": False, "out": "bf16"},
        # weight gradient of a short, odd batch
        {"name": "wg_odd", "op": "weight_grad", "M": 777, "K": 1000, "N": 1111, "fp8": "e4m3", "src": "f16", "out": "f16"},
        # weight gradient into a 32-bit gradient buffer
        {"name": "wg_train", "op": "weight_grad", "M": 4096, "K": 4096, "N": 14336, "fp8": "e4m3", "src": "bf16", "out": "f32"},
        # weight gradient over a long batch
        {"name": "wg_long", "op": "weight_grad", "M": 16384, "K": 4096, "N": 4096, "fp8": "e4m3", "src": "bf16", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["quantize", "matmul", "matmul", "weight_grad"])
        c = {"op": op, "M": _log(rng, 1, 16384), "K": _log(rng, 100, 16384)}
        c["fp8"] = rng.choice(["e4m3", "e4m3", "e5m2"])
        if op == "quantize":
            c["src"] = rng.choice(["bf16", "f16", "f32"])
            c["block"] = rng.choice(["rows", "rows", "tiles"])
            c["pow2"] = rng.random() < 0.5
            if c["M"] * c["K"] > 16384 * 4096:
                continue
            return c
        c["N"] = _log(rng, 100, 16384)
        if op == "matmul":
            c["trans"], c["bias"] = rng.random() < 0.5, rng.random() < 0.5
            c["out"] = rng.choice(["bf16", "f16"])
        else:
            c["src"] = rng.choice(["bf16", "bf16", "f16"])
            c["out"] = rng.choice(["f32", c["src"]])
        if c["M"] * c["K"] * c["N"] > 8192 ** 3:
            continue
        return c


def _values(g, M, K, dtype, spread):
    """Normal values whose rows and columns differ in size, as activations, weights and gradients have them."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x *= torch.exp(spread * torch.randn(M, 1, generator=g, device="cuda"))
    x *= torch.exp(0.5 * torch.randn(1, K, generator=g, device="cuda"))
    return x.to(dtype)


def _pitched(codes):
    """The codes in rows that start on 16 bytes, as a program keeps them."""
    M, K = codes.shape
    buf = torch.zeros(M, (K + 15) // 16 * 16, dtype=torch.uint8, device=codes.device)
    buf[:, :K] = codes.view(torch.uint8)
    return buf.view(codes.dtype)[:, :K]


def _by_row(scales):
    """Scales of (M, K/128) blocks with the rows next to each other in memory."""
    return scales.t().contiguous().t()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, K = case["M"], case["K"]
    s = {"case": dict(case)}
    if case["op"] == "quantize":
        s["x"] = _values(g, M, K, _T[case["src"]], 1.0)
        rows = case["block"] == "rows"
        s["codes"] = torch.empty(M, (K + 15) // 16 * 16, dtype=_T[case["fp8"]], device="cuda")[:, :K]
        kb = (K + 127) // 128
        s["scales"] = (torch.empty(kb, M, device="cuda").t() if rows else torch.empty((M + 127) // 128, kb, device="cuda"))
        return s
    N = case["N"]
    a, sa = _quantize(_values(g, M, K, torch.bfloat16, 1.0), case["fp8"], True, case["op"] == "weight_grad")
    s["a"], s["sa"] = _pitched(a), _by_row(sa)
    if case["op"] == "matmul":
        w = _values(g, N, K, torch.bfloat16, 0.2) if case["trans"] else _values(g, K, N, torch.bfloat16, 0.2)
        w, sw = _quantize(w * 0.02, "e4m3", False, False)
        w = _pitched(w)
        s["b"], s["sb"] = (w.t(), sw.t()) if case["trans"] else (w, sw)
        s["bias"] = torch.randn(N, generator=g, device="cuda").to(_T[case["out"]]) if case["bias"] else None
        s["out"] = torch.empty(M, N, dtype=_T[case["out"]], device="cuda")
    else:
        s["dy"] = (_values(g, M, N, torch.float32, 1.0) * 1e-2).to(_T[case["src"]])
        s["out"] = torch.empty(K, N, dtype=_T[case["out"]], device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _pmin(src, fp8):
    """The smallest scale's exponent: with 16-bit floats the codes' steps then are no finer than the type's own."""
    return (-15 if fp8 == "e4m3" else -8) if src == torch.float16 else -100


def _quantize(x, fp8, rows, pow2):
    """Codes and scales of x by elementary 32-bit operations."""
    M, K = x.shape
    fmax, pmin = _FMAX[fp8], _pmin(x.dtype, fp8)
    kb, mb = (K + 127) // 128, (M + 127) // 128
    x = x.float()
    fine = torch.isfinite(x)
    v = torch.where(fine, x, torch.nan)
    size = torch.where(fine, x.abs(), 0.0)
    size = torch.nn.functional.pad(size, (0, kb * 128 - K, 0, 0 if rows else mb * 128 - M))
    if rows:
        amax = size.view(M, kb, 128).amax(2)
    else:
        amax = size.view(mb, 128, kb, 128).amax((1, 3))
    amax = amax.clamp_min(fmax * 2.0 ** pmin)
    if pow2:
        m, e = torch.frexp(amax)  # FMAX is 0.875 * 2^9 or 0.875 * 2^16
        p = e - (9 if fp8 == "e4m3" else 16) + (m > 0.875).int()
        scale, inv = torch.ldexp(torch.ones_like(amax), p), torch.ldexp(torch.ones_like(amax), -p)
    else:
        scale, inv = amax / fmax, fmax / amax
    wide = inv.repeat_interleave(128, 1)[:, :K]
    if not rows:
        wide = wide.repeat_interleave(128, 0)[:M]
    return (v * wide).to(_T[fp8]), scale


def _spread_a(codes, scale):
    return codes.float() * scale.repeat_interleave(128, 1)[:, :codes.shape[1]]


def _spread_b(codes, scale):
    K, N = codes.shape
    return codes.float() * scale.repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :N]


def run(s):
    c = s["case"]
    if own:
        import gemm_collective_tiles_gb300 as gct
        if c["op"] == "quantize":
            gct.quantize_fp8(s["x"], s["codes"], s["scales"], block=c["block"], pow2=c["pow2"])
            return {"codes": s["codes"], "scales": s["scales"]}
        if c["op"] == "matmul":
            s["ws"] = gct.matmul_fp8(s["a"], s["sa"], s["b"], s["sb"], s["out"], bias=s["bias"], workspace=s.get("ws"))
        else:
            s["ws"] = gct.weight_grad_fp8(s["a"], s["sa"], s["dy"], s["out"], workspace=s.get("ws"))
        return {"out": s["out"]}
    if c["op"] == "quantize":
        codes, scales = _quantize(s["x"], c["fp8"], c["block"] == "rows", c["pow2"])
        return {"codes": codes, "scales": scales}
    if c["op"] == "matmul":
        y = torch.matmul(_spread_a(s["a"], s["sa"]), _spread_b(s["b"], s["sb"]))
        if s["bias"] is not None:
            y = y + s["bias"].float()
    else:
        y = torch.matmul(_spread_a(s["a"], s["sa"]).t(), s["dy"].float())
    return {"out": y.to(s["out"].dtype)}


def work(case):
    M, K = case["M"], case["K"]
    kb = (K + 127) // 128
    if case["op"] == "quantize":
        blocks = kb * (M if case["block"] == "rows" else (M + 127) // 128)
        return {"bytes": M * K * (_SIZE[case["src"]] + 1) + 4 * blocks, "flops": 3 * M * K}
    N = case["N"]
    b = M * K + 4 * M * kb
    if case["op"] == "matmul":
        b += K * N + 4 * kb * ((N + 127) // 128) + M * N * 2 + (2 * N if case["bias"] else 0)
    else:
        b += M * N * 2 + K * N * _SIZE[case["out"]]
    return {"bytes": b, "flops": 2 * M * N * K}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _round8(v, fp8):
    """v to the nearest value of the code type, ties to the even one, in 64 bits."""
    bits, low = (3, -6) if fp8 == "e4m3" else (2, -14)
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))).clamp_min(low)
    step = torch.exp2(e - bits)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    M, K = case["M"], case["K"]
    starts = range(0, K, 128)
    if case["op"] == "quantize":
        x = s["x"].double()
        fmax, least = _FMAX[case["fp8"]], 2.0 ** _pmin(s["x"].dtype, case["fp8"])
        codes = torch.empty_like(x)
        scales = torch.empty(s["scales"].shape, dtype=torch.float64, device="cuda")
        tall = 1 if case["block"] == "rows" else 128
        group = torch.arange(M, device="cuda") // tall
        for i, k in enumerate(starts):
            part = x[:, k:k + 128]
            top = torch.zeros(scales.shape[0], dtype=torch.float64, device="cuda")
            top.scatter_reduce_(0, group, part.abs().amax(1), "amax")
            scale = (top / fmax).clamp_min(least)
            if case["pow2"]:
                two = torch.exp2(torch.ceil(torch.log2(scale)))
                scale = torch.where(two / 2 >= scale, two / 2, two)  # log2 of a power of two may come out a little over it
            scales[:, i] = scale
            codes[:, k:k + 128] = _round8(part / scale[group][:, None], case["fp8"])
        return {"codes": codes, "scales": scales}
    N = case["N"]
    if case["op"] == "matmul":
        y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        column = torch.arange(N, device="cuda") // 128
        for i, k in enumerate(starts):
            part = s["a"][:, k:k + 128].double() @ s["b"][k:k + 128].double()
            y += part * s["sa"][:, i].double()[:, None] * s["sb"][i].double()[column][None, :]
        if s["bias"] is not None:
            y += s["bias"].double()
        return {"out": y}
    y = torch.empty(K, N, dtype=torch.float64, device="cuda")
    dy = s["dy"].double()
    for i, k in enumerate(starts):
        y[k:k + 128] = s["a"][:, k:k + 128].double().t() @ (dy * s["sa"][:, i].double()[:, None])
    return {"out": y}
