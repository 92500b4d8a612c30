"""64-bit references of the block-scaled 8-bit float operators, from their
definitions (numpy only; nothing of the library)."""
import numpy as np

FMAX = {"e4m3": 448.0, "e5m2": 57344.0}


def blocks(n):
    return -(-n // 128)


def round8(v, fp8):
    """To the nearest value of the code type, ties to even (NaN stays)."""
    bits, low = (3, -6) if fp8 == "e4m3" else (2, -14)
    v = np.asarray(v, np.float64)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.where(np.isfinite(v), v, 0.0))
    step = np.ldexp(1.0, np.maximum(e - 1, low) - bits)
    return np.rint(v / step) * step


def pmin(src, fp8):
    return (-15 if fp8 == "e4m3" else -8) if src == "f16" else -100


def block_amax(x, rows):
    """Largest finite magnitude of each block of x (float64)."""
    M, K = x.shape
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    a = np.pad(a, ((0, 0 if rows else -M % 128), (0, -K % 128)))
    a = a.reshape(a.shape[0], -1, 128).max(2)
    return a if rows else a.reshape(-1, 128, a.shape[1]).max(1)


def spread(s, M, K, rows):
    w = np.repeat(s, 128, 1)[:, :K]
    return w if rows else np.repeat(w, 128, 0)[:M]


def quantize(x, src, fp8, rows, pow2):
    """(codes, scales) of x as float64; x holds values of the source type."""
    M, K = x.shape
    amax = np.maximum(block_amax(x, rows), FMAX[fp8] * 2.0 ** pmin(src, fp8))
    v = np.where(np.isfinite(x), x, np.nan)
    if pow2:
        p = np.ceil(np.log2(amax / FMAX[fp8]))
        p = np.where(np.ldexp(FMAX[fp8], (p - 1).astype(int)) >= amax, p - 1, p)
        p = np.where(np.ldexp(FMAX[fp8], p.astype(int)) < amax, p + 1, p)
        scale = np.ldexp(1.0, p.astype(int))
        return round8(v / spread(scale, M, K, rows), fp8), scale
    a32 = amax.astype(np.float32)
    scale = a32 * (np.float32(1.0) / np.float32(FMAX[fp8]))
    inv = (np.float32(1.0) / a32) * np.float32(FMAX[fp8])
    assert scale.dtype == inv.dtype == np.float32
    with np.errstate(invalid="ignore"):
        scaled = v.astype(np.float32) * spread(inv, M, K, rows)
    return round8(scaled.astype(np.float64), fp8), scale.astype(np.float64)
