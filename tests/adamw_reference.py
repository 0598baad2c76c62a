"""AdamW as include/gs/training.h defines it, in numpy: FP32 operation by
FP32 operation (step32, whose results a correct implementation has bit for
bit), and the update in 64 bits (step64)."""
import numpy as np

F = np.float32
MASK = np.uint64(0xFFFFFFFF)


def mix32(x):
    """lowbias32 on uint64 arrays holding 32-bit values."""
    x = np.asarray(x, dtype=np.uint64)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x7FEB352D)) & MASK
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0x846CA68B)) & MASK
    return x ^ (x >> np.uint64(16))


def hashes(n, tensor, seed, t, first=0):
    i = np.arange(n, dtype=np.uint64) + np.uint64(first)
    key = mix32(mix32(mix32(seed) ^ np.uint64(t)) ^ np.uint64(tensor))
    return mix32((i & MASK) ^ mix32(key ^ (i >> np.uint64(32))))


# values of the non-negative E4M3 codes 0..126, from the format
CODES = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                  for c in range(127)], dtype=np.float32)


def decode(codes, scales, n):
    """code * scale in FP32, one scale per 128 elements."""
    c = codes.astype(np.int64)
    v = np.where((c & 0x7F) == 0x7F, np.float32(np.nan), CODES[np.minimum(c & 0x7F, 126)])
    v = np.where(c & 0x80, -v, v).astype(F)
    return v * np.repeat(scales, 128)[:n]


def encode(x, h16, squared):
    """(codes, scales) of the stored form of x (FP32 [n])."""
    n = x.size
    nb = -(-n // 128)
    pad = np.zeros(nb * 128, dtype=F)
    pad[:n] = np.where(np.isfinite(x), np.abs(x), 0)
    s = (np.maximum(pad.reshape(nb, 128).max(1), F(1e-12)) / F(448)).astype(F)
    with np.errstate(all="ignore"):
        y = np.minimum((np.abs(x) / np.repeat(s, 128)[:n]).astype(F), F(448))
    y = np.where(np.isnan(y), F(0), y)
    at = np.searchsorted(CODES, y, side="right") - 1
    y0 = CODES[at]
    q = CODES[np.minimum(at + 1, 126)] - y0
    q = np.where(at == 126, F(32), q).astype(F)
    u = ((2 * h16.astype(np.int64) + 1).astype(F) * F(2.0 ** -17)).astype(F)
    d = y - y0
    if squared:
        up = d * (y + y0) > u * (q * ((y0 + y0) + q))
    else:
        up = d > u * q
    code = at + up
    if squared:
        code = np.where((code == 0) & (x > 0), 1, code)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8), s


def scalars(t, lr, beta1, beta2, scale, norm_sq, max_norm):
    inv = F(1) / F(scale) if scale is not None else F(1)
    c = min(1.0, max_norm / (np.sqrt(norm_sq) + 1e-6)) if norm_sq is not None else 1.0
    return (F(np.float64(inv) * c), F(np.float64(F(lr)) / (1.0 - beta1 ** t)),
            F(1.0 / np.sqrt(1.0 - beta2 ** t)))


def update32(p, g, m, v, wd, lr, t, beta1, beta2, eps, scale=None, norm_sq=None, max_norm=0.0):
    """(p', m', v', r') of FP32 arrays."""
    mul, size, c2 = scalars(t, lr, beta1, beta2, scale, norm_sq, max_norm)
    b1, ob1, b2, ob2 = F(beta1), F(1.0 - beta1), F(beta2), F(1.0 - beta2)
    with np.errstate(all="ignore"):
        g = g.astype(F) * mul
        m = b1 * m + ob1 * g
        v = b2 * v + ob2 * (g * g)
        r = np.sqrt(v)
        keep = F(1) - F(lr) * F(wd)
        p = p * keep - size * (m / (r * c2 + F(eps)))
    assert p.dtype == m.dtype == v.dtype == F
    return p, m, v, r


def update64(p, g, m, v, wd, lr, t, beta1, beta2, eps, scale=None, norm_sq=None, max_norm=0.0):
    D = np.float64
    c = min(1.0, max_norm / (np.sqrt(norm_sq) + 1e-6)) if norm_sq is not None else 1.0
    g = g.astype(D) * (c / (1.0 if scale is None else float(scale)))
    m = beta1 * m.astype(D) + (1 - beta1) * g
    v = beta2 * v.astype(D) + (1 - beta2) * g * g
    lr = float(F(lr))
    p = p.astype(D) * (1 - lr * float(F(wd))) - lr / (1 - beta1 ** t) * m / (
        np.sqrt(v) / np.sqrt(1 - beta2 ** t) + eps)
    return p, m, v
