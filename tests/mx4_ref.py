"""Plain 64-bit implementations of the MXFP4 operators and the block norms, and
the error bounds that their arithmetic allows (numpy, no code of the library)."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1])
assert E4M3[-1] == 448.0 and len(E4M3) == 127


def bf16(a):
    """fp32 or fp64 values rounded once to bf16 (nearest, ties to even), as fp32 values."""
    a = np.asarray(a, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore", under="ignore"):
        m, e = np.frexp(a)
        step = np.ldexp(1.0, np.maximum(e - 8, -133))
        r = np.rint(a / step) * step
    r = np.where(np.isfinite(a), r, a)
    return np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, r), r).astype(np.float32)


def bf16_of_bits(u):
    return (np.asarray(u).astype(np.uint32) << 16).view(np.float32)


def _round_to(table, a):
    """Index of the table's nearest member, ties to the even index, the last one for what is above."""
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def quant(v, fmt):
    """[M, K] values -> (codes, scale codes): packed nibbles [M, K/2] for "mxfp4", bytes [M, K] for "mxfp8"."""
    with np.errstate(invalid="ignore"):  # signalling NaNs become quiet ones
        v = np.asarray(v, dtype=np.float64)
    M, K = v.shape
    b = v.reshape(M, K // 32, 32)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(amax)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.where(bad, 1.0, amax))
    X = np.where(amax == 0, -127, np.clip(e - 1 - (2 if fmt == "mxfp4" else 8), -127, 127))
    a = np.ldexp(np.abs(np.where(bad[..., None], 0.0, b)), -X[..., None])
    code = _round_to(E2M1 if fmt == "mxfp4" else E4M3, a).astype(np.uint8)
    neg = np.signbit(b) & ~bad[..., None]
    scale = np.where(bad, 255, X + 127).astype(np.uint8)
    if fmt == "mxfp8":
        return (code | (neg.astype(np.uint8) << 7)).reshape(M, K), scale
    code = (code | (neg.astype(np.uint8) << 3)).reshape(M, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale


def values(q, s, fmt="mxfp4"):
    """The values of rows, in fp64: q [.., K/2] (mxfp4) or [.., K] (mxfp8), s [.., K/32]."""
    s = np.asarray(s)
    if fmt == "mxfp4":
        n = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], q.shape[-1] * 2)
        v = E2M1[n & 7] * np.where(n & 8, -1.0, 1.0)
    else:
        v = np.append(E4M3, np.nan)[q & 127] * np.where(q & 128, -1.0, 1.0)
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return v * np.repeat(scale, 32, axis=-1)


# The matrix cores' additions are taken as roundings of 2^-23 each (a directed
# rounding of fp32 at worst): a sum of K products is off by at most
# gamma = n u / (1 - n u) of the sum of their magnitudes, n = K + 4.
def gamma(K):
    n = (K + 4) * 2.0 ** -23
    return n / (1 - n)


HALF = {"bf16": 2.0 ** -8, "fp32": 0.0}  # one rounding to bf16; fp32 sums are stored as they are


def product(x, w, out="bf16"):
    """x [T, K] w [N, K]^T in fp64 and the largest error of the stored output."""
    y, a = x @ w.T, gamma(x.shape[1]) * (np.abs(x) @ np.abs(w).T)
    return y, a + HALF[out] * (np.abs(y) + a)


def glu(x, w, u, out="bf16"):
    """silu(x w^T) (x u^T) and its largest error.  SiLU's slope is below 1.1; its exponential has an
    argument rounded to 2^-24 of its size and, like the reciprocal, an error of an ulp or two: together below
    (|g| + 8) 2^-22 of the result."""
    K = x.shape[1]
    g, v = x @ w.T, x @ u.T
    ag, av = gamma(K) * (np.abs(x) @ np.abs(w).T), gamma(K) * (np.abs(x) @ np.abs(u).T)
    with np.errstate(over="ignore"):
        s = g / (1 + np.exp(-g))
    h = s * v
    err = 1.1 * ag * (np.abs(v) + av) + np.abs(s) * av + (np.abs(g) + 8) * 2.0 ** -22 * (np.abs(h) + 1.1 * ag * np.abs(v))
    return h, err + HALF[out] * (np.abs(h) + err)


f32 = np.float32


def inv_rms(x, eps):
    with np.errstate(over="ignore", invalid="ignore"):
        return (1 / np.sqrt((x.astype(np.float64) ** 2).sum(-1, keepdims=True) / x.shape[-1] + np.float64(f32(eps)))).astype(f32)


def norm_before(x, w, eps):
    """z as the operator defines it: the mean square in 64 bits, each other step one fp32 operation."""
    with np.errstate(over="ignore", invalid="ignore"):
        return bf16((x.astype(f32) * inv_rms(x, eps)).astype(f32) * w.astype(f32))


def norm_after(y, res, w_post, gate, alpha, beta, eps, res_bf16):
    """out as the operator defines it."""
    with np.errstate(over="ignore", invalid="ignore"):
        b = y.astype(f32)
        if w_post is not None:
            b = (b * inv_rms(b, eps)).astype(f32) * w_post.astype(f32)
        if gate is not None:
            b = b * gate.astype(f32)
        out = res.astype(f32) * f32(beta) + b * f32(alpha)
    assert out.dtype == f32
    return bf16(out) if res_bf16 else out
