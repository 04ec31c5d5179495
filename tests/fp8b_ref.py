"""Plain 64-bit implementations of the FP8 operators with block scales of 128, and the error bounds that their
arithmetic allows (torch in float64, no code of the library)."""
import torch

E4M3 = torch.tensor([m * 2.0 ** -9 for m in range(8)]
                    + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1], dtype=torch.float64)
assert E4M3[-1] == 448.0 and len(E4M3) == 127
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def code_values(q):
    """Values of e4m3 codes."""
    t = torch.cat([E4M3, torch.tensor([float("nan")], dtype=torch.float64)]).to(q.device)
    v = t[(q & 127).long()]
    return torch.where(q > 127, -v, v)


def quant(v):
    """fp32 operations as the operator defines them -> (codes [M, K], scales [K/128, M])."""
    v = v.float()
    M, K = v.shape
    b = v.view(M, K // 128, 128)
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    a = torch.where(bad, torch.ones_like(top), top).clamp(min=2.0 ** -110)
    # (64 bits, rounded: a correctly rounded fp32 division, where torch multiplies by a number's reciprocal)
    s, mul = (a.double() / 448).float(), (448 / a.double()).float()
    x = torch.where(bad.unsqueeze(-1), torch.zeros_like(b), b) * mul.unsqueeze(-1)
    t = E4M3.to(v.device)
    mid = (t[1:] + t[:-1]) / 2
    m = x.abs().double()
    lo, hi = torch.bucketize(m, mid), torch.bucketize(m, mid, right=True)
    code = torch.where(lo % 2 == 0, lo, hi).to(torch.uint8)
    code = code | (torch.signbit(x) & ~bad.unsqueeze(-1)).to(torch.uint8) << 7
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    return code.view(M, K), s.t().contiguous()


def rows(q, s):
    """Values of rows [M, K] with scales [K/128, M]."""
    return code_values(q) * s.t().double().repeat_interleave(128, 1)


def weights(q, s):
    """Values of matrices [.., N, K] with scales [.., N/128 rounded up, K/128]."""
    N = q.shape[-2]
    return code_values(q) * s.double().repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)


# The additions are taken as roundings of 2^-23 each (a directed rounding of fp32 at worst): K products, the sums of
# up to 16 waves, and the roundings of the scales' product.
def gamma(K):
    n = (K + 32) * 2.0 ** -23
    return n / (1 - n)


def product(x, w, half=0.0):
    """x [T, K] w [N, K]^T and the largest error of the stored sum."""
    y = x @ w.T.contiguous()
    a = gamma(x.shape[1]) * (x.abs() @ w.abs().T.contiguous())
    return y, a + half * (y.abs() + a)


def held(h, err):
    """Largest error of the values that quantised rows stand for, of fp32 values off by at most err from h: half a
    step is 2^-4 of a value and 2^-10 of the scale below 2^-6 scales; scale and product are three fp32 operations."""
    M, K = h.shape
    big = h.abs() + err
    scale = big.view(M, K // 128, 128).amax(-1, keepdim=True).expand(M, K // 128, 128).reshape(M, K) / 448 * (1 + 2.0 ** -20)
    return err + torch.maximum(big * 2.0 ** -4, scale * 2.0 ** -10) + big * 2.0 ** -20


def glu(x, w, u):
    """gate, up, h and their largest errors (h: SiLU's slope is below 1.1, its exponential's argument is rounded to
    2^-24 of its size, it and the reciprocal have an error of an ulp or two)."""
    g, ag = product(x, w)
    v, av = product(x, u)
    s = g * torch.sigmoid(g)
    h = s * v
    err = (1.1 * ag * (v.abs() + av) + s.abs() * av
           + (g.abs() + 8) * 2.0 ** -22 * (h.abs() + 1.1 * ag * v.abs()))
    return (g, ag), (v, av), (h, err)


def glu_grad(dh, adh, g, u):
    """dg, du and their largest errors for dh off by at most adh: sig and 1 - sig are good to (|g| + 8) 2^-22, and the
    sum 1 + g (1 - sig) to that of its terms."""
    sig = torch.sigmoid(g)
    rel = (g.abs() + 8) * 2.0 ** -22
    slope = sig * (1 + g * (1 - sig))
    aslope = sig * (1 + g.abs() * (1 - sig)) * 3 * rel
    dg, du = dh * u * slope, dh * g * sig
    big = dh.abs() + adh
    return ((dg, adh * (u * slope).abs() + big * u.abs() * (aslope + slope.abs() * 2.0 ** -21)),
            (du, adh * (g * sig).abs() + big * (g * sig).abs() * 2 * rel))
