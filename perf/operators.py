"""The MXFP4 operators and the block norms: what is measured, and their plain form.

Sizes are those of the repository's workloads: hidden 4096 with experts of 1536
(64 experts, top-6, 8 tokens), hidden 7168 with experts of 2048 (256 experts,
top-8, 64, 4604 and 16384 tokens) and the 16384 -> 7168 dense projection.

Formats: e2m1 nibbles two per byte (even element in the low nibble), one E8M0
scale (2^(c - 127)) per 32 consecutive elements of a row; rows that a kernel
holds in 4 or 8 bits are returned as the bf16 values that they stand for.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's activations before a 4-bit projection: latency counts
        {"name": "quant decode T8", "op": "quant", "M": 8, "K": 4096, "dtype": "bf16"},
        # one projection of all 64 experts quantised at load time
        {"name": "quant expert weights", "op": "quant", "M": 64 * 1536, "K": 4096, "dtype": "bf16"},
        # the attention output projection for one decode step of 8 requests
        {"name": "dense decode T8", "op": "dense", "T": 8, "K": 16384, "N": 7168, "out": "bf16"},
        # an odd number of tokens of a small prompt through a 4096 -> 1536 projection, fp32 out
        {"name": "dense ragged T333", "op": "dense", "T": 333, "K": 4096, "N": 1536, "out": "fp32"},
        # the attention output projection for a whole prompt
        {"name": "dense prefill T4604", "op": "dense", "T": 4604, "K": 16384, "N": 7168, "out": "bf16"},
        # gate/up of a decode step: most experts see one token or none
        {"name": "grouped glu decode T8", "op": "grouped", "T": 8, "k": 6, "E": 64, "K": 4096, "N": 1536, "glu": True,
         "zipf": False},
        # down projection of a decode batch: rows already in expert order
        {"name": "grouped decode T64", "op": "grouped", "T": 64, "k": 8, "E": 256, "K": 2048, "N": 7168, "glu": False,
         "zipf": False},
        # gate/up of a whole prompt
        {"name": "grouped glu prefill T4604", "op": "grouped", "T": 4604, "k": 8, "E": 256, "K": 7168, "N": 2048,
         "glu": True, "zipf": False},
        # down projection of a long prompt whose routing is skewed: a few experts hold most rows, many hold none
        {"name": "grouped zipf T16384", "op": "grouped", "T": 16384, "k": 8, "E": 256, "K": 2048, "N": 7168,
         "glu": False, "zipf": True},
        # in front of a block in a decode step, the experts' MXFP8 rows beside the router's bf16 ones
        {"name": "norm before T8", "op": "before", "T": 8, "H": 4096, "x": "bf16", "quant": "mxfp8"},
        # behind a block of a prompt: post-norm, a gate for each token, residual scale, the next block's 4-bit rows
        {"name": "norm after T4604", "op": "after", "T": 4604, "H": 7168, "y": "fp32", "post": True, "gate": "token",
         "quant": "mxfp4"},
        # behind a block of a long prompt: a learned scale for each channel and no post-norm, MXFP8 rows
        {"name": "norm after T16384", "op": "after", "T": 16384, "H": 7168, "y": "fp32", "post": False,
         "gate": "channel", "quant": "mxfp8"},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` from [lo, hi], even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    op = rng.choice(["quant", "dense", "dense", "grouped", "grouped", "before", "after"])
    if op == "quant":
        return {"op": op, "M": _log(rng, 1, 30000), "K": _log(rng, 32, 8192, 32),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "dense":
        return {"op": op, "T": _log(rng, 1, 4604), "K": _log(rng, 128, 16384, 128), "N": _log(rng, 32, 7168, 32),
                "out": rng.choice(["bf16", "fp32"])}
    if op == "grouped":
        E = _log(rng, 2, 64)
        return {"op": op, "T": _log(rng, 1, 4604), "k": rng.randint(1, min(E, 8)), "E": E,
                "K": _log(rng, 128, 7168, 128), "N": _log(rng, 32, 2048, 32), "glu": rng.random() < 0.5,
                "zipf": rng.random() < 0.5}
    if op == "before":
        return {"op": op, "T": _log(rng, 1, 16384), "H": _log(rng, 32, 7168, 32), "x": rng.choice(["bf16", "fp32"]),
                "quant": rng.choice(["mxfp8", "mxfp4"])}
    return {"op": op, "T": _log(rng, 1, 16384), "H": _log(rng, 32, 7168, 32), "y": rng.choice(["bf16", "fp32"]),
            "post": rng.random() < 0.5, "gate": rng.choice(["none", "token", "channel"]),
            "quant": rng.choice(["mxfp8", "mxfp4"])}


def _popularity(E, zipf, g):
    """Share of the routing that each expert draws: even, or Zipf (1.2) in a random order of the experts."""
    p = torch.ones(E, dtype=torch.float64) if not zipf else torch.arange(1, E + 1, dtype=torch.float64) ** -1.2
    p = p / p.sum()
    return p[torch.randperm(E, generator=g)] if zipf else p


def work(case):
    op = case["op"]
    if op == "quant":
        n, b = case["M"] * case["K"], 4 if case["dtype"] == "fp32" else 2
        return {"bytes": n * (b + 17 / 32 * 2 + 2), "flops": 0}  # read, codes written and read back, values written
    if op == "dense":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": (T + N) * K * 17 / 32 + T * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * T * N * K}
    if op == "grouped":
        P, N, K = case["T"] * case["k"], case["N"], case["K"]
        wide = N * (2 if case["glu"] else 1)
        p = _popularity(case["E"], case["zipf"], torch.Generator().manual_seed(1))
        used = float((1 - (1 - p).clamp(min=0) ** P).sum())
        rows = case["T"] if case["glu"] else P
        return {"bytes": used * wide * K * 17 / 32 + rows * K * 17 / 32 + P * N * 2, "flops": 2 * P * wide * K}
    T, H = case["T"], case["H"]
    q = 17 / 32 if case["quant"] == "mxfp4" else 33 / 32
    tail = 2 + 2 * q + 2  # z written; codes written and read back; their values written
    if op == "before":
        return {"bytes": T * H * ((4 if case["x"] == "fp32" else 2) + tail), "flops": 0}
    return {"bytes": T * H * ((4 if case["y"] == "fp32" else 2) + 2 + 2 + tail), "flops": 0}


# --------------------------------------------------------------------- inputs
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _tables(dev):
    """[256, 2] values of a byte's two e2m1 codes, and the 256 E8M0 scales."""
    v = _E2M1 + [-x for x in _E2M1]
    pairs = torch.tensor([[v[b & 15], v[b >> 4]] for b in range(256)], dtype=torch.float64)
    scales = torch.tensor([2.0 ** (c - 127) for c in range(255)] + [math.nan], dtype=torch.float64)
    return {"pairs": pairs.to(dev), "scales": scales.to(dev), "pairs32": pairs.float().to(dev),
            "scales32": scales.float().to(dev)}


def _rows4(x):
    """MXFP4 codes and scales of rows that a program has in hand (made by the plain quantiser)."""
    X, mag = _quant4(x.double(), torch.float64)
    code = torch.searchsorted(torch.tensor(_E2M1, dtype=torch.float64, device=x.device), mag).to(torch.uint8)
    code = code | (torch.signbit(x).to(torch.uint8) << 3)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), (X + 127).to(torch.uint8).contiguous()


def _weights4(g, E, N, K, dev):
    """Expert weights as the repository's workloads draw them: all codes alike, scales such that a product of K
    terms with unit activations stays near one."""
    q = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=dev, generator=g)
    mid = 127 - round(math.log2(2.9 * math.sqrt(K)))
    s = torch.randint(mid - 1, mid + 2, (E, N, K // 32), dtype=torch.uint8, device=dev, generator=g)
    return q, s


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    st = {"case": case, "tab": _tables(dev)}
    if own:
        import fp4_routed_expert_amd as moe
        st["moe"] = moe

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=g)

    if op == "quant":
        # rows of different magnitude, as the tokens of a model have
        M, K = case["M"], case["K"]
        x = torch.empty(M, K, dtype=_DTYPES[case["dtype"]], device=dev)
        for i in range(0, M, 16384):
            n = min(16384, M - i)
            x[i:i + n] = (normal(n, K) * torch.exp(normal(n, 1))).to(x.dtype)
        st["x"] = x
        if own:
            st["q"] = torch.empty(M, K // 2, dtype=torch.uint8, device=dev)
            st["s"] = torch.empty(M, K // 32, dtype=torch.uint8, device=dev)
            st["y"] = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    elif op == "dense":
        T, K, N = case["T"], case["K"], case["N"]
        st["xq"], st["xs"] = _rows4(normal(T, K).bfloat16())
        wq, ws = _weights4(g, 1, N, K, dev)
        st["wq"], st["ws"] = wq[0], ws[0]
        if own:
            st["w"] = st["moe"].mxfp4_prepack(st["wq"], st["ws"])
            st["y"] = torch.empty(T, N, dtype=_DTYPES[case["out"]], device=dev)
    elif op == "grouped":
        T, k, E, K, N = (case[v] for v in ("T", "k", "E", "K", "N"))
        P = T * k
        host = torch.Generator().manual_seed(seed)
        bias = torch.log(_popularity(E, case["zipf"], host) * E).float().to(dev)
        ids = torch.topk(normal(T, E) + bias, k, dim=1).indices.reshape(-1)
        st["pair"] = torch.sort(ids, stable=True).indices.int()
        counts = torch.bincount(ids, minlength=E)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
        st["sizes"] = counts.tolist()
        # gate/up reads a token's row for each of its k experts; down reads rows already in expert order
        st["xq"], st["xs"] = _rows4(normal(T if case["glu"] else P, K).bfloat16())
        st["wq"], st["ws"] = _weights4(g, E, N, K, dev)
        if case["glu"]:
            st["uq"], st["us"] = _weights4(g, E, N, K, dev)
        if own:
            moe = st["moe"]
            st["w"] = (moe.mxfp4_prepack_glu(st["wq"], st["ws"], st["uq"], st["us"]) if case["glu"]
                       else moe.mxfp4_prepack(st["wq"], st["ws"]))
            st["y"] = torch.empty(P, N, dtype=torch.bfloat16, device=dev)
            st["workspace"] = torch.empty(moe.mxfp4_grouped_workspace_size(P, E, N, K, case["glu"]),
                                          dtype=torch.uint8, device=dev)
    else:
        T, H = case["T"], case["H"]
        # the residual stream: channels of different size
        res = (normal(T, H) * torch.exp(0.5 * normal(1, H)))
        if op == "before":
            st["x"] = res.to(_DTYPES[case["x"]])
        else:
            st["res"] = res.bfloat16()
            st["y"] = (normal(T, H) * torch.exp(0.5 * normal(T, 1))).to(_DTYPES[case["y"]])
            st["post"] = 1 + 0.1 * normal(H) if case["post"] else None
            st["gate"] = (torch.sigmoid(normal(T, 1)) if case["gate"] == "token" else
                          0.5 + 0.1 * normal(H) if case["gate"] == "channel" else None)
        st["w"] = 1 + 0.1 * normal(H)
        if own:
            st["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
            st["z"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
            st["q"] = torch.empty(T, H // 2 if case["quant"] == "mxfp4" else H, dtype=torch.uint8, device=dev)
            st["s"] = torch.empty(T, H // 32, dtype=torch.uint8, device=dev)
            st["v"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    return st


# The residual scale and the norms' epsilon of every case.
_ALPHA, _EPS = 0.7, 1e-6


# ----------------------------------------------------------------- plain form
def _scale_exponent(v, emax):
    """X of each block of 32: floor(log2 of the largest magnitude) - emax, kept in [-127, 127]; -127 for zeros."""
    amax = v.abs().amax(-1)
    X = torch.frexp(amax).exponent - 1 - emax
    return torch.where(amax == 0, torch.full_like(X, -127), X.clamp(-127, 127))


def _two_to(n, dtype):
    """2^n of whole numbers inside the type's normal range, by its bits."""
    if dtype == torch.float64:
        return ((n.long() + 1023) << 52).view(dtype)
    return ((n.int() + 127) << 23).view(dtype)


def _quant4(x, dtype):
    """Scale exponents [M, K/32] and the magnitudes that e2m1 holds (nearest, ties to even, at most 6) of rows."""
    M, K = x.shape
    v = x.to(dtype).view(M, K // 32, 32)
    X = _scale_exponent(v, 2)
    a = v.abs() * _two_to(-X, dtype).unsqueeze(-1)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(dtype)
    return X, (torch.round(a / step) * step).clamp(max=6.0).view(M, K)


def _plain4(x, tab):
    X, mag = _quant4(x, torch.float32)
    scale = tab["scales32"][(X + 127).long()].repeat_interleave(32, dim=1)
    return (torch.copysign(mag, x.float()) * scale).bfloat16()


def _plain8(x, tab):
    """The values of x's MXFP8 rows: e4m3 steps by 2^-3 of the binade, by 2^-9 below 2^-6, at most 448."""
    M, K = x.shape
    v = x.float().view(M, K // 32, 32)
    X = _scale_exponent(v, 8)
    a = v.abs() * _two_to(-X, torch.float32).unsqueeze(-1)
    e = (torch.frexp(a).exponent - 1).clamp(min=-6)
    step = _two_to(e - 3, torch.float32)
    mag = (torch.round(a / step) * step).clamp(max=448.0).view(M, K)
    return (torch.copysign(mag, x.float()) * tab["scales32"][(X + 127).long()].repeat_interleave(32, dim=1)).bfloat16()


def _values(q, s, pairs, scales):
    v = pairs[q.int()].view(*s.shape, 32)
    return (v * scales[s.int()].unsqueeze(-1)).view(*q.shape[:-1], q.shape[-1] * 2)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _norm(x, w, eps):
    """x / rms(x) * w: the mean square in 64 bits, every later step rounded to fp32."""
    r = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + eps)
    return (x.float() * r.float()) * w


def _run_plain(st):
    case, tab, op = st["case"], st["tab"], st["case"]["op"]
    if op == "quant":
        return _plain4(st["x"], tab)
    if op == "dense":
        w = _values(st["wq"], st["ws"], tab["pairs32"], tab["scales32"])
        x = _values(st["xq"], st["xs"], tab["pairs32"], tab["scales32"])
        return (x @ w.T).to(_DTYPES[case["out"]])
    if op == "grouped":
        rows = st["pair"] // case["k"] if case["glu"] else None
        return _grouped(st, rows, tab["pairs32"], tab["scales32"], torch.bfloat16)
    if op == "before":
        z = _norm(st["x"], st["w"], _EPS).bfloat16()
        return {"z": z, "q": (_plain4 if case["quant"] == "mxfp4" else _plain8)(z, tab)}
    b = st["y"].float() if st["post"] is None else _norm(st["y"], st["post"], _EPS)
    if st["gate"] is not None:
        b = b * st["gate"]
    out = (st["res"].float() + b * _ALPHA).bfloat16()
    z = _norm(out, st["w"], _EPS).bfloat16()
    return {"out": out, "z": z, "q": (_plain4 if case["quant"] == "mxfp4" else _plain8)(z, tab)}


def _grouped(st, rows, pairs, scales, dtype):
    """One product for each expert that has rows: the groups are ragged and their weights too large to decode at once."""
    case = st["case"]
    y = torch.empty(st["pair"].numel(), case["N"], dtype=dtype, device=st["xq"].device)
    at = 0
    for e, n in enumerate(st["sizes"]):
        if n:
            xq, xs = ((st["xq"][at:at + n], st["xs"][at:at + n]) if rows is None else
                      (st["xq"][rows[at:at + n]], st["xs"][rows[at:at + n]]))
            x = _values(xq, xs, pairs, scales)
            part = x @ _values(st["wq"][e], st["ws"][e], pairs, scales).T
            if case["glu"]:
                part = _silu(part) * (x @ _values(st["uq"][e], st["us"][e], pairs, scales).T)
            y[at:at + n] = part
            at += n
    return y


# ------------------------------------------------------------- the framework's
def _run_own(st):
    case, moe, op = st["case"], st["moe"], st["case"]["op"]
    if op == "quant":
        q, s = moe.quant_mxfp4(st["x"], q=st["q"], s=st["s"])
        return moe.dequant_mx(q, s, "mxfp4", out=st["y"])
    if op == "dense":
        return moe.mxfp4_dense(st["w"], st["xq"], st["xs"], y=st["y"])
    if op == "grouped":
        if case["glu"]:
            return moe.mxfp4_grouped(st["w"], st["xq"], st["xs"], st["offsets"], rows=st["pair"], row_div=case["k"],
                                     y=st["y"], workspace=st["workspace"])
        return moe.mxfp4_grouped(st["w"], st["xq"], st["xs"], st["offsets"], y=st["y"], workspace=st["workspace"])
    if op == "before":
        z, q, s = moe.norm_before(st["x"], st["w"], _EPS, quant=case["quant"], z=st["z"], q=st["q"], s=st["s"])
        return {"z": z, "q": moe.dequant_mx(q, s, case["quant"], out=st["v"])}
    out, z, q, s = moe.norm_after(st["y"], st["res"], st["post"], gate=st["gate"], alpha=_ALPHA, eps=_EPS,
                                  next_weight=st["w"], quant=case["quant"], out=st["out"], z=st["z"], q=st["q"],
                                  s=st["s"])
    return {"out": out, "z": z, "q": moe.dequant_mx(q, s, case["quant"], out=st["v"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- from 64 bits
def _nearest(values, a):
    """The member of `values` (ascending, at least two) nearest to each a, ties to the even place in the list."""
    t = torch.tensor(values, dtype=torch.float64, device=a.device)
    mid = (t[1:] + t[:-1]) / 2
    lo, hi = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    return t[torch.where(lo % 2 == 0, lo, hi)]


def _held(x, quant, tab):
    """The values that the MXFP4 or MXFP8 rows of x stand for, by the nearest member of the format's list."""
    values = _E2M1
    if quant == "mxfp8":
        values = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)]
        values = values[:values.index(448.0) + 1]
    M, K = x.shape
    got = torch.empty(M, K, dtype=torch.float64, device=x.device)
    for i in range(0, M, 8192):
        v = x[i:i + 8192].double().view(-1, K // 32, 32)
        top = v.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(top))
        e = e - (torch.exp2(e) > top).double() + (torch.exp2(e + 1) <= top).double()  # log2 rounds next to a border
        one = tab["scales"][((e - (2 if quant == "mxfp4" else 8)).clamp(-127, 127) + 127).long()]
        got[i:i + 8192] = (_nearest(values, v.abs() / one) * one * torch.sign(v)).view(-1, K)
    return got


def exact(case, seed):
    st = prepare(case, seed)
    tab, op = st["tab"], case["op"]
    if op == "quant":
        return _held(st["x"], "mxfp4", tab)
    if op == "dense":
        w = _values(st["wq"], st["ws"], tab["pairs"], tab["scales"])
        return _values(st["xq"], st["xs"], tab["pairs"], tab["scales"]) @ w.T
    if op == "grouped":
        rows = torch.div(st["pair"].long(), case["k"], rounding_mode="floor") if case["glu"] else None
        return _grouped(st, rows, tab["pairs"], tab["scales"], torch.float64)

    def norm(x, w):
        x = x.double()
        return x * torch.rsqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS) * w.double()

    if op == "before":
        z = norm(st["x"], st["w"])
        return {"z": z, "q": _held(z.bfloat16(), case["quant"], tab)}
    b = st["y"].double() if st["post"] is None else norm(st["y"], st["post"])
    out = st["res"].double() + _ALPHA * b * (1.0 if st["gate"] is None else st["gate"].double())
    z = norm(out.bfloat16(), st["w"])  # the next norm reads the residual as it is stored, the codes z as it is stored
    return {"out": out, "z": z, "q": _held(z.bfloat16(), case["quant"], tab)}
