"""The MXFP4 products on sums that fp32 holds exactly: every output has to be
equal, whatever the order of the additions.

Codes are any; scales are 2^0 or 2^1 on both sides (times one power of two for a
whole side), so that a product of two elements is a multiple of a quarter unit of at
most 6 * 6 * 4 = 144, and a sum of K <= 16384 of them, like each of its parts, is a
whole number of quarters of at most 144 * 4 * 16384 < 2^24.  A single wrong element,
scale or K-step shows.

The tiled product's workgroups walk several items each here, with stages that run on
from one item into the next: with items of up to 256 rows x 256 weight rows, there
are more of them than workgroups however the rows are cut."""
import pytest
import torch

import fp4_routed_expert_amd as moe

pytestmark = pytest.mark.gpu

DECODE, PREFILL = moe.MOE_FLAG_FORCE_DECODE, moe.MOE_FLAG_FORCE_PREFILL
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1 += [-v for v in E2M1]


def rows4(g, *shape, shift=0):
    """Codes and scales of [.., K]."""
    q = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), dtype=torch.uint8, device=g.device, generator=g)
    s = torch.randint(127 + shift, 129 + shift, (*shape[:-1], shape[-1] // 32), dtype=torch.uint8, device=g.device,
                      generator=g)
    return q, s


def values(q, s):
    table = torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], dtype=torch.float64, device=q.device)
    v = table[q.int()].view(*s.shape, 32) * torch.exp2(s.double() - 127).unsqueeze(-1)
    return v.view(*q.shape[:-1], 2 * q.shape[-1])


def gen(dev, *seed):
    n = 0
    for v in seed:
        n = (1000003 * n + v) % (1 << 31)
    return torch.Generator(device=dev).manual_seed(n)


def gate_shift(K):
    """Power of two that brings a gate's sums near one: an element's mean square is 8.6 (codes) times 2.5 (scales)."""
    return -round(torch.tensor(21.4 * K ** 0.5).log2().item())


def expect(x, w, u=None):
    """The exact sums x w^T, or silu(x w^T) (x u^T) in 64 bits and its error in fp32: the exponential's argument
    is rounded to 2^-24 of its size, and it, the reciprocal and three operations are off by an ulp or two each:
    together below (|g| + 8) 2^-22 of the result (the sums are exact)."""
    a = x @ w.T
    if u is None:
        return a, torch.zeros((), dtype=torch.float64, device=x.device)
    h = a / (1 + torch.exp(-a)) * (x @ u.T)
    return h, (a.abs() + 8) * 2.0 ** -22 * h.abs()


def check(y, want, err, what):
    d = (y.double() - want).abs()
    if y.dtype == torch.bfloat16:
        err = err + 2.0 ** -8 * (want.abs() + err)
    bad = ~(d <= err)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0].tolist()}"


def chained(dev, row_tiles, columns):
    """More items than workgroups, with the tallest tiles even."""
    cus = torch.cuda.get_device_properties(dev).multi_processor_count // 8 * 8
    assert row_tiles * columns > cus, (row_tiles, columns, cus)


def dense(dev, T, K, N, flags, glu=False, out=torch.float32):
    g = gen(dev, T, K, N, int(glu))
    x, w, u = rows4(g, T, K), rows4(g, N, K, shift=gate_shift(K) if glu else 0), rows4(g, N, K)
    pw = moe.mxfp4_prepack_glu(*w, *u) if glu else moe.mxfp4_prepack(*w)
    y = torch.full((T + 2, N), 7.0, dtype=out, device=dev)
    moe.mxfp4_dense(pw, *x, flags=flags, y=y[:T])
    check(y[:T], *expect(values(*x), values(*w), values(*u) if glu else None), f"T {T} K {K} N {N}")
    assert (y[T:] == 7.0).all()


@pytest.mark.parametrize("T,K,N", [(1, 128, 32), (8, 16384, 96), (40, 7168, 160), (33, 2048, 64), (300, 16384, 288),
                                   (257, 1408, 544)])
@pytest.mark.parametrize("flags", [DECODE, PREFILL])
def test_dense_exact(dev, T, K, N, flags):
    dense(dev, T, K, N, flags)


# Stages (of 256 K) per item: 1, 2 and 3 with an odd number of K-steps, 5, 6 odd, 8, 28.
@pytest.mark.parametrize("K", [128, 384, 640, 1280, 1408, 2048, 7168])
@pytest.mark.parametrize("T,N", [(2600, 7168), (2817, 7200)])
def test_dense_items_run_on(dev, T, K, N):
    chained(dev, (T + 255) // 256, (N + 255) // 256)
    dense(dev, T, K, N, PREFILL)


@pytest.mark.parametrize("K", [128, 640, 1280, 1408, 2048])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_dense_glu_items_run_on(dev, K, out):
    T, N = 2600, 3616
    chained(dev, (T + 255) // 256, (N + 127) // 128)
    dense(dev, T, K, N, PREFILL, glu=True, out=out)


SIZES = [700, 0, 1, 530, 256, 33, 900, 5]


@pytest.mark.parametrize("gather", [None, (500, 4)])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("K", [128, 384, 1280, 1408, 2048])
def test_grouped_items_run_on(dev, K, glu, gather):
    """Groups that are empty, of one row and of several tiles; rows in front of the first group and behind the
    last one are left as they were.  gather: (rows of x, row_div)."""
    N, lead, tail = (3616 if glu else 7200), 2, 3
    chained(dev, sum((n + 255) // 256 for n in SIZES), (N + 127) // 128 if glu else (N + 255) // 256)
    E, P = len(SIZES), lead + sum(SIZES) + tail
    g = gen(dev, K, int(glu), 0 if gather is None else 1)
    X = P if gather is None else gather[0]
    rows = None if gather is None else torch.randint(0, X * gather[1], (P,), dtype=torch.int32, device=dev, generator=g)
    x, w, u = rows4(g, X, K), rows4(g, E, N, K, shift=gate_shift(K) if glu else 0), rows4(g, E, N, K)
    pw = moe.mxfp4_prepack_glu(*w, *u) if glu else moe.mxfp4_prepack(*w)
    off = lead + torch.tensor([0] + SIZES).cumsum(0)
    read = values(*x)
    if gather:
        read = read[(rows // gather[1]).long()]
    for flags in (PREFILL, DECODE):
        y = torch.full((P, N), 7.0, dtype=torch.float32, device=dev)
        moe.mxfp4_grouped(pw, *x, off.int().to(dev), rows=rows, row_div=gather[1] if gather else 1, flags=flags, y=y)
        for e in range(E):
            i = slice(int(off[e]), int(off[e + 1]))
            if i.start < i.stop:
                check(y[i], *expect(read[i], values(w[0][e], w[1][e]), values(u[0][e], u[1][e]) if glu else None),
                      f"expert {e}, flags {flags}")
        assert (y[:lead] == 7.0).all() and (y[off[E]:] == 7.0).all()


@pytest.mark.parametrize("flags", [DECODE, PREFILL])
def test_glu_gates_to_their_end(dev, flags):
    """Gates from 0 to +-103 beside an up sum of 2^100: within the error of the exponential and the reciprocal down
    to -87, where 1 + exp(-g) passes 2^125; below it 0 is as good (the reciprocal has no subnormals)."""
    a, b, c = (t.reshape(-1) for t in torch.meshgrid(torch.arange(8), torch.arange(8), torch.arange(2), indexing="ij"))
    T, K, N = a.numel(), 128, 32
    q, s = torch.zeros(T, K // 2, dtype=torch.uint8), torch.full((T, K // 32), 127, dtype=torch.uint8)
    q[:, 0], q[:, 16], q[:, 32], q[:, 48] = a, b, c, 2          # elements 0, 32, 64 and 96 (1.0)
    s[:, 0] = 131                                               # 2^4
    wq, uq = torch.zeros(N, K // 2, dtype=torch.uint8), torch.zeros(N, K // 2, dtype=torch.uint8)
    ws, us = torch.full((N, K // 32), 127, dtype=torch.uint8), torch.full((N, K // 32), 227, dtype=torch.uint8)
    wq[:, [0, 16, 32]] = 2                                      # 1.0
    wq[::2, [0, 16, 32]] = 10                                   # -1.0
    uq[:, 48] = 2
    x, w, u = ([t.to(dev) for t in p] for p in ((q, s), (wq, ws), (uq, us)))
    want, err = expect(values(*x), values(*w), values(*u))
    g = values(*x) @ values(*w).T
    assert g.min() == -g.max() and g.max() > 102
    y = moe.mxfp4_dense(moe.mxfp4_prepack_glu(*w, *u), *x, torch.float32, flags)
    check(y, want, err + torch.where(g < -87, want.abs(), 0.0), f"flags {flags}")
