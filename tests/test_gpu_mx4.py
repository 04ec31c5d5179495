"""The MXFP4 operators and the block norms on the GPU against the 64-bit
reference (mx4_ref), on both paths, at the sizes where each can go wrong."""
import threading

import numpy as np
import pytest
import torch

import fp4_routed_expert_amd as moe
import mx4_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DECODE, PREFILL = moe.MOE_FLAG_FORCE_DECODE, moe.MOE_FLAG_FORCE_PREFILL


def rng(*seed):
    return np.random.default_rng(seed)


def dev_t(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def host(t):
    return t.float().cpu().numpy() if t.dtype in (torch.bfloat16, torch.float16) else t.cpu().numpy()


def rows4(r, M, K):
    """MXFP4 rows of normal data: codes, scales and their values."""
    q, s = ref.quant(r.standard_normal((M, K)) * np.exp(r.standard_normal((M, 1))), "mxfp4")
    return q, s, ref.values(q, s)


def weights4(r, *shape):
    """Weights with every code alike and scales around 1/sqrt(K) of their own."""
    q = r.integers(0, 256, (*shape[:-1], shape[-1] // 2), dtype=np.uint8)
    mid = 126 - int(np.log2(shape[-1])) // 2
    s = r.integers(mid - 2, mid + 3, (*shape[:-1], shape[-1] // 32), dtype=np.uint8)
    return q, s, ref.values(q, s)


def check(got, want, err, what=""):
    d = np.abs(host(got).astype(np.float64) - want)
    assert np.isfinite(host(got)).all(), what
    assert (d <= err).all(), f"{what}: {np.max(d / np.maximum(err, 1e-300)):.3f} of the bound"


# ------------------------------------------------------------- quantisation
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (8, 4096), (257, 160), (1000, 2080)])
def test_quant_rows(dev, dtype, M, K):
    r = rng(M, K)
    x = (r.standard_normal((M, K)) * np.exp2(r.integers(-12, 13, (M, K // 32)).repeat(32, 1))).astype(np.float32)
    x[r.random((M, K)) < 0.02] = 0.0
    t = torch.from_numpy(x).to(DT[dtype]).to(dev)
    q, s = moe.quant_mxfp4(t)
    qr, sr = ref.quant(host(t), "mxfp4")
    assert np.array_equal(host(s), sr) and np.array_equal(host(q), qr)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quant_every_pattern(dev, dtype):
    """Every 16-bit pattern, each in a block of neighbouring patterns and alone in a block of zeros."""
    bits = np.arange(65536, dtype=np.uint16)
    alone = np.zeros((65536, 32), np.uint16)
    alone[np.arange(65536), bits % 32] = bits
    for b in (bits.reshape(-1, 32), alone, rng(5).permutation(bits).reshape(-1, 64)):
        t = torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(DT[dtype]).to(dev)
        q, s = moe.quant_mxfp4(t)
        v = ref.bf16_of_bits(b) if dtype == "bf16" else b.view(np.float16).astype(np.float32)
        qr, sr = ref.quant(v, "mxfp4")
        assert np.array_equal(host(s), sr) and np.array_equal(host(q), qr)


def test_quant_borders_fp32(dev):
    """Values on, just below and just above every rounding border, at scales over the whole range, and
    blocks with NaN, infinities, zeros of both signs and subnormals."""
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], np.float32)
    near = np.concatenate([border, np.nextafter(border, f32(9)), np.nextafter(border, f32(0))])
    near = np.concatenate([near, [4.0, 7.9999995, 0.0, -0.0, 1e-30]]).astype(np.float32)[:32]
    rows = []
    for e in list(range(-149, 126, 7)) + [125]:
        with np.errstate(over="ignore", under="ignore"):
            rows.append(np.ldexp(near, e).astype(np.float32))
            rows.append(-rows[-1])
    x = np.stack(rows)
    x[~np.isfinite(x)] = 1.0
    special = np.ones((6, 32), np.float32)
    special[0, 3], special[1, 31], special[2, 0] = np.nan, np.inf, -np.inf
    special[3], special[4], special[5] = 0.0, -0.0, 2.0 ** -149
    x = np.concatenate([x, special, np.full((1, 32), np.finfo(np.float32).max, np.float32)])
    q, s = moe.quant_mxfp4(dev_t(x, dev))
    qr, sr = ref.quant(x, "mxfp4")
    assert np.array_equal(host(s), sr) and np.array_equal(host(q), qr)


f32 = np.float32


def test_quant_strided_rows_and_no_rows(dev):
    r = rng(7)
    for dtype, ld in (("bf16", 264), ("fp32", 300), ("fp16", 1024)):
        full = torch.from_numpy(r.standard_normal((37, ld)).astype(np.float32)).to(DT[dtype]).to(dev)
        q, s = moe.quant_mxfp4(full[:, 8:8 + 224])
        qr, sr = ref.quant(host(full)[:, 8:8 + 224], "mxfp4")
        assert np.array_equal(host(s), sr) and np.array_equal(host(q), qr)
    q, s = moe.quant_mxfp4(torch.empty(0, 64, dtype=torch.bfloat16, device=dev))
    assert q.shape == (0, 32) and s.shape == (0, 2)
    with pytest.raises(moe.MoeError):                                      # rows not 16-byte aligned
        moe.quant_mxfp4(torch.zeros(4, 68, dtype=torch.bfloat16, device=dev)[:, :64])


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_dequant_every_code_and_scale(dev, fmt, dtype):
    s = np.arange(256, dtype=np.uint8).repeat(8).reshape(256, 8)
    q = np.broadcast_to(np.arange(128 if fmt == "mxfp4" else 256, dtype=np.uint8), (256, 128 if fmt == "mxfp4" else 256))
    got = moe.dequant_mx(dev_t(q, dev), dev_t(s, dev), fmt, DT[dtype])
    want = ref.values(q, s, fmt)
    with np.errstate(over="ignore"):
        want32 = want.astype(np.float32)
    want_t = torch.from_numpy(want32).to(DT[dtype])
    assert torch.equal(got.cpu().isnan(), want_t.isnan())
    assert torch.equal(got.cpu().nan_to_num(nan=0.0), want_t.nan_to_num(nan=0.0))


# ------------------------------------------------------------------ products
def dense_case(dev, T, K, N, out, flags, seed=1):
    r = rng(T, K, N, seed)
    xq, xs, x = rows4(r, T, K)
    wq, ws, w = weights4(r, N, K)
    pw = moe.mxfp4_prepack(dev_t(wq, dev), dev_t(ws, dev))
    y = torch.full((T + 3, N), 7.0, dtype=DT[out], device=dev)
    moe.mxfp4_dense(pw, dev_t(xq, dev), dev_t(xs, dev), flags=flags, y=y[:T])
    check(y[:T], *ref.product(x, w, out), f"T {T} K {K} N {N}")
    assert (y[T:] == 7.0).all()


@pytest.mark.parametrize("flags", [DECODE, PREFILL, 0])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("T,K,N", [(1, 128, 32), (2, 256, 64), (8, 384, 96), (31, 512, 128), (32, 640, 160), (33, 768, 288),
                                   (64, 128, 1056), (100, 1024, 224), (255, 256, 32), (256, 384, 320), (257, 128, 96),
                                   (300, 512, 256), (513, 640, 544), (1000, 896, 64)])
def test_dense(dev, T, K, N, out, flags):
    dense_case(dev, T, K, N, out, flags)


@pytest.mark.parametrize("T,K,N,flags", [(8, 16384, 512, 0), (1, 7168, 2048, 0), (1100, 2048, 7168, PREFILL),
                                         (2300, 512, 4096, PREFILL), (2300, 384, 7168, 0), (4600, 256, 7168, 0),
                                         (1024, 1024, 2048, 0), (1500, 2048, 1056, 0)])
def test_dense_large(dev, T, K, N, flags):
    """Long sums, tiles of every height, and more work items than workgroups (each walks several)."""
    dense_case(dev, T, K, N, "bf16", flags)


def test_dense_scale_extremes_and_nan(dev):
    """Scales at both ends of the range, a NaN block in a row of x and one in a row of W: NaN exactly
    where such a row takes part."""
    r = rng(9)
    T, K, N = 70, 384, 96
    xq, xs, _ = rows4(r, T, K)
    wq, ws, _ = weights4(r, N, K)
    xs[3], xs[4] = 0, 254
    ws[:, :] = r.integers(120, 124, ws.shape)
    ws[5] = 0
    ws[6, ::2] = 1
    x, w = ref.values(xq, xs), ref.values(wq, ws)
    xs[10, 11], ws[50, 0] = 255, 255
    want, err = ref.product(x, w, "fp32")
    pw = moe.mxfp4_prepack(dev_t(wq, dev), dev_t(ws, dev))
    for flags in (DECODE, PREFILL):
        got = host(moe.mxfp4_dense(pw, dev_t(xq, dev), dev_t(xs, dev), torch.float32, flags))
        nan = np.zeros((T, N), bool)
        nan[10], nan[:, 50] = True, True
        # Row 4's scales are 2^127: where the magnitudes of a sum's terms reach 2^127 together, partial sums
        # (and, of terms with both signs, their difference) can leave fp32's range, 2^128, whatever the exact
        # sum is; such a value says nothing.  Everywhere else it has to be right.
        over = np.abs(x) @ np.abs(w).T >= 2.0 ** 127
        assert not over[np.arange(T) != 4].any()
        assert np.array_equal(np.isnan(got)[~over], nan[~over]) and np.isnan(got[4, 50])
        fine = ~nan & ~over
        # products below the smallest fp32 may come out as zero
        assert (np.abs(got - want)[fine] <= (err + 2.0 ** -126)[fine]).all()


def test_dense_glu(dev):
    for T, K, N in ((5, 256, 32), (40, 384, 96), (300, 128, 160), (270, 640, 64)):
        r = rng(T, N)
        xq, xs, x = rows4(r, T, K)
        wq, ws, w = weights4(r, N, K)
        uq, us, u = weights4(r, N, K)
        pw = moe.mxfp4_prepack_glu(*(dev_t(a, dev) for a in (wq, ws, uq, us)))
        for out in ("bf16", "fp32"):
            for flags in (DECODE, PREFILL):
                y = moe.mxfp4_dense(pw, dev_t(xq, dev), dev_t(xs, dev), DT[out], flags)
                check(y, *ref.glu(x, w, u, out), f"T {T} K {K} N {N} {out} {flags}")


@pytest.mark.parametrize("flags", [DECODE, PREFILL])
def test_dense_glu_far_gates(dev, flags):
    """Gate and up sums of 2^100 (their product is past fp32's range): a closed gate gives zero, an open one
    its product.  Each sum is one product of powers of two, so the outputs are exact."""
    K, N, T = 128, 32, 40
    xq, xs = np.zeros((T, K // 2), np.uint8), np.full((T, K // 32), 127, np.uint8)
    xq[:, 0] = 2                                                            # element 0: 1.0
    wq, uq = np.zeros((N, K // 2), np.uint8), np.zeros((N, K // 2), np.uint8)
    ws, us = np.full((N, K // 32), 227, np.uint8), np.full((N, K // 32), 227, np.uint8)
    wq[:, 0], uq[:, 0] = 10, 2                                              # -2^100, 2^100
    uq[1::3, 0] = 10                                                        # -2^100, -2^100
    wq[2::3, 0], us[2::3] = 2, 27                                           # 2^100, 2^-100
    pw = moe.mxfp4_prepack_glu(*(dev_t(a, dev) for a in (wq, ws, uq, us)))
    want = np.where(np.arange(N) % 3 == 2, 1.0, 0.0)
    for out in ("bf16", "fp32"):
        y = host(moe.mxfp4_dense(pw, dev_t(xq, dev), dev_t(xs, dev), DT[out], flags))
        assert (y == want).all()


def group_case(dev, sizes, K, N, glu=False, gather=None, out="bf16", flags=0, lead=0, tail=0, seed=0):
    """Groups of the given sizes in rows [lead, lead + sum) of P = lead + sum + tail; gather: (X, div)."""
    r = rng(len(sizes), K, N, seed)
    E, P = len(sizes), lead + sum(sizes) + tail
    off = lead + np.concatenate([[0], np.cumsum(sizes)])
    X = gather[0] if gather else P
    rows = r.integers(0, X * gather[1], P).astype(np.int32) if gather else None
    xq, xs, x = rows4(r, X, K)
    wq, ws, w = weights4(r, E, N, K)
    args = [dev_t(wq, dev), dev_t(ws, dev)]
    if glu:
        uq, us, u = weights4(r, E, N, K)
        args += [dev_t(uq, dev), dev_t(us, dev)]
    pw = (moe.mxfp4_prepack_glu if glu else moe.mxfp4_prepack)(*args)
    y = torch.full((P, N), 7.0, dtype=DT[out], device=dev)
    moe.mxfp4_grouped(pw, dev_t(xq, dev), dev_t(xs, dev), dev_t(off.astype(np.int32), dev),
                      rows=None if rows is None else dev_t(rows, dev), row_div=gather[1] if gather else 1, flags=flags, y=y)
    xr = x[rows // gather[1]] if gather else x
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a < b:
            want, err = ref.glu(xr[a:b], w[e], u[e], out) if glu else ref.product(xr[a:b], w[e], out)
            check(y[a:b], want, err, f"expert {e} of {sizes}")
    assert (y[:lead] == 7.0).all() and (y[off[E]:] == 7.0).all()


RAGGED = [[1], [0, 5, 0], [33, 0, 1, 256, 31, 0, 257], [64, 64], [0, 0, 700], [1] * 40, [130, 2, 300, 0, 513]]


@pytest.mark.parametrize("flags", [DECODE, PREFILL, 0])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("i", range(len(RAGGED)))
def test_grouped_ragged(dev, i, glu, flags):
    K, N = [(128, 64), (256, 96), (384, 32), (512, 288), (640, 128), (1024, 32), (256, 544)][i]
    group_case(dev, RAGGED[i], K, N, glu, None if i % 2 else (97, 3), "fp32" if i % 3 == 1 else "bf16", flags,
               lead=i % 3, tail=5 * (i % 2))


@pytest.mark.parametrize("gather", [None, (500, 4)])
@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 896])
def test_grouped_many_items(dev, K, gather):
    """More work items than workgroups, with fewer, as many and more K-steps than the ring has slots:
    the loads run on from one item into the next, or over several."""
    sizes = [(37 * i) % 190 for i in range(24)]
    group_case(dev, sizes, K, 4096 + 32, False, gather, "bf16", PREFILL, lead=2, tail=3)


@pytest.mark.parametrize("glu", [False, True])
def test_grouped_tall_tiles(dev, glu):
    """Items enough for the tallest tiles, whole and with their last rows missing."""
    group_case(dev, [1024, 768, 256, 250], 256, 3584 if glu else 7168, glu, None, "bf16", PREFILL, lead=1, tail=2)


@pytest.mark.parametrize("flags", [DECODE, PREFILL])
def test_scales_at_any_dword(dev, flags):
    """Activation scales need 4-byte alignment only: shifted copies give the same bits."""
    r = rng(43)
    P, K = 70, 1024
    xq, xs, _ = rows4(r, P, K)
    wq, ws, _ = weights4(r, 2, 64, K)
    pw, one = moe.mxfp4_prepack(dev_t(wq, dev), dev_t(ws, dev)), moe.mxfp4_prepack(dev_t(wq[0], dev), dev_t(ws[0], dev))
    q, s, off = dev_t(xq, dev), dev_t(xs, dev), dev_t(np.array([0, 33, P], np.int32), dev)
    want, dense = moe.mxfp4_grouped(pw, q, s, off, flags=flags), moe.mxfp4_dense(one, q, s, flags=flags)
    for shift in (4, 8, 12):
        t = torch.empty(s.numel() + shift, dtype=torch.uint8, device=dev)[shift:].view(s.shape)
        t.copy_(s)
        assert torch.equal(moe.mxfp4_grouped(pw, q, t, off, flags=flags), want)
        assert torch.equal(moe.mxfp4_dense(one, q, t, flags=flags), dense)


def test_grouped_no_rows(dev):
    r = rng(3)
    wq, ws, _ = weights4(r, 4, 64, 256)
    pw = moe.mxfp4_prepack(dev_t(wq, dev), dev_t(ws, dev))
    off = torch.zeros(5, dtype=torch.int32, device=dev)
    e = torch.empty
    y = moe.mxfp4_grouped(pw, e(0, 128, dtype=torch.uint8, device=dev), e(0, 8, dtype=torch.uint8, device=dev), off)
    assert y.shape == (0, 64)
    xq, xs, _ = rows4(r, 9, 256)
    for flags in (DECODE, PREFILL):                                        # rows, but all groups empty
        y = torch.full((9, 64), 7.0, dtype=torch.bfloat16, device=dev)
        moe.mxfp4_grouped(pw, dev_t(xq, dev), dev_t(xs, dev), off, flags=flags, y=y)
        assert (y == 7.0).all()


def test_grouped_after_route_and_sort(dev):
    """The routing's own offsets and sorted pairs; tokens gathered by pair / k."""
    r = rng(11)
    T, E, k, K, N = 200, 16, 3, 256, 128
    ids, _ = moe.route_topk(dev_t(r.standard_normal((T, E)).astype(np.float32), dev), k)
    _, off, sp, _ = moe.sort_permute(ids, E)
    xq, xs, x = rows4(r, T, K)
    wq, ws, w = weights4(r, E, N, K)
    pw = moe.mxfp4_prepack(dev_t(wq, dev), dev_t(ws, dev))
    o, tok = host(off), host(sp) // k
    for flags in (DECODE, PREFILL):
        y = moe.mxfp4_grouped(pw, dev_t(xq, dev), dev_t(xs, dev), off, rows=sp, row_div=k, flags=flags)
        for e in range(E):
            if o[e] < o[e + 1]:
                check(y[o[e]:o[e + 1]], *ref.product(x[tok[o[e]:o[e + 1]]], w[e]), f"expert {e}")


def test_products_repeat_their_bits(dev):
    """The same inputs give the same bits, with other work between."""
    r = rng(13)
    xq, xs, _ = rows4(r, 600, 1024)
    wq, ws, _ = weights4(r, 6, 512, 1024)
    pw = moe.mxfp4_prepack(dev_t(wq, dev), dev_t(ws, dev))
    off = dev_t(np.array([0, 100, 100, 350, 351, 590, 600], np.int32), dev)
    for flags in (DECODE, PREFILL):
        first = moe.mxfp4_grouped(pw, dev_t(xq, dev), dev_t(xs, dev), off, flags=flags)
        for _ in range(5):
            torch.randn(1 << 20, device=dev).sort()
            assert torch.equal(first, moe.mxfp4_grouped(pw, dev_t(xq, dev), dev_t(xs, dev), off, flags=flags))


def some_rows(dev, y, x_of, w_of, rows, out="bf16"):
    for e, i in rows:
        w = w_of(e)
        want, err = ref.product(x_of(i), w, out)
        check(y[i:i + 1], want, err, f"row {i}")


@pytest.mark.parametrize("flags", [DECODE, PREFILL])
def test_grouped_offsets_past_32_bits(dev, flags):
    """Weights, activations and outputs of more than 4 GiB each: the last rows and experts."""
    g = torch.Generator(device=dev).manual_seed(3)
    # 4.3 GiB of weights: 70 experts of 16384 x 7680 codes
    E, N, K = 70, 16384, 7680
    wq = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=dev, generator=g)
    ws = torch.randint(118, 122, (E, N, K // 32), dtype=torch.uint8, device=dev, generator=g)
    pw = moe.mxfp4_prepack(wq, ws)
    assert pw.buffer.numel() > 1 << 32
    r = rng(29)
    xq, xs, x = rows4(r, 40, K)
    off = np.zeros(E + 1, np.int32)
    off[1:-1], off[-1] = 3, 40                                              # expert 0: 3 rows, the last one: 37
    y = moe.mxfp4_grouped(pw, dev_t(xq, dev), dev_t(xs, dev), dev_t(off, dev), flags=flags)
    some_rows(dev, y, lambda i: x[i:i + 1], lambda e: ref.values(host(wq[e]), host(ws[e])), [(0, 2), (E - 1, 3), (E - 1, 39)])
    del wq, ws, pw, y
    # 4.5 GiB of outputs, and activation rows up to the largest byte offset
    N, K = 7168, 256
    P, X = 340000, ((1 << 33) - 8192) // K
    xq = torch.empty(X, K // 2, dtype=torch.uint8, device=dev).random_(0, 256, generator=g)
    xs = torch.randint(120, 124, (X, K // 32), dtype=torch.uint8, device=dev, generator=g)
    wq, ws, w = weights4(r, 2, N, K)
    rows = torch.arange(X - P, X, dtype=torch.int32, device=dev)
    off = torch.tensor([0, 5, P], dtype=torch.int32, device=dev)
    y = moe.mxfp4_grouped(moe.mxfp4_prepack(dev_t(wq, dev), dev_t(ws, dev)), xq, xs, off, rows=rows, flags=flags)
    assert y.numel() * 2 > 1 << 32
    some_rows(dev, y, lambda i: ref.values(host(xq[X - P + i:X - P + i + 1]), host(xs[X - P + i:X - P + i + 1])), lambda e: w[e],
              [(0, 0), (0, 4), (1, 5), (1, 200000), (1, P - 1)])
    with pytest.raises(moe.MoeError):                                       # one row more
        moe.mxfp4_grouped(moe.mxfp4_prepack(dev_t(wq, dev), dev_t(ws, dev)), xq.new_empty(X + 1, K // 2),
                          xs.new_empty(X + 1, K // 32), off, rows=rows)


def test_quant_and_norm_past_32_bits(dev):
    """More than 2^32 bytes of rows: the last ones."""
    g = torch.Generator(device=dev).manual_seed(5)
    M, K = 300000, 8192
    x = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    x.normal_(generator=g)
    q, s = moe.quant_mxfp4(x)
    v = moe.dequant_mx(q, s, "mxfp4")
    z, q8, s8 = moe.norm_before(x, torch.ones(K, device=dev), quant="mxfp8")
    for i in (0, 150000, M - 1):
        a = host(x[i:i + 1])
        qr, sr = ref.quant(a, "mxfp4")
        assert np.array_equal(host(q[i:i + 1]), qr) and np.array_equal(host(s[i:i + 1]), sr)
        assert np.array_equal(host(v[i:i + 1]), ref.values(qr, sr).astype(np.float32))
        zr = ref.norm_before(a, np.ones(K, np.float32), 1e-6)
        assert np.array_equal(host(z[i:i + 1]), zr)
        qr, sr = ref.quant(zr, "mxfp8")
        assert np.array_equal(host(q8[i:i + 1]), qr) and np.array_equal(host(s8[i:i + 1]), sr)


# --------------------------------------------------------------------- norms
def norm_data(r, T, H, dtype):
    x = torch.from_numpy((r.standard_normal((T, H)) * np.exp(r.standard_normal((T, 1)))).astype(np.float32))
    return x.to(DT[dtype])


def same(got, want):
    got, want = host(got), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.nan_to_num(got, nan=0.0), np.nan_to_num(want, nan=0.0))


@pytest.mark.parametrize("x_type,w_type", [("bf16", "fp32"), ("fp32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 32), (5, 40), (8, 4096), (2, 512), (3, 520), (4, 2048), (5, 2056), (9, 7168),
                                 (3, 8192), (2, 8224), (2, 16384), (700, 256)])
def test_norm_before(dev, T, H, x_type, w_type):
    r = rng(T, H)
    x, w = norm_data(r, T, H, x_type), norm_data(r, 1, H, w_type)[0]
    want = ref.norm_before(host(x), host(w), 1e-5)
    z, q, s = moe.norm_before(x.to(dev), w.to(dev), 1e-5)
    same(z, want)
    assert q is None and s is None
    for quant in ("mxfp8", "mxfp4") if H % 32 == 0 else ():
        for want_z in (True, False):
            z, q, s = moe.norm_before(x.to(dev), w.to(dev), 1e-5, quant, want_z)
            qr, sr = ref.quant(want, quant)
            assert np.array_equal(host(q), qr) and np.array_equal(host(s), sr)
            assert z is None if not want_z else np.array_equal(host(z), want)


@pytest.mark.parametrize("y_type,res_type", [("fp32", "bf16"), ("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("gate", [None, "token", "channel", "both", "wide"])
@pytest.mark.parametrize("post,nxt,quant", [(True, True, "mxfp4"), (False, True, "mxfp8"), (True, False, None),
                                            (False, False, None), (True, True, None)])
def test_norm_after(dev, y_type, res_type, gate, post, nxt, quant):
    for T, H in ((1, 32), (5, 544), (4, 4096), (6, 7168), (2, 9216)):
        r = rng(T, H, 2)
        y, res = norm_data(r, T, H, y_type), norm_data(r, T, H, res_type)
        wp = norm_data(r, 1, H, "fp32")[0] if post else None
        wn = norm_data(r, 1, H, "fp32")[0] if nxt else None
        shape = {None: None, "token": (T, 1), "channel": (H,), "both": (T, H), "wide": (T, H)}[gate]
        g = None if gate is None else torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(dev)
        if gate == "wide":                                                 # rows further apart than they are long
            g = torch.cat([g, g], 1)[:, :H]
        to = lambda t: None if t is None else t.to(dev)  # noqa: E731
        out, z, q, s = moe.norm_after(to(y), to(res), to(wp), g, 0.7, 0.5, 1e-6, to(wn), quant)
        want = ref.norm_after(host(y), host(res), None if wp is None else host(wp), None if g is None else host(g), 0.7, 0.5,
                              1e-6, res_type == "bf16")
        same(out, want)
        if not nxt:
            assert z is None and q is None and s is None
            continue
        zr = ref.norm_before(want, host(wn), 1e-6)
        same(z, zr)
        if quant:
            qr, sr = ref.quant(zr, quant)
            assert np.array_equal(host(q), qr) and np.array_equal(host(s), sr)


def test_norm_against_64_bits(dev):
    """The defined steps stay within their roundings of the formula: r, x r and (x r) w in fp32 (2^-24 each) and the
    one to bf16 (2^-8)."""
    r = rng(17)
    x, w = norm_data(r, 50, 7168, "bf16"), norm_data(r, 1, 7168, "fp32")[0]
    z, _, _ = moe.norm_before(x.to(dev), w.to(dev), 1e-6)
    v = host(x).astype(np.float64)
    want = v / np.sqrt((v ** 2).mean(-1, keepdims=True) + 1e-6) * host(w)
    assert (np.abs(host(z) - want) <= np.abs(want) * (2.0 ** -8 + 4 * 2.0 ** -24) + 2.0 ** -133).all()


def test_norm_in_place_and_special_rows(dev):
    """out may be the residual; a NaN or an infinity stays in its row; a row of zeros gives zeros; no rows."""
    r = rng(19)
    T, H = 6, 1024
    y, res, w = norm_data(r, T, H, "fp32"), norm_data(r, T, H, "bf16"), norm_data(r, 1, H, "fp32")[0]
    y[1, 100], y[2, 5], y[3] = float("nan"), float("inf"), 0.0
    res[3] = 0.0
    want = ref.norm_after(host(y), host(res), host(w), None, 1.0, 1.0, 1e-6, True)
    with np.errstate(invalid="ignore"):
        zr = ref.norm_before(want, host(w), 1e-6)
    for quant in ("mxfp8", "mxfp4"):
        t = res.to(dev)
        out, z, q, s = moe.norm_after(y.to(dev), t, w.to(dev), next_weight=w.to(dev), quant=quant, out=t)
        assert out is t
        same(out, want)
        same(z, zr)
        qr, sr = ref.quant(zr, quant)
        assert np.array_equal(host(s), sr) and np.array_equal(host(q), qr)
        assert (host(s)[1] == 255).all() and (host(s)[3] == 0).all() and not host(z)[3].any()
    e = torch.empty(0, H, dtype=torch.bfloat16, device=dev)
    z, q, s = moe.norm_before(e, w.to(dev), quant="mxfp8")
    assert z.shape == (0, H) and q.shape == (0, H) and s.shape == (0, H // 32)


def test_norm_codes_are_the_quantisers(dev):
    r = rng(23)
    x, w = norm_data(r, 33, 2048, "bf16").to(dev), norm_data(r, 1, 2048, "fp32")[0].to(dev)
    z, q, s = moe.norm_before(x, w, quant="mxfp8")
    q8, s8 = moe.quant_act_mxfp8(z)
    assert torch.equal(q, q8) and torch.equal(s, s8)
    z, q, s = moe.norm_before(x, w, quant="mxfp4")
    q4, s4 = moe.quant_mxfp4(z)
    assert torch.equal(q, q4) and torch.equal(s, s4)


# --------------------------------------------------------------- the block
def block_setup(dev, seed, E=8, H=512, I=256, ns=1):
    r = rng(seed)
    w = []
    for shape in ((E, I, H), (E, I, H), (E, H, I)):
        q, s, _ = weights4(r, *shape)
        w += [dev_t(q, dev), dev_t(s, dev)]
    pw = moe.prepack_weights(*w)
    wg = torch.from_numpy((r.standard_normal((E - ns, H)) / np.sqrt(H)).astype(np.float32)).bfloat16().to(dev)
    n = [torch.from_numpy((1 + 0.1 * r.standard_normal(H)).astype(np.float32)).to(dev) for _ in range(2)]
    return r, pw, wg, n


@pytest.mark.parametrize("T", [1, 8, 16, 17, 100, 300])
@pytest.mark.parametrize("ns,post,x_type", [(0, True, "bf16"), (1, False, "fp32"), (1, True, "bf16")])
def test_block_is_its_chain(dev, T, ns, post, x_type):
    r, pw, wg, (pre, after) = block_setup(dev, T, ns=ns)
    x = norm_data(r, T, 512, x_type).to(dev)
    gate = torch.from_numpy(r.random((T, 1)).astype(np.float32)).to(dev)
    wp = after if post else None
    z, _, _ = moe.norm_before(x, pre, 1e-5)
    y = moe.layer_forward_full(pw, ns, wg, z, 2)
    want, _, _, _ = moe.norm_after(y, x, wp, gate, 0.7, 1.0, 1e-5)
    got = moe.block_forward(pw, ns, wg, x, 2, pre, wp, gate, 0.7, 1.0, 1e-5)
    assert torch.equal(got, want)
    moe.block_forward(pw, ns, wg, x, 2, pre, wp, gate, 0.7, 1.0, 1e-5, out=x)
    assert torch.equal(x, want)


def four_bit_block(x, w, k, buf=None):
    """A block with 4-bit activations: norm -> route -> gate/up -> down -> combine -> norm + residual."""
    z, q, s = moe.norm_before(x, w["pre"], quant="mxfp4")
    ids, gates = moe.route_topk(moe.router_logits(z, w["router"]), k)
    _, off, sp, pp = moe.sort_permute(ids, w["up"].E)
    h = moe.mxfp4_grouped(w["up"], q, s, off, rows=sp, row_div=k)
    hq, hs = moe.quant_mxfp4(h)
    o = moe.mxfp4_grouped(w["down"], hq, hs, off)
    y = moe.combine(o, gates, pp, x.shape[0], k, x.shape[1])
    out, z2, q2, s2 = moe.norm_after(y, x, w["post"], next_weight=w["pre"], quant="mxfp4")
    proj = moe.mxfp4_dense(w["proj"], q2, s2)
    return dict(z=z, q=q, s=s, gates=gates, off=off, sp=sp, pp=pp, h=h, hq=hq, hs=hs, o=o, y=y, out=out, z2=z2, q2=q2,
                s2=s2, proj=proj)


def four_bit_weights(dev, seed, E=8, H=512, I=256, N=384):
    r = rng(seed)
    vals = {"w1": weights4(r, E, I, H), "w3": weights4(r, E, I, H), "w2": weights4(r, E, H, I), "proj": weights4(r, N, H)}
    t = {n: (dev_t(v[0], dev), dev_t(v[1], dev)) for n, v in vals.items()}
    w = {"up": moe.mxfp4_prepack_glu(*t["w1"], *t["w3"]), "down": moe.mxfp4_prepack(*t["w2"]),
         "proj": moe.mxfp4_prepack(*t["proj"]),
         "router": torch.from_numpy((r.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32)).bfloat16().to(dev),
         "pre": torch.from_numpy((1 + 0.1 * r.standard_normal(H)).astype(np.float32)).to(dev),
         "post": torch.from_numpy((1 + 0.1 * r.standard_normal(H)).astype(np.float32)).to(dev)}
    return r, w, {n: v[2] for n, v in vals.items()}


@pytest.mark.parametrize("T", [1, 7, 64, 333])
def test_run_of_the_operators(dev, T):
    """The whole 4-bit block, each stage against the reference on the stage before it."""
    k = 2
    r, w, v = four_bit_weights(dev, T)
    x = norm_data(r, T, 512, "bf16")
    b = {n: host(t) for n, t in four_bit_block(x.to(dev), w, k).items()}
    zr = ref.norm_before(host(x), host(w["pre"]), 1e-6)
    qr, sr = ref.quant(zr, "mxfp4")
    assert np.array_equal(b["z"], zr) and np.array_equal(b["q"], qr) and np.array_equal(b["s"], sr)
    xv, tok = ref.values(qr, sr), b["sp"] // k
    hv = ref.values(b["hq"], b["hs"])
    for e in range(8):
        i = slice(b["off"][e], b["off"][e + 1])
        if i.start < i.stop:
            want, err = ref.glu(xv[tok[i]], v["w1"][e], v["w3"][e])
            assert (np.abs(b["h"][i] - want) <= err).all()
            want, err = ref.product(hv[i], v["w2"][e])
            assert (np.abs(b["o"][i] - want) <= err).all()
    hq, hs = ref.quant(b["h"], "mxfp4")
    assert np.array_equal(b["hq"], hq) and np.array_equal(b["hs"], hs)
    out = ref.norm_after(b["y"], host(x), host(w["post"]), None, 1.0, 1.0, 1e-6, True)
    assert np.array_equal(b["out"], out)
    q2, s2 = ref.quant(ref.norm_before(out, host(w["pre"]), 1e-6), "mxfp4")
    assert np.array_equal(b["q2"], q2) and np.array_equal(b["s2"], s2)
    want, err = ref.product(ref.values(q2, s2), v["proj"])
    assert (np.abs(b["proj"] - want) <= err).all()


# ------------------------------------------- streams, graphs, host threads
def test_other_stream(dev):
    r, w, _ = four_bit_weights(dev, 31)
    x = norm_data(r, 50, 512, "bf16").to(dev)
    want = four_bit_block(x, w, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = four_bit_block(x, w, 2)
    side.synchronize()
    for n in ("h", "o", "out", "proj"):
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("T", [5, 300])
def test_graph_replays(dev, T):
    """Two graphs with their own buffers, replayed with new inputs and eager work between."""
    r, w, _ = four_bit_weights(dev, 37)
    rb, pw, wg, (pre, post) = block_setup(dev, 37)
    xs = [norm_data(r, T, 512, "bf16").to(dev) for _ in range(4)]
    static = [xs[0].clone(), xs[1].clone()]
    four_bit_block(static[0], w, 2)
    moe.block_forward(pw, 1, wg, static[0], 2, pre, post)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((four_bit_block(static[i], w, 2), moe.block_forward(pw, 1, wg, static[i], 2, pre, post)))
        graphs.append(g)
    for step in range(4):
        for i in range(2):
            static[i].copy_(xs[(step + i) % 4])
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            want = four_bit_block(xs[(step + i) % 4], w, 2)
            for n in ("h", "o", "out", "q2", "proj"):
                assert torch.equal(outs[i][0][n], want[n]), (step, i, n)
            assert torch.equal(outs[i][1], moe.block_forward(pw, 1, wg, xs[(step + i) % 4], 2, pre, post))


def test_host_threads(dev):
    r, w, _ = four_bit_weights(dev, 41)
    xs = [norm_data(r, 40 + 60 * i, 512, "bf16").to(dev) for i in range(4)]
    want = [four_bit_block(x, w, 2) for x in xs]
    torch.cuda.synchronize()
    got, failed = [None] * 4, []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    got[i] = four_bit_block(xs[i], w, 2)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    ts = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not failed, failed
    for i in range(4):
        for n in ("h", "o", "out", "proj"):
            assert torch.equal(got[i][n], want[i][n]), (i, n)
