"""The FP8 operators with block scales of 128 on the GPU against their definitions in 64 bits."""
import pytest
import torch

import fp4_routed_expert_amd as moe
import fp8b_ref as ref

pytestmark = pytest.mark.gpu
DEC, PRE = moe.MOE_FLAG_FORCE_DECODE, moe.MOE_FLAG_FORCE_PREFILL
BF, FH, FS = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def make_rows(g, M, K):
    return ref.quant((normal(g, M, K) * torch.exp(normal(g, M, 1))).to(BF))


def make_weights(g, E, N, K):
    """Codes of every magnitude, scales of every block its own."""
    q = (normal(g, E, N, K) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.exp(normal(g, E, (N + 127) // 128, K // 128)) * K ** -0.5 / 100
    return q, s


def within(got, want, err, what=""):
    d = (got.double() - want).abs()
    bad = ~(d <= err)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d / err).nan_to_num(9e9).max()):.3g}x"


# ------------------------------------------------------------- quantisation
@pytest.mark.parametrize("dtype", [BF, FH, FS])
@pytest.mark.parametrize("M,K", [(1, 128), (5, 384), (16, 512), (17, 640), (130, 7168)])
def test_quant(dtype, M, K):
    g = gen(M + K)
    x = (normal(g, M, K) * torch.exp(2 * normal(g, M, 1))).to(dtype)
    x[0, :128] = 0
    if M > 4:
        x[1, 3], x[2, 130], x[3, 1], x[4, 200] = float("nan"), float("inf"), -0.0, float("-inf")
    q, s = moe.quant_fp8_block(x)
    wq, ws = ref.quant(x)
    assert torch.equal(q, wq)
    assert torch.equal(s.isnan(), ws.isnan()) and torch.equal(s.nan_to_num(0), ws.nan_to_num(0))
    for out in (BF, FH, FS):
        v = moe.dequant_fp8_block(q, s, dtype=out)
        want = (ref.code_values(wq).float() * ws.t().repeat_interleave(128, 1)).to(out)
        assert torch.equal(v.isnan(), want.isnan()) and torch.equal(v.nan_to_num(0), want.nan_to_num(0))


@pytest.mark.parametrize("scale", [2.0 ** -149, 2.0 ** -120, 2.0 ** -100, 2.0 ** 100, 2.0 ** 126])
def test_quant_ends_of_the_range(scale):
    x = torch.linspace(-1, 1, 256, device="cuda").view(2, 128) * scale
    q, s = moe.quant_fp8_block(x)
    wq, ws = ref.quant(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)


def test_quant_strided_rows_and_views():
    g = gen(7)
    x = normal(g, 9, 520).to(BF)[:, 8:264]
    q, s = moe.quant_fp8_block(x)
    wq, ws = ref.quant(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)
    x = normal(g, 1, 256)
    assert torch.equal(moe.quant_fp8_block(x)[0], ref.quant(x)[0])
    q, s = moe.quant_fp8_block(torch.empty(0, 256, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (2, 0)


def test_quant_more_than_2_to_28_rows():
    """More workgroups than a launch dimension holds threads for."""
    M = 2 ** 28 + 2 ** 24 + 5
    x = torch.zeros(M, 128, dtype=BF, device="cuda")
    at = torch.tensor([0, 2 ** 24 - 1, 2 ** 24, 2 ** 28 - 1, 2 ** 28, M - 1], device="cuda")
    rows = normal(gen(51), 6, 128).to(BF)
    x[at] = rows
    q, s = moe.quant_fp8_block(x)
    want = ref.quant(rows)
    assert torch.equal(q[at], want[0]) and torch.equal(s[:, at], want[1])
    assert int((s != 2.0 ** -110 / 448).sum()) == 6
    moe.dequant_fp8_block(q, s, out=x)
    assert torch.equal(x[at].double(), ref.rows(*want).to(BF).double())
    del x, q, s
    torch.cuda.empty_cache()


def test_quant_codes_of_torchs_type():
    x = normal(gen(8), 4, 256)
    q = torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="cuda")
    s = moe.quant_fp8_block(x, q=q)[1]
    assert torch.equal(q.float() * s.t().repeat_interleave(128, 1), moe.dequant_fp8_block(q, s, dtype=FS))


# ------------------------------------------------------------ dense product
@pytest.mark.parametrize("flags", [DEC, PRE])
@pytest.mark.parametrize("dtype", [BF, FS])
@pytest.mark.parametrize("T,K,N", [(1, 128, 32), (3, 256, 160), (16, 384, 128), (17, 128, 288), (40, 1024, 256),
                                   (257, 640, 352), (600, 256, 512), (50, 384, 5120), (230, 4096, 4096)])
def test_dense(flags, dtype, T, K, N):
    g = gen(T * 7 + K + N)
    xq, xs = make_rows(g, T, K)
    wq, ws = make_weights(g, 1, N, K)
    w = moe.fp8_block_prepack(wq[0], ws[0])
    y = torch.full((T + 1, N), 7.0, dtype=dtype, device="cuda")
    moe.fp8_block_dense(w, xq, xs, flags=flags, y=y[:T])
    want, err = ref.product(ref.rows(xq, xs), ref.weights(wq[0], ws[0]), ref.HALF[dtype])
    within(y[:T], want, err)
    assert (y[T] == 7).all()
    assert torch.equal(moe.fp8_block_dense(w, xq, xs, flags=flags, dtype=dtype), y[:T])


@pytest.mark.parametrize("flags", [DEC, PRE])
@pytest.mark.parametrize("dtype", [BF, FS])
def test_dense_all_codes(flags, dtype):
    """Every code.  In fp32 the products are exact; in bf16 eight neighbouring ones are added with 14 bits below the
    largest, each off by less than 2^-13 of the largest one then."""
    g = gen(41)
    T, N, K = 70, 160, 512
    xq = torch.randint(0, 256, (T, K), generator=g, device="cuda", dtype=torch.uint8)
    wq = torch.randint(0, 256, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    xq[(xq & 127) == 127] = 0x80
    wq[(wq & 127) == 127] = 0x7E
    xs, ws = torch.rand(K // 128, T, generator=g, device="cuda") + 0.1, torch.rand(2, K // 128, generator=g, device="cuda") - 0.5
    y = moe.fp8_block_dense(moe.fp8_block_prepack(wq, ws), xq, xs, dtype=dtype, flags=flags)
    x, w = ref.rows(xq, xs), ref.weights(wq, ws)
    want, err = ref.product(x, w, ref.HALF[dtype])
    if dtype == BF:
        for k in range(0, K, 8):
            top = (x[:, None, k:k + 8] * w[None, :, k:k + 8]).abs().amax(-1)
            err = err + 8 * 2.0 ** -13 * (1 + ref.HALF[BF]) * top
    within(y, want, err)


@pytest.mark.parametrize("flags", [DEC, PRE])
def test_dense_nan_stays_in_its_row(flags):
    g = gen(3)
    x = normal(g, 20, 256).to(BF)
    x[4, 200] = float("nan")
    xq, xs = moe.quant_fp8_block(x)
    wq, ws = make_weights(g, 1, 64, 256)
    y = moe.fp8_block_dense(moe.fp8_block_prepack(wq[0], ws[0]), xq, xs, flags=flags)
    bad = y.isnan()
    assert bad[4].all() and not bad[:4].any() and not bad[5:].any()


@pytest.mark.parametrize("flags", [DEC, PRE])
def test_dense_nan_weight_stays_in_its_column(flags):
    g = gen(4)
    xq, xs = make_rows(g, 20, 256)
    wq, ws = make_weights(g, 1, 64, 256)
    wq[0, 37, 140] = 0x7F
    y = moe.fp8_block_dense(moe.fp8_block_prepack(wq[0], ws[0]), xq, xs, flags=flags)
    bad = y.isnan()
    assert bad[:, 37].all() and int(bad.sum()) == 20


def test_dense_transposed_weights():
    g = gen(11)
    xq, xs = make_rows(g, 33, 512)
    wq, ws = make_weights(g, 2, 256, 384)
    for pair, K in ((False, 256), (True, 512)):
        w = (moe.fp8_block_prepack_t(wq[0], ws[0], wq[1], ws[1]) if pair else moe.fp8_block_prepack_t(wq[0], ws[0]))
        full = torch.cat([ref.weights(wq[0], ws[0]), ref.weights(wq[1], ws[1])])[:K]
        y = moe.fp8_block_dense(w, xq[:, :K].contiguous(), xs[:K // 128].contiguous(), dtype=FS)
        want, err = ref.product(ref.rows(xq, xs)[:, :K], full.T.contiguous())
        within(y, want, err)


# ---------------------------------------------------------- grouped product
# sizes of the groups (0: no rows), rows in front of and behind them
GROUPS = {"one each": ([1, 1, 1], 0, 0), "ragged": ([0, 17, 1, 0, 40, 16, 0], 0, 0), "left alone": ([5, 0, 33], 3, 4),
          "large": ([300, 0, 70, 513], 0, 9), "all in one": ([0, 0, 260], 1, 0), "none": ([0, 0], 2, 3)}


def grouping(name, k=1, seed=0):
    """offsets, the pair of each row (in a random order of X = rows / k tokens), the expert of each row or -1."""
    sizes, front, back = GROUPS[name]
    P = front + sum(sizes) + back
    P = (P + k - 1) // k * k
    off = torch.tensor([front] + sizes).cumsum(0).int().cuda()
    expert = torch.full((P,), -1)
    at = front
    for e, n in enumerate(sizes):
        expert[at:at + n] = e
        at += n
    pair = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).int().cuda()
    return off, pair, expert.cuda(), P, len(sizes)


@pytest.mark.parametrize("flags", [DEC, PRE])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("K,N,dtype", [(128, 32, FS), (640, 416, BF)])
def test_grouped(flags, gather, name, K, N, dtype):
    k = 2 if gather else 1
    off, pair, expert, P, E = grouping(name, k)
    g = gen(P + K)
    xq, xs = make_rows(g, P // k, K)
    wq, ws = make_weights(g, E, N, K)
    y = torch.full((P, N), 7.0, dtype=dtype, device="cuda")
    w = moe.fp8_block_prepack(wq, ws)
    moe.fp8_block_grouped(w, xq, xs, off, **({"rows": pair, "row_div": k} if gather else {}), flags=flags, y=y)
    x = ref.rows(xq, xs)
    if gather:
        x = x[(pair // k).long()]
    assert (y[expert < 0] == 7).all()
    for e in range(E):
        at = expert == e
        want, err = ref.product(x[at], ref.weights(wq[e], ws[e]), ref.HALF[dtype])
        within(y[at], want, err, f"expert {e}")


def many_groups(seed, E=40, most=260):
    """Ragged groups whose items are several to each workgroup: offsets, pairs (two a token), expert of each row."""
    sizes = torch.randint(0, most, (E,), generator=torch.Generator().manual_seed(seed))
    sizes[::7] = 0
    P = (int(sizes.sum()) + 5) // 2 * 2
    off = torch.cat([torch.tensor([2]), 2 + sizes.cumsum(0)]).int().cuda()
    expert = torch.full((P,), -1)
    expert[2:2 + int(sizes.sum())] = torch.repeat_interleave(torch.arange(E), sizes)
    pair = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).int().cuda()
    return off, pair, expert.cuda(), P, E


@pytest.mark.parametrize("dtype", [BF, FS])
@pytest.mark.parametrize("K", [128, 256, 384, 512, 1280])
def test_grouped_items_that_run_on_into_the_next(dtype, K):
    """Several items to a workgroup: loads of the next one under the last stages, no wait for the stores."""
    N = 2080
    off, pair, expert, P, E = many_groups(K)
    g = gen(K)
    xq, xs = make_rows(g, P // 2, K)
    wq, ws = make_weights(g, E, N, K)
    w, x = moe.fp8_block_prepack(wq, ws), ref.rows(xq, xs)
    for gather in (False, True):
        y = torch.full((P, N), 7.0, dtype=dtype, device="cuda")
        if gather:
            moe.fp8_block_grouped(w, xq, xs, off, rows=pair, row_div=2, flags=PRE, y=y)
            r = (pair // 2).long()
        else:  # the same rows in expert order
            r = (pair // 2).long()
            moe.fp8_block_grouped(w, xq[r].contiguous(), xs[:, r].contiguous(), off, flags=PRE, y=y)
        assert (y[expert < 0] == 7).all()
        for e in range(E):
            at = expert == e
            want, err = ref.product(x[r[at]], ref.weights(wq[e], ws[e]), ref.HALF[dtype])
            within(y[at], want, err, f"expert {e}, gather {gather}")


@pytest.mark.parametrize("K", [128, 256, 384, 1024])
def test_gated_items_that_run_on_into_the_next(K):
    N = 1024
    off, pair, expert, P, E = many_groups(K + 1)
    g = gen(K)
    xq, xs = make_rows(g, P // 2, K)
    (wq, ws), (uq, us) = make_weights(g, E, N, K), make_weights(g, E, N, K)
    x, r = ref.rows(xq, xs), (pair // 2).long()
    for save in (False, True):
        q, s = torch.full((P, N), 9, dtype=torch.uint8, device="cuda"), torch.full((N // 128, P), 7.0, device="cuda")
        _, _, gate, up = moe.fp8_block_glu(moe.fp8_block_prepack_glu(wq, ws, uq, us), xq, xs, off, rows=pair, row_div=2,
                                           flags=PRE, q=q, s=s, save=save)
        assert (q[expert < 0] == 9).all() and (s[:, expert < 0] == 7).all()
        for e in range(E):
            at = expert == e
            if at.any():
                (a, ea), (b, eb), (h, eh) = ref.glu(x[r[at]], ref.weights(wq[e], ws[e]), ref.weights(uq[e], us[e]))
                within(ref.rows(q[at], s[:, at]), h, ref.held(h, eh), f"expert {e}")
                if save:
                    within(gate[at], a, ea + ref.HALF[BF] * (a.abs() + ea), "gate")
                    within(up[at], b, eb + ref.HALF[BF] * (b.abs() + eb), "up")
    wq, ws = make_weights(g, E, K, N)
    gate, up = (2 * normal(g, P, N)).to(BF), normal(g, P, N).to(BF)
    xq, xs = xq[r].contiguous(), xs[:, r].contiguous()
    q, s = moe.fp8_block_glu_backward(moe.fp8_block_prepack_t(wq, ws), xq, xs, gate, up, off, flags=PRE)
    for e in range(E):
        at = expert == e
        if at.any():
            dh, adh = ref.product(ref.rows(xq, xs)[at], ref.weights(wq[e], ws[e]).T.contiguous())
            (dg, ag), (du, au) = ref.glu_grad(dh, adh, gate[at].double(), up[at].double())
            v = ref.rows(q[at], s[:, at])
            within(v[:, :N], dg, ref.held(dg, ag), f"dg, expert {e}")
            within(v[:, N:], du, ref.held(du, au), f"du, expert {e}")


def test_rows_of_y_past_32_bits():
    """Outputs of more than 2^32 elements: the first and the last rows."""
    g = gen(21)
    P, N = 270000, 16384
    xq, xs = make_rows(g, 300, 128)
    wq, ws = make_weights(g, 2, N, 128)
    w = moe.fp8_block_prepack(wq, ws)
    rows = (torch.arange(P, device="cuda", dtype=torch.int32) * 7) % 300
    off = torch.tensor([0, P - 40, P], dtype=torch.int32, device="cuda")
    x = ref.rows(xq, xs)[rows.long()]
    for flags in (DEC, PRE):
        y = moe.fp8_block_grouped(w, xq, xs, off, rows=rows, flags=flags)
        for e, a, b in ((0, 0, 300), (0, P - 300, P - 40), (1, P - 40, P)):
            want, err = ref.product(x[a:b], ref.weights(wq[e], ws[e]), ref.HALF[BF])
            within(y[a:b], want, err, f"rows {a}")
        del y


@pytest.mark.parametrize("flags", [DEC, PRE])
def test_codes_up_to_the_limit_of_32_bits(flags):
    """The last rows of as many as a call takes (T K = 2^32 - 16384), and one more refused."""
    g = gen(22)
    T, K, N = 2 ** 18 - 1, 16384, 32
    xq = torch.zeros(T, K, dtype=torch.uint8, device="cuda")
    xs = torch.ones(K // 128, T, device="cuda")
    at = torch.tensor([0, T // 2, T - 257, T - 2, T - 1], device="cuda")
    xq[at], s = make_rows(g, 5, K)
    xs[:, at] = s
    wq, ws = make_weights(g, 1, N, K)
    w = moe.fp8_block_prepack(wq, ws)
    y = moe.fp8_block_dense(w, xq, xs, flags=flags)
    want, err = ref.product(ref.rows(xq[at], s), ref.weights(wq[0], ws[0]), ref.HALF[BF])
    within(y[at], want, err)
    assert int((y != 0).any(1).sum()) == 5
    with pytest.raises(moe.MoeError):
        moe.fp8_block_dense(w, torch.cat([xq, xq[:1]]), torch.ones(K // 128, T + 1, device="cuda"), flags=flags)


def test_weight_grad_rows_past_32_bits():
    """Codes of more than 2^32 bytes: the last group's rows."""
    g = gen(23)
    P, N, K = 300000, 16384, 128
    yq = torch.zeros(P, N, dtype=torch.uint8, device="cuda")
    ys, xs = torch.ones(N // 128, P, device="cuda"), torch.ones(1, P, device="cuda")
    xq = torch.zeros(P, K, dtype=torch.uint8, device="cuda")
    yq[P - 50:], ys[:, P - 50:] = make_rows(g, 50, N)
    xq[P - 50:], xs[:, P - 50:] = make_rows(g, 50, K)
    off = torch.tensor([0, P - 50, P], dtype=torch.int32, device="cuda")
    dw = moe.fp8_block_weight_grad(yq, ys, xq, xs, off)
    s = ys[:, P - 50:].contiguous(), xs[:, P - 50:].contiguous()
    want, err = grad_bound(ref.rows(yq[P - 50:], s[0]), ref.rows(xq[P - 50:], s[1]), ref.HALF[BF])
    assert (dw[0] == 0).all()
    within(dw[1], want, err + grad_floor(*s, 50))


def test_grouped_offsets_and_rows_out_of_range_stay_inside():
    g = gen(5)
    xq, xs = make_rows(g, 40, 256)
    wq, ws = make_weights(g, 3, 64, 256)
    w = moe.fp8_block_prepack(wq, ws)
    y = torch.zeros(48, 64, device="cuda")
    off = torch.tensor([-4, 10, 1 << 30, (1 << 31) - 1], dtype=torch.int32, device="cuda")
    rows = torch.arange(40, device="cuda", dtype=torch.int32)
    rows[3], rows[20] = 1 << 30, -5
    for flags in (DEC, PRE):
        y.fill_(7)
        moe.fp8_block_grouped(w, xq, xs, off, rows=rows, flags=flags, y=y[:40])
        assert (y[40:] == 7).all()
        r = rows.long().where((rows >= 0) & (rows < 40), torch.tensor(39, device="cuda"))
        x = ref.rows(xq, xs)[r]
        for e, a, b in ((0, 0, 10), (1, 10, 40)):
            want, err = ref.product(x[a:b], ref.weights(wq[e], ws[e]))
            within(y[a:b], want, err)


# ------------------------------------------------- gated feed-forward block
@pytest.mark.parametrize("flags", [DEC, PRE])
@pytest.mark.parametrize("name", ["ragged", "left alone", "large", "none"])
@pytest.mark.parametrize("K,N,save", [(128, 128, True), (768, 384, False), (256, 640, True)])
def test_glu(flags, name, K, N, save):
    k = 2
    off, pair, expert, P, E = grouping(name, k)
    g = gen(P + N)
    xq, xs = make_rows(g, P // k, K)
    (wq, ws), (uq, us) = make_weights(g, E, N, K), make_weights(g, E, N, K)
    q, s = torch.full((P, N), 9, dtype=torch.uint8, device="cuda"), torch.full((N // 128, P), 7.0, device="cuda")
    gate, up = (torch.full((P, N), 7.0, dtype=BF, device="cuda") for _ in range(2)) if save else (None, None)
    moe.fp8_block_glu(moe.fp8_block_prepack_glu(wq, ws, uq, us), xq, xs, off, rows=pair, row_div=k, flags=flags, q=q,
                      s=s, gate=gate, up=up)
    out = expert < 0
    assert (q[out] == 9).all() and (s[:, out] == 7).all()
    x = ref.rows(xq, xs)[(pair // k).long()]
    for e in range(E):
        at = expert == e
        (a, ea), (b, eb), (h, eh) = ref.glu(x[at], ref.weights(wq[e], ws[e]), ref.weights(uq[e], us[e]))
        if at.any():
            within(ref.rows(q[at], s[:, at]), h, ref.held(h, eh), f"expert {e}")
        if save:
            within(gate[at], a, ea + ref.HALF[BF] * (a.abs() + ea), "gate")
            within(up[at], b, eb + ref.HALF[BF] * (b.abs() + eb), "up")
    if save:
        assert (gate[out] == 7).all() and (up[out] == 7).all()


@pytest.mark.parametrize("flags", [DEC, PRE])
@pytest.mark.parametrize("T", [1, 20, 300])
def test_glu_without_groups(flags, T):
    g = gen(T)
    xq, xs = make_rows(g, T, 384)
    (wq, ws), (uq, us) = make_weights(g, 1, 256, 384), make_weights(g, 1, 256, 384)
    q, s, gate, up = moe.fp8_block_glu(moe.fp8_block_prepack_glu(wq[0], ws[0], uq[0], us[0]), xq, xs, flags=flags)
    assert gate is None and up is None
    _, _, (h, eh) = ref.glu(ref.rows(xq, xs), ref.weights(wq[0], ws[0]), ref.weights(uq[0], us[0]))
    within(ref.rows(q, s), h, ref.held(h, eh))


@pytest.mark.parametrize("flags", [DEC, PRE])
def test_glu_closed_gates_and_bad_rows(flags):
    """Gates far below zero close; a NaN row is NaN, its neighbours are not."""
    g = gen(2)
    x = normal(g, 18, 128).to(BF)
    x[5, 0] = float("inf")
    xq, xs = moe.quant_fp8_block(x)
    wq = torch.full((1, 128, 128), 0x7E, dtype=torch.uint8, device="cuda")  # 448
    ws = torch.ones(1, 1, 1, device="cuda")
    uq, us = make_weights(g, 1, 128, 128)
    q, s, gate, up = moe.fp8_block_glu(moe.fp8_block_prepack_glu(wq, ws, uq, us), xq, xs, flags=flags, save=True)
    v = ref.rows(q, s)
    assert s[0, 5].isnan() and (q[5] == 0).all() and int(s.isnan().sum()) == 1
    for i in range(18):
        if i != 5 and gate[i, 0] < -100:
            assert (v[i] == 0).all()
        elif i != 5:
            assert v[i].isfinite().all()


# ------------------------------------------------------------ backward pass
@pytest.mark.parametrize("flags", [DEC, PRE])
@pytest.mark.parametrize("name", ["ragged", "left alone", "large", "none"])
@pytest.mark.parametrize("K,N", [(128, 128), (256, 384), (640, 256)])
def test_glu_backward(flags, name, K, N):
    off, _, expert, P, E = grouping(name)
    g = gen(P + K)
    yq, ys = make_rows(g, P, K)
    wq, ws = make_weights(g, E, K, N)
    gate, up = (4 * normal(g, P, N)).to(BF), normal(g, P, N).to(BF)
    q, s = torch.full((P, 2 * N), 9, dtype=torch.uint8, device="cuda"), torch.full((2 * N // 128, P), 7.0, device="cuda")
    moe.fp8_block_glu_backward(moe.fp8_block_prepack_t(wq, ws), yq, ys, gate, up, off, flags=flags, q=q, s=s)
    out = expert < 0
    assert (q[out] == 9).all() and (s[:, out] == 7).all()
    dy = ref.rows(yq, ys)
    for e in range(E):
        at = expert == e
        if not at.any():
            continue
        dh, adh = ref.product(dy[at], ref.weights(wq[e], ws[e]).T.contiguous())
        (dg, ag), (du, au) = ref.glu_grad(dh, adh, gate[at].double(), up[at].double())
        v = ref.rows(q[at], s[:, at])
        within(v[:, :N], dg, ref.held(dg, ag), f"dg, expert {e}")
        within(v[:, N:], du, ref.held(du, au), f"du, expert {e}")


@pytest.mark.parametrize("flags", [DEC, PRE])
def test_glu_backward_gates_of_all_sizes(flags):
    """Gates up to the ends of bf16, each in a block of its own.  Below -87.3 sig may be 0, which leaves out |g| e^g <
    2^-118; blocks of so small values have the least scale there is.  Past 100 the exponential's argument, whose
    rounding grows with g, no longer matters."""
    g = gen(61)
    sizes = [-3e38, -1e38, -1e30, -1e20, -1e5, -1e3, -200.0, -100.0, -88.0, -87.5, -87.0, -80.0, -20.0, -1.5, -1e-30, 0.0,
             1e-30, 2.0, 50.0, 90.0, 1e4, 1e20, 1e30]
    P, K, N = len(sizes), 128, 128
    yq, ys = make_rows(g, P, K)
    wq, ws = make_weights(g, 1, K, N)
    gate = torch.tensor(sizes, device="cuda").to(BF).unsqueeze(1).repeat(1, N)
    up = normal(g, P, N).to(BF)
    q, s = moe.fp8_block_glu_backward(moe.fp8_block_prepack_t(wq[0], ws[0]), yq, ys, gate, up, flags=flags)
    dh, adh = ref.product(ref.rows(yq, ys), ref.weights(wq[0], ws[0]).T.contiguous())
    sig, gd, ud = torch.sigmoid(gate.double()), gate.double(), up.double()
    rel = (gd.abs().clamp(max=100) + 8) * 2.0 ** -22
    slope, big, tiny = sig * (1 + gd * (1 - sig)), dh.abs() + adh, 2.0 ** -118
    bend = sig * (1 + gd.abs() * (1 - sig)) * 3 * rel + slope.abs() * 2.0 ** -21 + tiny
    dg, du = dh * ud * slope, dh * gd * sig
    v, least = ref.rows(q, s), 2.0 ** -110 / 448 * 2.0 ** -10
    within(v[:, :N], dg, ref.held(dg, adh * (ud * slope).abs() + big * ud.abs() * bend) + least, "dg")
    within(v[:, N:], du, ref.held(du, adh * (gd * sig).abs() + big * ((gd * sig).abs() * 2 * rel + tiny)) + least, "du")


def test_glu_backward_sums_alike_either_way():
    """Streamed or tiled, dh of one block of K is the same matrix instruction's sum, so that the codes are the same
    bits: for every code, and where large products cancel and leave small ones, which those sums may drop."""
    g = gen(64)
    P, K, N = 75, 128, 256
    wq = torch.randint(0, 256, (K, N), generator=g, device="cuda", dtype=torch.uint8)
    yq = torch.randint(0, 256, (P, K), generator=g, device="cuda", dtype=torch.uint8)
    wq[(wq & 127) == 127], yq[(yq & 127) == 127] = 0x7E, 0x80
    wq[1::8], yq[40:, 1::8] = wq[::8], yq[40:, ::8] ^ 0x80
    ys, ws = torch.rand(1, P, generator=g, device="cuda") + 0.1, torch.rand(1, 2, generator=g, device="cuda") + 0.1
    gate, up = (2 * normal(g, P, N)).to(BF), normal(g, P, N).to(BF)
    w = moe.fp8_block_prepack_t(wq, ws)
    a, b = (moe.fp8_block_glu_backward(w, yq, ys, gate, up, flags=f) for f in (DEC, PRE))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_glu_grad_against_differences():
    """The formula that the kernel is tested against is the derivative of silu(g) u."""
    g, u = torch.linspace(-6, 6, 49, dtype=torch.float64), torch.linspace(2, -3, 49, dtype=torch.float64)
    one = torch.ones_like(g)
    (dg, _), (du, _) = ref.glu_grad(one, 0 * one, g, u)
    f = lambda a, b: a * torch.sigmoid(a) * b  # noqa: E731
    d = 1e-5
    assert ((f(g + d, u) - f(g - d, u)) / (2 * d) - dg).abs().max() < 1e-8
    assert ((f(g, u + d) - f(g, u - d)) / (2 * d) - du).abs().max() < 1e-8


def grad_bound(y, x, half):
    """dw, and its largest error.  The scales' product is rounded to fp16 (2^-11 of it), dy's code times that again
    (2^-11; together below 2^-10 (1 + 2^-11)), behind two fp32 roundings.  Below fp16's normal numbers, 2^-14, where the
    first of them rounds to 2^-25: the largest product of scales is at least 2^4 there (its two factors lie in [1/2, 1)
    2^6 together), so that this is 2^-29 of the largest row's scales, times 448 squared at most; a row's own product then
    rounds to 2^-25 too, times a code of x of 448.  The sum of n products in fp32."""
    n = y.shape[0]
    want, mags = y.T.contiguous() @ x, y.abs().T.contiguous() @ x.abs()
    a = (2.0 ** -10 * (1 + 2.0 ** -10) + ref.gamma(n)) * mags
    return want, a + half * (want.abs() + a)


def grad_floor(ys, xs, n):
    """What the range of fp16 may cost n rows' sums: n (2^-29 448 448 + 2^-29 448) times the largest scales of the
    blocks, [N, K] (both largest ones, of any rows: at least the largest product)."""
    if n == 0:
        return 0.0
    top = ys.abs().double().amax(1).repeat_interleave(128).unsqueeze(1) * xs.abs().double().amax(1).repeat_interleave(128)
    return n * 2.0 ** -29 * (448 * 448 + 448) * top


@pytest.mark.parametrize("dtype", [BF, FS])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K", [(128, 128), (384, 256), (256, 640)])
def test_weight_grad(dtype, gather, name, N, K):
    k = 2 if gather else 1
    off, pair, expert, P, E = grouping(name, k)
    g = gen(P + N)
    yq, ys = make_rows(g, P, N)
    xq, xs = make_rows(g, P // k, K)
    dw = moe.fp8_block_weight_grad(yq, ys, xq, xs, off, **({"rows": pair, "row_div": k} if gather else {}), dtype=dtype)
    y, x = ref.rows(yq, ys), ref.rows(xq, xs)
    if gather:
        x = x[(pair // k).long()]
    for e in range(E):
        at = expert == e
        want, err = grad_bound(y[at], x[at], ref.HALF[dtype])
        within(dw[e], want, err + grad_floor(ys, xs, int(at.sum())) + 1e-300, f"expert {e}")


@pytest.mark.parametrize("T", [0, 1, 33, 700, 2100])
@pytest.mark.parametrize("dtype", [BF, FS])
def test_weight_grad_of_one_group(T, dtype):
    """Few tiles: the rows are split and their sums joined."""
    g = gen(T)
    yq, ys = make_rows(g, T, 256)
    xq, xs = make_rows(g, T, 128)
    dw = moe.fp8_block_weight_grad(yq, ys, xq, xs, dtype=dtype)
    want, err = grad_bound(ref.rows(yq, ys), ref.rows(xq, xs), ref.HALF[dtype])
    assert dw.shape == (256, 128)
    within(dw, want, err + grad_floor(ys, xs, T) + 1e-300)
    assert torch.equal(dw, moe.fp8_block_weight_grad(yq, ys, xq, xs, dtype=dtype))


@pytest.mark.parametrize("parts", [False, True])
def test_weight_grad_scales_of_all_sizes(parts):
    """Rows whose scales lie up to 2^-60 apart, and the range of fp32 itself."""
    g = gen(31)
    P, N, K = (3000, 128, 256) if parts else (400, 256, 384)
    (yq, ys), (xq, xs) = make_rows(g, P, N), make_rows(g, P, K)
    for low, high in ((-30, 0), (-8, 0), (0, 40), (-100, -90)):
        y2 = ys * torch.exp2(torch.randint(low, high, ys.shape, generator=g, device="cuda").float())
        x2 = xs * torch.exp2(torch.randint(-20, 20, xs.shape, generator=g, device="cuda").float())
        dw = moe.fp8_block_weight_grad(yq, y2, xq, x2, dtype=FS)
        want, err = grad_bound(ref.rows(yq, y2), ref.rows(xq, x2), ref.HALF[FS])
        within(dw, want, err + grad_floor(y2, x2, P) + 2.0 ** -149, f"{low} {high}")


def row_floor(ys, xs):
    """What the range of fp16 may cost the rows' sums, [N, K]: n (2^-29 448 448 + 2^-29 448) times the largest product of
    one row's scales."""
    top = (ys.abs().double().unsqueeze(1) * xs.abs().double().unsqueeze(0)).amax(-1)
    return ys.shape[1] * 2.0 ** -29 * (448 * 448 + 448) * top.repeat_interleave(128, 0).repeat_interleave(128, 1)


@pytest.mark.parametrize("P", [60, 1500])
@pytest.mark.parametrize("gather", [False, True])
def test_weight_grad_outliers_in_different_rows(P, gather):
    """A row of large gradients and another of large activations, whose codes are zero in half of the channels, leave
    the other rows' bits alone: no row's scales are both large."""
    g = gen(62)
    for e in (0, 6, 12, 16, 20, 40):
        y, x = normal(g, P, 384), normal(g, P, 256)
        for n in range(0, 384, 128):
            y[3, n:n + 64] = 0
        for n in range(0, 256, 128):
            x[5, n:n + 64] = 0
        y[3] *= 2.0 ** e
        x[5] *= 2.0 ** e
        (yq, ys), (xq, xs) = moe.quant_fp8_block(y), moe.quant_fp8_block(x)
        v = ref.rows(xq, xs)
        off = torch.tensor([0, P], dtype=torch.int32, device="cuda")
        if gather:  # an odd row of x stands for two neighbouring rows of dy
            rows = torch.arange(P, device="cuda", dtype=torch.int32) // 2 * 2 + 1
            dw = moe.fp8_block_weight_grad(yq, ys, xq, xs, off, rows=rows, dtype=FS)[0]
            v, xs = v[rows.long()], xs[:, rows.long()]
        else:
            dw = moe.fp8_block_weight_grad(yq, ys, xq, xs, off, dtype=FS)[0]
        want, err = grad_bound(ref.rows(yq, ys), v, ref.HALF[FS])
        within(dw, want, err + row_floor(ys, xs), f"2^{e}")


def test_weight_grad_scales_at_the_ends_of_fp32():
    """One scale near 2^127 beside one near 2^-126 in a row, zeros, and scales below the normal numbers."""
    g = gen(63)
    P = 64
    (yq, _), (xq, _) = make_rows(g, P, 128), make_rows(g, P, 128)
    e = torch.linspace(-126, 126, P, device="cuda")
    for lift in (0.0, -20.0, 20.0):
        ys, xs = torch.exp2(e).unsqueeze(0), torch.exp2((lift - e).clamp(-126, 127)).unsqueeze(0)
        xs[0, 7], ys[0, 50] = 0.0, 0.0
        want, err = grad_bound(ref.rows(yq, ys), ref.rows(xq, xs), ref.HALF[FS])
        within(moe.fp8_block_weight_grad(yq, ys, xq, xs, dtype=FS), want, err + row_floor(ys, xs), f"lift {lift}")
    ys, xs = torch.full((1, P), 2.0 ** -135, device="cuda"), torch.full((1, P), 2.0 ** 100, device="cuda")
    want, err = grad_bound(ref.rows(yq, ys), ref.rows(xq, xs), ref.HALF[FS])
    within(moe.fp8_block_weight_grad(yq, ys, xq, xs, dtype=FS), want, err + row_floor(ys, xs), "subnormal")


def test_weight_grad_all_codes():
    """Every code of e4m3, and the not-a-numbers where they belong: a row of dw and a column of it."""
    g = gen(32)
    P, N, K = 130, 256, 128
    yq = torch.randint(0, 256, (P, N), generator=g, device="cuda", dtype=torch.uint8)
    xq = torch.randint(0, 256, (P, K), generator=g, device="cuda", dtype=torch.uint8)
    yq[(yq & 127) == 127] = 1
    xq[(xq & 127) == 127] = 0x81
    ys, xs = torch.rand(N // 128, P, generator=g, device="cuda") + 0.5, torch.rand(K // 128, P, generator=g, device="cuda")
    want, err = grad_bound(ref.rows(yq, ys), ref.rows(xq, xs), ref.HALF[BF])
    within(moe.fp8_block_weight_grad(yq, ys, xq, xs), want, err + grad_floor(ys, xs, P))
    yq[7, 33], xq[129, 100] = 0x7F, 0xFF
    dw = moe.fp8_block_weight_grad(yq, ys, xq, xs)
    bad = torch.zeros(N, K, dtype=torch.bool, device="cuda")
    bad[33], bad[:, 100] = True, True
    assert torch.equal(dw.isnan(), bad)
    within(dw[~bad], want[~bad], (err + grad_floor(ys, xs, P))[~bad])


def test_weight_grad_nan_row_stays_in_its_group():
    off, _, expert, P, E = grouping("ragged")
    g = gen(1)
    x = normal(g, P, 128)
    x[int(off[4]), 3] = float("nan")
    yq, ys = make_rows(g, P, 128)
    dw = moe.fp8_block_weight_grad(yq, ys, *moe.quant_fp8_block(x), off)
    assert dw[4].isnan().any() and not dw[:4].isnan().any() and not dw[5:].isnan().any()


# ------------------------------------------------------------- as it is used
def feed_forward(w, x, do, off, pair, k, flags=0):
    """One expert layer's forward and backward pass as a program makes them."""
    xq, xs = moe.quant_fp8_block(x)
    hq, hs, gate, up = moe.fp8_block_glu(w["w13"], xq, xs, off, rows=pair, row_div=k, save=True, flags=flags)
    o = moe.fp8_block_grouped(w["w2"], hq, hs, off, flags=flags)
    dq, ds = moe.quant_fp8_block(do)
    gq, gs = moe.fp8_block_glu_backward(w["w2_t"], dq, ds, gate, up, off, flags=flags)
    dx = moe.fp8_block_grouped(w["w13_t"], gq, gs, off, dtype=FS, flags=flags)
    dw2 = moe.fp8_block_weight_grad(dq, ds, hq, hs, off)
    dw13 = moe.fp8_block_weight_grad(gq, gs, xq, xs, off, rows=pair, row_div=k)
    return o, dx, dw2, dw13


def training_case(T=70, k=2, E=5, H=256, I=128, seed=0):
    g = gen(seed)
    x = normal(g, T, H).to(BF)
    ids, _ = moe.route_topk(normal(g, T, E), k)
    _, off, pair, pos = moe.sort_permute(ids, E)
    m = {n: make_weights(g, E, *s) for n, s in (("w1", (I, H)), ("w3", (I, H)), ("w2", (H, I)))}
    w = {"w13": moe.fp8_block_prepack_glu(*m["w1"], *m["w3"]), "w2": moe.fp8_block_prepack(*m["w2"]),
         "w2_t": moe.fp8_block_prepack_t(*m["w2"]), "w13_t": moe.fp8_block_prepack_t(*m["w1"], *m["w3"])}
    return w, m, x, normal(g, T * k, H).to(BF), off, pair, k, E


@pytest.mark.parametrize("T", [3, 70, 400])
def test_forward_and_backward_chain(T):
    """The chain's results against the unquantised layer's in 64 bits: what e4m3 rounds (a step of 2^-4 relative at
    most, 2^-5 on average of a binade's values) enters twice in each result's factors, so norms agree to a tenth."""
    w, m, x, do, off, pair, k, E = training_case(T)
    got = feed_forward(w, x, do, off, pair, k)
    v = {n: ref.weights(*m[n]).requires_grad_() for n in m}
    xd = x.double()[(pair // k).long()].requires_grad_()
    parts = []
    for e in range(E):
        a = xd[int(off[e]):int(off[e + 1])]
        gate = a @ v["w1"][e].T
        parts.append((gate * torch.sigmoid(gate) * (a @ v["w3"][e].T)) @ v["w2"][e].T)
    o = torch.cat(parts)
    o.backward(do.double())
    want = (o.detach(), xd.grad, v["w2"].grad, torch.cat([v["w1"].grad, v["w3"].grad], 1))
    for a, b, what in zip(got, want, ("o", "dx", "dw2", "dw13")):
        assert (a.double() - b).norm() < 0.1 * b.norm(), what


@pytest.mark.parametrize("flags", [DEC, PRE])
def test_chain_in_a_graph_and_on_another_stream(flags):
    w, m, x, do, off, pair, k, E = training_case()
    want = feed_forward(w, x, do, off, pair, k, flags)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        again = feed_forward(w, x, do, off, pair, k, flags)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    graph = torch.cuda.CUDAGraph()
    xs, dos = x.clone(), do.clone()
    with torch.cuda.graph(graph):
        out = feed_forward(w, xs, dos, off, pair, k, flags)
    for i in range(3):
        xs.copy_(x * (i + 1))
        dos.copy_(do * 0.5 ** i)
        graph.replay()
        eager = feed_forward(w, xs, dos, off, pair, k, flags)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i


@pytest.mark.parametrize("flags", [DEC, PRE])
def test_two_calls_and_two_graphs_at_once(flags):
    """On two streams, each with outputs and workspaces of its own; then both captured, and replayed side by side."""
    cases = [training_case(T=90, seed=1), training_case(T=70, seed=2)]
    run = [lambda c=c: feed_forward(c[0], c[2], c[3], c[4], c[5], c[6], flags) for c in cases]
    want = [f() for f in run]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(run[i]())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for out in got[i] for a, b in zip(out, want[i]))
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], [None, None]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            outs[i] = run[i]()
    for _ in range(3):
        for i in range(2):
            for t in outs[i]:
                t.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))


def test_decode_step_beside_the_fp4_layer():
    """A token's row through the experts and the combine, as the FP4 layer's stages are chained."""
    g = gen(9)
    T, k, E, H, I = 4, 2, 6, 256, 256
    x = normal(g, T, H).to(BF)
    ids, gates = moe.route_topk(normal(g, T, E), k)
    _, off, pair, pos = moe.sort_permute(ids, E)
    m = {n: make_weights(g, E, *s) for n, s in (("w1", (I, H)), ("w3", (I, H)), ("w2", (H, I)))}
    xq, xs = moe.quant_fp8_block(x)
    hq, hs, _, _ = moe.fp8_block_glu(moe.fp8_block_prepack_glu(*m["w1"], *m["w3"]), xq, xs, off, rows=pair, row_div=k)
    o = moe.fp8_block_grouped(moe.fp8_block_prepack(*m["w2"]), hq, hs, off)
    y = moe.combine(o, gates, pos, T, k, H)
    xv = ref.rows(xq, xs)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            _, _, (h, _) = ref.glu(xv[t:t + 1], ref.weights(m["w1"][0][e], m["w1"][1][e]),
                                   ref.weights(m["w3"][0][e], m["w3"][1][e]))
            want[t] += float(gates[t, j]) * (ref.weights(m["w2"][0][e], m["w2"][1][e]) @ h[0])
    # h is off by half an e4m3 step (2^-4) at most, o by half a bf16 step
    assert (y.double() - want).norm() < (2.0 ** -4 + 2.0 ** -8) * want.norm()


def test_one_workspace_for_a_large_batch_and_smaller_ones():
    """The size for rows that take the tiled product serves fewer rows, which are streamed through it."""
    g = gen(12)
    E, N, K = 8, 512, 256
    large = 2400
    w13 = moe.fp8_block_prepack_glu(*make_weights(g, E, N, K), *make_weights(g, E, N, K))
    w2_t = moe.fp8_block_prepack_t(*make_weights(g, E, K, N))
    ws = torch.empty(moe.fp8_block_glu_workspace_size(large, E, N, K), dtype=torch.uint8, device="cuda")
    for P in (large, 2309, 2200, 700, 40, 1):
        off = torch.linspace(0, P, E + 1, device="cuda").int()
        xq, xs = make_rows(g, P, K)
        got = moe.fp8_block_glu(w13, xq, xs, off, save=True, workspace=ws)
        want = moe.fp8_block_glu(w13, xq, xs, off, save=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), P
        back = moe.fp8_block_glu_backward(w2_t, xq, xs, *got[2:], off, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(back, moe.fp8_block_glu_backward(w2_t, xq, xs, *got[2:], off))), P


# -------------------------------------------- forms that only larger sizes take
def tall_groups(low, high, seed, E=128):
    """Ragged groups of low to high rows, every ninth empty: offsets, pairs (two a token), expert of each row."""
    gc = torch.Generator().manual_seed(seed)
    sizes = torch.randint(low, high + 1, (E,), generator=gc)
    sizes[4::9] = 0
    P = (int(sizes.sum()) + 7) // 2 * 2
    off = torch.cat([torch.tensor([3]), 3 + sizes.cumsum(0)]).int().cuda()
    expert = torch.full((P,), -1)
    expert[3:3 + int(sizes.sum())] = torch.repeat_interleave(torch.arange(E), sizes)
    return off, torch.randperm(P, generator=gc).int().cuda(), expert.cuda(), P, E


def tile_rows(workspace):
    """Rows of the tiles that the tiled product listed in its workspace."""
    w = workspace.view(torch.int32)
    return w[4:4 + 4 * int(w[0])].view(-1, 4)[:, 2]


# rows of a group, and the heights of tile that they are to be cut to (three and four token tiles a wave)
TALL = {"three": (110, 190, 129, 192), "four": (200, 256, 193, 256), "four, several tiles": (150, 700, 193, 256)}


def assert_tall(workspace, name):
    top = int(tile_rows(workspace).max())
    assert TALL[name][2] <= top <= TALL[name][3], top


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K", [128, 256, 384, 1152])
@pytest.mark.parametrize("name", list(TALL))
def test_grouped_tall_tiles(name, K, gather):
    N = 1056
    off, pair, expert, P, E = tall_groups(*TALL[name][:2], seed=K)
    g = gen(K + 5)
    xq, xs = make_rows(g, P // 2 if gather else P, K)
    wq, ws = make_weights(g, E, N, K)
    ws_ = torch.empty(moe.fp8_block_grouped_workspace_size(P, E, N, K), dtype=torch.uint8, device="cuda")
    y = torch.full((P, N), 7.0, dtype=BF, device="cuda")
    moe.fp8_block_grouped(moe.fp8_block_prepack(wq, ws), xq, xs, off, **({"rows": pair, "row_div": 2} if gather else {}),
                          flags=PRE, y=y, workspace=ws_)
    assert_tall(ws_, name)
    x = ref.rows(xq, xs)
    x = x[(pair // 2).long()] if gather else x
    assert (y[expert < 0] == 7).all()
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        want, err = ref.product(x[a:b], ref.weights(wq[e], ws[e]), ref.HALF[BF])
        within(y[a:b], want, err, f"expert {e}")


@pytest.mark.parametrize("T", [2300, 3000])
def test_dense_tall_tiles(T):
    """Three and four token tiles a wave of one group (256 CUs: heights of 192 and 256 rows are the fewest rounds)."""
    K, N = 384, 4096 + 96
    g = gen(T)
    xq, xs = make_rows(g, T, K)
    wq, ws = make_weights(g, 1, N, K)
    y = moe.fp8_block_dense(moe.fp8_block_prepack(wq[0], ws[0]), xq, xs, flags=PRE)
    want, err = ref.product(ref.rows(xq, xs), ref.weights(wq[0], ws[0]), ref.HALF[BF])
    within(y, want, err)


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("K", [128, 256, 384, 1152])
@pytest.mark.parametrize("name", list(TALL))
def test_gated_tall_tiles(name, K, save):
    N = 512
    off, pair, expert, P, E = tall_groups(*TALL[name][:2], seed=K + 1)
    g = gen(K + 6)
    xq, xs = make_rows(g, P // 2, K)
    (wq, ws), (uq, us) = make_weights(g, E, N, K), make_weights(g, E, N, K)
    x = ref.rows(xq, xs)[(pair // 2).long()]
    q, s = torch.full((P, N), 9, dtype=torch.uint8, device="cuda"), torch.full((N // 128, P), 7.0, device="cuda")
    room = torch.empty(moe.fp8_block_glu_workspace_size(P, E, N, K, PRE), dtype=torch.uint8, device="cuda")
    gate, up = (torch.full((P, N), 7.0, dtype=BF, device="cuda") for _ in range(2)) if save else (None, None)
    moe.fp8_block_glu(moe.fp8_block_prepack_glu(wq, ws, uq, us), xq, xs, off, rows=pair, row_div=2, flags=PRE, q=q, s=s,
                      gate=gate, up=up, workspace=room)
    assert_tall(room, name)
    out = expert < 0
    assert (q[out] == 9).all() and (s[:, out] == 7).all()
    assert not save or ((gate[out] == 7).all() and (up[out] == 7).all())
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a < b:
            (vg, eg), (vu, eu), (h, eh) = ref.glu(x[a:b], ref.weights(wq[e], ws[e]), ref.weights(uq[e], us[e]))
            within(ref.rows(q[a:b], s[:, a:b]), h, ref.held(h, eh), f"expert {e}")
            if save:
                within(gate[a:b], vg, eg + ref.HALF[BF] * (vg.abs() + eg), "gate")
                within(up[a:b], vu, eu + ref.HALF[BF] * (vu.abs() + eu), "up")


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K", [128, 256, 384, 1152])
@pytest.mark.parametrize("name", list(TALL))
def test_glu_backward_tall_tiles(name, K, gather):
    N = 896
    off, pair, expert, P, E = tall_groups(*TALL[name][:2], seed=K + 2)
    g = gen(K + 7)
    yq, ys = make_rows(g, P // 2 if gather else P, K)
    wq, ws = make_weights(g, E, K, N)
    gate, up = (2 * normal(g, P, N)).to(BF), normal(g, P, N).to(BF)
    q, s = torch.full((P, 2 * N), 9, dtype=torch.uint8, device="cuda"), torch.full((2 * N // 128, P), 7.0, device="cuda")
    room = torch.empty(moe.fp8_block_glu_workspace_size(P, E, N, K, PRE), dtype=torch.uint8, device="cuda")
    moe.fp8_block_glu_backward(moe.fp8_block_prepack_t(wq, ws), yq, ys, gate, up, off,
                               **({"rows": pair, "row_div": 2} if gather else {}), flags=PRE, q=q, s=s, workspace=room)
    assert_tall(room, name)
    out = expert < 0
    assert (q[out] == 9).all() and (s[:, out] == 7).all()
    dy = ref.rows(yq, ys)
    dy = dy[(pair // 2).long()] if gather else dy
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a < b:
            dh, adh = ref.product(dy[a:b], ref.weights(wq[e], ws[e]).T.contiguous())
            (dg, ag), (du, au) = ref.glu_grad(dh, adh, gate[a:b].double(), up[a:b].double())
            v = ref.rows(q[a:b], s[:, a:b])
            within(v[:, :N], dg, ref.held(dg, ag), f"dg, expert {e}")
            within(v[:, N:], du, ref.held(du, au), f"du, expert {e}")


@pytest.mark.parametrize("dtype", [BF, FS])
@pytest.mark.parametrize("K", [2176, 8192])
@pytest.mark.parametrize("T", [1, 8, 16])
def test_dense_few_rows_of_many_tiles(T, K, dtype):
    """More weight tiles than CUs and several K-steps in flight, with and without a remainder of them."""
    N = 4128
    g = gen(T + K)
    xq, xs = make_rows(g, T, K)
    wq, ws = make_weights(g, 1, N, K)
    w = moe.fp8_block_prepack(wq[0], ws[0])
    want, err = ref.product(ref.rows(xq, xs), ref.weights(wq[0], ws[0]), ref.HALF[dtype])
    for flags in (0, DEC):
        within(moe.fp8_block_dense(w, xq, xs, flags=flags, dtype=dtype), want, err)


@pytest.mark.parametrize("flags", [0, DEC])
def test_dense_fp32_of_a_few_hundred_rows(flags):
    g = gen(333)
    xq, xs = make_rows(g, 333, 4096)
    wq, ws = make_weights(g, 1, 1536, 4096)
    y = moe.fp8_block_dense(moe.fp8_block_prepack(wq[0], ws[0]), xq, xs, flags=flags, dtype=FS)
    within(y, *ref.product(ref.rows(xq, xs), ref.weights(wq[0], ws[0])))


@pytest.mark.parametrize("sizes", [[1, 0, 16, 7, 9, 2, 16, 16], [40, 0, 31, 17, 33, 64, 1, 25]])
def test_streamed_groups_of_many_tiles(sizes):
    """The products, the gated block and its backward pass: few rows a group and 16 of them or more on average, with
    more weight tiles than CUs and several K-steps to a wave."""
    E, P = len(sizes), sum(sizes)
    K, N = 2176, 1152
    g = gen(P)
    off = torch.tensor([0] + sizes).cumsum(0).int().cuda()
    xq, xs = make_rows(g, P, K)
    (wq, ws), (uq, us) = make_weights(g, E, N, K), make_weights(g, E, N, K)
    tq, ts = make_weights(g, E, K, N)
    gate, up = (2 * normal(g, P, N)).to(BF), normal(g, P, N).to(BF)
    w = moe.fp8_block_prepack(wq, ws)
    sums = {t: moe.fp8_block_grouped(w, xq, xs, off, flags=DEC, dtype=t) for t in (BF, FS)}
    hq, hs, hg, hu = moe.fp8_block_glu(moe.fp8_block_prepack_glu(wq, ws, uq, us), xq, xs, off, flags=DEC, save=True)
    q, s = moe.fp8_block_glu_backward(moe.fp8_block_prepack_t(tq, ts), xq, xs, gate, up, off, flags=DEC)
    x = ref.rows(xq, xs)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a == b:
            continue
        (vg, eg), (vu, eu), (h, eh) = ref.glu(x[a:b], ref.weights(wq[e], ws[e]), ref.weights(uq[e], us[e]))
        for t, y in sums.items():
            within(y[a:b], vg, eg + ref.HALF[t] * (vg.abs() + eg), f"{t}, expert {e}")
        within(ref.rows(hq[a:b], hs[:, a:b]), h, ref.held(h, eh), f"h, expert {e}")
        within(hg[a:b], vg, eg + ref.HALF[BF] * (vg.abs() + eg), "gate")
        within(hu[a:b], vu, eu + ref.HALF[BF] * (vu.abs() + eu), "up")
        dh, adh = ref.product(x[a:b], ref.weights(tq[e], ts[e]).T.contiguous())
        (dg, ag), (du, au) = ref.glu_grad(dh, adh, gate[a:b].double(), up[a:b].double())
        v = ref.rows(q[a:b], s[:, a:b])
        within(v[:, :N], dg, ref.held(dg, ag), f"dg, expert {e}")
        within(v[:, N:], du, ref.held(du, au), f"du, expert {e}")


@pytest.mark.parametrize("dtype", [BF, FS])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(640, 2176), (384, 4480), (2304, 2048)])
def test_weight_grad_of_several_panels(N, K, gather, dtype):
    """More than eight tiles of columns of x: a narrow last panel, half tiles, tile counts that eight does not divide."""
    sizes = [70, 0, 33, 1]
    off = torch.tensor([2] + [2 + sum(sizes[:i + 1]) for i in range(4)], dtype=torch.int32, device="cuda")
    P = 110
    g = gen(N + K)
    yq, ys = make_rows(g, P, N)
    xq, xs = make_rows(g, P // 2 if gather else P, K)
    pair = torch.randperm(P, generator=torch.Generator().manual_seed(1)).int().cuda()
    dw = moe.fp8_block_weight_grad(yq, ys, xq, xs, off, **({"rows": pair, "row_div": 2} if gather else {}), dtype=dtype)
    y, x = ref.rows(yq, ys), ref.rows(xq, xs)
    if gather:
        x, xs = x[(pair // 2).long()], xs[:, (pair // 2).long()]
    for e in range(4):
        a, b = int(off[e]), int(off[e + 1])
        if a == b:
            assert (dw[e] == 0).all()
            continue
        want, err = grad_bound(y[a:b], x[a:b], ref.HALF[dtype])
        within(dw[e], want, err + row_floor(ys[:, a:b], xs[:, a:b]), f"expert {e}")


@pytest.mark.parametrize("flags", [0, DEC, PRE])
@pytest.mark.parametrize("T,K,N", [(1, 256, 256), (20, 384, 640), (33, 2176, 128), (128, 256, 4096), (300, 128, 384)])
def test_glu_backward_without_groups(flags, T, K, N):
    """One group, as a shared expert has; 128 rows of 256 weight tiles are streamed 64 rows a pass."""
    g = gen(T + K)
    yq, ys = make_rows(g, T, K)
    wq, ws = make_weights(g, 1, K, N)
    gate, up = (2 * normal(g, T, N)).to(BF), normal(g, T, N).to(BF)
    q, s = moe.fp8_block_glu_backward(moe.fp8_block_prepack_t(wq[0], ws[0]), yq, ys, gate, up, flags=flags)
    dh, adh = ref.product(ref.rows(yq, ys), ref.weights(wq[0], ws[0]).T.contiguous())
    (dg, ag), (du, au) = ref.glu_grad(dh, adh, gate.double(), up.double())
    v = ref.rows(q, s)
    within(v[:, :N], dg, ref.held(dg, ag), "dg")
    within(v[:, N:], du, ref.held(du, au), "du")
