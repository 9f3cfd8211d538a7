"""The residual RMS norm, 8-bit matrices and their product on the GPU against fp64
references.

Roundings counted: bf16 2^-8 of the value, e4m3 2^-4 (half a step of 448 / 2^18 =
2^-10 among its subnormal values), fp32 2^-24."""
import numpy as np
import pytest
import torch

import gated_delta_rule_124_b200 as kda
from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(seed, *shape, dtype="f32", scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(DT[dtype])


def check_codes(y8, scale, want, block_rows, rel=0.0):
    """Codes and scales of an 8-bit matrix of `want` (fp64), itself known to the
    relative error `rel` (per value and per block maximum): the scale is within
    that and two fp32 roundings, a dequantised value within half a step of e4m3
    (and the relative errors of value and factor, which cannot add more than
    their own size), the padding zero."""
    R, K = want.shape
    codes = f64(y8)
    assert codes.shape == (R, kda.kda_fp8_pitch(K)) and not codes[:, K:].any()
    amax = np.maximum(ofp8.block_max(want, block_rows), ofp8.AMAX_FLOOR)
    s = f64(scale)
    assert s.shape == amax.shape
    assert (np.abs(s - amax / 448) <= (rel + 2 * U) * amax / 448).all()
    back = ofp8.dequantize(codes[:, :K], s, block_rows)
    # half a step at the value, or at the smallest normal number 2^-6
    exact = np.abs(want) / ofp8.spread(amax / 448, block_rows, R, K)
    step = np.maximum(exact, 2.0 ** -6) * 2.0 ** -4
    tol = step * ofp8.spread(s, block_rows, R, K) + (2 * rel + 8 * U) * np.abs(want)
    assert (np.abs(back - want) <= tol).all()


# ------------------------------------------------------------------ the norm

SIZES = [(1, 8), (3, 64), (5, 136), (2, 512), (7, 520), (9, 1000), (130, 1024), (33, 2048),
         (16, 2056), (301, 4096), (6, 4104), (4, 8192), (3, 12288), (2, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", SIZES)
def test_norm_matches_the_definition(rows, D, dtype):
    x, r = randn(1, rows, D, dtype=dtype), randn(2, rows, D, dtype=dtype, scale=4.0)
    w = 1 + randn(3, D, scale=0.1)
    s, y = kda.add_rms_norm(x.cuda(), w.cuda(), r.cuda(), eps=EPS)
    total = f64(x) + f64(r)
    assert (np.abs(f64(s) - total) <= HALF[dtype] * np.abs(total)).all()
    # the sum of D squares in fp32: at most D / 256 + 24 additions in a row, half
    # of that in the root; three more roundings
    rel = ((D / 256 + 24) / 2 + 6) * U
    want = ofp8.rms_norm(f64(s), f64(w), EPS)
    assert (np.abs(f64(y) - want) <= (rel + HALF[dtype] * (1 + rel)) * np.abs(want)).all()
    s2, y8, scale = kda.add_rms_norm(x.cuda(), w.cuda(), r.cuda(), eps=EPS, quantize=True)
    assert torch.equal(s, s2)
    check_codes(y8, scale, want, 1, rel)
    # without a residual, s is x itself
    x3, y3 = kda.add_rms_norm(s, w.cuda(), eps=EPS)
    assert x3 is s and torch.equal(y3, y)


def test_norm_writes_the_sum_in_place_and_both_outputs():
    rows, D = 37, 1032
    x, r, w = randn(4, rows, D, dtype="bf16").cuda(), randn(5, rows, D, dtype="bf16").cuda(), \
        torch.ones(D, device="cuda")
    s, y = kda.add_rms_norm(x, w, r)
    _, y8, scale = kda.add_rms_norm(x, w, r, quantize=True)
    for target in (x.clone(), r.clone()):
        xs, rs = (target, r) if torch.equal(target, x) else (x, target)
        yb, y8b, scb = torch.empty_like(y), torch.empty_like(y8), torch.empty_like(scale)
        kda.kda_add_rms_norm(xs, rs, w, rows, D, "bf16", 1e-6, target, yb, y8b, scb)
        assert torch.equal(target, s) and torch.equal(yb, y)
        assert torch.equal(y8b.view(torch.uint8), y8.view(torch.uint8)) and torch.equal(scb, scale)
    for pick in (0, 1):
        xs, rs = x.clone(), r.clone()
        target = (xs, rs)[pick]
        got, yb = kda.add_rms_norm(xs, w, rs, sum=target)
        assert got is target and torch.equal(target, s) and torch.equal(yb, y)
    both, twice = kda.add_rms_norm(x, w, x)      # the same tensor twice
    assert torch.equal(both, x + x)


def test_padding_behind_a_row_of_nan_is_zero():
    x = torch.full((2, 24), float("nan"), device="cuda")
    x[1] = 1.0
    _, y8, _ = kda.add_rms_norm(x, torch.ones(24, device="cuda"), quantize=True)
    assert y8.shape == (2, 32) and not y8.view(torch.uint8)[:, 24:].any()
    assert (y8.view(torch.uint8)[:, :24] & 0x7F)[0].eq(0x7F).all()


def test_norm_of_zero_rows_large_values_and_nan():
    D = 256
    x = torch.zeros(5, D)
    x[1] = 1e15                       # squares near 1e30
    x[2] = torch.arange(D) * 1e-30    # far below eps
    x[3, 7] = float("nan")
    x[4] = 1.0
    w = torch.ones(D)
    s, y8, scale = kda.add_rms_norm(x.cuda(), w.cuda(), quantize=True)
    _, y = kda.add_rms_norm(x.cuda(), w.cuda())
    assert not y[0].any() and not f64(y8)[0].any() and (scale[:, 0] > 0).all()
    assert torch.allclose(y[1].cpu(), torch.ones(D), atol=1e-6)
    want = ofp8.rms_norm(f64(x[2:3]), f64(w), 1e-6)
    assert np.allclose(f64(y[2:3]), want, rtol=1e-6, atol=0)
    assert torch.isnan(y[3]).all() and torch.isnan(y8[3].float()).all()
    assert torch.equal(y[4], torch.full_like(y[4], float(y[4, 0])))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(1, 8), (5, 136), (600, 512), (1300, 1000), (33, 2048),
                                    (700, 4096), (4, 8192), (3, 16384), (0, 64)])
def test_norm_backward_matches_the_formula(rows, D, dtype):
    s, dy = randn(6, rows, D, dtype=dtype, scale=3.0), randn(7, rows, D, dtype=dtype)
    ds, w = randn(8, rows, D, dtype=dtype), 1 + randn(9, D, scale=0.1)
    S, W, DY, DS = s.cuda(), w.cuda(), dy.cuda(), ds.cuda()
    for dsum in (DS, None):
        dx, dw = kda.add_rms_norm_bwd(S, W, DY, dsum, eps=EPS)
        rx, rw = ofp8.rms_norm_bwd(f64(s), f64(w), f64(dy), None if dsum is None else f64(ds), EPS)
        if rows == 0:
            assert dx.shape == (0, D) and not dw.any()
            continue
        # terms of dx: r w dy, r^3 s mean(s w dy) (bounded by r |s| r rms |w dy|), dsum
        r = 1 / np.sqrt((f64(s) ** 2).mean(-1, keepdims=True) + EPS)
        wdy = np.abs(f64(w) * f64(dy))
        mag = r * wdy + r * np.abs(f64(s)) * r * np.sqrt((wdy ** 2).mean(-1, keepdims=True))
        rel = (1.5 * (D / 256 + 24) + 10) * U
        tol = rel * mag + HALF[dtype] * (np.abs(rx) + rel * mag) + 2 * U * np.abs(rx)
        assert (np.abs(f64(dx) - rx) <= tol).all()
        terms = np.abs(f64(dy) * f64(s) * r).sum(0)
        # at most rows / 4 + 80 additions in a row
        assert (np.abs(f64(dw) - rw) <= (rows / 4 + 80 + rel / U) * U * terms).all()


def test_norm_backward_into_the_sums_gradient():
    rows, D = 700, 520
    s, dy = randn(60, rows, D, dtype="bf16").cuda(), randn(61, rows, D, dtype="bf16").cuda()
    ds, w = randn(62, rows, D, dtype="bf16").cuda(), (1 + randn(63, D, scale=0.1)).cuda()
    want_dx, want_dw = kda.add_rms_norm_bwd(s, w, dy, ds)
    dw = torch.empty_like(w)
    ws = torch.empty(kda.kda_add_rms_norm_bwd_workspace_size(rows, D), dtype=torch.uint8,
                     device="cuda")
    kda.kda_add_rms_norm_bwd(s, w, dy, ds, rows, D, "bf16", 1e-6, ds, dw, ws)
    assert torch.equal(ds, want_dx) and torch.equal(dw, want_dw)


def test_norm_backward_is_the_difference_quotient():
    rows, D, h = 3, 40, 1e-5
    s, dy, ds = f64(randn(10, rows, D)), f64(randn(11, rows, D)), f64(randn(12, rows, D))
    w = 1 + 0.1 * f64(randn(13, D))
    dx, dw = (f64(t) for t in kda.add_rms_norm_bwd(*(torch.tensor(v, dtype=torch.float32).cuda()
                                                     for v in (s, w, dy, ds)), eps=EPS))
    loss = lambda s_, w_: (ofp8.rms_norm(s_, w_, EPS) * dy).sum() + (s_ * ds).sum()  # noqa: E731
    rng = np.random.default_rng(0)
    for _ in range(10):
        u, v = rng.standard_normal(s.shape), rng.standard_normal(D)
        num = (loss(s + h * u, w + h * v) - loss(s - h * u, w - h * v)) / (2 * h)
        # h^2 third derivatives (~1e-10 * 120) and fp32 gradients
        assert abs(num - (dx * u).sum() - (dw * v).sum()) <= 1e-4


def test_norm_autograd():
    x, r = randn(14, 6, 128).cuda().requires_grad_(), randn(15, 6, 128).cuda().requires_grad_()
    w = (1 + randn(16, 128, scale=0.1)).cuda().requires_grad_()
    a, b = randn(17, 6, 128).cuda(), randn(18, 6, 128).cuda()
    s, y = kda.residual_rms_norm(x, w, r, EPS)
    gx, gw, gr = torch.autograd.grad([s, y], [x, w, r], [a, b])
    x64, r64, w64 = (t.detach().double().requires_grad_() for t in (x, r, w))
    s64 = x64 + r64
    y64 = s64 * torch.rsqrt(s64.pow(2).mean(-1, keepdim=True) + EPS) * w64
    want = torch.autograd.grad([s64, y64], [x64, w64, r64], [a.double(), b.double()])
    for got, ref in zip((gx, gw, gr), want):
        assert torch.allclose(got.double(), ref, rtol=1e-5, atol=1e-5)
    s, y = kda.residual_rms_norm(x, w)
    gx, = torch.autograd.grad([s, y], [x], [a, b])
    y64 = x64 * torch.rsqrt(x64.pow(2).mean(-1, keepdim=True) + EPS) * w64
    ref, = torch.autograd.grad([x64 * 1, y64], [x64], [a.double(), b.double()])
    assert torch.allclose(gx.double(), ref, rtol=1e-5, atol=1e-5)


# -------------------------------------------------------------- the quantiser

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (127, 129), (128, 128), (300, 72),
                                       (17, 1001), (1025, 16)])
def test_quantize(rows, cols, transpose, block_rows, dtype):
    x = randn(20, rows, cols, dtype=dtype) * torch.exp(randn(21, rows, 1)).to(DT[dtype])
    y8, scale = kda.quantize_fp8(x.cuda(), block_rows=block_rows, transpose=transpose)
    want = f64(x).T if transpose else f64(x)
    check_codes(y8, scale, want, block_rows)


@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_zeros_extremes_and_nan(transpose):
    x = torch.zeros(4, 512)
    x[1, :128] = 2.0 ** -120            # below the floor: zero
    x[1, 128:256] = 3e38
    x[2, :128] = torch.arange(128) * 1e-38
    x[3, 0], x[3, 1] = float("nan"), 2.0
    x[3, 130] = float("inf")
    if transpose:   # blocks run along the other side
        x = x.T.contiguous()
    y8, scale = kda.quantize_fp8(x.cuda(), transpose=transpose)
    y, s = y8.float().cpu(), scale.cpu()
    assert torch.isfinite(s[:, :3]).all() and (s > 0).all()
    assert not y[0].any() and not y[1, :128].any() and (y[1, 128:256] == 448).all()
    assert torch.isnan(y[3, 0]) and y[3, 1] == 448 and s[0, 3] == 2.0 / 448
    assert torch.isnan(y[3, 130] * s[1, 3])


def test_quantize_strided_views_are_refused_and_empty_is_nothing():
    with pytest.raises(ValueError, match="contiguous"):
        kda.quantize_fp8(torch.zeros(8, 16, device="cuda").t())
    y8, scale = kda.quantize_fp8(torch.zeros(0, 100, device="cuda"))
    assert y8.shape == (0, 112) and scale.shape == (1, 0)


# -------------------------------------------------------------- the product

def operands(seed, M, N, K, block):
    gen = torch.Generator().manual_seed(seed)
    a = torch.randn(M, K, generator=gen) * torch.exp(torch.randn(M, 1, generator=gen))
    b = torch.randn(N, K, generator=gen)
    a8, sa = kda.quantize_fp8(a.cuda())
    b8, sb = kda.quantize_fp8(b.cuda(), block_rows=block)
    return a8, sa, b8, sb


def check_product(out, a8, sa, b8, sb, K, block, out_dtype):
    a = ofp8.dequantize(f64(a8)[:, :K], f64(sa), 1)
    b = ofp8.dequantize(f64(b8)[:, :K], f64(sb), block)
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    # e4m3 products are exact; at most 128 additions within a block, K / 128
    # blocks, 8 parts, three roundings of scales: each of them at most 2 u (the
    # tensor cores may cut off instead of rounding) of the sum of magnitudes
    tol = 2 * (128 + K / 128 + 8 + 3) * U * mag + HALF[out_dtype] * np.abs(want)
    err = np.abs(f64(out) - want)
    assert (err <= tol).all(), (err / np.maximum(mag, 1e-30)).max()


PRODUCTS = [(1, 1, 1), (1, 128, 128), (7, 100, 40), (16, 256, 1024), (17, 384, 130),
            (33, 129, 1000), (64, 1000, 512), (100, 513, 257), (129, 128, 4096), (256, 384, 384),
            (300, 257, 640), (2, 4096, 2048), (513, 1100, 300)]


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product_matches_fp64(M, N, K, block, out_dtype):
    a8, sa, b8, sb = operands(M + N + K, M, N, K, block)
    out = torch.full((M + 2, N), float("nan"), dtype=DT[out_dtype], device="cuda")
    kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=block, out=out[:M])
    check_product(out[:M], a8, sa, b8, sb, K, block, out_dtype)
    assert torch.isnan(out[M:]).all()     # rows behind the last one stay as they were


@pytest.mark.parametrize("block,out_dtype", [(128, "bf16"), (1, "f32")])
@pytest.mark.parametrize("M,N,K", [(1700, 3100, 300), (128 * 16, 256 * 10, 256), (40 * 128, 1024, 130),
                                   (9500, 520, 128)])
def test_product_of_a_full_round_of_tiles_and_a_part(M, N, K, block, out_dtype):
    """160 to 225 tiles of 128 x 256 on 148 SMs."""
    a8, sa, b8, sb = operands(M + N, M, N, K, block)
    out = kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=block, out_dtype=DT[out_dtype])
    check_product(out, a8, sa, b8, sb, K, block, out_dtype)


@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("M,N,K", [(20, 1000, 4100), (70, 2050, 4096), (20, 5120, 4096),
                                   (130, 2500, 4096), (200, 4096, 3000)])
def test_product_of_a_split_k(M, N, K, block):
    """Eight, four, three and two ways."""
    a8, sa, b8, sb = operands(M + N, M, N, K, block)
    out = kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=block, out_dtype=torch.float32)
    check_product(out, a8, sa, b8, sb, K, block, "f32")


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("M,N,K", [(16, 5000, 1100), (9, 300, 9000), (13, 4901, 3100),
                                   (8, 9500, 4100), (12, 20000, 130), (1, 513, 12001),
                                   (16, 9601, 8200), (10, 130, 5000)])
def test_product_of_few_rows_and_a_large_weight(M, N, K, block, out_dtype):
    """Split eight, four, two ways and not at all; the last tile and block ragged."""
    a8, sa, b8, sb = operands(M + N, M, N, K, block)
    out = torch.full((M + 2, N), float("nan"), dtype=DT[out_dtype], device="cuda")
    kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=block, out=out[:M])
    check_product(out[:M], a8, sa, b8, sb, K, block, out_dtype)
    assert torch.isnan(out[M:]).all()
    first = out[:M].clone()
    raw = b8.view(torch.uint8)
    raw[:, K:] = 0x7F                                  # NaN codes behind the last column
    raw[N // 2, 3] = 0x7F
    kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=block, out=out[:M])
    assert torch.isnan(out[:M, N // 2]).all()
    keep = torch.arange(N) != N // 2
    assert torch.equal(out[:M][:, keep], first[:, keep])


@pytest.mark.parametrize("M", [16, 300, 1500])
def test_product_is_the_same_every_time(M):
    args = operands(3, M, 1024, 2048, 128)
    first = kda.fp8_matmul(*args, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(kda.fp8_matmul(*args, out_dtype=torch.float32), first)


def test_product_ignores_the_padding_and_keeps_nan_in_its_row():
    M, N, K = 40, 200, 100
    a8, sa, b8, sb = operands(5, M, N, K, 128)
    out = kda.fp8_matmul(a8, sa, b8, sb, K=K, out_dtype=torch.float32)
    raw = a8.view(torch.uint8)
    raw[:, K:] = 0x7F                                  # NaN codes behind the last column
    assert torch.equal(kda.fp8_matmul(a8, sa, b8, sb, K=K, out_dtype=torch.float32), out)
    raw[3, 5] = 0x7F
    got = kda.fp8_matmul(a8, sa, b8, sb, K=K, out_dtype=torch.float32)
    assert torch.isnan(got[3]).all()
    keep = torch.arange(M) != 3
    assert torch.equal(got[keep], out[keep])
    sa[0, 7] = float("inf")
    got = kda.fp8_matmul(a8, sa, b8, sb, K=K, out_dtype=torch.float32)
    assert not torch.isfinite(got[7]).any() and torch.isfinite(got[8:]).all()


def test_product_empty_and_captured():
    a8, sa, b8, sb = operands(6, 20, 256, 512, 128)
    empty = kda.fp8_matmul(a8[:0], sa[:, :0].contiguous(), b8, sb)
    assert empty.shape == (0, 256)
    want = kda.fp8_matmul(a8, sa, b8, sb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kda.fp8_matmul(a8, sa, b8, sb)
    out.zero_()
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = kda.fp8_matmul(a8, sa, b8, sb, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(other, want)


def test_linear_and_its_gradients():
    """Against fp64 products of the quantised operands' values."""
    M, K, N = 150, 200, 136
    x, w, dy = randn(30, M, K, dtype="bf16"), randn(31, N, K, dtype="bf16"), \
        randn(32, M, N, dtype="bf16")
    X, W = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = kda.fp8_linear(X, W)
    dx, dw = torch.autograd.grad(y, [X, W], dy.cuda())
    q = lambda v, b: ofp8.dequantize(*ofp8.quantize(v, b), b)  # noqa: E731
    for got, a, b in ((y, q(f64(x), 1), q(f64(w), 128)),
                      (dx, q(f64(dy), 1), q(f64(w).T, 128)),
                      (dw, q(f64(dy).T, 1), q(f64(x).T, 1))):
        want = a @ b.T
        # a code at the border between two may round either way in fp32: one
        # step, 2^-3 of one term in thousands; bf16 rounding
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -3 * 3 * np.abs(a).max(1, keepdims=True) * np.abs(b).max()
        assert (np.abs(f64(got) - want) <= tol).all()
        assert np.abs(f64(got) - want).mean() <= 2.0 ** -8 * np.abs(want).mean()


def test_gradients_captured_into_a_graph():
    """Forward and backward of the three differentiable calls in one graph, replayed
    on new inputs; refused while an eager graph of the same leaves lives."""
    T, D = 70, 256
    x, r = (randn(70 + i, T, D, dtype="bf16").cuda().requires_grad_() for i in range(2))
    w_norm = torch.ones(D, device="cuda", requires_grad=True)
    w = randn(72, D, D, dtype="bf16", scale=D ** -0.5).cuda().requires_grad_()
    g = -torch.rand(T, 2, D // 2, device="cuda")
    dy = randn(73, T, D, dtype="bf16").cuda()

    def step():
        s, y = kda.residual_rms_norm(x, w_norm, r)
        h, _ = kda.gated_linear_scan(kda.fp8_linear(y, w).view(T, 2, D // 2), g)
        grads = torch.autograd.grad([h.reshape(T, D), s], [x, w_norm, r, w], [dy, dy])
        return [t.detach() for t in (h, s, *grads)]
    alive = kda.fp8_linear(x, w)
    with pytest.raises(RuntimeError, match="eager graph"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            step()
    del alive
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.no_grad():
        x.copy_(randn(74, T, D, dtype="bf16"))
        dy.copy_(randn(75, T, D, dtype="bf16"))
    graph.replay()
    want = step()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def test_second_derivatives_are_refused():
    x = randn(80, 4, 64, dtype="f32").cuda().requires_grad_()
    w = torch.ones(64, device="cuda")
    w2 = randn(81, 64, 64).cuda()
    for y in (kda.residual_rms_norm(x, w)[1], kda.fp8_linear(x, w2),
              kda.gated_linear_scan(x.view(4, 1, 64), torch.zeros(4, 1, 64, device="cuda"))[0]):
        dy = torch.ones_like(y).requires_grad_()
        grad, = torch.autograd.grad(y, x, dy, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            grad.sum().backward()


@pytest.mark.parametrize("M", [5, 40, 300])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_product_into_outputs_that_start_on_16_bytes(M, out_dtype):
    N, K = 256, 200
    a8, sa = kda.quantize_fp8(randn(82, M, K).cuda())
    for rows in (1, 128):
        b8, sb = kda.quantize_fp8(randn(83, N, K).cuda(), block_rows=rows)
        want = kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=rows, out_dtype=DT[out_dtype])
        skip = 16 // want.element_size()
        buf = torch.zeros(M * N + 2 * skip, dtype=DT[out_dtype], device="cuda")
        out = buf[skip:skip + M * N].view(M, N)
        kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=rows, out=out)
        assert torch.equal(out, want) and not buf[:skip].any() and not buf[-skip:].any()


def test_a_layer_from_its_parts():
    """Residual norm in 8 bits -> projections -> conv + norm -> the operator and,
    beside it, the gated linear recurrence -> output norm + gate -> projection
    back, against the same chain in fp64 on the GPU's own intermediate inputs."""
    import oracle
    from oracle import layer as olayer, scan as oscan
    T, H, d, D = 130, 2, 128, 256
    x, r = randn(40, T, D, dtype="bf16").cuda(), randn(41, T, D, dtype="bf16").cuda()
    w_norm = (1 + randn(42, D, scale=0.1)).cuda()
    wq, wk, wv, wg = (kda.quantize_fp8((randn(43 + i, H * d, D, scale=D ** -0.5)).cuda(),
                                       block_rows=128) for i in range(4))
    wo = kda.quantize_fp8(randn(47, D, H * d, scale=(H * d) ** -0.5).cuda(), block_rows=128)
    s, y8, sc = kda.add_rms_norm(x, w_norm, r, quantize=True)
    q, k, v, gate = (kda.fp8_matmul(y8, sc, *w).view(T, H, d) for w in (wq, wk, wv, wg))
    yq = ofp8.dequantize(f64(y8), f64(sc), 1)
    ref = yq @ ofp8.dequantize(f64(wv[0]), f64(wv[1]), 128).T
    assert np.abs(f64(v).reshape(T, -1) - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
    conv = [randn(50 + i, H * d, 4, scale=0.5).cuda() for i in range(3)]
    q2, k2, v2 = (torch.empty_like(q) for _ in range(3))
    kda.kda_qkv_conv_norm(q, k, v, *conv, None, 1, T, 1, H, d, d, "bf16", 1e-6, q2, k2, v2)
    g = -torch.nn.functional.softplus(gate.float())
    beta = torch.sigmoid(randn(53, T, H)).cuda()
    o, _ = kda.chunk_fwd(q2.view(1, T, H, d), k2.view(1, T, H, d), v2.view(1, T, H, d),
                         g.view(1, T, H, d), beta.view(1, T, H))
    ro, _ = oracle.forward(q2.cpu(), k2.cpu(), v2.cpu(), g.cpu(), beta.cpu(),
                           torch.zeros(1, H, d, d), None)
    assert np.abs(f64(o).reshape(T, H, d) - ro).max() <= 2e-2 * np.abs(ro).max()
    h, _ = kda.linear_scan(v2, g)
    rh, _ = oscan.forward(v2, g)
    assert np.abs(f64(h) - rh).max() <= 2.0 ** -8 * np.abs(rh).max() + 1e-5
    mixed = torch.empty_like(v2)
    kda.kda_output_norm_gate(h, gate, torch.ones(d, device="cuda"), T, H, d, "bf16", 1e-6, mixed)
    rm = olayer.output_norm_gate(h.cpu(), gate.cpu(), torch.ones(d), eps=1e-6)
    assert np.abs(f64(mixed) - rm).max() <= 1e-2 * np.abs(rm).max()
    m8, ms = kda.quantize_fp8(mixed.view(T, H * d))
    out = kda.fp8_matmul(m8, ms, *wo)
    ref = ofp8.dequantize(f64(m8), f64(ms), 1) @ ofp8.dequantize(f64(wo[0]), f64(wo[1]), 128).T
    assert np.abs(f64(out) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-4
    assert out.shape == s.shape
