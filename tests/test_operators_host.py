"""Host-only checks of the gated linear recurrence, the residual RMS norm and the
8-bit calls: refusals before anything is enqueued, sizes, and the fp64 references
themselves (against explicit sums and differences)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_124_b200 as kda
from gated_delta_rule_124_b200 import build as kbuild
from oracle import fp8 as ofp8, scan as oscan

FAKE = 1 << 20  # a 16-byte-aligned non-NULL address; never dereferenced on these paths
INVALID, UNSUPPORTED, WORKSPACE, OK = (kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED,
                                       kda.KDA_ERR_WORKSPACE, kda.KDA_OK)


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kda.load()


def refusals(call, ok, cases):
    for change, want in cases:
        assert call(**{**ok, **change}) == want, change


def test_linear_scan_refusals():
    ok = dict(x=FAKE, g=FAKE, initial_state=None, cu_seqlens=None, B=1, T=64, num_seqs=1, H=2,
              d=20, dtype="bf16", h=FAKE, final_state=None, entry_states=None, workspace=2 * FAKE,
              workspace_bytes=16, stream=0, check=False)
    common = [(dict(), WORKSPACE), (dict(workspace=None), WORKSPACE), (dict(x=None), INVALID),
              (dict(g=FAKE + 4), INVALID), (dict(T=-1), INVALID), (dict(B=0), INVALID),
              (dict(num_seqs=2), INVALID), (dict(H=0), INVALID), (dict(d=0), INVALID),
              (dict(H=1 << 13, d=1 << 12), INVALID), (dict(initial_state=FAKE + 8), INVALID),
              (dict(cu_seqlens=FAKE, B=2, num_seqs=2), INVALID),
              (dict(workspace=FAKE + 16, workspace_bytes=1 << 40), INVALID),
              (dict(cu_seqlens=FAKE, T=0x7fffffff, workspace_bytes=1 << 60), INVALID)]
    refusals(kda.kda_linear_scan_fwd, ok, common + [
        (dict(h=None), INVALID), (dict(final_state=FAKE + 4), INVALID),
        (dict(entry_states=FAKE + 4), INVALID)])
    bwd = dict(x=FAKE, g=FAKE, initial_state=None, dout=FAKE, dfinal_state=None,
               entry_states=None, cu_seqlens=None, B=1, T=64, num_seqs=1, H=2, d=20, dtype="f32",
               dx=FAKE, dg=FAKE, dinitial_state=None, workspace=2 * FAKE, workspace_bytes=16,
               stream=0, check=False)
    refusals(kda.kda_linear_scan_bwd, bwd, common + [
        (dict(dout=None), INVALID), (dict(dx=FAKE + 2), INVALID), (dict(dg=None), INVALID),
        (dict(workspace_bytes=1 << 40, dfinal_state=FAKE, dinitial_state=FAKE), INVALID),
        (dict(workspace_bytes=1 << 40, initial_state=FAKE, dinitial_state=FAKE), INVALID)])
    with pytest.raises(ValueError):
        kda.kda_linear_scan_fwd(**{**ok, "dtype": 7})
    step = dict(x=FAKE, g=FAKE, state_in=FAKE, state_out=FAKE, h=FAKE, N=4, H=2, d=3, dtype="f32",
                stream=0, check=False)
    refusals(kda.kda_linear_scan_step, step, [
        (dict(x=None), INVALID), (dict(state_out=FAKE + 4), INVALID), (dict(N=-1), INVALID),
        (dict(H=0), INVALID), (dict(N=0), OK), (dict(N=0, x=None), OK)])


def test_linear_scan_sizes():
    assert [kda.kda_linear_scan_num_entries(n) for n in (-1, 0, 1, 64, 65)] == [0, 1, 1, 1, 2]
    f, b = kda.kda_linear_scan_workspace_size, kda.kda_linear_scan_bwd_workspace_size
    assert f(64, 4, 32) == 256                       # one tile: the status word
    assert f(65, 4, 32) > f(64, 4, 32) and f(1 << 20, 4, 32) > f(1 << 19, 4, 32)
    assert b(1000, 4, 32) >= f(1000, 4, 32) + 4 * 128 * kda.kda_linear_scan_num_entries(1000)
    assert f(-1, 1, 1) == 0 and f(1, 0, 1) == 0 and b(1, 1, 0) == 0 and b(1, 1 << 20, 1 << 20) == 0


def test_norm_refusals():
    ok = dict(x=FAKE, residual=None, w=FAKE, rows=4, D=64, dtype="bf16", eps=1e-6, sum=None,
              y=FAKE, y8=None, y8_scale=None, stream=0, check=False)
    refusals(kda.kda_add_rms_norm, ok, [
        (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
        (dict(y8=FAKE), INVALID), (dict(y8_scale=FAKE), INVALID), (dict(rows=-1), INVALID),
        (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(D=0), INVALID),
        (dict(D=12), UNSUPPORTED), (dict(D=16392), UNSUPPORTED), (dict(residual=FAKE + 2), INVALID),
        (dict(rows=0, x=None), OK)])
    bwd = dict(s=FAKE, w=FAKE, dy=2 * FAKE, dsum=None, rows=4, D=64, dtype="bf16", eps=1e-6,
               dx=3 * FAKE, dw=FAKE, workspace=FAKE, workspace_bytes=16, stream=0, check=False)
    refusals(kda.kda_add_rms_norm_bwd, bwd, [
        (dict(), WORKSPACE), (dict(workspace=None), WORKSPACE), (dict(s=None), INVALID),
        (dict(dx=FAKE, workspace_bytes=1 << 40), INVALID), (dict(dw=None), INVALID),
        (dict(dx=2 * FAKE, workspace_bytes=1 << 40), INVALID), (dict(D=20), UNSUPPORTED),
        (dict(workspace=FAKE + 16, workspace_bytes=1 << 40), INVALID), (dict(eps=-1.0), INVALID)])
    size = kda.kda_add_rms_norm_bwd_workspace_size
    assert size(1, 64) >= 4 * 64 and size(10 ** 6, 64) >= size(296, 64) and size(4, 12) == 0


def test_eight_bit_refusals():
    q = dict(x=FAKE, rows=4, cols=64, dtype="bf16", block_rows=1, transpose=False, y8=FAKE,
             scale=FAKE, stream=0, check=False)
    refusals(kda.kda_quantize_fp8, q, [
        (dict(x=None), INVALID), (dict(y8=FAKE + 8), INVALID), (dict(scale=None), INVALID),
        (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(block_rows=64), UNSUPPORTED),
        (dict(rows=0x7fffff00, cols=0x7fffff00), UNSUPPORTED), (dict(rows=0, x=None), OK)])
    m = dict(a8=FAKE, a_scale=FAKE, b8=FAKE, b_scale=FAKE, M=4, N=64, K=64, b_block_rows=128,
             out_dtype="bf16", out=FAKE, stream=0, check=False)
    refusals(kda.kda_fp8_matmul, m, [
        (dict(a8=None), INVALID), (dict(b8=FAKE + 8), INVALID), (dict(out=None), INVALID),
        (dict(b_scale=FAKE + 4), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID),
        (dict(K=0), INVALID), (dict(b_block_rows=2), UNSUPPORTED), (dict(M=0, a8=None), OK)])
    assert [kda.kda_fp8_pitch(k) for k in (-1, 0, 1, 16, 17, 4099)] == [0, 0, 16, 16, 32, 4112]


def test_wrappers_refuse_shapes_the_library_would_misread():
    x, g = torch.zeros(8, 2, 4), torch.zeros(8, 2, 4)
    with pytest.raises(ValueError, match="g is"):
        kda.linear_scan(x, g[:7])
    with pytest.raises(ValueError, match="initial_state"):
        kda.linear_scan(x, g, torch.zeros(2, 2, 4))
    with pytest.raises(ValueError, match="packed"):
        kda.linear_scan(x[None], g[None], cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="dout"):
        kda.linear_scan_bwd(x, g, g[:, :1])
    with pytest.raises(ValueError, match="entry_states"):
        kda.linear_scan_bwd(x, g, x, entry_states=torch.zeros(2, 2, 4))
    with pytest.raises(ValueError, match="float32"):
        kda.kda_linear_scan_step(x[0], g[0].half(), x[0], x[0], x[0], 2, 1, 4, "f32")
    with pytest.raises(ValueError, match="residual"):
        kda.add_rms_norm(x[0], torch.ones(4), x[0, :1])
    with pytest.raises(ValueError, match="w is"):
        kda.add_rms_norm(x[0], torch.ones(5))
    with pytest.raises(ValueError, match="rows, cols"):
        kda.quantize_fp8(x)
    a8, b8 = torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(5, 32, dtype=torch.uint8)
    sa, sb = torch.zeros(1, 3), torch.zeros(1, 1)
    with pytest.raises(ValueError, match="a8 is"):
        kda.fp8_matmul(a8, sa, b8, sb, K=10)
    with pytest.raises(ValueError, match="b_scale"):
        kda.fp8_matmul(a8, sa, b8, sb, b_block_rows=1)
    with pytest.raises(ValueError, match="float8"):
        kda.kda_fp8_matmul(a8.float(), sa, b8, sb, 3, 5, 32, 128, "f32", torch.zeros(3, 5))
    with pytest.raises(ValueError, match="fp8_linear"):   # (rows of 112 bytes both)
        kda.fp8_linear(torch.zeros(2, 97), torch.zeros(8, 112))


def test_wrappers_refuse_tensors_that_are_not_on_a_gpu():
    x, g, w = torch.zeros(8, 2, 4), torch.zeros(8, 2, 4), torch.ones(8)
    y = x.view(8, 8)
    a8, sa = torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(1, 3)
    for call in (lambda: kda.linear_scan(x, g), lambda: kda.linear_scan_bwd(x, g, x),
                 lambda: kda.linear_scan_step(x, g, x), lambda: kda.add_rms_norm(y, w),
                 lambda: kda.add_rms_norm_bwd(y, w, y), lambda: kda.quantize_fp8(y),
                 lambda: kda.fp8_matmul(a8, sa, a8, sa, b_block_rows=1)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


def test_scan_reference_is_the_explicit_sum_and_its_gradient_a_difference():
    rng = np.random.default_rng(1)
    lens, H, d = [4, 0, 3], 1, 2
    x, g = rng.standard_normal((7, H, d)), -np.abs(rng.standard_normal((7, H, d)))
    h0 = rng.standard_normal((3, H, d))
    h, final = oscan.forward(x, g, h0, lens)
    for t in range(4):  # h_t = sum_s exp(g_{s+1} + .. + g_t) x_s + exp(g_0 + .. + g_t) h_0
        want = np.exp(g[:t + 1].sum(0)) * h0[0] + sum(
            np.exp(g[s + 1:t + 1].sum(0)) * x[s] for s in range(t + 1))
        assert np.allclose(h[t], want, rtol=1e-13)
    assert np.array_equal(final[1], h0[1]) and np.array_equal(final[2], h[6])
    do, df = rng.standard_normal(x.shape), rng.standard_normal(h0.shape)

    def loss(x_, g_, h_):
        a, b = oscan.forward(x_, g_, h_, lens)
        return (a * do).sum() + (b * df).sum()
    grads = oscan.backward(x, g, do, h0, df, lens)
    for i, v in enumerate((x, g, h0)):
        u, e = rng.standard_normal(v.shape), 1e-6
        args = [[x, g, h0], [x, g, h0]]
        args[0][i], args[1][i] = v + e * u, v - e * u
        assert abs((loss(*args[0]) - loss(*args[1])) / (2 * e) - (grads[i] * u).sum()) < 1e-7


def test_eight_bit_reference():
    x = np.array([0.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 1.0625, 1.1875, -17.0, 448.0, 1e9])
    assert ofp8.e4m3(x).tolist() == [0.0, 2.0 ** -9, 0.0, 2.0 ** -8, 1.0, 1.25, -16.0, 448.0, 448.0]
    t = torch.linspace(-448, 448, 5001)
    assert np.array_equal(ofp8.e4m3(t.numpy()), t.to(torch.float8_e4m3fn).double().numpy())
    rng = np.random.default_rng(2)
    a = rng.standard_normal((130, 260))
    for block in (1, 128):
        codes, scale = ofp8.quantize(a, block)
        assert scale.shape == (3, 130 if block == 1 else 2) and np.abs(codes).max() == 448
        back = ofp8.dequantize(codes, scale, block)
        # half a step of 2^-3, or of e4m3's smallest step 2^-9
        assert (np.abs(back - a) <= np.maximum(2.0 ** -4 * np.abs(a),
                                               2.0 ** -10 * scale.max())).all()
    s, w, dy, ds = (rng.standard_normal(v) for v in ((3, 16), 16, (3, 16), (3, 16)))
    dx, dw = ofp8.rms_norm_bwd(s, w, dy, ds, 1e-6)
    loss = lambda s_, w_: (ofp8.rms_norm(s_, w_, 1e-6) * dy).sum() + (s_ * ds).sum()  # noqa: E731
    u, v, e = rng.standard_normal(s.shape), rng.standard_normal(16), 1e-6
    num = (loss(s + e * u, w + e * v) - loss(s - e * u, w - e * v)) / (2 * e)
    assert abs(num - (dx * u).sum() - (dw * v).sum()) < 1e-6
