"""The gated linear recurrence on the GPU against the fp64 recurrence: forward,
backward, the one-token step, and the ways in which a caller uses them.

Error bounds.  With u = 2^-24, M_t = alpha_t M_{t-1} + |x_t| (M_{-1} = |h_{-1}|)
bounds every partial sum.  A step's gate is within 3 u (the exponential is within
2 units in the last place of fp32, counted as 2^-23 each, and g is exact), its
multiply-add within u: E_t = alpha_t (E_{t-1} + 6 u M_{t-1}) + u M_t.  A state
that crosses a tile goes through exp2 of a sum G of up to 64 logarithms per tile:
the sum is off by at most 64 u |G| and |G| exp(G) <= 1 / e, exp2 by 4 u, the sum
with the tile's part by 2 u: 64 u M more at each tile.  bf16 outputs are one
rounding further, 2^-8 of the value.  Gradients obey the same recurrence from the
other side; dg is e_t h_{t-1}, a product of two such values.

Below 2^-126 errors are absolute: a gate that small may be taken as zero, 2^-126
times a state (at most 16 here), and in dg once more times a state: 2^-118; fp32's
subnormal roundings (2^-150 each) are far below that."""
import numpy as np
import pytest
import torch

import gated_delta_rule_124_b200 as kda
from oracle import scan as oscan

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -117
BF16 = 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TILE = 64


def make(seed, lens, H, d, dtype, gate=0.0, h0=True):
    gen = torch.Generator().manual_seed(seed)
    total, N = sum(lens), len(lens)
    x = torch.randn(total, H, d, generator=gen).to(DT[dtype])
    z = torch.randn(total, H, d, generator=gen)
    if gate == "zero":
        g = torch.zeros_like(z)                       # a plain running sum
    elif gate == "strong":
        g = -50.0 * z.abs()                           # products far below the fp32 range
    elif gate == "growth":
        g = 0.02 + 0.01 * z                           # gates above one
    else:
        g = -torch.nn.functional.softplus(z + gate)
    init = torch.randn(N, H, d, generator=gen) if h0 else None
    dout = torch.randn(total, H, d, generator=gen).to(DT[dtype])
    dfin = torch.randn(N, H, d, generator=gen)
    return x, g, init, dout, dfin


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def error_bound(alpha, x, start, first_row=0):
    """E_t over one sequence whose first token is packed row `first_row`; `alpha`
    multiplies the state before a row, `start` is the state that enters."""
    M, E = np.abs(start), np.zeros_like(start)
    out = np.empty_like(x)
    for t in range(x.shape[0]):
        if t and (first_row + t) % TILE == 0:
            E = E + 64 * U * M
        E = alpha[t] * (E + 6 * U * M)
        M = alpha[t] * M + np.abs(x[t])
        E = E + U * M
        out[t] = E + TINY
    return out


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def seq_slices(lens):
    at = 0
    for n, length in enumerate(lens):
        yield n, at, length
        at += length


def check_forward(x, g, init, lens, h, final, dtype):
    rh, rf = oscan.forward(x, g, init, lens)
    x64, a64 = f64(x), np.exp(f64(g))
    h, final = f64(h), f64(final)
    for n, at, length in seq_slices(lens):
        start = np.zeros(x.shape[1:]) if init is None else f64(init)[n]
        if length == 0:
            assert np.array_equal(final[n], start)
            continue
        sl = slice(at, at + length)
        tol = error_bound(a64[sl], x64[sl], start, at)
        assert (np.abs(final[n] - rf[n]) <= tol[-1]).all()
        if dtype == "bf16":
            tol = tol * (1 + BF16) + BF16 * np.abs(rh[sl])
        assert (np.abs(h[sl] - rh[sl]) <= tol).all(), (n, np.abs(h[sl] - rh[sl]).max())


def check_backward(x, g, init, dout, dfin, lens, got, dtype):
    dx, dg, dh0 = (f64(t) for t in got)
    rx, rg, rh0 = oscan.backward(x, g, dout, init, dfin, lens)
    rh, _ = oscan.forward(x, g, init, lens)
    x64, a64, d64 = f64(x), np.exp(f64(g)), f64(dout)
    for n, at, length in seq_slices(lens):
        end = np.zeros(x.shape[1:]) if dfin is None else f64(dfin)[n]
        start = np.zeros(x.shape[1:]) if init is None else f64(init)[n]
        if length == 0:
            assert np.array_equal(dh0[n], end)
            continue
        sl = slice(at, at + length)
        # dx from the right: dx_t = dout_t + alpha_{t+1} dx_{t+1}; the tiles'
        # bounds lie between the same rows, so the same count of crossings
        right = np.concatenate([np.ones_like(a64[:1]), a64[sl][:0:-1]])
        mag = error_bound(right, d64[sl][::-1], end, 0)[::-1]
        tol = 2 * mag + 64 * U * np.abs(end)   # (where the crossings fall differs)
        want = rx[sl]
        assert (np.abs(dx[sl] - want) <=
                tol * (1 + BF16) + (BF16 if dtype == "bf16" else U) * np.abs(want)).all()
        e, e_tol = a64[sl] * want, a64[sl] * (tol + 8 * U * np.abs(want))
        assert (np.abs(dh0[n] - rh0[n]) <= e_tol[0] + U * np.abs(rh0[n]) + TINY).all()
        before = np.concatenate([start[None], rh[sl][:-1]])
        h_tol = np.concatenate([np.zeros_like(start)[None],
                                error_bound(a64[sl], x64[sl], start, at)[:-1]])
        dg_tol = (e_tol * (np.abs(before) + h_tol) + np.abs(e) * h_tol + 2 * U * np.abs(e * before)
                  + TINY)
        assert (np.abs(dg[sl] - rg[sl]) <= dg_tol).all()


LENGTHS = [[1], [63], [64], [65], [0], [0, 1, 0, 200, 64, 0, 0], [5, 59, 64, 1, 127, 3],
           [1] * 130, [2000]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,d", [(1, 1), (1, 3), (2, 64), (3, 44), (1, 131), (2, 128)])
@pytest.mark.parametrize("lens", LENGTHS, ids=lambda v: "-".join(map(str, v[:7])) + f"x{len(v)}")
def test_forward_and_backward_match_the_recurrence(lens, H, d, dtype):
    x, g, init, dout, dfin = make(sum(lens) + d, lens, H, d, dtype)
    X, G, I, D, F = cuda(x, g, init, dout, dfin)
    cu = offsets(lens)
    h, final, entry = kda.linear_scan(X, G, I, cu_seqlens=cu, output_entry_states=True)
    check_forward(x, g, init, lens, h, final, dtype)
    kept = kda.linear_scan_bwd(X, G, D, I, F, cu_seqlens=cu, entry_states=entry)
    check_backward(x, g, init, dout, dfin, lens, kept, dtype)
    again = kda.linear_scan_bwd(X, G, D, I, F, cu_seqlens=cu)   # entry states recomputed
    check_backward(x, g, init, dout, dfin, lens, again, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,d", [(1, 2052), (32, 64), (9, 128), (1, 301), (3, 128)])
def test_rows_of_every_length(H, d, dtype):
    """Tiles in groups of three and without groups, the backward pass's long rows."""
    lens = [110, 133, 162, 0, 26, 343]
    x, g, init, dout, dfin = make(d, lens, H, d, dtype)
    X, G, I, D, F = cuda(x, g, init, dout, dfin)
    cu = offsets(lens)
    h, final, entry = kda.linear_scan(X, G, I, cu_seqlens=cu, output_entry_states=True)
    check_forward(x, g, init, lens, h, final, dtype)
    got = kda.linear_scan_bwd(X, G, D, I, F, cu_seqlens=cu, entry_states=entry)
    check_backward(x, g, init, dout, dfin, lens, got, dtype)


@pytest.mark.parametrize("gate", ["zero", "strong", "growth", -4.0])
def test_gates_of_every_size(gate):
    lens = [700, 1, 500]
    x, g, init, dout, dfin = make(3, lens, 2, 20, "f32", gate)
    X, G, I, D, F = cuda(x, g, init, dout, dfin)
    h, final = kda.linear_scan(X, G, I, cu_seqlens=offsets(lens))
    check_forward(x, g, init, lens, h, final, "f32")
    got = kda.linear_scan_bwd(X, G, D, I, F, cu_seqlens=offsets(lens))
    check_backward(x, g, init, dout, dfin, lens, got, "f32")


def test_product_of_gates_beyond_fp32_meets_a_small_state():
    """exp(g) over 640 tokens is e^96, the state e^-60: the product of the gates
    alone (and of several tiles) would overflow, their states do not."""
    T, C = 640, 8
    g = torch.full((T, 1, C), 0.15)
    x = torch.zeros(T, 1, C)
    init = torch.full((1, 1, C), float(np.exp(-60.0)))
    h, final = kda.linear_scan(*cuda(x, g, init))
    rh, rf = oscan.forward(x, g, init)
    # every step's error is relative here, and so is every tile's (64 u |G|, |G| <= 14)
    rel = T * 8 * U + (T // TILE) * 64 * 14 * U
    assert (np.abs(f64(h) - rh) <= rel * rh).all() and (np.abs(f64(final) - rf) <= rel * rf).all()
    h, _ = kda.linear_scan(*cuda(x, g, torch.zeros_like(init)))
    assert not h.any()


def test_batch_by_time_layout_without_states():
    B, T, H, d = 3, 150, 2, 24
    x, g, _, dout, _ = make(5, [T] * B, H, d, "bf16", h0=False)
    X, G, D = (t.cuda().view(B, T, H, d) for t in (x, g, dout))
    h, final = kda.linear_scan(X, G)
    assert h.shape == X.shape and final.shape == (B, H, d)
    check_forward(x, g, None, [T] * B, h.view(-1, H, d), final, "bf16")
    dx, dg, dh0 = kda.linear_scan_bwd(X, G, D)
    check_backward(x, g, None, dout, None, [T] * B,
                   (dx.view(-1, H, d), dg.view(-1, H, d), dh0), "bf16")
    empty = kda.linear_scan(X[:, :0], G[:, :0], init3 := torch.randn(B, H, d, device="cuda"))
    assert empty[0].shape == (B, 0, H, d) and torch.equal(empty[1], init3)
    h2, none = kda.linear_scan(X, G, output_final_state=False)
    assert none is None and torch.equal(h, h2)


def test_final_state_in_the_initial_states_buffer():
    lens = [300, 0, 2, 640]
    x, g, init, _, _ = make(6, lens, 2, 64, "bf16")
    X, G, I = cuda(x, g, init)
    total, H, d = x.shape
    h = torch.empty_like(X)
    ws = torch.empty(kda.kda_linear_scan_workspace_size(total, H, d), dtype=torch.uint8,
                     device="cuda")
    for _ in range(3):
        state = I.clone()
        kda.kda_linear_scan_fwd(X, G, state, offsets(lens), 1, total, len(lens), H, d, "bf16", h,
                                state, None, ws)
        check_forward(x, g, init, lens, h, state, "bf16")


def test_long_sequence_on_few_channels():
    """Far more tiles than fit on the device at once; against the same recurrence
    in fp64 by doubling."""
    T, H, d = 300_001, 1, 8
    x, g, init, _, _ = make(8, [T], H, d, "f32", -4.0)
    X, G, I = cuda(x, g, init)
    h, final = kda.linear_scan(X, G, I)
    a, b = G.double().exp(), X.double()
    b[0] += a[0] * I[0]
    a[0] = 0
    span = 1
    while span < T:
        b = torch.cat([b[:span], b[span:] + a[span:] * b[:-span]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    # sum of magnitudes by the same recurrence is at most max |x| / (1 - mean gate)
    # ~ 55 * 5; a bound of 64 u a tile over its memory of a few tiles
    assert (h.double() - b).abs().max().item() <= 275 * (64 + 6 * 55) * U
    assert torch.equal(final[0], h[-1])


@pytest.mark.parametrize("T,H,d,dtype", [(30_000, 1, 128, "bf16"), (6_000, 16, 128, "bf16"),
                                         (30_000, 1, 24, "f32"), (20_000, 1, 33, "bf16"),
                                         (30_000, 4, 128, "bf16"), (20_000, 9, 128, "f32"),
                                         (40_000, 1, 155, "f32"), (9_000, 1, 301, "bf16")])
def test_results_have_the_same_bits_in_every_run(T, H, d, dtype):
    """Few channels (tiles in groups of six and of three), many, one channel per lane;
    more tiles than fit on the device at once."""
    lens = [T // 2 + 7, T - T // 2 - 7]
    X, G, I, D, F = cuda(*make(14, lens, H, d, dtype, -3.0))
    cu = offsets(lens)

    def call():
        h, final, entry = kda.linear_scan(X, G, I, cu_seqlens=cu, output_entry_states=True)
        return (h, final, entry, *kda.linear_scan_bwd(X, G, D, I, F, cu_seqlens=cu,
                                                      entry_states=entry))
    first = call()
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(first, call()))


def test_nan_and_infinity_stay_in_their_sequence_and_channel():
    lens = [100, 70, 90]
    x, g, init, _, _ = make(9, lens, 1, 8, "f32")
    x[150, 0, 3] = float("nan")
    x[110, 0, 5] = float("inf")
    init[0, 0, 6] = float("nan")
    h, final = kda.linear_scan(*cuda(x, g, init), cu_seqlens=offsets(lens))
    bad = ~torch.isfinite(h[:, 0].cpu())
    want = torch.zeros_like(bad)
    want[150:170, 3] = want[110:170, 5] = want[0:100, 6] = True
    assert torch.equal(bad, want)
    assert torch.isfinite(final[2]).all()


@pytest.mark.parametrize("bad_gate", [float("nan"), 3e38])
@pytest.mark.parametrize("C", [8, 7, 128, 400, 1100, 2500])
def test_a_nan_gate_stays_in_its_sequence(C, bad_gate):
    """Sequences that begin inside the tile, and the group of tiles, of the NaN."""
    lens = [90, 20, 200, 1000, 700, 300, 1]
    x, g, init, dout, dfin = make(15, lens, 1, C, "f32")
    starts = np.cumsum([0] + lens)
    for n in (0, 2, 4):
        g[starts[n] + lens[n] // 2, 0, 1] = bad_gate
    X, G, I, D, F = cuda(x, g, init, dout, dfin)
    cu = offsets(lens)
    h, final, entry = kda.linear_scan(X, G, I, cu_seqlens=cu, output_entry_states=True)
    dx, dg, dh0 = kda.linear_scan_bwd(X, G, D, I, F, cu_seqlens=cu, entry_states=entry)
    for n, at, length in seq_slices(lens):
        mid, end = at + length // 2, at + length
        for out, a, b in ((h, mid, end), (dx, at, mid), (dg, at, end)):
            bad = torch.zeros(length, C, dtype=torch.bool)
            if n in (0, 2, 4):
                bad[a - at:b - at, 1] = True
            got = ~torch.isfinite(out[at:end, 0].cpu())
            assert torch.equal(got, bad), (n, torch.nonzero(got != bad)[:4])
    bad = torch.zeros(len(lens), C, dtype=torch.bool)
    bad[[0, 2, 4], 1] = True
    assert torch.equal(~torch.isfinite(final[:, 0].cpu()), bad)
    assert torch.equal(~torch.isfinite(dh0[:, 0].cpu()), bad)


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min, -1e9])
@pytest.mark.parametrize("C", [8, 5, 1024])
def test_gates_of_zero_start_the_state_again(C, low):
    """As sequences of their own do: the same values, within the bounds."""
    lens = [130, 64, 1, 500, 305]
    total = sum(lens)
    x, g, init, dout, _ = make(16, [total], 1, C, "f32")
    for _, at, _ in list(seq_slices(lens))[1:]:
        g[at] = low
    X, G, I, D = cuda(x, g, init, dout)
    h, final = kda.linear_scan(X, G, I)
    check_forward(x, g, init, [total], h, final, "f32")
    check_backward(x, g, init, dout, None, [total], kda.linear_scan_bwd(X, G, D, I), "f32")


def test_gates_beyond_the_range_of_exp():
    x, g = torch.ones(3, 1, 4), torch.tensor([0.0, 90.0, 3e38]).view(3, 1, 1).expand(3, 1, 4)
    h, _ = kda.linear_scan(*cuda(x, g.contiguous(), torch.ones(1, 1, 4)))
    assert (h[0] == 2).all() and not torch.isfinite(h[1:]).any()


@pytest.mark.parametrize("C,every", [(8, 97), (128, 384), (128, 161), (33, 1531), (400, 193),
                                     (400, 320), (1100, 161), (155, 700)])
def test_many_sequences_on_few_channels(C, every):
    """Starts in every place of a tile and of a group of tiles, far more tiles than
    run at once."""
    T = 120_000 if C < 200 else 30_000
    lens = [every] * (T // every) + [T % every]
    x, g, init, _, _ = make(17, lens, 1, C, "f32", -3.0)
    X, G, I = cuda(x, g, init)
    for _ in range(3):
        h, final = kda.linear_scan(X, G, I, cu_seqlens=offsets(lens))
    n = T // every * every      # the whole sequences, side by side
    H64 = I[:-1].double()
    a = G[:n].view(-1, every, 1, C).double().exp()
    b = X[:n].view(-1, every, 1, C).double()
    E, M = torch.zeros_like(H64), H64.abs()
    at = torch.arange(0, n, every, device="cuda")
    for t in range(every):
        if t:
            E = torch.where(((at + t) % TILE == 0).view(-1, 1, 1), E + 64 * U * M, E)
        H64 = a[:, t] * H64 + b[:, t]
        E = a[:, t] * (E + 6 * U * M)
        M = a[:, t] * M + b[:, t].abs()
        E = E + U * M
        assert ((h[:n].view(-1, every, 1, C)[:, t].double() - H64).abs() <= E + TINY).all()
    assert ((final[:-1].double() - H64).abs() <= E + TINY).all()


def test_step_continues_a_prefill():
    N, H, d, T = 5, 3, 20, 70
    x, g, init, _, _ = make(10, [T] * N, H, d, "bf16")
    X, G, I = cuda(x, g, init)
    X, G = X.view(N, T, H, d), G.view(N, T, H, d)
    h, final = kda.linear_scan(X, G, I)
    _, state = kda.linear_scan(X[:, :-2].contiguous(), G[:, :-2].contiguous(), I)
    keep = state.clone()
    for t in (T - 2, T - 1):
        out = kda.linear_scan_step(X[:, t].contiguous(), G[:, t].contiguous(), state)
        assert torch.equal(out, state.to(torch.bfloat16))
    assert not torch.equal(state, keep)
    rh, rf = oscan.forward(x, g, init, [T] * N)
    tol = np.stack([error_bound(np.exp(f64(g))[n * T:n * T + T], f64(x)[n * T:n * T + T],
                                f64(init)[n])[-1] + 64 * U * np.abs(rf[n]) for n in range(N)])
    assert (np.abs(f64(state) - rf) <= tol).all()
    other = torch.empty_like(state)
    kda.linear_scan_step(X[:, 0].contiguous(), G[:, 0].contiguous(), state, state_out=other)
    assert not torch.equal(other, state)


@pytest.mark.parametrize("n,d", [(1, 1), (7, 3), (256, 128)])
def test_step_sizes(n, d):
    x, g, init, _, _ = make(11, [1] * n, 2, d, "f32")
    X, G, S = cuda(x, g, init)
    h = kda.linear_scan_step(X, G, S)
    want = np.exp(f64(g)) * f64(init) + f64(x)
    assert (np.abs(f64(S) - want) <= 8 * U * (np.abs(f64(init)) + np.abs(f64(x)))).all()
    assert torch.equal(h, S)


def test_bad_offsets_are_reported():
    x, g, init, dout, dfin = make(12, [100, 100], 1, 8, "f32")
    X, G, I, D, F = cuda(x, g, init, dout, dfin)
    ws = torch.empty(kda.kda_linear_scan_bwd_workspace_size(200, 1, 8), dtype=torch.uint8,
                     device="cuda")
    h, final = torch.empty_like(X), torch.empty_like(I)
    for cu, want in (([0, 100, 200], kda.KDA_OK), ([0, 150, 100], kda.KDA_ERR_BAD_SEQLENS),
                     ([0, 100, 190], kda.KDA_ERR_BAD_SEQLENS),
                     ([1, 100, 200], kda.KDA_ERR_BAD_SEQLENS), ([0, 0, 200], kda.KDA_OK)):
        off = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kda.linear_scan(X, G, I, cu_seqlens=off, workspace=ws)
        assert kda.kda_get_device_status(ws) == want
        kda.linear_scan_bwd(X, G, D, I, F, cu_seqlens=off, workspace=ws)
        assert kda.kda_get_device_status(ws) == want


def test_captured_calls_replay_beside_others():
    """Two captured graphs and an eager call on another stream, each with its own
    workspace; replays on new inputs give the new results."""
    lens = [500, 33]
    cu = offsets(lens)
    sets = [make(20 + i, lens, 2, 64, "bf16") for i in range(3)]
    bufs = [cuda(*s) for s in sets[:2]]
    graphs, outs = [], []
    kda.linear_scan(bufs[0][0], bufs[0][1], bufs[0][2], cu_seqlens=cu)
    for b in bufs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append((kda.linear_scan(b[0], b[1], b[2], cu_seqlens=cu),
                         kda.linear_scan_bwd(b[0], b[1], b[3], b[2], b[4], cu_seqlens=cu)))
        graphs.append(gr)
    side, c = torch.cuda.Stream(), cuda(*sets[2])
    torch.cuda.synchronize()
    for gr in graphs:
        gr.replay()
    eager = kda.linear_scan(c[0], c[1], c[2], cu_seqlens=cu, stream=side)
    graphs[0].replay()
    torch.cuda.synchronize()
    for s, o in zip(sets, outs):
        check_forward(s[0], s[1], s[2], lens, *o[0], "bf16")
        check_backward(*s, lens, o[1], "bf16")
    check_forward(sets[2][0], sets[2][1], sets[2][2], lens, *eager, "bf16")
    for dst, src in zip(bufs[0], c):
        dst.copy_(src)
    graphs[0].replay()
    torch.cuda.synchronize()
    check_forward(sets[2][0], sets[2][1], sets[2][2], lens, *outs[0][0], "bf16")


def test_autograd_gradients():
    lens = [90, 0, 41]
    x, g, init, dout, dfin = make(13, lens, 2, 12, "f32")
    X, G, I, D, F = cuda(x, g, init, dout, dfin)
    for t in (X, G, I):
        t.requires_grad_()
    h, final = kda.gated_linear_scan(X, G, I, offsets(lens))
    grads = torch.autograd.grad([h, final], [X, G, I], [D, F])
    check_backward(x, g, init, dout, dfin, lens, grads, "f32")
    h, _ = kda.gated_linear_scan(X, G, I, offsets(lens))        # the final state unused
    grads = torch.autograd.grad(h, [X, G, I], D.transpose(1, 2).contiguous().transpose(1, 2))
    check_backward(x, g, init, dout, None, lens, grads, "f32")
