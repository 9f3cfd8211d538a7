"""The variants of the 8-bit product, each at sizes that reach it: which one a size
takes is asserted on the host, so that the GPU tests below cannot lose their variant.

Error bound as for the other products: e4m3 products are exact, at most 128
additions inside a block, K / 128 blocks, 8 parts and three roundings of scales,
each at most 2 u (u = 2^-24; the tensor cores may cut off instead of rounding) of
the sum of magnitudes; then the output's rounding (bf16 2^-8, fp32 2^-24)."""
import pytest
import torch

import gated_delta_rule_124_b200 as kda
from gated_delta_rule_124_b200 import build as kbuild

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# (M, N, K, b_block_rows): rows of b per tile, CTAs per tile.  Down projections and
# weight gradients over long batches among them, and sizes that end inside a tile, a
# block of 128 and a 16-byte piece.
SPLIT_256 = {
    (512, 4096, 8192, 128): 2, (512, 4096, 8192, 1): 2, (500, 4001, 8190, 128): 2,
    (500, 4001, 8190, 1): 2, (256, 5120, 6144, 128): 3, (250, 5001, 6100, 1): 3,
    (250, 5001, 6100, 128): 3, (1024, 1024, 16384, 1): 4, (1000, 1010, 16401, 128): 4,
    (64, 6101, 8200, 128): 4, (64, 6101, 8200, 1): 4, (128, 2048, 14336, 128): 8,
    (128, 2048, 14336, 1): 8, (70, 2001, 14401, 128): 8, (17, 2001, 14301, 1): 8,
}
WHOLE_256 = {(4090, 4090, 4101, 1): 1, (3900, 4001, 1000, 1): 1, (2100, 4090, 300, 1): 1,
             (4090, 4090, 4101, 128): 1, (2100, 4090, 300, 128): 1}
OTHERS = {  # the variants of other tests: (rows of b per tile, CTAs per tile)
    (20, 1000, 4100, 128): (128, 8), (130, 2500, 4096, 128): (128, 3),
    (200, 4096, 3000, 1): (128, 2), (513, 1100, 300, 1): (128, 1),
    (16, 5000, 1100, 128): (0, 1), (9, 300, 9000, 128): (0, 8), (13, 4901, 3100, 1): (0, 4),
    (16, 9601, 8200, 1): (0, 2), (8, 9500, 4100, 128): (0, 1), (16, 256, 1024, 128): (-1, 1),
    (2, 4096, 2048, 1): (-1, 1),
}


def test_sizes_take_the_variant_that_they_test():
    kbuild.build()
    for sizes, split in {**SPLIT_256, **WHOLE_256}.items():
        assert kda.kda_test_fp8_matmul_plan(*sizes) == (256, split), sizes
    for sizes, want in OTHERS.items():
        assert kda.kda_test_fp8_matmul_plan(*sizes) == want, sizes


def test_plan_refusals():
    kbuild.build()
    for sizes in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 1, 0)):
        with pytest.raises(RuntimeError):
            kda.kda_test_fp8_matmul_plan(*sizes)
    with pytest.raises(RuntimeError):
        kda.kda_test_fp8_matmul_plan(1, 1, 1, 64)
    # the largest sizes that the library takes, on devices of other sizes
    for sms in (1, 2, 148, 160, 1024):
        for M in (1, 16, 17, 0x7fffff00):
            rows, split = kda.kda_test_fp8_matmul_plan(M, 0x7fffff00, 0x7fffff00, 1, sms)
            assert rows in (-1, 0, 128, 256) and split in (1, 2, 3, 4, 8)


def operands(seed, M, N, K, block):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randn(M, K, generator=gen, device="cuda")
    a *= torch.exp(torch.randn(M, 1, generator=gen, device="cuda"))
    b = torch.randn(N, K, generator=gen, device="cuda")
    return (*kda.quantize_fp8(a), *kda.quantize_fp8(b, block_rows=block))


def values(y8, scale, K, block):
    """The matrix that the codes stand for, in 64 bits."""
    s = scale.double().t().repeat_interleave(block, 0)[:y8.shape[0]]
    return y8[:, :K].double() * s.repeat_interleave(128, 1)[:, :K]


def check(out, a8, sa, b8, sb, K, block, out_dtype):
    a, b = values(a8, sa, K, 1), values(b8, sb, K, block)
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    tol = 2 * (128 + K / 128 + 8 + 3) * U * mag + HALF[out_dtype] * want.abs()
    err = (out.double() - want).abs()
    assert (err <= tol).all(), (err / mag.clamp_min(1e-30)).max()


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,block", [*SPLIT_256, *WHOLE_256])
def test_wide_tiles(M, N, K, block, out_dtype):
    """Tiles of 256 rows of b, whole and split two, three, four and eight ways, with
    the same bits every time."""
    a8, sa, b8, sb = operands(M + N + K, M, N, K, block)
    out = torch.full((M + 2, N), float("nan"), dtype=DT[out_dtype], device="cuda")
    kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=block, out=out[:M])
    check(out[:M], a8, sa, b8, sb, K, block, out_dtype)
    assert torch.isnan(out[M:]).all()     # rows behind the last one stay as they were
    again = torch.empty_like(out[:M])
    for _ in range(20):
        again.zero_()
        kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=block, out=again)
        assert torch.equal(again, out[:M])


@pytest.mark.gpu
@pytest.mark.parametrize("block", [128, 1])
def test_wide_split_tiles_beside_other_work(block):
    """Two products at once, on two streams, each with the bits it has alone."""
    first, second = operands(1, 512, 4096, 8192, block), operands(2, 128, 2048, 14336, block)
    alone = [kda.fp8_matmul(*args, b_block_rows=block, out_dtype=torch.float32)
             for args in (first, second)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(10):
        for stream, args in zip(streams, (first, second)):
            with torch.cuda.stream(stream):
                outs.append(kda.fp8_matmul(*args, b_block_rows=block, out_dtype=torch.float32))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, alone[i % 2])


def test_timeout_hook_refusals():
    kbuild.build()
    fake = 1 << 20
    ok = dict(a8=fake, a_scale=fake, b8=fake, b_scale=fake, M=20, N=64, K=64, b_block_rows=128,
              out_dtype="bf16", out=fake, withheld_cta=0, withheld_block=0, stream=0,
              check=False)
    for change in (dict(withheld_cta=-1), dict(withheld_block=-1), dict(out=None), dict(K=0)):
        assert kda.kda_test_fp8_matmul_timeout(**{**ok, **change}) == kda.KDA_ERR_INVALID_ARG, change
    assert kda.kda_test_fp8_matmul_timeout(**{**ok, "M": 0}) == kda.KDA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,block,cta,withheld", [
    (2100, 4090, 300, 1, 3, 1), (2100, 4090, 300, 128, 3, 4),   # both tiles of a CTA, the second
    (5120, 1024, 130, 1, 4, 3), (9500, 520, 700, 128, 5, 8),
    (20, 1000, 4100, 128, 9, 1), (250, 5001, 6100, 1, 7, 3), (64, 6101, 8200, 128, 2, 0),
    (16, 5000, 1100, 1, 6, 8), (13, 4901, 3100, 128, 5, 2), (9, 300, 9000, 128, 17, 8)])
def test_tiles_whose_waits_give_up_are_nan(M, N, K, block, cta, withheld):
    """One block of one CTA is never loaded: the tile that lacks it and the CTA's later
    ones are NaN throughout, everything else has the bits of the ordinary call, and
    the next call is right again."""
    a8, sa, b8, sb = operands(M + K, M, N, K, block)
    want = kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=block, out_dtype=torch.float32)
    got = torch.zeros_like(want)
    kda.kda_test_fp8_matmul_timeout(a8, sa, b8, sb, M, N, K, block, "f32", got, cta, withheld)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows, split = kda.kda_test_fp8_matmul_plan(M, N, K, block, sms)
    KB, ntm, bn = -(-K // 128), -(-M // 128), rows or 128
    tiles = ntm * -(-N // bn)
    lost = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    if split > 1 or rows == 0:
        rank = cta % split
        assert withheld < KB * (rank + 1) // split - KB * rank // split
        mine = [cta // split]
    else:
        mine = list(range(cta, tiles, min(tiles, sms)))[withheld // KB:]
    assert mine and mine[-1] < tiles
    for t in mine:
        m, n = t % ntm * 128, t // ntm * bn
        lost[m:m + 128, n:n + bn] = True
    assert torch.isnan(got[lost]).all() and torch.equal(got[~lost], want[~lost])
    got.zero_()
    kda.fp8_matmul(a8, sa, b8, sb, K=K, b_block_rows=block, out=got)
    assert torch.equal(got, want)


# sizes of each kernel: without stages (8 and 16 rows), of changed places, 128 and 256
# rows of b a tile, whole and split
EDGE = [(5, 200, 300), (13, 200, 300), (16, 5000, 1100), (9, 300, 9000), (60, 200, 300),
        (20, 1000, 4100), (2100, 4090, 300), (130, 1000, 14500)]


@pytest.mark.gpu
@pytest.mark.parametrize("block", [128, 1])
@pytest.mark.parametrize("sa_log2,sb_log2", [(-63, -63), (-17, -109), (-109, -17), (63, 50), (-100, 119)])
def test_scales_at_the_edges_of_their_range(sa_log2, sb_log2, block):
    """Products of scales that are just normal numbers, and large ones, on codes whose
    sums are small whole numbers: the result is exact."""
    plans = set()
    for M, N, K in EDGE:
        gen = torch.Generator(device="cuda").manual_seed(M)
        pitch, KB = kda.kda_fp8_pitch(K), -(-K // 128)

        def codes(rows):
            y = torch.zeros(rows, pitch, device="cuda")
            y[:, :K] = torch.randint(-1, 2, (rows, K), generator=gen, device="cuda")
            return y
        a, b = codes(M), codes(N)
        sa = torch.full((KB, M), 2.0 ** sa_log2, device="cuda")
        sb = torch.full((KB, N if block == 1 else -(-N // 128)), 2.0 ** sb_log2, device="cuda")
        out = kda.fp8_matmul(a.to(torch.float8_e4m3fn), sa, b.to(torch.float8_e4m3fn), sb, K=K,
                             b_block_rows=block, out_dtype=torch.float32)
        want = (a.double() @ b.double().t()) * 2.0 ** (sa_log2 + sb_log2)
        assert torch.equal(out.double(), want)
        plans.add(kda.kda_test_fp8_matmul_plan(M, N, K, block))
    assert {rows for rows, _ in plans} == {-1, 0, 128, 256}
