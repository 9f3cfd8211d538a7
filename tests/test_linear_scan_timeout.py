"""The bounded waits of the gated linear recurrence, without any fault: one tile is
never run, and the calls that need it report KDA_ERR_TIMEOUT."""
import pytest
import torch

import gated_delta_rule_124_b200 as kda
from gated_delta_rule_124_b200 import build as kbuild


def test_timeout_hook_refusals():
    kbuild.build()
    fake = 1 << 20
    ok = dict(x=fake, g=fake, dout=None, entry_states=None, T=300, H=1, d=4, dtype="bf16", out=fake,
              dg=None, workspace=fake, wait_ns=1000, workspace_bytes=1 << 30, stream=0, check=False)
    for change in (dict(wait_ns=0), dict(wait_ns=2 * 10 ** 9 + 1), dict(T=256), dict(out=None),
                   dict(dout=fake), dict(H=0), dict(workspace=fake + 16)):
        assert kda.kda_test_linear_scan_timeout(**{**ok, **change}) == kda.KDA_ERR_INVALID_ARG, change
    assert (kda.kda_test_linear_scan_timeout(**{**ok, "workspace_bytes": 16})
            == kda.KDA_ERR_WORKSPACE)


# one channel a lane, groups of six, of three and of one tile
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,d", [(700, 1, 31), (500, 2, 64), (1000, 5, 128), (300, 16, 128)])
@pytest.mark.parametrize("form", ["forward", "backward", "backward without entry states"])
def test_a_tile_that_never_comes_is_reported(form, T, H, d, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, dout = (torch.randn(T, H, d, generator=gen, device="cuda").to(dtype) for _ in range(2))
    g = -torch.rand(T, H, d, generator=gen, device="cuda")
    h, _, entry = kda.linear_scan(x, g, output_entry_states=True)
    dx, dg, _ = kda.linear_scan_bwd(x, g, dout, entry_states=entry)
    forward = form == "forward"
    size = (kda.kda_linear_scan_workspace_size if forward
            else kda.kda_linear_scan_bwd_workspace_size)(T, H, d)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    out, out_g = torch.empty_like(x), torch.empty_like(g)
    given = entry if form == "backward" else None
    kda.kda_test_linear_scan_timeout(x, g, None if forward else dout, given, T, H, d, dtype, out,
                                     None if forward else out_g, ws, wait_ns=20_000_000)
    assert kda.kda_get_device_status(ws) == kda.KDA_ERR_TIMEOUT
    # the next call on the same workspace starts clean
    if forward:
        got, _ = kda.linear_scan(x, g, workspace=ws)
        assert torch.equal(got, h)
    else:
        got, got_g, _ = kda.linear_scan_bwd(x, g, dout, entry_states=given, workspace=ws)
        assert torch.equal(got, dx) and torch.equal(got_g, dg)
    assert kda.kda_get_device_status(ws) == kda.KDA_OK


@pytest.mark.gpu
def test_bad_offsets_are_reported_by_a_backward_without_entry_states():
    T, H, d = 300, 2, 64
    x = torch.ones(T, H, d, device="cuda")
    g = -torch.ones(T, H, d, device="cuda")
    ws = torch.zeros(kda.kda_linear_scan_bwd_workspace_size(T, H, d), dtype=torch.uint8,
                     device="cuda")
    for offsets, want in (([0, 200, 100, T], kda.KDA_ERR_BAD_SEQLENS), ([0, 100, 200, T], kda.KDA_OK)):
        cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        kda.linear_scan_bwd(x, g, x, cu_seqlens=cu, workspace=ws)
        assert kda.kda_get_device_status(ws) == want
