"""Workspaces of the selective scan and of draft verification, on the host: the
shapes below are split by the library's rules, so that too small, missing,
misaligned and overlapping workspaces have to be refused (no GPU needed)."""
import pytest

import mamba_ssd_scan_06_amd as ssd
from test_layer_refusals import BF16, ERR_ALIAS, ERR_ALIGN, ERR_WORKSPACE, F32, Scan, Verify


def queries():
    scan = Scan(b=1, T=4096, D=64, G=1)
    verify = Verify(b=1, V=200000)
    verify.dtype = F32
    return {"scan": (scan, ssd.ssd_selective_scan_workspace_bytes(scan.shape, BF16), ("y", "final", "u", "init")),
            "verify": (verify, ssd.ssd_verify_workspace_bytes(verify.shape, F32), ("n", "tokens", "p", "u"))}


@pytest.mark.parametrize("op", ["scan", "verify"])
def test_workspaces_are_refused(op):
    call, need, others = queries()[op]
    assert need > 0
    call.scalars["ws_bytes"] = need - 1
    assert call() == ERR_WORKSPACE
    call.scalars["ws_bytes"] = 0
    assert call() == ERR_WORKSPACE
    call.scalars["ws_bytes"] = need
    where, call.p["ws"] = call.p["ws"], None
    assert call() == ERR_WORKSPACE
    call.p["ws"] = where + 8
    assert call() == ERR_ALIGN
    for k in others:
        call.p["ws"] = call.p[k]
        assert call() == ERR_ALIAS, k
        call.p["ws"] = call.p[k] - need + 16             # its last bytes reach into the other
        if call.p["ws"] % 16 == 0:
            assert call() == ERR_ALIAS, k


def ranges_of(b, T, D, N, G):
    """The number of token ranges, from the workspace: each range's states and
    sums of steps, the states rounded up to 256 bytes."""
    need = ssd.ssd_selective_scan_workspace_bytes(Scan(b=b, T=T, D=D, N=N, G=G).shape, BF16)
    for r in range(2, 800):
        if (4 * r * b * D * N + 255) // 256 * 256 + 4 * r * b * D == need:
            return r
    assert need == 0
    return 1


@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_ranges_fit_the_workspace_and_the_tiles(N):
    # Either no ranges or three and more, each but the last of whole tiles of
    # 32 tokens, none of them empty; none for sixteen tokens and fewer, none
    # where the channels fill the GPU.
    for b, D in ((1, 64), (1, 1536), (2, 1000), (1, 5120), (2, 3584), (2, 5120), (3, 4096), (8, 5120)):
        wgs = b * ((D + 63) // 64)
        for T in [1, 16, 17, 32, 33, 64, 65, 127, 128, 129, 160, 161, 192, 193, 255, 288, 289, 320, 513, 515, 1000, 2048, 4093]:
            r = ranges_of(b, T, D, N, 1)
            assert r != 2 and (r == 1 or T > 16 and wgs < 193), (b, D, T, r)
            if r > 1:
                assert any(-(-T // (32 * k)) == r for k in range(1, T // 32 + 2)), (b, D, T, r)
