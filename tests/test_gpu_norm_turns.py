"""Gated norms with more parts than one launch has workgroups: the workgroups
take turns.  The input is one row for all tokens (a stride of 0), so that only
the output takes memory and every one of its rows is the same."""
import pytest
import torch

import mamba_ssd_scan_06_amd as ssd
from test_gpu_layer_ops import announce, gen, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,dim", [
    (8 * (1 << 21) + 77, 8),            # 8 lanes per row, eight rows per workgroup
    ((1 << 21) + 3, 2568),              # 128 lanes: sums meet in LDS every turn
    ((1 << 22) + 1, 20488),             # 1024 lanes: 2^32 threads and more without turns
])
def test_parts_beyond_one_launch(rows, dim):
    announce(rows, dim)
    need = 2 * rows * dim
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip(f"needs {need >> 30} GiB of free GPU memory")
    g = gen(121)
    x, w = rnd(g, (1, dim), "bf16"), 1 + rnd(g, (dim,), scale=0.2)
    some = x.expand(8192, dim)           # rows enough for the same lanes per row
    want = ssd.ssd_gated_norm_fwd(some, some, w)[:1].clone()
    out = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    wide = x.expand(rows, dim)
    ssd.ssd_gated_norm_fwd(wide, wide, w, out=out)
    torch.cuda.synchronize()
    step = max(1, (1 << 30) // dim)
    assert torch.isfinite(want).all() and want.any()
    wrong = sum((out[k:k + step] != want).any(1).sum() for k in range(0, rows, step))
    assert int(wrong) == 0
    del out
    torch.cuda.empty_cache()
