"""GPU test of the rotation beside values that are not finite: dimensions behind
the rotated part come back as they are, whatever they or their neighbours hold."""
import math

import numpy as np
import pytest

from gpu_util import announce, bits
from test_gpu_single import DT, _part, nt  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 32), (40, 10), (64, 48), (16, 2), (128, 16)])
def test_unrotated_dimensions_stay(nt, D, R, interleaved, dtype):  # noqa: F811
    announce(f"rotation beside infinities {D} {R} {interleaved} {dtype}")
    t = getattr(torch, DT[dtype])
    gen = torch.Generator().manual_seed(71)
    x = torch.randn((9, 3, D), generator=gen).to(t).cuda()
    for i, v in enumerate((math.inf, -math.inf, math.nan)):
        x[1 + i, :, R] = v
        x[5, i, D - 1 - i] = v
    p = _part(nt, [9])
    table = nt.nt_rotary_table(9, R)
    out, _ = nt.nt_qk_norm_rotary(p, x, table=table, interleaved=interleaved)
    g, _, _, _ = nt.nt_qk_norm_rotary_backward(p, x, None, x, table=table, interleaved=interleaved)
    clean = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    want, _ = nt.nt_qk_norm_rotary(p, clean, table=table, interleaved=interleaved)
    back, _, _, _ = nt.nt_qk_norm_rotary_backward(p, clean, None, clean, table=table,
                                                  interleaved=interleaved)
    torch.cuda.synchronize()
    for y, z in ((out, want), (g, back)):
        assert torch.equal(torch.isnan(y[..., R:]), torch.isnan(x[..., R:]))
        fine = ~torch.isnan(x[..., R:])
        assert torch.equal(y[..., R:][fine], x[..., R:][fine])
        # the rotated part does not see them
        np.testing.assert_array_equal(bits(y[..., :R].contiguous(), torch),
                                      bits(z[..., :R].contiguous(), torch))
