"""GPU test of the 8-bit states bit by bit: scales and codes are those that the
formulas give in separately rounded fp32, here formed in numpy on the host."""
import numpy as np
import pytest

from gpu_util import announce
from test_gpu_single import nt  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

F = np.float32
UNIT = F(1.0) / F(448.0)  # a scale is the block's largest magnitude times this number


def _codes(x, positive):
    """(codes, scales) of fp32 values, 256 to a block."""
    n = len(x)
    b = np.concatenate([x, np.zeros(-n % 256, F)]).reshape(-1, 256)
    scale = np.abs(b).max(1) * UNIT
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(scale[:, None] > 0, b / scale[:, None], F(0.0))
    y = np.clip(y, F(-448.0), F(448.0))
    if positive:
        y = np.where(b > 0, np.maximum(y, F(2.0 ** -9)), y)
    c = torch.from_numpy(y.reshape(-1)[:n].copy()).to(torch.float8_e4m3fn)
    return c, scale


def _values(c, scale):
    return c.float().numpy() * np.repeat(scale, 256)[:len(c)]


@pytest.mark.parametrize("seed", range(3))
def test_states_bit_by_bit(nt, seed):  # noqa: F811
    announce(f"adamw codes bit by bit {seed}")
    rng = np.random.default_rng(80 + seed)
    n, b1, b2 = 256 * 400 + 77, 0.9, 0.99
    w = torch.zeros(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    m, v, ms, vs = nt.nt_adamw_states([w], 8)
    h = nt.nt_adamw_tensors([w], [g], m, v, ms, vs)
    cm = cv = torch.zeros(n, dtype=torch.float8_e4m3fn)
    sm = sv = np.zeros(401, F)
    inexact = 0
    for step in (1, 2, 3):
        x = (rng.normal(size=n) * 10.0 ** rng.integers(-4, 3, n)).astype(F)
        g.copy_(torch.from_numpy(x))
        nt.nt_adamw_step(h, step, lr=0.0, beta1=b1, beta2=b2)
        a = F(b1) * _values(cm, sm) + F(1.0 - b1) * x
        r = _values(cv, sv)
        q = F(b2) * (r * r) + F(1.0 - b2) * x * x
        cm, sm = _codes(a, False)
        cv, sv = _codes(np.sqrt(q), True)
        top = np.abs(np.concatenate([a, np.zeros(-n % 256, F)])).reshape(-1, 256).max(1)
        inexact += int((top * UNIT != top / F(448.0)).sum())
        torch.cuda.synchronize()
        for got, want in ((ms[0], sm), (vs[0], sv)):
            np.testing.assert_array_equal(got.cpu().numpy().view(np.uint32), want.view(np.uint32))
        for got, want in ((m[0], cm), (v[0], cv)):
            np.testing.assert_array_equal(got.view(torch.uint8).cpu().numpy(),
                                          want.view(torch.uint8).numpy())
    assert inexact > 400  # the product with the reciprocal and the quotient are not the same
