"""The norms' gradients of rows of 1 and -1, whose rms is 1 exactly (eps = 0): with whole numbers besides,
dweight and dgate are sums that fp32 holds exactly in any order, and a lost or doubled row shows."""
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


def _whole(shape, top, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(dtype)


# widths of every number of threads a row, whole and not; rows from one to many turns of the blocks
@pytest.mark.parametrize("T,D", [(1, 8), (5000, 8), (20001, 64), (20000, 72), (40001, 128), (9000, 264), (81920, 512),
                                 (3, 520), (9001, 1024), (5000, 1544), (3001, 2048), (2500, 2056), (1999, 4096),
                                 (1300, 5000), (1217, 8192)])
@pytest.mark.parametrize("gate,dtype", [(False, BF), (True, F16)])
def test_gradients_of_whole_numbers(T, D, gate, dtype):
    h = _whole((T, D), 1, 1, dtype)
    h = torch.where(h > 0, 1.0, -1.0).to(dtype)
    w, dy = _whole((D,), 3, 2, dtype), _whole((T, D), 3, 3, dtype)
    g = _whole((T, 4 * D), 2, 4, dtype)[:, :D] if gate else None
    y, _, rstd = hb.rms_norm(h, w, gate=g, eps=0.0)
    H, W, DY, G = h.double(), w.double(), dy.double(), g.double() if gate else 1.0
    assert (rstd == 1).all() and torch.equal(y, (H * W * G).to(dtype))
    dx, dw, dg = hb.rms_norm_bwd(dy, h, rstd, w, gate=g)
    assert torch.equal(dw, (DY * G * H).sum(0).to(dtype))
    assert dg is None if not gate else torch.equal(dg, (DY * H * W).to(dtype))
    if D & (D - 1) == 0:  # the mean is exact too: a sum of whole numbers over a power of two
        t = DY * G * W
        assert torch.equal(dx, (t - H * (t * H).mean(1, keepdim=True)).to(dtype))
