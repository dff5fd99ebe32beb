"""Sums of the linear maps' gradients: the bias gradient against sums of terms that no rounding
to 16 bits touched, and whole numbers, whose sums are exact."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import layer_testutil as lt

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("T,N", [(300, 264), (61, 2584), (1200, 8)])
@pytest.mark.parametrize("act,dtype", [("silu", BF), ("gelu", F16), ("gelu", BF), ("silu", F16)])
def test_bias_gradient_sums_before_the_rounding_to_16_bits(T, N, act, dtype):
    x, w = lt.randn((T, 16), dtype, 1), lt.randn((N, 16), dtype, 2)
    z, dy = lt.randn((T, N), dtype, 3, 2.0), lt.randn((T, N), dtype, 4)
    db = hb.linear_bwd(dy, z, x, w, act=act)[2]
    Z, DY = lt.f64(z), lt.f64(dy)
    g = DY * lt.act_grad(Z, act)
    eg = np.abs(DY) * lt.act_grad_err(Z, act) + 2 * lt.STEP32 * np.abs(g)
    # a thread's chain of rows (at most T / 152 + 4 of these sizes), halves of 256 threads, 152 / 32
    # chunks a warp, 32 warps: below 64 sums behind one another, an fp32 rounding each
    err = eg.sum(0) + 64 * lt.STEP32 * (np.abs(g) + eg).sum(0)
    ref = g.sum(0)
    tol = err + lt.half_step(dtype) * (np.abs(ref) + err) + lt.smallest_half_step(dtype)
    assert lt.worst(lt.f64(db), ref, tol) <= 1.0


def test_bias_gradient_of_terms_below_the_smallest_half():
    """Each term would round to zero in fp16; their sum does not."""
    T, N = 4096, 64
    x, w = lt.randn((T, 16), F16, 1), lt.randn((N, 16), F16, 2)
    dy = torch.full((T, N), 2.0 ** -24, dtype=F16, device="cuda")  # the smallest subnormal
    z = torch.full((T, N), -0.5, dtype=F16, device="cuda")
    db = lt.f64(hb.linear_bwd(dy, z, x, w, act="silu")[2])
    ref = T * 2.0 ** -24 * float(lt.act_grad(np.float64(-0.5), "silu"))  # 6.3e-5, a normal fp16 number
    assert np.abs(db - ref).max() <= 2.0 ** -11 * ref + 1e-5 * ref
