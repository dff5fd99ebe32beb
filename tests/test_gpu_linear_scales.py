"""8-bit linear maps whose rows lie far from one another in magnitude: a scale of 2^119 against one of
2^-20 and the like, whose product is ordinary."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import layer_testutil as lt

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _check(qx, qw, y):
    X = lt.e4m3(qx.codes) * lt.scale_of(qx.scale)[:, None]
    W = lt.e4m3(qw.codes) * lt.scale_of(qw.scale)[:, None]
    ref, err = X @ W.T, lt.product_err(X, W.T)
    # past the range of the type: infinities of the sign
    top = float(torch.finfo(BF).max)
    inside = np.abs(ref) + err <= top
    got = lt.f64(y)
    tol = err + lt.half_step(BF) * (np.abs(ref) + err) + lt.smallest_half_step(BF)
    assert lt.worst(got[inside], ref[inside], tol[inside]) <= 1.0
    past = np.abs(ref) - err > top * (1 + 2.0 ** -8)
    assert np.isinf(got[past]).all()
    return inside


# few rows, pairs of SMs
@pytest.mark.parametrize("T,K,N", [(9, 64, 72), (600, 256, 1032)])
def test_rows_that_hold_the_lowest_value(T, K, N):
    """A mask's value in one place of every third row; the weights are small."""
    x, w = lt.randn((T, K), BF, 1), lt.randn((N, K), BF, 2, 2.0 ** -20)
    x[::3, 5] = torch.finfo(BF).min
    qx, qw = hb.quantise_rows(x), hb.quantise_rows(w)
    y, z = hb.linear(qx, qw, act="relu", want_z=True)
    assert _check(qx, qw, z).all() and torch.equal(y, z.clamp(min=0))


@pytest.mark.parametrize("T,K,N", [(9, 64, 72), (600, 256, 1032)])
def test_scales_of_all_sizes(T, K, N):
    x, w = lt.randn((T, K), BF, 3).float(), lt.randn((N, K), BF, 4).float()
    r = np.random.default_rng(5)
    to = lambda n, lo, hi: torch.tensor(np.exp2(r.integers(lo, hi, n)), dtype=torch.float32, device="cuda")[:, None]  # noqa: E731
    # x anywhere in the type's range, w where the header says that the sums stay exact
    qx, qw = hb.quantise_rows((x * to(T, -120, 125)).to(BF)), hb.quantise_rows((w * to(N, -98, 97)).to(BF))
    assert 19 <= int(qw.scale.min()) and int(qw.scale.max()) <= 221
    inside = _check(qx, qw, hb.linear(qx, qw)[0])
    assert 0.4 < inside.mean() < 1.0
