"""The table's gradient of whole numbers, whose sums are exact: runs of sorted tokens that begin and end
anywhere; and embedding rows under unusual scales."""
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import layer_testutil as lt

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("T,D", [(5, 16), (41000, 256)])
def test_rows_that_are_not_named_are_zeros_under_any_scale(T, D):
    t = lt.randn((7, D), BF, 1)
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % 11) - 2  # -2 to 8
    off = (ids < 0) | (ids >= 7)
    for scale in (-2.0, 0.0, 3e38):
        y = hb.embed(t, ids, scale)
        assert (y[off] == 0).all() and torch.equal(y[~off], (t.float() * scale).to(BF)[ids[~off].long()])
    for scale in (float("inf"), float("nan"), 1e300):  # not a float
        with pytest.raises(hb.HstuError) as e:
            hb.embed(t, ids, scale)
        assert e.value.status == 1
