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


def _runs(lengths, seed):
    """ids of `lengths[v]` tokens each, in a random order."""
    ids = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths))
    g = torch.Generator()
    g.manual_seed(seed)
    return ids[torch.randperm(len(ids), generator=g)]


C = 16  # tokens of a chunk at these sizes (64 for the longest runs of the widest rows)
# Runs of sorted tokens by where they begin and end in chunks: within one, over the end of one, whole chunks
# with and without ends, 15, 16 and 17 whole chunks (16 are joined by one group of threads), more than 1024.
RUNS = {
    "short": [3, 0, 14, 16, 15, 17, 1, 31, 16, 16, 32, 5, 0, 48, 33],
    "sixteen chunks": [5, C * 15, C * 16, C * 17, 3, C * 15 + 7, C * 16 + 9, C * 17 + 1, 12, C * 14 + 31, C * 15 + 31, 0,
                       C * 16 + 31, 4, C * 15, C * 16, C * 17],
    "sixteen chunks, many tokens": [5, C * 15, C * 16, C * 17, 3, C * 15 + 7, C * 16 + 9, C * 17 + 1, 12] * 4,
    "aligned": [C * 16, C * 15, C * 17, C, 2 * C, C * 1025],
    "long": [7, C * 1024, 2, C * 1025 + 3, C * 1030 + 15, 0, 9, C * 2100, C * 16, 1],
    "one": [0, C * 1500 + 5],
}


@pytest.mark.parametrize("D,dtype,grad", [(8, BF, F32), (520, F16, F32), (72, BF, BF), (2056, F16, F16)])
@pytest.mark.parametrize("runs", list(RUNS))
@pytest.mark.parametrize("padding", [0, 37])
def test_gradient_of_whole_numbers(D, dtype, grad, runs, padding):
    """Sums of whole numbers below 2^24, and a scale that is a power of two: exact in any order, one
    rounding to a 16-bit gradient, and a lost or doubled chunk shows."""
    lengths = RUNS[runs]
    V = len(lengths)
    ids = _runs(lengths + [padding], 1).int().cuda()
    ids[ids == V] = -1
    T = len(ids)
    dy = torch.randint(-8, 9, (T, D), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(dtype)
    ref = torch.zeros((V + 1, D), dtype=torch.float64, device="cuda").index_add_(0, ids.long() % (V + 1), dy.double())[:V]
    got = hb.embed_bwd(dy, ids, V, 0.5, dtype=grad)
    assert torch.equal(got, (0.5 * ref).to(grad))
    if grad == F32:
        base = torch.arange(V * D, device="cuda", dtype=torch.float32).view(V, D)
        out = base.clone()
        hb.embed_bwd(dy, ids, V, 0.5, out=out, accumulate=True)
        assert torch.equal(out, (base.double() + 0.5 * ref).float())
