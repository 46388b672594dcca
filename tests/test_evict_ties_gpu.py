"""Weights that are equal as numbers are ties, whatever their sign bit: of zeros of either sign the lower index stays."""
import pytest
import torch

from test_evict_gpu import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", ([300, 65, 90], [9000]))
def test_zeros_of_either_sign_are_ties(lens):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    values = torch.tensor([0.0, -0.0, -0.0, 0.0, -0.0, 1e-45, -1e-45, 2.0])
    for top in (2, 5, 8):  # zeros only; a few weights beside them
        p = Pool("int8", len(lens), 1, 64, 16, lens, seed=top)
        p.w = values[torch.randint(0, top, p.w.shape, generator=torch.Generator().manual_seed(top))]
        want = p.expect(60, first=1, recent=4)
        got, _, flag = p.evict(pd, 60, first=1, recent=4)
        assert flag == 0 and torch.equal(got, want[2])
        p.check(want)
