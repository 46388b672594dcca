"""Which calls of the differential decode split their units: a unit that its own CTA
finishes writes no partials, so the workspace shows it."""
import pytest
import torch

from paged_split_decode_gb300 import inputs
from test_diff_gpu import DEV, parity

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


# tables of at most eight steps of a CTA (two tiles a step for a warp that takes two,
# times the key groups) stay whole where the SMs are many units' -- three row tiles, four
# tiles a step; one row tile at D = 128, two tiles -- and few units are cut
@pytest.mark.parametrize("B,Hq,Hkv,D,qlen,L,whole", [
    (38, 24, 4, 256, 3, 512, True), (38, 24, 4, 256, 3, 528, False), (100, 24, 4, 256, 2, 400, True),
    (76, 32, 8, 128, 1, 256, True), (76, 32, 8, 128, 1, 272, False), (1, 24, 4, 256, 3, 256, False),
    (1, 32, 8, 128, 1, 128, False)])
def test_units_of_short_tables(pd, B, Hq, Hkv, D, qlen, L, whole):
    w = inputs.make_workload(B=B, Hq=Hq, Hkv=Hkv, D=D, seq_lens=[L - i % 30 for i in range(B)], qlen=qlen, kv="f16",
                             seed=B + L, scale=(D // 2) ** -0.5)
    need = pd.diff_workspace_bytes(pd.dims_of(w.q, w.k_cache, w.block_table, qlen), qlen, 0)
    ws = torch.full((need,), 0xAB, dtype=torch.uint8, device=DEV)
    parity(pd, w, norm=True, workspace=ws)
    assert bool((ws == 0xAB).all()) == whole
