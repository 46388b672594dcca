"""The heads' norm of a row with a NaN: the whole row is NaN, as the formula's, elements that are zero too."""
import pytest
import torch

from paged_split_decode_gb300 import inputs
from test_diff_gpu import factors, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("kv,Hq,Hkv,D,qlen", [("f16", 24, 4, 256, 1), ("bf16", 6, 3, 128, 1), ("f16", 12, 2, 256, 3),
                                              ("fp8", 8, 4, 128, 1), ("fp8", 12, 2, 256, 3), ("fp8_bf16q", 12, 2, 128, 4)])
def test_a_nan_row_is_nan(pd, kv, Hq, Hkv, D, qlen, S):
    w = inputs.make_workload(B=3, Hq=Hq, Hkv=Hkv, D=D, seq_lens=[700, 91, 0], qlen=qlen, kv=kv, seed=7,
                             scale=(D // 2) ** -0.5)
    w.v_cache.view(torch.uint8 if w.kv_fp8 else torch.int16)[..., 3:9] = 0  # dims that are zero in every row
    lam, weight = factors(w)
    want = run(pd, w, lam, S, weight).clone()
    assert (want[..., 3:9] == 0).all()
    at = (int(w.block_table[0, 2]), 5, Hkv - 1, 77)
    if w.kv_fp8:
        w.v_cache.view(torch.uint8)[at] = 0x7F
    else:
        w.v_cache[at] = float("nan")
    got = run(pd, w, lam, S, weight)
    G = Hq // Hkv
    assert torch.isnan(got[:qlen, Hq - G:]).all()
    got[:qlen, Hq - G:] = want[:qlen, Hq - G:]
    assert torch.equal(got, want)
