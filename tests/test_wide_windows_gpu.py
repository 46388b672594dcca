"""Windows at and beyond a table's capacity, up to the largest integer: none at all, also for
sequences shorter than their query tokens."""
import pytest
import torch

from paged_split_decode_gb300 import inputs
from test_diff_gpu import DEV, caches, factors, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


@pytest.mark.parametrize("window", (48, 49, 2 ** 30, 2 ** 31 - 9, 2 ** 31 - 1))
@pytest.mark.parametrize("S", (0, 1, 2))
@pytest.mark.parametrize("kv,Hq,Hkv,D,qlen", [("f16", 4, 4, 128, 8), ("bf16", 4, 2, 256, 8), ("fp8", 8, 2, 256, 8), ("int8", 4, 1, 128, 8),
                                              ("fp8_bf16q", 2, 2, 128, 5)])
def test_a_wide_window_is_none(pd, kv, Hq, Hkv, D, qlen, S, window):
    w = inputs.make_workload(B=6, Hq=Hq, Hkv=Hkv, D=D, seq_lens=[1, 3, 0, 48, 17, 2], qlen=qlen, kv=kv, seed=3,
                             scale=(D // 2) ** -0.5)
    lam, weight = factors(w)
    want = run(pd, w, lam, S, weight)
    plain = lambda: pd.decode_paged(w.q.to(DEV), *caches(w), w.block_table.to(DEV), w.seq_lens.to(DEV), w.scale, w.window,
                                    qlen, S, k_scale=w.k_scale, v_scale=w.v_scale)
    plain_want = plain()
    w.window = window
    assert torch.equal(run(pd, w, lam, S, weight), want)
    assert torch.equal(plain(), plain_want)
