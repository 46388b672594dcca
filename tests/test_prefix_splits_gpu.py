"""The automatic split of a call with prefixes: how long they are is known on the device alone, so that a long prefix beside
a small window is spread as widely as the same keys without a window."""
import pytest
import torch

from ref_scored import Work, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


def pieces(pd, w, window, prefix):
    """How many partial rows of (m, l) the decode left in its workspace, and the call's outputs."""
    from paged_split_decode_gb300 import binding
    d = binding.make_dims(w.B, w.Hq, w.Hkv, w.D, w.bs, w.caches[0].shape[0], w.table.shape[1], kv_bf16=w.kv == "bf16")
    if w.kv == "fp4":
        d.kv_dtype = binding.PD_KV_FP4
    need = binding.scored_workspace_bytes(d, w.qlen, 0)
    ws = torch.full((need // 4,), -77.0, device="cuda")
    w.window, w.prefix = window, prefix
    got = w.run(pd, weights=False, workspace=ws)
    return int((ws != -77.0).sum()) / (w.D + 2) / (w.Hq // w.Hkv * w.qlen), got


@pytest.mark.parametrize("kv,Hq,Hkv,D,qlen", [("f16", 24, 4, 256, 1), ("bf16", 8, 2, 128, 3), ("fp4", 24, 4, 256, 1), ("fp4", 32, 8, 128, 1)])
@pytest.mark.parametrize("window", (16, 200))
def test_long_prefix_beside_a_window(pd, kv, Hq, Hkv, D, qlen, window):
    w = Work(kv, Hq, Hkv, D, [8192], qlen=qlen, seed=31)
    free, _ = pieces(pd, w, 0, None)
    wide, got = pieces(pd, w, window, torch.tensor([8000], dtype=torch.int32))
    assert wide >= 0.5 * free and free > 16  # (as many tiles but for the gap's)
    check(w, got)


@pytest.mark.parametrize("kv", ("f16", "fp4"))
def test_short_prefixes_and_long_tables(pd, kv):
    """A few keys at the start beside a window, in tables of many more."""
    w = Work(kv, 24, 4, 256, [5000, 40, 1], seed=32)
    w.table = torch.cat([w.table, torch.full((3, 2000), -1, dtype=torch.int32)], 1)
    for window in (1, 300):
        for prefix in ([4, 4, 0], [0, 0, 0]):
            w.window, w.prefix = window, torch.tensor(prefix, dtype=torch.int32)
            check(w, w.run(pd))
