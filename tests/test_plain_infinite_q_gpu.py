"""decode_paged with an infinite element of q, one and several query tokens, whole and split units: the row that has it is
NaN, and no bit of another row changes."""
import math

import pytest
import torch

from ref_scored import Work

pytestmark = pytest.mark.gpu

KINDS = [("f16", "f16"), ("bf16", "bf16"), ("fp8", "f16"), ("fp8", "bf16"), ("int8", "f16"), ("int8", "bf16")]
LENS = [500, 130, 700]


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


def plant(w, qlen):
    """An infinite element in one row of each sequence; the rows, [T, Hq]."""
    hit = torch.zeros(w.q.shape[:2], dtype=torch.bool)
    for b in range(len(LENS)):
        row, head = b * qlen + (b + 1) % qlen, (5 * b + 3) % w.Hq
        w.q[row, head, 17 + b] = -math.inf if b % 2 else math.inf
        hit[row, head] = True
    return hit


@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("qlen", (1, 3))
@pytest.mark.parametrize("kv,q", KINDS)
def test_rows(pd, kv, q, qlen, S):
    for Hq, Hkv, D in ((24, 4, 256), (12, 2, 128)):
        w = Work(kv, Hq, Hkv, D, LENS, qlen=qlen, q=q, seed=23)
        if kv == "fp8":  # (small codes: their multiples of a large finite number would not overflow by themselves)
            w.caches[0] = w.caches[0].float().clamp(-100, 100).to(w.caches[0].dtype)
        up = lambda t: t.cuda()
        run = lambda: pd.decode_paged(up(w.q), up(w.caches[0]), up(w.caches[1]), up(w.table), up(w.lens), w.scale, qlen=qlen,
                                      num_splits=S, k_scale=w.c_scale, v_scale=w.c_scale).cpu()
        want = run()
        hit = plant(w, qlen)
        got = run()
        assert torch.equal(torch.isnan(got), hit[..., None].expand(w.q.shape))
        assert torch.equal(got[~hit], want[~hit])
