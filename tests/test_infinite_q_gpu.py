"""Infinite elements of q, over every cache kind, one and several query tokens, whole and split units: the row that has
them comes out as the definition says, and no bit of another row changes."""
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


def plant(w, qlen, several):
    """An infinite element (or three) in one row of each sequence; the rows, [T, Hq]."""
    hit = torch.zeros(w.q.shape[:2], dtype=torch.bool)
    for b in range(len(LENS)):
        row, head = b * qlen + (b + 1) % qlen, (5 * b + 3) % w.Hq
        for i, d in enumerate((17, 100, 101) if several else (17 + b,)):
            w.q[row, head, d] = -math.inf if (b + i) % 2 else math.inf
        hit[row, head] = True
    return hit


@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("qlen", (1, 3))
@pytest.mark.parametrize("kv,q", KINDS + [("fp4", "f16"), ("fp4", "bf16")])
def test_scored(pd, kv, q, qlen, S):
    """Scores of +infinity are there (the keys' elements have either sign): the row is NaN."""
    for Hq, Hkv, D in ((24, 4, 256), (12, 2, 128)):
        for several in (False, True):
            w = Work(kv, Hq, Hkv, D, LENS, qlen=qlen, q=q, seed=21)
            want = w.run(pd, S)
            hit = plant(w, qlen, several)
            got = w.run(pd, S)
            assert torch.equal(torch.isnan(got[0]).cpu(), hit[..., None].expand(w.q.shape))
            assert torch.equal(got[0].cpu()[~hit], want[0].cpu()[~hit])
            assert torch.equal(got[1].cpu()[~hit], want[1].cpu()[~hit])
            assert not bool(torch.isfinite(got[1].cpu()[hit]).any()) and got[3] == 0


@pytest.mark.parametrize("qlen", (1, 3))
@pytest.mark.parametrize("kv,q", KINDS + [("fp4", "f16"), ("fp4", "bf16")])
def test_capped(pd, kv, q, qlen):
    """A cap makes scores of +-cap of infinite ones: numbers again, unless a visible key's element is zero (0 times infinity)."""
    w = Work(kv, 24, 4, 256, LENS, qlen=qlen, q=q, cap=3.0, seed=22)
    hit = plant(w, qlen, False)
    out, lse, _, flag = w.run(pd)
    r_out, bound, r_lse, b_lse, _, _ = w.reference()
    nan = torch.isnan(r_out)
    assert flag == 0 and torch.equal(torch.isnan(out).cpu(), nan)
    if kv in ("f16", "bf16", "fp8"):
        assert not bool(nan.any())  # (no zero among the keys' elements)
    else:
        assert bool(nan[hit].all())
    assert bool(((out.double().cpu() - r_out).abs()[~nan] <= bound[~nan]).all())
    rows = ~nan[..., 0]
    assert bool(((lse.double().cpu() - r_lse).abs()[rows] <= b_lse[rows]).all())
