"""NaN and infinities in V of keys that a query row does not see: they change no bit
of that row, and show in the rows that see them."""
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


def plant(w, b, key, head, dim, value):
    at = (int(w.block_table[b, key // 16]), key % 16, head, dim)
    if w.kv_fp8:
        w.v_cache.view(torch.uint8)[at] = 0x7F if dim % 2 else 0xFF
    else:
        w.v_cache[at] = value


def check(pd, w, planted, S, norm):
    """planted: (sequence, key, KV head, dim, value). Every row against the run without them."""
    lam, weight = factors(w)
    weight = weight if norm else None
    want = run(pd, w, lam, S, weight).clone()
    nan = torch.zeros(want.shape, dtype=torch.bool)
    G = w.Hq // w.Hkv
    starts = w.q_start.tolist() if w.q_start is not None else [b * w.qlen for b in range(w.B + 1)]
    for b, key, head, dim, value in planted:
        plant(w, b, key, head, dim, value)
        n, L = starts[b + 1] - starts[b], int(w.seq_lens[b])
        for i in range(n):
            last = L - n + i
            if key <= last and (w.window <= 0 or key > last - w.window):
                rows = nan[starts[b] + i, head * G:(head + 1) * G]
                rows[:, slice(None) if norm else dim] = True  # (the norm spreads it over the head)
    got = run(pd, w, lam, S, weight)
    assert torch.equal(torch.isnan(got).cpu(), nan)
    assert torch.equal(got[~nan], want[~nan])
    return int(nan.sum())


CASES = [("f16", 24, 4, 256, 3), ("f16", 8, 4, 128, 2), ("bf16", 12, 2, 128, 2), ("bf16", 6, 3, 256, 5),
         ("f16", 8, 2, 256, 8), ("bf16", 8, 1, 256, 4), ("fp8", 24, 4, 256, 3), ("fp8_bf16q", 12, 2, 128, 4),
         ("fp8", 8, 4, 128, 2), ("fp8", 4, 2, 256, 3), ("fp8", 8, 1, 128, 4), ("fp8", 12, 2, 256, 2), ("f16", 6, 2, 128, 1),
         ("fp8", 24, 4, 256, 1), ("fp8", 16, 1, 256, 1), ("bf16", 24, 2, 128, 1), ("fp8", 32, 2, 128, 2)]


@pytest.mark.parametrize("norm", (False, True))
@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("kv,Hq,Hkv,D,qlen", CASES)
def test_later_tokens_of_a_verify(pd, kv, Hq, Hkv, D, qlen, S, norm):
    """The newest keys, which the earlier query tokens do not see; sequences that end
    at a tile's start, its end and inside it, and one of new tokens only."""
    lens = [700, 705, 704, qlen, 1041]
    w = inputs.make_workload(B=5, Hq=Hq, Hkv=Hkv, D=D, seq_lens=lens, qlen=qlen, kv=kv, seed=3, scale=(D // 2) ** -0.5)
    bad = [(b, L - 1 - (b + k) % qlen, (b + k) % Hkv, (37 * b + 61 * k) % D, (float("nan"), float("inf"), -float("inf"))[k % 3])
           for b, L in enumerate(lens) for k in range(4)]
    assert check(pd, w, bad, S, norm) > 0


@pytest.mark.parametrize("window", (1, 2, 16, 90, 333))
@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("kv,Hq,Hkv,D,qlen", CASES)
def test_around_a_window(pd, kv, Hq, Hkv, D, qlen, window, S):
    """Keys just before the window of the first query token (seen by no row), and those that leave
    it between the first and the last."""
    lens = [700, 705, 704, 2, 1041]
    w = inputs.make_workload(B=5, Hq=Hq, Hkv=Hkv, D=D, seq_lens=[max(L, qlen) for L in lens], qlen=qlen, window=window,
                             kv=kv, seed=5, scale=(D // 2) ** -0.5)
    bad = []
    for b, L in enumerate(w.seq_lens.tolist()):
        first = L - qlen - window + 1
        for k, key in enumerate((first - 1, first - 2, first - 9, first, first + 1, first + qlen - 2, L - 1)):
            if 0 <= key < L:
                bad.append((b, key, (b + k) % Hkv, (29 * b + 17 * k) % D, float("nan") if k % 2 else float("inf")))
    check(pd, w, bad, S, False)


@pytest.mark.parametrize("kv", ("f16", "fp8", "fp8_bf16q"))
def test_varlen(pd, kv):
    w = inputs.make_varlen_workload(B=6, qlens=[1, 0, 4, 2, 3, 4], Hq=24, Hkv=4, D=256,
                                    seq_lens=[500, 40, 1200, 0, 3, 768], kv=kv, seed=19, scale=128 ** -0.5)
    bad = [(2, 1199, 0, 5, float("nan")), (2, 1198, 1, 6, float("inf")), (4, 2, 2, 100, float("nan")),
           (5, 767, 3, 255, float("nan")), (0, 499, 1, 0, float("nan")), (5, 765, 3, 128, float("inf"))]
    assert check(pd, w, bad, 0, True) > 0
