"""The differential decode where numbers are extreme: infinite queries and keys."""
import pytest
import torch

import ref_diff
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


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("S", (0, 1, 3))
@pytest.mark.parametrize("sign", (1.0, -1.0))
@pytest.mark.parametrize("kv,qlen", [("f16", 1), ("f16", 3), ("bf16", 1), ("bf16", 3), ("fp8", 1), ("fp8", 3),
                                     ("fp8_bf16q", 1), ("fp8_bf16q", 4), ("int8", 1), ("int8", 3), ("int8_bf16q", 3)])
@pytest.mark.parametrize("Hkv", (2, 4))
def test_an_infinite_query_silences_its_map(pd, Hkv, kv, qlen, sign, S):
    """An infinity in a half of a query row makes every score of that map +infinity,
    -infinity or NaN: no softmax exists, the map contributes zeros."""
    w = inputs.make_workload(B=2, Hq=6 * Hkv, Hkv=Hkv, D=256, seq_lens=[700, 91], qlen=qlen, kv=kv, seed=89,
                             scale=128 ** -0.5)
    lam, _ = factors(w)
    want, alone = run(pd, w, lam, S), run(pd, w, torch.zeros(6 * Hkv), S)
    w.q[1, 7, 200] = sign * float("inf")
    want[1, 7] = alone[1, 7]
    assert torch.equal(run(pd, w, lam, S), want)
    w.q[1, 7, 20] = -sign * float("inf")
    want[1, 7] = 0
    assert torch.equal(run(pd, w, lam, S), want)


@pytest.mark.parametrize("code", (0x00, 0x01, 0x81))
@pytest.mark.parametrize("kv,qlen", [("fp8", 1), ("fp8", 3), ("fp8_bf16q", 3), ("fp8", 5), ("int8", 1), ("int8", 3)])
def test_an_infinite_query_against_small_keys(pd, kv, qlen, code):
    """The same where every key's element beside the infinity is zero (NaN scores) or the smallest there is."""
    w = inputs.make_workload(B=2, Hq=12, Hkv=2, D=256, seq_lens=[700, 5], qlen=qlen, kv=kv, seed=89, scale=128 ** -0.5)
    w.k_cache.view(torch.uint8)[..., 200] = code
    lam, _ = factors(w)
    want, alone = run(pd, w, lam), run(pd, w, torch.zeros(12))
    for i in (0, qlen):  # the first token of each sequence
        w.q[i, 7, 200] = float("inf")
        want[i, 7] = alone[i, 7]
    assert torch.equal(run(pd, w, lam), want)


@pytest.mark.parametrize("qlen", (1, 3))
@pytest.mark.parametrize("kv", ("f16", "bf16"))
def test_an_infinite_key(pd, kv, qlen):
    """An infinity in the second half of a visible key: rows whose score it makes
    +infinity lose that map, the others' softmax gives the key no weight."""
    w = inputs.make_workload(B=2, Hq=12, Hkv=2, D=256, seq_lens=[700, 91], qlen=qlen, kv=kv, seed=93, scale=128 ** -0.5)
    lam, _ = factors(w)
    alone = run(pd, w, torch.zeros(12))
    blk, at = int(w.block_table[0, 5]), 3
    row = w.k_cache[blk, at, 1].clone()
    w.k_cache[blk, at, 1, 130] = float("inf")
    got = run(pd, w, lam)
    # a weight of zero: the same key with a score far below the others
    w.k_cache[blk, at, 1] = row
    plus = w.q[:qlen, 6:, 130] > 0
    for i in range(qlen):
        for h in range(6):
            if plus[i, h]:
                assert torch.equal(got[i, 6 + h], alone[i, 6 + h])
    k = w.k_cache.double()[w.block_table[0].long()].reshape(-1, 2, 256)[:700, 1]
    v = w.v_cache.double()[w.block_table[0].long()].reshape(-1, 2, 256)[:700, 1]
    rest = torch.arange(700) != 5 * 16 + at
    u = ref_diff.HALF_STEP[w.q.dtype]
    for i in range(qlen):
        for h in range(6):
            if plus[i, h]:
                continue
            q, seen = w.q[i, 6 + h].double(), torch.arange(700) <= 700 - qlen + i
            o = a = 0.0
            for m, c in ((0, 1.0), (1, -float(lam[6 + h]))):
                x = k[:, 128 * m:128 * m + 128] @ q[128 * m:128 * m + 128] * w.scale
                p = torch.softmax(torch.where(seen & (rest if m else seen), x, -torch.inf), 0)
                o, a = o + c * (p @ v), a + abs(c) * (p @ v.abs())
            err = (got[i, 6 + h].double().cpu() - o).abs()
            assert torch.all(err <= (u + 2.0 ** -12) * a + u * o.abs() + 2.0 ** -24)

