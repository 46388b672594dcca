"""The codes of the norm's 8-bit outputs are y / s rounded to the nearest, ties
to even, and s is max |y| / Q, both in fp32: on rows whose y is known bit for bit.

A row of +-1 has a mean square of 1, so with eps = 0 and gain = 1 its y is its
float32 weight, with the sign: the weights place the quotients on ties, beside
them and anywhere between."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


def weights(N, q, top, seed):
    """float32 [N]: quotients by s = top / q on ties and a few float32 steps beside them."""
    rng = np.random.RandomState(seed)
    s = np.float32(top) / np.float32(q)
    if q == 127.0:
        ties = rng.randint(0, 126, N) + 0.5
    else:  # a 3-bit fraction and a half step of it
        ties = (1 + (2 * rng.randint(0, 8, N) + 1) / 16) * 2.0 ** rng.randint(-6, 8, N)
        ties = np.minimum(ties, 440.0)
    w = (ties.astype(np.float32) * s).astype(np.float32)
    w = (w.view(np.int32) + rng.randint(-2, 3, N).astype(np.int32)).view(np.float32)
    w[rng.randint(N)] = np.float32(top)
    return w


@pytest.mark.parametrize("offset", (0, 1))  # 16-byte vectors, or one value at a time
@pytest.mark.parametrize("top", (1.0, 3.7, 448.0 / 3.0, 0.011))
@pytest.mark.parametrize("kind", (torch.float8_e4m3fn, torch.int8))
@pytest.mark.parametrize("N", (256, 6144))
def test_codes_are_the_rounded_quotients(pd, N, kind, top, offset):
    q = 448.0 if kind == torch.float8_e4m3fn else 127.0
    w = weights(N, q, top, N)
    sign = torch.where(torch.rand(3, N, generator=torch.Generator().manual_seed(N)) < 0.5, -1.0, 1.0)
    buf = torch.zeros(3 * N + 8, dtype=torch.bfloat16, device=DEV)
    x = buf[offset:offset + 3 * N].view(3, N)
    x.copy_(sign)
    codes, scale = pd.rms_norm(x, torch.from_numpy(w).to(DEV), 0.0, out_dtype=kind)
    torch.cuda.synchronize()
    s = np.float32(w.max()) / np.float32(q)
    assert np.all(scale.cpu().numpy() == s)
    t = torch.from_numpy(sign.numpy() * (w / s).astype(np.float32))
    want = t.to(torch.float8_e4m3fn).float() if q == 448.0 else t.round()
    bad = (codes.float().cpu() != want).nonzero()
    assert bad.shape[0] == 0, f"{bad.shape[0]} codes of {3 * N} are off, first {bad[0].tolist()}"


@pytest.mark.parametrize("kind", (torch.float8_e4m3fn, torch.int8))
@pytest.mark.parametrize("seed", range(12))
def test_codes_under_drawn_scales(pd, kind, seed):
    """Scales drawn over 60 powers of two, quotients anywhere and on ties, small and subnormal codes among them."""
    q = 448.0 if kind == torch.float8_e4m3fn else 127.0
    rng = np.random.RandomState(100 + seed)
    N = 4096
    top = np.float32(rng.uniform(1, 2) * 2.0 ** rng.randint(-30, 30))
    w = weights(N, q, top, seed)
    some = rng.rand(N) < 0.5
    w[some] = (top * rng.uniform(0, 1, N) * 2.0 ** -rng.uniform(0, 18, N)).astype(np.float32)[some]
    w[rng.randint(N)] = top
    assert w.max() == top
    codes, scale = pd.rms_norm(torch.ones(1, N, dtype=torch.float16, device=DEV), torch.from_numpy(w).to(DEV), 0.0,
                               out_dtype=kind)
    torch.cuda.synchronize()
    s = top / np.float32(q)
    assert float(scale) == s
    t = torch.from_numpy(w / s)
    want = t.to(torch.float8_e4m3fn).float() if q == 448.0 else t.round()
    bad = (codes[0].float().cpu() != want).nonzero()
    assert bad.shape[0] == 0, f"{bad.shape[0]} codes of {N} are off, first {bad[0].tolist()}"
