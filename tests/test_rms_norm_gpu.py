"""rms_norm against numpy in 64 bits.

Bounds. h = x + residual is one fp32 sum (relative 2^-24); the mean of n
squares, in any order of summation, is off by at most (n + 2) 2^-24, its
inverse root by half of that and the root's own 2 ulp, and the products with h, weight and
gain add three roundings, so y is off by r = (n / 2 + 16) 2^-24 relative. An
output in 16 bits adds half its step u (fp16 2^-11, bfloat16 2^-8; fp16
subnormals 2^-25 absolute). A scale is off by r + 2^-23. A code's value is
within half a step of y: e4m3 2^-4 |y| or 2^-10 scale (subnormals), int8
scale / 2; r again for y / scale.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


def draw(rows, N, n, dt, residual, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, N, generator=g)
    if spread:  # rows of different sizes
        x = x * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x = x.to(dt)
    res = torch.randn(rows, N, generator=g).to(dt) if residual else None
    w = (1 + 0.2 * torch.randn(n, generator=g)).to(dt)
    return x, res, w


def reference(x, res, w, eps, gain, n):
    h = x.double().numpy() + (res.double().numpy() if res is not None else 0.0)
    g = h.reshape(h.shape[0], -1, n)
    y = g / np.sqrt(np.mean(g * g, axis=-1, keepdims=True) + eps) * w.double().numpy() * gain
    return h, y.reshape(h.shape)


def check_16(got, ref, r, dt):
    g = got.float().cpu().numpy().astype(np.float64).reshape(ref.shape)
    excess = np.abs(g - ref) / ((U[dt] + r) * np.abs(ref) + 2.0 ** -25)
    assert np.all(np.isfinite(g)) and excess.max() <= 1.0, f"{excess.max():.2f}x the bound"


def check_codes(codes, scale, y, r, dt, s):
    rows, N = y.shape
    z = y.reshape(rows, N // s, s)
    q, sub = (448.0, 2.0 ** -10) if dt == torch.float8_e4m3fn else (127.0, 0.5)
    sc = scale.double().cpu().numpy().reshape(rows, N // s, 1)
    want = np.maximum(np.abs(z).max(-1, keepdims=True) / q, 2.0 ** -100)
    assert np.all(np.abs(sc - want) <= (r + 2.0 ** -23) * want)
    c = codes.float().cpu().numpy().astype(np.float64).reshape(z.shape)
    assert np.all(np.abs(c) <= q)
    half = (2.0 ** -4 * np.abs(z) if q == 448.0 else 0.0) + sub * sc * (1 + 2 ** -20)
    excess = np.abs(c * sc - z) / (half + 2 * r * np.abs(z))
    assert excess.max() <= 1.0, f"{excess.max():.2f}x the bound"


SHAPES = [(1, 1, 1, 1), (3, 7, 7, 1), (2, 100, 20, 50), (5, 128, 128, 128), (1, 6144, 256, 6144), (33, 6144, 6144, 128),
          (7, 4096, 4096, 4096), (4, 1000, 200, 8), (9, 24 * 80, 80, 160), (300, 256, 32, 64), (2, 8192, 8192, 64),
          (3, 32768, 32768, 32768), (2, 32768, 4, 2), (6, 1001, 1001, 7), (1, 2048, 2048, 1024), (700, 64, 64, 64),
          (2, 96 * 104, 104, 104), (3, 8 * 1031, 8 * 1031, 8)]


@pytest.mark.parametrize("out", ("same", "e4m3", "int8"))
@pytest.mark.parametrize("residual", (False, True))
@pytest.mark.parametrize("dt", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("rows,N,n,s", SHAPES)
def test_parity(pd, rows, N, n, s, dt, residual, out):
    x, res, w = draw(rows, N, n, dt, residual, rows + N)
    if rows > 2:
        x[1] = 0  # a row of zeros
        if res is not None:
            res[1] = 0
    odt = {"same": dt, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[out]
    rd = None if res is None else res.to(DEV)
    got = pd.rms_norm(x.to(DEV), w.to(DEV), 1e-5, residual=rd, gain=0.7, norm_size=n, out_dtype=odt, scale_size=s)
    torch.cuda.synchronize()
    h, y = reference(x, res, w, 1e-5, 0.7, n)
    r = (n / 2 + 16) * 2.0 ** -24
    if res is not None:  # replaced in place
        check_16(rd, h, 2.0 ** -24, dt)
    if out == "same":
        check_16(got, y, r, dt)
    else:
        assert got[1].shape == (rows, N // s) and got[0].dtype == odt
        check_codes(got[0], got[1], y, r, odt, s)


@pytest.mark.parametrize("f32", (False, True))
def test_layouts_weights_and_in_place(pd, f32):
    """Leading dimensions, a float32 weight, out over x, h over x."""
    x, res, w = draw(12, 512, 64, torch.bfloat16, True, 5)
    wd = (w.float() if f32 else w).to(DEV)
    h, y = reference(x, res, w, 0.0, 1.0, 64)
    r = (64 / 2 + 16) * 2.0 ** -24
    xd, rd = x.to(DEV).view(3, 4, 512), res.to(DEV).view(3, 4, 512)
    got = pd.rms_norm(xd, wd, 0.0, residual=rd, norm_size=64, out=xd)
    assert got is xd
    check_16(xd.view(12, 512), y, r, torch.bfloat16)
    check_16(rd.view(12, 512), h, 2.0 ** -24, torch.bfloat16)
    xd, rd = x.to(DEV), res.to(DEV)
    got, sc = pd.rms_norm(xd, wd, 0.0, residual=rd, residual_out=xd, norm_size=64, out_dtype=torch.float8_e4m3fn)
    check_codes(got, sc, y, r, torch.float8_e4m3fn, 512)
    check_16(xd, h, 2.0 ** -24, torch.bfloat16)
    assert torch.equal(rd.cpu(), res)


@pytest.mark.parametrize("offset", (1, 2, 4))
@pytest.mark.parametrize("N", (256, 1024))
def test_unaligned_rows(pd, N, offset):
    """Contiguous tensors that start off a 16-byte boundary."""
    x, res, w = draw(5, N, N, torch.float16, True, 9)

    def off(t):
        buf = torch.zeros(t.numel() + 8, dtype=t.dtype, device=DEV)
        v = buf[offset:offset + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    h, y = reference(x, res, w, 1e-6, 1.0, N)
    r = (N / 2 + 16) * 2.0 ** -24
    xd, rd, wd = off(x), off(res), off(w)
    check_16(pd.rms_norm(xd, wd, 1e-6, residual=rd), y, r, torch.float16)
    check_16(rd, h, 2.0 ** -24, torch.float16)
    codes = torch.zeros(5 * N + 8, dtype=torch.int8, device=DEV)
    out = codes[offset:offset + 5 * N].view(5, N)
    _, sc = pd.rms_norm(xd, wd, 1e-6, out=out, scale_size=N // 4)
    h, y = reference(x, None, w, 1e-6, 1.0, N)
    check_codes(out, sc, y, r, torch.int8, N // 4)
    assert int(codes[:offset].abs().sum()) == 0 and int(codes[offset + 5 * N:].abs().sum()) == 0


@pytest.mark.parametrize("out", (None, torch.float8_e4m3fn, torch.int8))
def test_infinities_nan_and_large_values(pd, out):
    """A row with an infinity or a NaN is not finite and disturbs no other
    row; the largest fp16 values neither overflow nor lose the row."""
    x, _, w = draw(6, 256, 256, torch.float16, False, 21, spread=False)
    x[1, 3], x[2, 4], x[4] = float("inf"), float("nan"), 65504.0
    got = pd.rms_norm(x.to(DEV), w.to(DEV), 1e-5, out_dtype=out)
    h, y = reference(x, None, w, 1e-5, 1.0, 256)
    r = (256 / 2 + 16) * 2.0 ** -24
    rows = [0, 3, 4, 5]
    if out is None:
        check_16(got[rows], y[rows], r, torch.float16)
        g = got.float().cpu()
        assert torch.isnan(g[2]).all() and torch.isnan(g[1, 3]) and (g[1, :3] == 0).all()
    else:
        check_codes(got[0][rows], got[1][rows], y[rows], r, out, 256)
        g = got[0].view(torch.uint8).cpu()
        nan = 0x7F if out == torch.float8_e4m3fn else 0
        assert int(g[1, 3]) == nan and (g[1, :3] == 0).sum() + (g[1, :3] == 0x80).sum() == 3
        assert (g[2] == nan).all() and torch.isfinite(got[1]).all()


def test_no_rows(pd):
    w = torch.ones(64, dtype=torch.float16, device=DEV)
    assert pd.rms_norm(torch.empty(0, 64, dtype=torch.float16, device=DEV), w).shape == (0, 64)
    codes, sc = pd.rms_norm(torch.empty(0, 64, dtype=torch.float16, device=DEV), w, out_dtype=torch.int8, scale_size=16)
    assert codes.shape == (0, 64) and sc.shape == (0, 4)


def test_graph_and_streams(pd):
    x, res, w = (t.to(DEV) for t in draw(40, 512, 512, torch.bfloat16, True, 31))
    want = pd.rms_norm(x, w, residual=res, residual_out=torch.empty_like(x), out_dtype=torch.float8_e4m3fn)
    out, sc, ro = torch.empty_like(want[0]), torch.empty_like(want[1]), torch.empty_like(x)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        pd.rms_norm(x, w, residual=res, residual_out=ro, out=out, out_scale=sc)
    for _ in range(3):
        out.view(torch.uint8).zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(sc, want[1])
    other = pd.rms_norm(x, w, residual=res, residual_out=ro, out_dtype=torch.float8_e4m3fn, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(other[0].view(torch.uint8), want[0].view(torch.uint8))
