"""The 4-bit writer against its definition, code by code, and the decode of what it wrote."""
import math

import pytest
import torch

from ref_scored import E2M1, Work, fp4_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


def quantise(x, g):
    """Codes [.., D/2] and scale bytes [.., D/16] of rows x, from the definition: fp32 quotients, nearest, ties to even."""
    f = x.float().unflatten(-1, (-1, 16))
    nan = torch.isnan(f).any(-1)
    g32 = torch.tensor(g, dtype=torch.float32)
    amax = torch.where(torch.isnan(f), 0.0, f.abs()).amax(-1)
    s = (amax / (6.0 * g32)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (s.float() * g32)[..., None]
    y = f / d
    mag = y.abs().double()
    # nearest of the eight magnitudes; between two at the same distance the even code
    dist = (mag[..., None] - E2M1[:8]).abs()
    order = dist + torch.tensor([0.0, 1e-12] * 4, dtype=torch.float64)
    code = torch.where(mag >= 6, 7, order.argmin(-1))
    code = torch.where(d > 0, code, 0).to(torch.uint8) | (torch.signbit(f).to(torch.uint8) << 3)
    code = torch.where(nan[..., None], 0, code).to(torch.uint8).flatten(-2)
    sf = torch.where(nan, 0x7F, s.view(torch.uint8)).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf


def write(pd, k, v, slots, shape, g=(1.0, 1.0), offset=0):
    n, Hkv, bs, D = shape
    caches = [torch.full((n, Hkv, bs, D // 2), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sfs = [torch.full((n, Hkv, bs, D // 16), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(2)]
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")

    def place(x):  # `offset` elements into a buffer: rows that begin at a multiple of 16 bytes only
        buf = torch.empty(x.numel() + offset, dtype=x.dtype, device="cuda")
        buf[offset:] = x.flatten().cuda()
        return buf[offset:].view(x.shape)

    pd.write_kv_cache_fp4(place(k), place(v), slots.cuda(), *caches, *sfs, k_scale=g[0], v_scale=g[1], error_flag=flag)
    torch.cuda.synchronize()
    return [c.cpu() for c in caches], [s.cpu() for s in sfs], int(flag.item())


def expect(x, slots, shape, g):
    n, Hkv, bs, D = shape
    codes, sf = quantise(x, g)
    c = torch.full((n, Hkv, bs, D // 2), 0xA5, dtype=torch.uint8)
    s = torch.full((n, Hkv, bs, D // 16), 0x5A, dtype=torch.uint8)
    for t, slot in enumerate(slots.tolist()):
        if 0 <= slot < n * bs:
            c[slot // bs, :, slot % bs], s[slot // bs, :, slot % bs] = codes[t], sf[t]
    return c, s


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("T,Hkv,D,bs", [(1, 1, 16, 16), (37, 4, 256, 16), (200, 3, 128, 32), (5, 8, 64, 48), (700, 2, 128, 16)])
@pytest.mark.parametrize("offset", (0, 8))
def test_codes(pd, dtype, T, Hkv, D, bs, offset):
    gen = torch.Generator().manual_seed(T)
    shape = (T // bs + 3, Hkv, bs, D)
    k, v = (torch.randn(T, Hkv, D, generator=gen).mul(3).to(dtype) for _ in range(2))
    slots = torch.randperm(shape[0] * bs, generator=gen)[:T]
    slots[::5] = -1
    slots[-1] = shape[0] * bs - 1 if T > 1 else 3
    slots = torch.where((torch.arange(T) < T - 1) & (slots == slots[-1]), -1, slots)
    g = (0.01, 0.37)
    caches, sfs, flag = write(pd, k, v, slots, shape, g, offset)
    assert flag == 0
    for i, x in enumerate((k, v)):
        c, s = expect(x, slots, shape, g[i])
        assert torch.equal(caches[i], c) and torch.equal(sfs[i], s)


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("g", (1.0, 2.0 ** -20, 2.0 ** 30, 1e-38, 3e38, 0.1))
def test_special_values(pd, dtype, g):
    """Zeros of either sign, infinities, NaN, the largest and smallest numbers, ties, groups whose scale vanishes or is at
    its end; scales of the cache beyond the corrected quotient's range."""
    big = torch.finfo(dtype).max
    rows = [[0.0, -0.0] * 8, [math.inf, -math.inf, 1.0, -1.0] * 4, [math.nan] + [1.0] * 15, [1.0] * 15 + [-math.nan],
            [big, -big, 1.0, 0.0] * 4, [torch.finfo(dtype).tiny, -torch.finfo(dtype).tiny] * 8,
            [torch.finfo(dtype).smallest_normal / 4] * 16, [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0],
            [48.0] + [4.0, 6.0, 10.0, 14.0, 20.0, 28.0, 40.0, 2.0, 1.99, 2.01, -6.0, -10.0, 39.9, 40.1, 0.0],
            [-1e-4, 1e-4] * 8, [3000.0, -2688.0, 2700.0, 100.0] * 4, [1.0] + [-0.0] * 15]
    x = torch.tensor(rows).to(dtype).view(1, 1, -1)
    pad = torch.zeros(1, 1, -(-x.shape[-1] // 128) * 128 - x.shape[-1], dtype=dtype)
    x = torch.cat([x, pad], -1)
    shape = (1, 1, 16, x.shape[-1])
    slots = torch.tensor([5])
    caches, sfs, _ = write(pd, x, -x, slots, shape, (g, g))
    for i, y in enumerate((x, -x)):
        c, s = expect(y, slots, shape, g)
        assert torch.equal(sfs[i], s)
        assert torch.equal(caches[i], c)


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
def test_every_value(pd, dtype):
    """Every 16-bit pattern, beside ones that set the group's scale."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    for top in (1.0, 5.3, 0.0):
        x = torch.cat([bits[:65535].view(-1, 15), torch.full((4369, 1), top, dtype=dtype)], -1).reshape(-1)
        x = torch.cat([x, torch.zeros(-x.numel() % 256, dtype=dtype)]).view(-1, 1, 256)
        T = x.shape[0]
        shape = (T // 16 + 1, 1, 16, 256)
        caches, sfs, _ = write(pd, x, x, torch.arange(T), shape, (0.05, 0.05))
        c, s = expect(x, torch.arange(T), shape, 0.05)
        assert torch.equal(sfs[0], s) and torch.equal(caches[0], c)


def test_bad_slots(pd):
    shape = (2, 2, 16, 64)
    x = torch.randn(4, 2, 64).half()
    slots = torch.tensor([-1, 32, 5, 2 ** 40])
    caches, sfs, flag = write(pd, x, x, slots, shape)
    assert flag == pd.DEVERR_SLOT
    c, s = expect(x, slots, shape, 1.0)
    assert torch.equal(caches[0], c) and torch.equal(sfs[1], s)


def test_refusals(pd):
    x = torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")
    c = torch.zeros(1, 2, 16, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(1, 2, 16, 4, dtype=torch.uint8, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    for kw in (dict(k_scale=0.0), dict(v_scale=-1.0), dict(k_scale=math.inf), dict(v_scale=math.nan)):
        with pytest.raises(pd.DecodeError):
            pd.write_kv_cache_fp4(x, x, slots, c, c.clone(), s, s.clone(), **kw)
    with pytest.raises(TypeError):
        pd.write_kv_cache_fp4(x.float(), x.float(), slots, c, c.clone(), s, s.clone())
    with pytest.raises(ValueError):
        pd.write_kv_cache_fp4(x[:, :1], x[:, :1], slots, c, c.clone(), s, s.clone())
    with pytest.raises(ValueError):
        pd.write_kv_cache_fp4(x, x, slots[:1], c, c.clone(), s, s.clone())
    with pytest.raises(ValueError):
        pd.write_kv_cache_fp4(x, x, slots, c, c.clone(), s[..., :2], s[..., :2])


def test_cache_past_four_gigabytes(pd):
    """Codes beyond 2^32 bytes: written and decoded."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    Hkv, D, bs = 8, 256, 16
    n = 340_000  # blocks: 5.6 GB of codes a cache
    g = torch.Generator().manual_seed(3)
    caches = [torch.zeros(n, Hkv, bs, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sfs = [torch.zeros(n, Hkv, bs, D // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    blocks = torch.tensor([n - 1, 5, n - 7, 300_001])
    T = 4 * bs
    k, v = (torch.randn(T, Hkv, D, generator=g).half() for _ in range(2))
    slots = (blocks[:, None] * bs + torch.arange(bs)).flatten()
    pd.write_kv_cache_fp4(k.cuda(), v.cuda(), slots.cuda(), *caches, *sfs, k_scale=0.1, v_scale=0.1)
    q = torch.randn(1, 16, D, generator=g).half()
    kw = torch.zeros(n, Hkv, bs, device="cuda")
    out = pd.decode_paged_scored(q.cuda(), *caches, blocks.int().view(1, 4).cuda(), torch.tensor([T], dtype=torch.int32).cuda(),
                                 D ** -0.5, k_block_scale=sfs[0], v_block_scale=sfs[1], k_scale=0.1, v_scale=0.1, key_weights=kw)
    vals = [fp4_values(*quantise(x, 0.1), torch.tensor(0.1, dtype=torch.float32).double()) for x in (k, v)]
    y = torch.einsum("hgd,jhd->hgj", q[0].double().view(Hkv, 2, D), vals[0]) * D ** -0.5
    p = torch.softmax(y, -1)
    ref = torch.einsum("hgj,jhd->hgd", p, vals[1]).reshape(16, D)
    A = torch.einsum("hgj,jhd->hgd", p, vals[1].abs()).reshape(16, D)
    bound = (2.0 ** -11 + 2.0 ** -20) * A + 2.0 ** -11 * ref.abs() + 2.0 ** -24
    assert bool(((out[0].double().cpu() - ref).abs() <= bound).all())
    got = kw[blocks.cuda()].cpu().permute(0, 2, 1).reshape(T, Hkv)
    assert bool(((got - p.sum(1).T).abs() <= 2.0 ** -11 * p.sum(1).T).all())
