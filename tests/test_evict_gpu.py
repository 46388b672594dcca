"""Eviction by key weight against a host model: which keys stay, where their rows, scales and weights go, the lengths,
the free list; in place and to other blocks."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_split_decode_gb300 as pd
    pd.load()
    return pd


def order(w):
    """Weights as numbers that order as the library orders them: NaN below all."""
    return torch.where(torch.isnan(w), -math.inf, w.double())


def kept_keys(w, keep, trigger, first, recent):
    """The kept keys of one head, in order; None: the sequence is not cut."""
    L = w.numel()
    if L <= trigger:
        return None
    m = keep - first - recent
    # NaN below -inf: two keys of the sort, the lower index first on a tie
    mid = sorted(range(first, L - recent), key=lambda j: (math.isnan(w[j]), -float(order(w[j:j + 1])), j))[:m]
    return sorted(list(range(first)) + mid + list(range(L - recent, L)))


class Pool:
    def __init__(self, kv, B, Hkv, D, bs, lens, seed=0, out_cols=0, zeros=0.3):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.bs, self.Hkv, self.lens = kv, bs, Hkv, torch.tensor(lens, dtype=torch.int32)
        cols = max(1, -(-max(lens) // bs)) + 1
        self.n = B * (cols + out_cols) + 3
        ids = torch.randperm(self.n, generator=g).int()
        self.table = ids[:B * cols].view(B, cols).clone()
        self.table_out = ids[B * cols:B * (cols + out_cols)].view(B, out_cols).clone() if out_cols else None
        self.spare = ids[B * (cols + out_cols):]
        width = {"f16": D, "bf16": D, "fp8": D, "int8": D, "fp4": D // 2}[kv]
        dt = {"f16": torch.int16, "bf16": torch.int16}.get(kv, torch.uint8)
        shape = (self.n, Hkv, bs, width) if kv == "fp4" else (self.n, bs, Hkv, width)
        top = 30000 if dt == torch.int16 else 256
        self.data = [torch.randint(0, top, shape, generator=g).to(dt) for _ in range(2)]
        if kv == "fp4":
            self.data += [torch.randint(0, 256, (self.n, Hkv, bs, D // 16), generator=g).to(torch.uint8) for _ in range(2)]
        w = torch.rand(self.n, Hkv, bs, generator=g) ** 6
        self.w = torch.where(torch.rand(self.n, Hkv, bs, generator=g) < zeros, 0.0, (w * 64).round() / 64 if seed % 2 else w)

    def view(self, i, t):
        t = t.cuda()
        if i < 2 and self.kv != "fp4":
            return t.view({"f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[self.kv])
        return t

    def evict(self, pd, keep, *, free=None, count=None, lens_out=False, **kw):
        self.gpu = [self.view(i, t) for i, t in enumerate(self.data)]
        self.gw, lens = self.w.cuda(), self.lens.cuda()
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(lens, -5) if lens_out else None
        sf = dict(k_block_scale=self.gpu[2], v_block_scale=self.gpu[3]) if self.kv == "fp4" else {}
        got = pd.evict_kv_cache(self.gpu[0], self.gpu[1], self.gw, self.table.cuda(), lens, keep, seq_lens_out=out,
                                block_table_out=None if self.table_out is None else self.table_out.cuda(), free_blocks=free,
                                free_count=count, error_flag=flag, **sf, **kw)
        torch.cuda.synchronize()
        return got.cpu(), lens.cpu(), int(flag.item())

    def expect(self, keep, trigger=None, first=0, recent=0):
        """Data, weights and lengths after it."""
        trigger = keep if trigger is None else trigger
        data, w, lens = [t.clone() for t in self.data], self.w.clone(), self.lens.clone()
        to = self.table if self.table_out is None else self.table_out
        for b, L in enumerate(self.lens.tolist()):
            if not 0 <= L <= self.table.shape[1] * self.bs:
                continue
            j = torch.arange(L)
            for h in range(self.Hkv):
                keys = kept_keys(self.w[self.table[b, j // self.bs].long(), h, j % self.bs], keep, trigger, first, recent)
                if keys is None:
                    if self.table_out is None:
                        continue
                    keys = list(range(L))
                src, i = torch.tensor(keys, dtype=torch.long), torch.arange(len(keys))
                sb, so = self.table[b, src // self.bs].long(), src % self.bs
                tb, t_o = to[b, i // self.bs].long(), i % self.bs
                w[tb, h, t_o] = self.w[sb, h, so]
                for k, d in enumerate(data):
                    if k < 2 and self.kv != "fp4":
                        d[tb, t_o, h] = self.data[k][sb, so, h]
                    else:
                        d[tb, h, t_o] = self.data[k][sb, h, so]
            lens[b] = keep if L > trigger else L
        return data, w, lens

    def check(self, want):
        data, w, lens = want
        for i, d in enumerate(data):
            assert torch.equal(self.gpu[i].view(d.dtype).cpu(), d), i
        assert torch.equal(self.gw.view(torch.int32).cpu(), w.view(torch.int32))


KINDS = ("f16", "bf16", "fp8", "int8", "fp4")


@pytest.mark.parametrize("copy", (False, True))
@pytest.mark.parametrize("D,Hkv,bs", [(128, 2, 16), (256, 4, 16), (128, 3, 48), (64, 1, 32)])
@pytest.mark.parametrize("kv", KINDS)
def test_kept_rows(pd, kv, D, Hkv, bs, copy):
    lens = [400, 0, 1, 130, 129, 128, 700, 333]
    for seed, (keep, kw) in enumerate([(128, dict(first=4, recent=32)), (129, dict(recent=129)), (1, dict()), (64, dict(first=64)),
                                       (100, dict(trigger=333, first=1))]):
        most = kw.get("trigger", keep)
        p = Pool(kv, len(lens), Hkv, D, bs, lens, seed=seed, out_cols=-(-most // bs) if copy else 0)
        want = p.expect(keep, **kw)
        got, old, flag = p.evict(pd, keep, lens_out=seed % 2 == 0, **kw)
        assert flag == 0 and torch.equal(got, want[2])
        assert torch.equal(old, p.lens if seed % 2 == 0 else want[2])
        p.check(want)


@pytest.mark.parametrize("kv", ("f16", "fp4"))
def test_weights_that_order_oddly(pd, kv):
    """Infinities, NaN, negative weights, zeros of either sign and nothing but ties."""
    values = torch.tensor([math.inf, -math.inf, math.nan, -math.nan, 0.0, -0.0, 1.0, -1.0, 1e-40, 3e38, 0.5])
    for seed in range(3):
        p = Pool(kv, 3, 2, 128, 16, [300, 200, 90], seed=seed)
        g = torch.Generator().manual_seed(seed)
        p.w = values[torch.randint(0, len(values), p.w.shape, generator=g)] if seed else torch.full_like(p.w, 2.0)
        p.w = torch.where(p.w == 0, 0.0, p.w)  # (zeros of either sign are ordered by their sign: taken out of the model)
        want = p.expect(77, first=3, recent=10)
        got, _, flag = p.evict(pd, 77, first=3, recent=10)
        assert flag == 0 and torch.equal(got, want[2])
        p.check(want)


def test_long_sequences(pd):
    """One sequence over a cluster of CTAs; many heads with more keys than a CTA's shared memory holds."""
    for B, Hkv, L, keep in ((1, 2, 30_000, 5000), (2, 1, 9_001, 1024), (80, 2, 51_000, 2000)):
        if B == 80 and torch.cuda.mem_get_info()[0] < 20 << 30:
            continue
        lens = [L - 13 * b for b in range(B)] if B < 80 else [L] + [5] * (B - 1)
        if B == 80:  # (the tables' capacity is what decides: one long sequence among short ones)
            p = Pool("fp4", B, Hkv, 64, 16, [L] + [5] * (B - 1), seed=3)
        else:
            p = Pool("fp4", B, Hkv, 64, 16, lens, seed=2)
        p.table = p.table.contiguous()
        dev = dict(first=7, recent=100)
        got, _, flag = p.evict(pd, keep, **dev)
        assert flag == 0
        w, L0 = p.w, int(p.lens[0])
        for b in range(min(B, 2)):
            Lb = int(p.lens[b])
            if Lb <= keep:
                assert int(got[b]) == Lb
                continue
            assert int(got[b]) == keep
            j = torch.arange(Lb)
            for h in range(Hkv):
                wh = w[p.table[b, j // 16].long(), h, j % 16]
                mid = wh[7:Lb - 100]
                idx = torch.sort(torch.sort(mid, descending=True, stable=True).indices[:keep - 107]).values + 7
                keys = torch.cat([torch.arange(7), idx, torch.arange(Lb - 100, Lb)])
                i = torch.arange(keep)
                at = p.table[b, i // 16].long()
                assert torch.equal(p.gw.cpu()[at, h, i % 16], wh[keys])
                src = p.data[0][p.table[b, keys // 16].long(), h, keys % 16]
                assert torch.equal(p.gpu[0].cpu()[at, h, i % 16], src)


def test_free_list(pd):
    lens = [400, 100, 0, 333, 96, 97]
    p = Pool("f16", 6, 2, 128, 16, lens, seed=5)
    free = torch.full((p.n,), -7, dtype=torch.int32, device="cuda")
    free[:3] = p.spare.cuda()
    count = torch.tensor([3], dtype=torch.int32, device="cuda")
    want = p.expect(96, recent=8)
    got, _, flag = p.evict(pd, 96, recent=8, free=free, count=count)
    assert flag == 0 and torch.equal(got, want[2])
    p.check(want)
    pushed = [int(x) for b, L in enumerate(lens) if L > 96 for x in p.table[b, 6:-(-L // 16)]]
    assert int(count.item()) == 3 + len(pushed)
    assert free[:int(count.item())].tolist() == p.spare.tolist() + pushed
    assert bool((free[int(count.item()):] == -7).all())


def test_free_list_errors(pd):
    p = Pool("f16", 2, 1, 128, 16, [100, 100], seed=6)
    free = torch.zeros(p.n, dtype=torch.int32, device="cuda")
    count = torch.tensor([p.n - 3], dtype=torch.int32, device="cuda")  # room for three of the eight
    _, _, flag = p.evict(pd, 40, free=free, count=count)
    assert flag == pd.DEVERR_FREE_LIST and int(count.item()) == p.n
    for bad in (-1, p.n + 1):
        count = torch.tensor([bad], dtype=torch.int32, device="cuda")
        _, _, flag = p.evict(pd, 40, free=free, count=count)
        assert flag == pd.DEVERR_FREE_LIST and int(count.item()) == bad


def test_bad_lengths_and_blocks(pd):
    for copy in (False, True):
        p = Pool("fp8", 4, 2, 128, 16, [200, 200, 200, 200], seed=7, out_cols=4 if copy else 0)
        p.lens[1], p.lens[2] = -3, 10 ** 6
        want = p.expect(64, recent=4)
        if copy:
            want[2][1] = want[2][2] = 0
        got, _, flag = p.evict(pd, 64, recent=4, lens_out=copy)
        assert flag == pd.DEVERR_SEQ_LEN and torch.equal(got, want[2])
        p.check(want)
    p = Pool("int8", 2, 2, 128, 16, [200, 200], seed=8)
    p.table[1, 2], p.table[1, 9] = -1, 10 ** 6
    before = [t.clone() for t in p.data]
    got, _, flag = p.evict(pd, 64, recent=64)  # the last 64 keys of sequence 1 lie in blocks 8 .. 12
    assert flag == pd.DEVERR_BLOCK_ID and got.tolist() == [64, 64]
    p2 = Pool("int8", 2, 2, 128, 16, [200, 200], seed=8)
    want = p2.expect(64, recent=64)
    rows = p2.table[0, :4].long()
    assert torch.equal(p.gpu[0].view(torch.uint8).cpu()[rows], want[0][0][rows])
    others = torch.ones(p.n, dtype=torch.bool)
    others[p.table[:, :4].clamp(0, p.n - 1).flatten().long()] = False
    assert torch.equal(p.gpu[1].view(torch.uint8).cpu()[others], before[1][others])


def test_again_and_in_a_graph(pd):
    """Cut, grown and cut once more: the second cut sees the first one's order; replayed from a graph."""
    p = Pool("f16", 5, 2, 128, 16, [300, 250, 90, 400, 64], seed=9)
    gpu = [p.view(i, t) for i, t in enumerate(p.data)]
    w, lens, table = p.w.cuda(), p.lens.cuda(), p.table.cuda()
    call = lambda: pd.evict_kv_cache(*gpu, w, table, lens, 60, trigger=80, first=2, recent=20)
    warm = [t.clone() for t in (*gpu, w, lens)]
    call()
    torch.cuda.synchronize()
    for t, s in zip((*gpu, w, lens), warm):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):
        p.data, p.w, p.lens = [t.view(torch.int16).cpu() for t in gpu], w.cpu(), lens.cpu()
        want = p.expect(60, trigger=80, first=2, recent=20)
        graph.replay()
        torch.cuda.synchronize()
        p.gpu, p.gw = gpu, w
        p.check(want)
        assert torch.equal(lens.cpu(), want[2])
        lens += 30  # what lies behind the kept keys counts as new ones
    assert int(lens.max()) == 90


def test_refusals(pd):
    p = Pool("f16", 2, 2, 128, 16, [50, 60], seed=1)
    gpu = [p.view(i, t) for i, t in enumerate(p.data)]
    args = (*gpu, p.w.cuda(), p.table.cuda(), p.lens.cuda())
    for keep, kw in ((0, {}), (8, dict(trigger=7)), (8, dict(first=5, recent=4)), (8, dict(first=-1)), (8, dict(recent=-1)),
                     (40, dict(block_table_out=p.table[:, :2].contiguous().cuda()))):
        with pytest.raises(pd.DecodeError):
            pd.evict_kv_cache(*args, keep, **kw)
    free, count = torch.zeros(p.n, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(pd.DecodeError):
        pd.evict_kv_cache(*args, 8, free_blocks=free)
    with pytest.raises(pd.DecodeError):
        pd.evict_kv_cache(*args, 8, free_blocks=free, free_count=count, block_table_out=p.table.cuda().clone())
    with pytest.raises(ValueError):
        pd.evict_kv_cache(*args, 8, free_blocks=free[:-1], free_count=count)
    with pytest.raises(ValueError):
        pd.evict_kv_cache(gpu[0], gpu[1], p.w.cuda()[:, :1], *args[3:], 8)
    with pytest.raises(TypeError):
        pd.evict_kv_cache(gpu[0], gpu[1], p.w.cuda().half(), *args[3:], 8)


def test_threads_on_one_stream(pd):
    """Calls of several threads on one stream share the stream's workspace; each call's launches stay together."""
    import threading
    pools = [Pool("fp8", 4, 2, 128, 16, [300, 280, 90, 200], seed=20 + i) for i in range(4)]
    wants = [p.expect(64, recent=4) for p in pools]
    stream, gpu, errors = torch.cuda.Stream(), [], []
    for p in pools:
        gpu.append([[p.view(i, t) for i, t in enumerate(p.data)] + [p.w.cuda(), p.table.cuda(), p.lens.cuda()] for _ in range(8)])
    torch.cuda.synchronize()

    def work(calls):
        try:
            with torch.cuda.stream(stream):
                for args in calls:
                    pd.evict_kv_cache(*args, 64, recent=4)
        except Exception as e:  # pragma: no cover
            errors.append(e)

    threads = [threading.Thread(target=work, args=(calls,)) for calls in gpu]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for p, want, calls in zip(pools, wants, gpu):
        for args in calls:
            p.gpu, p.gw = args[:2], args[2]
            p.check(want)
            assert torch.equal(args[4].cpu(), want[2])
