"""Scored decode and 4-bit caches in 64 bits on the CPU, written from the definitions, with the error bound of the
kernels.

Bound per output element. A row's weights w_j (summing to one) meet the product with V as two 16-bit operands, which
leave u = 2^-20 (fp16: a rest below half an fp16 step of half an fp16 step, with one binade to spare) or 2^-15
(bfloat16) of each, or as one fp16 operand, 2^-11, where the output is bfloat16 over 8- and 4-bit caches. Over e4m3
caches with more than 8 rows per KV head they are three e4m3 operands: three nearest roundings to 4 bits leave 2^-4 each,
2^-12 in all (beside a bfloat16 output less than the 2^-11 that it is given), and the last one's smallest step, 2^-9
times 2^-8, half of which is 2^-18 beside a largest weight of 2^4 or more: 2^-22, of either sign, so that 2^12 keys
add up to 2^-16. Elsewhere tiny weights are held to 2^-31 of the largest, of at most 2^11 keys here: 2^-20 of the sum, inside f. The fp32 parts move a weight
by a relative amount f: a score is a sum of D products, off by at most D 2^-24 sum |q_d k_d| scale, for the N(0, 1)
rows drawn here (D = 256, sum |q_d k_d| < 300, scale 1 / 16) 2^-12; tanh to 2^-21 of itself, times a cap of at most 50:
2^-15; a bias of up to 2^10 nats to 2^-14; f = 2^-11 stands for all of it. So with A = sum_j w_j |v_j|

    |out - ref| <= (u + f) A + u_out |ref|,   |lse - ref| <= f + 2^-22 |ref|,
    |key weight - ref| <= f (sum of its softmax weights) + 2^-22 |ref|.
"""
import math

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], dtype=torch.float64)
F = 2.0 ** -11


def fp4_values(codes, sf, scale):
    """[.., D/2] codes and [.., D/16] e4m3 scales as 64-bit values [.., D]."""
    x = torch.stack((E2M1[(codes & 15).long()], E2M1[(codes >> 4).long()]), -1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * sf.view(torch.float8_e4m3fn).double()[..., None]).flatten(-2) * scale


class Work:
    """Inputs of one call; caches as the library lays them out, and their values [num_blocks, block_size, Hkv, D]."""

    def __init__(self, kv, Hq, Hkv, D, lens, qlen=1, qlens=None, window=0, prefix=None, cap=0.0, alibi=False, bs=16, q="f16",
                 seed=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.Hq, self.Hkv, self.D, self.bs = kv, Hq, Hkv, D, bs
        self.qlen, self.window, self.cap = qlen, window, cap
        B, cols = len(lens), max(1, -(-max(lens) // bs))
        self.B = B
        n = B * cols + 2
        self.qt = torch.bfloat16 if kv == "bf16" or (q == "bf16" and kv != "f16") else torch.float16
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.table = torch.randperm(n, generator=g)[:B * cols].view(B, cols).int()
        self.starts = None
        rows = B * qlen
        if qlens is not None:
            self.starts = torch.tensor([0] + qlens).cumsum(0).int()
            rows = int(self.starts[-1])
        self.q = (spread * torch.randn(rows, Hq, D, generator=g)).to(self.qt)
        self.scale = D ** -0.5
        self.slopes = 2.0 ** (-8.0 * (1 + torch.arange(Hq)) / Hq) if alibi else None
        self.prefix = None if prefix is None else torch.tensor(prefix, dtype=torch.int32)
        self.c_scale = {"fp8": 0.0125, "int8": 0.0375, "fp4": 0.0059}.get(kv, 1.0)
        self.sf = [None, None]
        self.caches, self.values = [], []
        for i in range(2):
            if kv == "fp4":
                c = torch.randint(0, 256, (n, Hkv, bs, D // 2), generator=g, dtype=torch.uint8)
                self.sf[i] = (20 + 60 * torch.rand(n, Hkv, bs, D // 16, generator=g)).to(torch.float8_e4m3fn)
            else:
                x = torch.randn(n, bs, Hkv, D, generator=g)
                c = {"f16": lambda: x.half(), "bf16": lambda: x.bfloat16(),
                     "fp8": lambda: (x / 0.0125).clamp(-448, 448).to(torch.float8_e4m3fn),
                     "int8": lambda: (x / 0.0375).round().clamp(-127, 127).to(torch.int8)}[kv]()
            self.caches.append(c)
        self.key_weights = torch.rand(n, Hkv, bs, generator=g) * 3

    def value(self, i):
        c = self.caches[i]
        if self.kv == "fp4":
            return fp4_values(c, self.sf[i], self.c_scale).transpose(1, 2)
        return c.double() * self.c_scale

    def spans(self):
        if self.starts is None:
            return [(b * self.qlen, self.qlen) for b in range(self.B)]
        s = self.starts.tolist()
        return [(s[b], s[b + 1] - s[b]) for b in range(self.B)]

    def sees(self, b, pos, j):
        """Whether the token at `pos` of sequence b sees keys j."""
        prefix = 0 if self.prefix is None else int(self.prefix[b])
        ok = (j <= pos) & ((j > pos - self.window) if self.window > 0 else (j >= 0))
        return (ok | (j < prefix)) & (j < int(self.lens[b])) & (pos >= 0)

    def u(self):
        if self.qt == torch.bfloat16:
            return 2.0 ** -15 if self.kv == "bf16" else 2.0 ** -11
        three = self.kv == "fp8" and self.Hq // self.Hkv * self.qlen > 8
        return 2.0 ** -12 if three else 2.0 ** -20

    def reference(self):
        """out, its bound, lse, its bound, key weights, their bound; rows of no sequence are None-like NaN."""
        G = self.Hq // self.Hkv
        out = torch.full(self.q.shape, math.nan, dtype=torch.float64)
        A, lse = out.clone(), out[..., 0].clone()
        kw, kb = self.key_weights.double().clone(), torch.zeros_like(self.key_weights, dtype=torch.float64)
        K, V = self.value(0), self.value(1)
        for b, (r0, n) in enumerate(self.spans()):
            L = int(self.lens[b])
            j = torch.arange(L)
            rows = self.table[b, j // self.bs].long()
            k, v = K[rows, j % self.bs], V[rows, j % self.bs]  # [L, Hkv, D]
            got = torch.zeros(L, self.Hkv, dtype=torch.float64)
            for i in range(n):
                pos = L - n + i
                see = self.sees(b, pos, j)
                out[r0 + i], A[r0 + i], lse[r0 + i] = 0.0, 0.0, -math.inf
                if not bool(see.any()):
                    continue
                q = self.q[r0 + i].double().view(self.Hkv, G, self.D)
                y = torch.einsum("hgd,jhd->hgj", q, k[see]) * self.scale
                if self.cap:
                    y = self.cap * torch.tanh(y / self.cap)
                if self.slopes is not None:
                    y = y - self.slopes.double().view(self.Hkv, G, 1) * (pos - j[see]).abs()
                lse[r0 + i] = torch.logsumexp(y, -1).flatten()
                w = torch.softmax(y, -1)
                out[r0 + i] = torch.einsum("hgj,jhd->hgd", w, v[see]).reshape(self.Hq, self.D)
                A[r0 + i] = torch.einsum("hgj,jhd->hgd", w, v[see].abs()).reshape(self.Hq, self.D)
                got[see] += w.sum(1).T
            at = (rows, slice(None), j % self.bs)
            old = kw[at].clone()
            old[max(0, L - n):] = 0
            kw[at] = old + got
            kb[at] = F * got + 2.0 ** -22 * (old + got)
        bound = (self.u() + F) * A + HALF_STEP[self.qt] * out.abs() + 2.0 ** -24
        return out, bound, lse, F + 2.0 ** -22 * lse.abs(), kw, kb

    def run(self, pd, S=0, weights=True, in_place=False, out=None, **kw):
        """(out, lse, key weights, error flag) of the library."""
        dev = "cuda"
        up = lambda t: None if t is None else t.to(dev)
        flag = torch.zeros(1, dtype=torch.int32, device=dev)
        lse = torch.full(self.q.shape[:2], 7.0, device=dev)
        w_in = up(self.key_weights) if weights else None
        w_out = w_in if in_place or not weights else w_in.clone()
        out = pd.decode_paged_scored(
            up(self.q), up(self.caches[0]), up(self.caches[1]), up(self.table), up(self.lens), self.scale, self.window,
            self.qlen, S, out, query_start_loc=up(self.starts), score_cap=self.cap, alibi_slopes=up(self.slopes),
            prefix_lens=up(self.prefix), k_block_scale=up(self.sf[0]), v_block_scale=up(self.sf[1]), k_scale=self.c_scale,
            v_scale=self.c_scale, lse=lse, key_weights=w_in, key_weights_out=w_out, error_flag=flag, **kw)
        torch.cuda.synchronize()
        return out, lse, w_out, int(flag.item())


def check(w, got, ref=None):
    """Every output within its bound; rows of no sequence (NaN in the reference) are not looked at."""
    out, lse, kw, flag = got
    r_out, b_out, r_lse, b_lse, r_kw, b_kw = ref or w.reference()
    assert flag == 0
    live = ~torch.isnan(r_lse)
    err = (out.double().cpu() - r_out).abs()[live]
    assert bool((err <= b_out[live]).all()), f"out: {float((err / b_out[live]).max()):.3g} of its bound"
    l, r = lse.double().cpu()[live], r_lse[live]
    empty = torch.isinf(r)
    assert bool((l[empty] == -math.inf).all())
    assert bool(((l - r).abs()[~empty] <= b_lse[live][~empty]).all())
    if kw is not None:
        err = (kw.double().cpu() - r_kw).abs()
        assert bool((err <= b_kw).all()), f"key weights: off by {float(err.max()):.3g}"
