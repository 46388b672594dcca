"""Cases of attention over 4-bit paged caches and its writer, of decodes with
capped scores, distance biases and prefix masks, of the attention weight that
keys collect, and of the eviction that goes by it.

Each case runs in a plain form (elementary torch operations in 32 bits) or,
with ``own`` set, through this package's calls on the same state. The passes
write to buffers that the state keeps; the weights' sums and the keys that an
eviction keeps go to buffers of their own, so that a pass leaves its inputs as
they were.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": F8, "int8": torch.int8, "fp4": torch.uint8}
# (query heads, KV heads, head size) of this repository's workloads and tests
HEADS = ((24, 4, 256), (32, 8, 128), (28, 4, 128), (8, 2, 128), (6, 6, 128), (12, 2, 256))
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _decode(name, kv, q, B, heads, longest, **kw):
    case = dict(name=name, op="decode", kv=kv, q=q, B=B, heads=heads, longest=longest, ragged=False, qlen=1, window=0,
                prefix=0, cap=0.0, alibi=False, weights=False, block_size=16)
    case.update(kw)
    return case


def listed():
    return [
        # a single request decoding under capped scores: latency
        _decode("cap_f16_b1", "f16", "f16", 1, 0, 4096, cap=50.0),
        # the headline batch of 32 sequences, scores capped
        _decode("cap_f16_b32", "f16", "f16", 32, 0, 4096, cap=50.0),
        # ragged lengths in [512, 16384], heads with slopes of their own, bfloat16
        _decode("alibi_bf16_ragged_b32", "bf16", "bf16", 32, 1, 16384, ragged=True, alibi=True),
        # speculative verify of three tokens: a window and the prompt's first keys, e4m3 cache
        _decode("prefix_e4m3_verify_b8", "e4m3", "bf16", 8, 0, 8192, qlen=3, window=4096, prefix=128),
        # a single request over a 4-bit cache: latency
        _decode("fp4_b1", "fp4", "f16", 1, 0, 4096),
        # the headline batch over a 4-bit cache
        _decode("fp4_b32", "fp4", "f16", 32, 0, 4096),
        # ragged lengths over a 4-bit cache with capped scores, every key's weight summed for a later eviction
        _decode("fp4_weights_ragged_b32", "fp4", "bf16", 32, 1, 16384, ragged=True, cap=30.0, weights=True),
        # the headline batch with its keys' weights summed
        _decode("weights_f16_b32", "f16", "f16", 32, 0, 4096, weights=True),
        # one new token for each of 32 sequences: every decode step
        dict(name="write_fp4_t32", op="write", q="f16", T=32, heads=0, block_size=16),
        # a prefill step of 32768 tokens
        dict(name="write_fp4_t32768", op="write", q="bf16", T=32768, heads=0, block_size=16),
        # a batch at its limit drops half of its keys
        dict(name="evict_f16_b32", op="evict", kv="f16", B=32, heads=0, longest=4096, keep=2048, first=4, recent=256,
             ragged=False, block_size=16),
        # one long request shrinks to an eighth, 4-bit cache
        dict(name="evict_fp4_b1", op="evict", kv="fp4", B=1, heads=1, longest=32768, keep=4096, first=4, recent=512,
             ragged=False, block_size=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("decode", "decode", "decode", "write", "evict"))
    h = rng.randrange(len(HEADS))
    Hq, Hkv, D = HEADS[h]
    bs = rng.choice((16, 32, 64))
    if op == "write":
        return dict(op=op, q=rng.choice(("f16", "bf16")), T=_log(rng, 1, (32768 * 4 * 256) // (Hkv * D)), heads=h,
                    block_size=bs)
    kv = rng.choice(("f16", "bf16", "e4m3", "int8", "fp4", "fp4", "fp4"))
    B = _log(rng, 1, 48)
    most = (32 * 4096 * 4 * 256) // (B * Hkv * D)  # keys a sequence: at most the headline batch's cache
    longest = _log(rng, 1, min(32768, most))
    if op == "evict":
        keep = _log(rng, 1, longest)
        first = rng.randrange(0, min(16, keep) + 1)
        return dict(op=op, kv=kv, B=B, heads=h, longest=longest, keep=keep, first=first,
                    recent=rng.randrange(0, keep - first + 1), ragged=rng.random() < 0.5, block_size=bs)
    qlen = min(rng.choice((1, 1, 1, 2, 3, 5)), 32 // (Hq // Hkv), longest)
    q = kv if kv in ("f16", "bf16") else rng.choice(("f16", "bf16"))
    case = _decode(None, kv, q, B, h, longest, ragged=rng.random() < 0.5, qlen=qlen,
                   window=rng.choice((0, 0, _log(rng, 1, longest))), prefix=rng.choice((0, 0, _log(rng, 1, longest))),
                   cap=rng.choice((0.0, 15.0, 30.0, 50.0)), alibi=rng.random() < 0.3, weights=rng.random() < 0.4,
                   block_size=bs)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
def _ragged(g, B, lo, hi):
    return torch.randint(lo, hi + 1, (B,), generator=g, device=DEV)


def _rand(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _codes4(g, *shape):
    """4-bit codes of N(0, 1) values scaled to a largest magnitude of about 6."""
    y = (_rand(g, *shape) * 2.2).abs()
    code = sum((y > t).to(torch.uint8) for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0))
    code |= (torch.randint(0, 2, shape, generator=g, device=DEV, dtype=torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _caches(s, g, num_blocks, Hkv, D, bs):
    kv = s["kv"]
    for n in ("k", "v"):
        s[n + "_block_scale"] = None
        if kv == "fp4":  # heads before keys
            s[n + "_cache"] = _codes4(g, num_blocks, Hkv, bs, D)
            s[n + "_block_scale"] = (40 + 80 * torch.rand(num_blocks, Hkv, bs, D // 16, generator=g, device=DEV)).to(F8)
        else:
            x = _rand(g, num_blocks, bs, Hkv, D, dtype=torch.float32 if kv in ("e4m3", "int8") else TYPES[kv])
            s[n + "_cache"] = ((x / 0.0125).clamp(-448, 448).to(F8) if kv == "e4m3" else
                               (x / 0.0375).round().clamp(-127, 127).to(torch.int8) if kv == "int8" else x)
    s["cache_scale"] = {"e4m3": 0.0125, "int8": 0.0375, "fp4": 0.0059}.get(kv, 1.0)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    (Hq, Hkv, D), bs = HEADS[case["heads"]], case["block_size"]
    s["error_flag"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if case["op"] == "write":
        T, xt = case["T"], TYPES[case["q"]]
        num_blocks = -(-T // bs) + 3
        for n in ("k", "v"):
            s[n + "_new"] = _rand(g, T, Hkv, D, dtype=xt)
            s[n + "_cache"] = torch.randint(0, 256, (num_blocks, Hkv, bs, D // 2), generator=g, device=DEV, dtype=torch.uint8)
            s[n + "_block_scale"] = (40 + 80 * torch.rand(num_blocks, Hkv, bs, D // 16, generator=g, device=DEV)).to(F8)
        slots = torch.randperm(num_blocks * bs, generator=g, device=DEV)[:T]
        # the token buffer is padded behind the last token of the step
        s.update(slot_mapping=torch.where(torch.arange(T, device=DEV) < max(1, T - T // 16), slots, -1), cache_scale=0.0059)
        return s
    B, L = case["B"], case["longest"]
    lens = torch.full((B,), L, device=DEV)
    if case["ragged"]:
        least = case["qlen"] if case["op"] == "decode" else 1
        lens = torch.where(torch.rand(B, generator=g, device=DEV) < 0.06, 0, _ragged(g, B, max(least, L // 32), L))
        lens[0] = L
    cols = -(-L // bs)
    if case["op"] == "evict":
        out_cols = -(-case["keep"] // bs)
        num_blocks = B * (cols + out_cols) + 1
        order = torch.randperm(num_blocks, generator=g, device=DEV, dtype=torch.int32)
        _caches(s, g, num_blocks, Hkv, D, bs)
        # most keys hardly ever seen, some never, few heavy
        w = torch.rand(num_blocks, Hkv, bs, generator=g, device=DEV) ** 12 * 40
        s.update(lens=lens.int(), lens_out=torch.zeros(B, dtype=torch.int32, device=DEV),
                 key_weights=torch.where(w < 1e-6, 0.0, w),
                 block_table=order[:B * cols].view(B, cols).contiguous(),
                 table_out=order[B * cols:B * (cols + out_cols)].view(B, out_cols).contiguous())
        return s
    num_blocks = B * cols + 1
    qt, T = TYPES[case["q"]], B * case["qlen"]
    _caches(s, g, num_blocks, Hkv, D, bs)
    slopes = 2.0 ** (-8.0 * (1 + torch.arange(Hq, device=DEV)) / Hq)
    prefix = torch.minimum(_ragged(g, B, (case["prefix"] + 1) // 2, case["prefix"]), lens) if case["prefix"] else None
    s.update(q=_rand(g, T, Hq, D).to(qt), lens=lens.int(), scale=D ** -0.5,
             block_table=torch.randperm(num_blocks, generator=g, device=DEV, dtype=torch.int32)[:B * cols].view(B, cols).contiguous(),
             slopes=slopes if case["alibi"] else None, prefix_lens=None if prefix is None else prefix.int(),
             out=torch.empty(T, Hq, D, dtype=qt, device=DEV), lse=None, key_weights=None, key_weights_out=None)
    if case["weights"]:
        w = torch.rand(num_blocks, Hkv, bs, generator=g, device=DEV) ** 8
        s.update(lse=torch.empty(T, Hq, device=DEV), key_weights=w, key_weights_out=w.clone())
    return s


# ---------------------------------------------------------------------------
def run(s):
    return {"decode": _run_decode, "write": _run_write, "evict": _run_evict}[s["op"]](s)


def _values(s, n):
    """The cache as 32-bit values, [num_blocks, block_size, Hkv, D]."""
    c = s[n + "_cache"]
    if s["kv"] != "fp4":
        return c.float() * s["cache_scale"]
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=c.device)
    x = torch.stack((table[(c & 15).int()], table[(c >> 4).int()]), -1)
    x = x.reshape(*c.shape[:3], -1, 16) * (s[n + "_block_scale"].float() * s["cache_scale"])[..., None]
    return x.flatten(-2).transpose(1, 2)


def _run_decode(s):
    if own:
        import paged_split_decode_gb300 as pd
        pd.decode_paged_scored(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"], s["scale"], s["window"],
                               s["qlen"], out=s["out"], score_cap=s["cap"], alibi_slopes=s["slopes"],
                               prefix_lens=s["prefix_lens"], k_block_scale=s["k_block_scale"],
                               v_block_scale=s["v_block_scale"], k_scale=s["cache_scale"], v_scale=s["cache_scale"],
                               lse=s["lse"], key_weights=s["key_weights"], key_weights_out=s["key_weights_out"],
                               error_flag=s["error_flag"])
        return [t for t in (s["out"], s["lse"], s["key_weights_out"]) if t is not None]
    table, lens, qlen = s["block_table"].long(), s["lens"].long(), s["qlen"]
    B, (Hq, D), bs = table.shape[0], s["q"].shape[1:], s["block_size"]
    k, v = (_values(s, n)[table].flatten(1, 2) for n in ("k", "v"))
    Hkv = k.shape[2]
    q = s["q"].float().view(B, qlen, Hkv, Hq // Hkv, D)
    x = torch.einsum("bihgd,bjhd->bhgij", q, k) * s["scale"]
    if s["cap"] > 0:
        x = s["cap"] * torch.tanh(x / s["cap"])
    j = torch.arange(k.shape[1], device=k.device)
    p = lens[:, None] - qlen + torch.arange(qlen, device=k.device)  # position of each query token
    far = j - p[..., None]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(Hkv, -1, 1, 1) * far.abs()[:, None, None].float()
    seen = far <= 0
    if s["window"] > 0:
        seen = seen & (far > -s["window"])
    if s["prefix_lens"] is not None:
        seen = seen | (j < s["prefix_lens"].long()[:, None, None])
    seen = (seen & (j < lens[:, None, None]) & (p[..., None] >= 0))[:, None, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(x - top), 0.0)
    total = e.sum(-1, keepdim=True)
    e = torch.where(total > 0, e / total, 0.0)
    o = torch.einsum("bhgij,bjhd->bihgd", e, v)
    out = [o.reshape(B * qlen, Hq, D).to(s["q"].dtype)]
    if s["lse"] is not None:
        lse = torch.where(total > 0, torch.where(total > 0, top, 0.0) + torch.log(total), -math.inf)
        out.append(lse[..., 0].permute(0, 3, 1, 2).reshape(B * qlen, Hq))
    if s["key_weights"] is not None:
        live = j < lens[:, None]
        blocks = table.repeat_interleave(bs, 1)
        old = s["key_weights"][blocks, :, j % bs]  # [B, keys, Hkv]
        old = torch.where((j < lens[:, None] - qlen)[..., None], old, 0.0)  # the step's own keys start from nothing
        new = old + e.sum((2, 3)).transpose(1, 2)
        w = s["key_weights_out"].clone()
        w[blocks[live], :, (j % bs).expand(B, -1)[live]] = new[live]
        out.append(w)
    return out


def _run_write(s):
    names = ("k_cache", "k_block_scale", "v_cache", "v_block_scale")
    if own:
        import paged_split_decode_gb300 as pd
        pd.write_kv_cache_fp4(s["k_new"], s["v_new"], s["slot_mapping"], s["k_cache"], s["v_cache"], s["k_block_scale"],
                              s["v_block_scale"], k_scale=s["cache_scale"], v_scale=s["cache_scale"],
                              error_flag=s["error_flag"])
        return [s[n] for n in names]
    slots, bs = s["slot_mapping"], s["block_size"]
    live = slots >= 0
    block, at = slots[live] // bs, slots[live] % bs
    scale = torch.tensor(s["cache_scale"], device=slots.device)
    for n in ("k", "v"):
        x = s[n + "_new"][live].float()
        x = x.view(*x.shape[:2], -1, 16)
        f = (x.abs().amax(-1) / (6.0 * scale)).clamp(max=448.0).to(F8)
        d = (f.float() * scale)[..., None]
        y = (x / d).abs()
        code = ((y > 0.25).to(torch.uint8) + (y >= 0.75).to(torch.uint8) + (y > 1.25).to(torch.uint8)
                + (y >= 1.75).to(torch.uint8) + (y > 2.5).to(torch.uint8) + (y >= 3.5).to(torch.uint8) + (y > 5).to(torch.uint8))
        code = torch.where(d > 0, code, 0) | (torch.signbit(x).to(torch.uint8) << 3)
        code = code.flatten(-2)
        s[n + "_cache"][block, :, at] = code[..., 0::2] | (code[..., 1::2] << 4)
        s[n + "_block_scale"].view(torch.uint8)[block, :, at] = f.view(torch.uint8)
    return [s[n] for n in names]


def _run_evict(s):
    names = ["k_cache", "v_cache", "key_weights", "lens_out"] + (["k_block_scale", "v_block_scale"] if s["kv"] == "fp4" else [])
    if own:
        import paged_split_decode_gb300 as pd
        pd.evict_kv_cache(s["k_cache"], s["v_cache"], s["key_weights"], s["block_table"], s["lens"], s["keep"],
                          first=s["first"], recent=s["recent"], block_table_out=s["table_out"], seq_lens_out=s["lens_out"],
                          k_block_scale=s["k_block_scale"], v_block_scale=s["v_block_scale"], error_flag=s["error_flag"])
        return [s[n] for n in names]
    table, lens, keep, bs = s["block_table"].long(), s["lens"].long(), s["keep"], s["block_size"]
    B, Hkv = table.shape[0], s["key_weights"].shape[1]
    j = torch.arange(table.shape[1] * bs, device=table.device)
    blocks = table.repeat_interleave(bs, 1)
    w = s["key_weights"][blocks, :, j % bs].transpose(1, 2)  # [B, Hkv, keys]
    n = lens[:, None, None]
    w = torch.where((j < s["first"]) | (j >= n - s["recent"]), math.inf, w)
    w = torch.where(j < n, w, -math.inf)
    m = min(keep, j.numel())
    kept = torch.sort(torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :m], dim=-1).values
    short = torch.arange(m, device=table.device).expand(B, Hkv, m)
    kept = torch.where(n > keep, kept, short)
    live = short < n.clamp(max=keep)
    b, h, i = live.nonzero(as_tuple=True)
    src = kept[live]
    src_block, src_at = table[b, src // bs], src % bs
    dst_block, dst_at = s["table_out"].long()[b, i // bs], i % bs
    for name in ("k_cache", "v_cache", "k_block_scale", "v_block_scale"):
        c = s[name]
        if c is None:
            continue
        if c.dtype == F8:
            c = c.view(torch.uint8)
        if s["kv"] == "fp4":
            c[dst_block, h, dst_at] = c[src_block, h, src_at]
        else:
            c[dst_block, dst_at, h] = c[src_block, src_at, h]
    s["key_weights"][dst_block, h, dst_at] = s["key_weights"][src_block, h, src_at]
    s["lens_out"].copy_(lens.clamp(max=keep))
    return [s[n] for n in names]


# ---------------------------------------------------------------------------
def work(case):
    Hq, Hkv, D = HEADS[case["heads"]]
    if case["op"] == "write":
        n = case["T"] * Hkv * D * 2
        return {"bytes": n * (2 + 9 / 16) + 8 * case["T"], "flops": 4 * n}
    kv, L, B = case["kv"], case["longest"], case["B"]
    row = D * {"fp4": 9 / 16, "e4m3": 1, "int8": 1}.get(kv, 2)
    mean = L * (33 / 64 if case["ragged"] and L > 32 else 1)
    if case["op"] == "evict":
        kept = min(mean, case["keep"])
        return {"bytes": B * Hkv * (4 * mean + kept * (4 * row + 4)) + 8 * B, "flops": 0}
    if case["window"]:
        mean = min(mean, case["window"] + case["qlen"] - 1 + 0.75 * case["prefix"])
    keys = B * mean
    qo = 2 * 2 * B * case["qlen"] * Hq * D
    return {"bytes": keys * Hkv * (2 * row + (8 if case["weights"] else 0)) + keys / case["block_size"] * 4 + qo,
            "flops": keys * case["qlen"] * Hq * D * 4}


# ---------------------------------------------------------------------------
def exact(case, seed):
    """The decodes' outputs and the 4-bit writer's scales in 64 bits, sequence by sequence and token by token's
    place; codes and moved keys have no other value."""
    if case["op"] == "evict":
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "write":
        got = []
        to = s["slot_mapping"][s["slot_mapping"] >= 0]
        for name in ("k", "v"):
            f = s[name + "_block_scale"].to(f64).transpose(1, 2).flatten(0, 1)  # a row for each slot
            x = s[name + "_new"][s["slot_mapping"] >= 0].to(f64)
            groups = x.unflatten(-1, (-1, 16))
            f[to] = torch.maximum(groups.max(-1).values, -groups.min(-1).values) / 6 / s["cache_scale"]
            got += [None, f.unflatten(0, (-1, case["block_size"])).transpose(1, 2)]
        return got
    Hq, Hkv, D = HEADS[case["heads"]]
    G, qlen, bs, kv = Hq // Hkv, case["qlen"], case["block_size"], case["kv"]
    out = torch.zeros(case["B"] * qlen, Hq, D, dtype=f64, device=DEV)
    lse = torch.full((case["B"] * qlen, Hq), -math.inf, dtype=f64, device=DEV)
    sums = s["key_weights_out"].to(f64) if case["weights"] else None

    def rows(name, blocks, L):
        c = s[name + "_cache"][blocks]
        if kv == "fp4":
            lo, hi = (c & 15).to(torch.int64), (c >> 4).to(torch.int64)
            code = torch.stack((lo, hi), -1).flatten(-2)
            mag, e = (code & 1).to(f64), (code >> 1) & 3
            x = torch.where(e == 0, mag / 2, (1 + mag / 2) * torch.exp2((e - 1).to(f64)))
            x = torch.where(code >= 8, -x, x)
            x = x * s[name + "_block_scale"][blocks].to(f64).repeat_interleave(16, -1)
            c = x.permute(0, 2, 1, 3)
        return c.to(f64).reshape(-1, Hkv, D)[:L] * s["cache_scale"]

    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        blocks = s["block_table"][b, :-(-L // bs)].long()
        K, V = rows("k", blocks, L), rows("v", blocks, L)
        prefix = int(s["prefix_lens"][b]) if case["prefix"] else 0
        at = torch.arange(L, device=DEV)
        got = torch.zeros(L, Hkv, dtype=f64, device=DEV)
        for i in range(qlen):
            pos = L - qlen + i
            if pos < 0:
                continue
            ok = (at < prefix) | ((at <= pos) & ((at > pos - case["window"]) if case["window"] > 0 else at >= 0))
            if not bool(ok.any()):
                continue
            for h in range(Hkv):
                heads = slice(h * G, (h + 1) * G)
                y = s["q"][b * qlen + i, heads].to(f64) @ K[ok, h].T * s["scale"]
                if case["cap"]:
                    y = torch.tanh(y / case["cap"]) * case["cap"]
                if case["alibi"]:
                    y = y - s["slopes"][heads, None].to(f64) * (pos - at[ok]).abs()
                lse[b * qlen + i, heads] = torch.logsumexp(y, -1)
                p = torch.softmax(y, -1)
                out[b * qlen + i, heads] = p @ V[ok, h]
                got[ok, h] += p.sum(0)
        if case["weights"]:
            old = s["key_weights"][blocks].to(f64).permute(0, 2, 1).reshape(-1, Hkv)[:L].clone()
            old[max(L - qlen, 0):] = 0
            full = sums[blocks].permute(0, 2, 1).reshape(-1, Hkv)
            full[:L] = old + got
            sums[blocks] = full.view(len(blocks), bs, Hkv).permute(0, 2, 1)
    return [out, lse, sums] if case["weights"] else [out]
