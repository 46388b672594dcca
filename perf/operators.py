"""Cases of the serving step around the paged cache: block tables and slot maps
built on the GPU, differential attention over the paged cache, and the
root-mean-square norm with its 8-bit output.

Each case runs in a plain form (elementary torch operations in 32 bits) or,
with ``own`` set, through this package's calls on the same state. The passes
write to buffers that the state keeps, as a program that replays its step in a
CUDA graph does, and read the free list's count from one buffer and write it
to another, so that a pass leaves its inputs as they were.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": F8, "int8": torch.int8}
# (query heads, KV heads, head size) of this repository's workloads and tests
HEADS = ((24, 4, 256), (32, 8, 128), (28, 4, 128), (8, 2, 128), (6, 6, 128), (12, 2, 256))
MIN_SCALE = 2.0 ** -100


def listed():
    return [
        # one token for each of 32 running sequences of about 4096 keys: every decode step
        dict(name="tables_decode_b32", op="tables", B=32, T=32, cols=256, block_size=16, longest=4096, chunk=1),
        # a continuous batch: most sequences decode, some bring a chunk of their prompt; the token buffer is padded
        dict(name="tables_mixed_b256", op="tables", B=256, T=8192, cols=1024, block_size=16, longest=16384, chunk=997),
        # a prefill step of 32768 tokens over long tables
        dict(name="tables_prefill_b64", op="tables", B=64, T=32768, cols=2048, block_size=16, longest=32768, chunk=0),
        # a few of 32 sequences end in a step
        dict(name="release_b32", op="release", B=32, cols=256, block_size=16, longest=4096, every=7),
        # a large batch is dropped: half of 1024 sequences of up to 16384 keys
        dict(name="release_b1024", op="release", B=1024, cols=1024, block_size=16, longest=16384, every=2),
        # a single request decoding: latency
        dict(name="diff_f16_b1", op="diff", kv="f16", q="f16", B=1, heads=0, longest=4096, ragged=False, qlen=1,
             window=0, block_size=16, norm=False),
        # the headline batch of 32 sequences
        dict(name="diff_f16_b32", op="diff", kv="f16", q="f16", B=32, heads=0, longest=4096, ragged=False, qlen=1,
             window=0, block_size=16, norm=True),
        # ragged lengths in [512, 16384], bfloat16
        dict(name="diff_bf16_ragged_b32", op="diff", kv="bf16", q="bf16", B=32, heads=1, longest=16384, ragged=True,
             qlen=1, window=0, block_size=16, norm=False),
        # speculative verify of three tokens over an e4m3 cache
        dict(name="diff_e4m3_verify_b8", op="diff", kv="e4m3", q="bf16", B=8, heads=0, longest=8192, ragged=False,
             qlen=3, window=0, block_size=16, norm=True),
        # the heads of one decode step normalised one by one, quantised for the output projection
        dict(name="norm_heads_b32", op="norm", dtype="bf16", out="e4m3", rows=32, N=6144, norm=256, scale=6144,
             residual=False),
        # a block's norm in a prefill step: residual added, 8-bit output with a scale for every 128 values
        dict(name="norm_residual_t8192", op="norm", dtype="bf16", out="e4m3", rows=8192, N=6144, norm=6144, scale=128,
             residual=True),
        # the widest step, output in the input's type
        dict(name="norm_residual_t32768", op="norm", dtype="f16", out="f16", rows=32768, N=4096, norm=4096, scale=0,
             residual=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("tables", "release", "diff", "diff", "norm", "norm"))
    if op == "tables":
        B, longest, bs = _log(rng, 1, 1024), _log(rng, 64, 32768), rng.choice((16, 32, 64))
        T = _log(rng, 1, 32768)
        return dict(op=op, B=B, T=max(T, B), cols=-(-longest // bs) + rng.randrange(3), block_size=bs,
                    longest=longest, chunk=rng.choice((0, 1, _log(rng, 1, 2048))))
    if op == "release":
        longest, bs = _log(rng, 64, 16384), rng.choice((16, 32, 64))
        return dict(op=op, B=_log(rng, 1, 1024), cols=-(-longest // bs) + rng.randrange(3), block_size=bs,
                    longest=longest, every=rng.randrange(1, 9))
    if op == "diff":
        h = rng.randrange(len(HEADS))
        Hq, Hkv, D = HEADS[h]
        kv = rng.choice(("f16", "bf16", "e4m3", "int8"))
        q = kv if kv in ("f16", "bf16") else rng.choice(("f16", "bf16"))
        B = _log(rng, 1, 48)
        most = (32 * 4096 * 4 * 256) // (B * Hkv * D)  # keys a sequence: at most the headline batch's cache
        longest = _log(rng, 1, min(32768, most))
        qlen = min(rng.choice((1, 1, 1, 2, 3, 5)), 32 // (Hq // Hkv), longest)
        window = rng.choice((0, 0, _log(rng, 1, longest)))
        return dict(op=op, kv=kv, q=q, B=B, heads=h, longest=longest, ragged=rng.random() < 0.5, qlen=qlen,
                    window=window, block_size=rng.choice((16, 32, 64)), norm=rng.random() < 0.5)
    while True:
        rows, unit = _log(rng, 1, 32768), rng.choice((32, 64, 80, 104, 128, 256))
        groups = _log(rng, 1, 8192 // unit)
        N = unit * groups
        if rows * N <= 32768 * 4096:
            break
    x, out = rng.choice(("f16", "bf16")), rng.choice(("same", "e4m3"))
    return dict(op=op, dtype=x, out=x if out == "same" else out, rows=rows, N=N, norm=rng.choice((unit, N)),
                scale=0 if out == "same" else rng.choice((unit, N)), residual=rng.random() < 0.7)


# ---------------------------------------------------------------------------
def _ragged(g, B, lo, hi):
    return torch.randint(lo, hi + 1, (B,), generator=g, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] in ("tables", "release"):
        B, cols, bs = case["B"], case["cols"], case["block_size"]
        num_blocks = B * cols + 7
        if case["op"] == "tables":
            T, longest = case["T"], case["longest"]
            if case["chunk"] == 1:  # every sequence decodes one token
                query = torch.ones(B, dtype=torch.long, device=DEV)
            elif case["chunk"] == 0:  # prompts only: equal shares of the step's tokens
                query = torch.full((B,), max(1, min(T // B, longest)), dtype=torch.long, device=DEV)
            else:  # one sequence in eight brings a chunk of its prompt
                chunk = torch.where(torch.rand(B, generator=g, device=DEV) < 0.125,
                                    _ragged(g, B, 1, max(1, min(case["chunk"], longest))), 1)
                fits = torch.cumsum(chunk, 0) + (B - 1 - torch.arange(B, device=DEV)) <= T
                query = torch.where(fits, chunk, 1)
            context = (torch.rand(B, generator=g, device=DEV) * (longest - query + 1)).long()
            context = torch.minimum(context, longest - query)
        else:
            context = _ragged(g, B, 0, case["longest"])
            s["released"] = _ragged(g, B, 0, case["every"] - 1) == 0
        order = torch.randperm(num_blocks, generator=g, device=DEV, dtype=torch.int32)
        held = (context + bs - 1) // bs
        start = torch.cumsum(held, 0) - held
        c = torch.arange(cols, device=DEV)
        table = order[(start[:, None] + c).clamp(max=num_blocks - 1)]
        table = torch.where(c < held[:, None], table, -1)
        used = held.sum()  # blocks in use come first in `order`, the free ones after them
        free = order.roll(-int(used.item())).contiguous()
        s.update(block_table=table, free_blocks=free, num_blocks=num_blocks,
                 free_count=(num_blocks - used).to(torch.int32).reshape(1), free_count_out=torch.empty(1, dtype=torch.int32, device=DEV),
                 seq_lens=torch.empty(B, dtype=torch.int32, device=DEV),
                 error_flag=torch.zeros(1, dtype=torch.int32, device=DEV))
        if case["op"] == "tables":
            s.update(context_lens=context.int(), query_lens=query.int(),
                     query_start_loc=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                     slot_mapping=torch.empty(case["T"], dtype=torch.long, device=DEV),
                     positions=torch.empty(case["T"], dtype=torch.int32, device=DEV))
        else:
            s.update(lens=context.int())
        return s
    if case["op"] == "diff":
        (Hq, Hkv, D), B, L, bs = HEADS[case["heads"]], case["B"], case["longest"], case["block_size"]
        lens = torch.full((B,), L, device=DEV)
        if case["ragged"]:
            lens = torch.where(torch.rand(B, generator=g, device=DEV) < 0.06, 0, _ragged(g, B, max(case["qlen"], L // 32), L))
            lens[0] = L
        cols = -(-L // bs)
        num_blocks = B * cols + 1
        qt = TYPES[case["q"]]

        def cache():
            x = torch.randn(num_blocks, bs, Hkv, D, generator=g, device=DEV, dtype=torch.float32 if case["kv"] in ("e4m3", "int8") else TYPES[case["kv"]])
            if case["kv"] == "e4m3":
                return (x / 0.0125).to(F8)
            return (x / 0.0375).round().clamp(-127, 127).to(torch.int8) if case["kv"] == "int8" else x

        s["k_cache"], s["v_cache"] = cache(), cache()
        s["cache_scale"] = {"e4m3": 0.0125, "int8": 0.0375}.get(case["kv"], 1.0)
        s.update(q=torch.randn(B * case["qlen"], Hq, D, generator=g, device=DEV).to(qt),
                 lam=0.2 + 0.6 * torch.rand(Hq, generator=g, device=DEV),
                 block_table=torch.randperm(num_blocks, generator=g, device=DEV, dtype=torch.int32)[:B * cols].view(B, cols).contiguous(),
                 lens=lens.int(), attn_scale=(D // 2) ** -0.5, eps=1e-5, gain=0.4,
                 weight=(1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(qt) if case["norm"] else None,
                 out=torch.empty(B * case["qlen"], Hq, D, dtype=qt, device=DEV),
                 error_flag=torch.zeros(1, dtype=torch.int32, device=DEV))
        return s
    xt, rows, N = TYPES[case["dtype"]], case["rows"], case["N"]
    s.update(x=torch.randn(rows, N, generator=g, device=DEV, dtype=xt),
             weight=(1 + 0.1 * torch.randn(case["norm"], generator=g, device=DEV)).to(xt),
             added=torch.randn(rows, N, generator=g, device=DEV, dtype=xt) if case["residual"] else None,
             residual_out=torch.empty(rows, N, dtype=xt, device=DEV) if case["residual"] else None,
             y=torch.empty(rows, N, dtype=TYPES[case["out"]], device=DEV),
             y_scale=torch.empty(rows, N // case["scale"], device=DEV) if case["scale"] else None,
             eps=1e-5)
    return s


# ---------------------------------------------------------------------------
def run(s):
    return {"tables": _tables, "release": _release, "diff": _diff, "norm": _norm}[s["op"]](s)


def _tables(s):
    if own:
        import paged_split_decode_gb300 as pd
        pd.build_block_tables(s["context_lens"], s["query_lens"], s["block_table"], s["free_blocks"], s["free_count"],
                              s["block_size"], seq_lens=s["seq_lens"], query_start_loc=s["query_start_loc"],
                              slot_mapping=s["slot_mapping"], positions=s["positions"],
                              free_count_out=s["free_count_out"], error_flag=s["error_flag"])
        return [s[k] for k in ("seq_lens", "query_start_loc", "block_table", "slot_mapping", "positions", "free_count_out")]
    bs, table, free = s["block_size"], s["block_table"], s["free_blocks"]
    context, query = s["context_lens"].long(), s["query_lens"].long()
    seq = context + query
    held, want = (context + bs - 1) // bs, (seq + bs - 1) // bs
    off = torch.cumsum(want - held, 0) - (want - held)
    ends = torch.cumsum(query, 0)
    start = torch.cat([ends.new_zeros(1), ends])
    # the k-th block that the step takes is the k-th from the free list's top
    c = torch.arange(table.shape[1], device=table.device)
    at = s["free_count"].long() - 1 - (off[:, None] + c - held[:, None])
    new = (c >= held[:, None]) & (c < want[:, None])
    table = torch.where(new, free[at.clamp(0, free.numel() - 1)], table)
    t = torch.arange(s["T"], device=table.device)
    b = torch.searchsorted(ends, t, right=True)
    live = b < ends.numel()
    b = b.clamp(max=ends.numel() - 1)
    pos = torch.where(live, context[b] + t - start[b], 0)
    slot = torch.where(live, table[b, (pos // bs).clamp(max=table.shape[1] - 1)].long() * bs + pos % bs, -1)
    count = s["free_count"] - (want - held).sum()
    return [seq.int(), start.int(), table, slot, pos.int(), count.int()]


def _release(s):
    if own:
        import paged_split_decode_gb300 as pd
        pd.release_blocks(s["block_table"], s["lens"], s["released"], s["free_blocks"], s["free_count"], s["block_size"],
                          seq_lens_out=s["seq_lens"], free_count_out=s["free_count_out"], error_flag=s["error_flag"])
        return [s[k] for k in ("seq_lens", "free_blocks", "free_count_out")]
    bs, table, free = s["block_size"], s["block_table"], s["free_blocks"]
    lens = s["lens"].long()
    n = torch.where(s["released"], (lens + bs - 1) // bs, 0)
    off = torch.cumsum(n, 0) - n
    c = torch.arange(table.shape[1], device=table.device)
    # blocks return in the order of the sequences, on top of the list; the others land behind its end
    at = torch.where(c < n[:, None], s["free_count"].long() + off[:, None] + c, free.numel())
    out = torch.cat([free, free.new_zeros(1)])
    out[at.reshape(-1)] = table.reshape(-1)
    return [torch.where(s["released"], 0, lens).int(), out[:-1], (s["free_count"] + n.sum()).int()]


def _diff(s):
    if own:
        import paged_split_decode_gb300 as pd
        return pd.decode_paged_diff(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"], s["lam"],
                                    s["attn_scale"], s["window"], s["qlen"], out=s["out"], norm_weight=s["weight"],
                                    norm_eps=s["eps"], norm_gain=s["gain"], k_scale=s["cache_scale"],
                                    v_scale=s["cache_scale"], error_flag=s["error_flag"])
    table, lens, qlen = s["block_table"].long(), s["lens"].long(), s["qlen"]
    B, (Hq, D), Hkv = table.shape[0], s["q"].shape[1:], s["k_cache"].shape[2]
    k = s["k_cache"][table].float().view(B, -1, Hkv, 2, D // 2) * s["cache_scale"]
    v = s["v_cache"][table].float().view(B, -1, Hkv, D) * s["cache_scale"]
    q = s["q"].float().view(B, qlen, Hkv, Hq // Hkv, 2, D // 2)
    x = torch.einsum("bihgmd,bjhmd->bhgmij", q, k) * s["attn_scale"]
    j = torch.arange(k.shape[1], device=k.device)
    p = lens[:, None] - qlen + torch.arange(qlen, device=k.device)  # position of each query token
    seen = j <= p[..., None]
    if s["window"] > 0:
        seen &= j > p[..., None] - s["window"]
    x = torch.where(seen[:, None, None, None], x, -math.inf)
    e = torch.where(seen[:, None, None, None], torch.exp(x - x.amax(-1, keepdim=True)), 0.0)
    total = e.sum(-1, keepdim=True)
    e = torch.where(total > 0, e / total, 0.0)
    o = torch.einsum("bhgmij,bjhd->bihgmd", e, v)
    o = o[..., 0, :] - s["lam"].view(Hkv, -1, 1) * o[..., 1, :]
    if s["weight"] is not None:
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float() * s["gain"]
    return o.reshape(B * qlen, Hq, D).to(s["q"].dtype)


def _norm(s):
    if own:
        import paged_split_decode_gb300 as pd
        pd.rms_norm(s["x"], s["weight"], s["eps"], residual=s["added"], residual_out=s["residual_out"],
                    norm_size=s["norm"], scale_size=s["scale"] or None, out=s["y"], out_scale=s["y_scale"])
        return [t for t in (s["y"], s["y_scale"], s["residual_out"]) if t is not None]
    x = s["x"].float()
    rows, N = x.shape
    if s["added"] is not None:
        x = x + s["added"].float()
    h = x.view(rows, -1, s["norm"])
    y = (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()).view(rows, N)
    if s["y_scale"] is None:
        out = [y.to(s["y"].dtype)]
    else:
        z = y.view(rows, -1, s["scale"])
        scale = (z.abs().amax(-1, keepdim=True) / 448.0).clamp(min=MIN_SCALE)
        out = [(z / scale).view(rows, N).to(F8), scale[..., 0]]
    return out if s["added"] is None else out + [x.to(s["x"].dtype)]


# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "tables":
        B, T = case["B"], case["T"]
        # lengths, the blocks' ids (at least one entry a sequence read), the maps written
        return {"bytes": 4 * (5 * B + 2) + 4 * B + 12 * T, "flops": 0}
    if case["op"] == "release":
        blocks = case["B"] / case["every"] * (case["longest"] / 2 / case["block_size"])
        return {"bytes": 9 * case["B"] + 8 * blocks + 8, "flops": 0}
    if case["op"] == "diff":
        Hq, Hkv, D = HEADS[case["heads"]]
        mean = case["longest"] * (33 / 64 if case["ragged"] and case["longest"] > 32 else 1)
        if case["window"]:
            mean = min(mean, case["window"] + case["qlen"] - 1)
        keys = case["B"] * mean
        size = 1 if case["kv"] in ("e4m3", "int8") else 2
        qo = 2 * 2 * case["B"] * case["qlen"] * Hq * D
        return {"bytes": keys * Hkv * D * 2 * size + keys / case["block_size"] * 4 + qo,
                "flops": keys * case["qlen"] * Hq * D * 6}
    n = case["rows"] * case["N"]
    size = 2 + (1 if case["out"] == "e4m3" else 2) + (4 if case["residual"] else 0)
    return {"bytes": n * size + (4 * n / case["scale"] if case["scale"] else 0) + 2 * case["norm"], "flops": 8 * n}


# ---------------------------------------------------------------------------
def exact(case, seed):
    """The same outputs in 64 bits, sequence by sequence; None for whole numbers."""
    if case["op"] in ("tables", "release"):
        return None
    s = prepare(case, seed)
    if case["op"] == "diff":
        Hq, Hkv, D = HEADS[case["heads"]]
        half, G, qlen = D // 2, Hq // Hkv, case["qlen"]
        out = torch.zeros(case["B"] * qlen, Hq, D, dtype=torch.float64, device=DEV)
        for b, L in enumerate(s["lens"].tolist()):
            if L == 0:
                continue
            rows = s["block_table"][b].long()
            K = s["k_cache"][rows].to(torch.float64).reshape(-1, Hkv, D)[:L] * s["cache_scale"]
            V = s["v_cache"][rows].to(torch.float64).reshape(-1, Hkv, D)[:L] * s["cache_scale"]
            for i in range(qlen):
                last = L - qlen + i
                first = max(0, last - case["window"] + 1) if case["window"] > 0 else 0
                if last < first:
                    continue
                for h in range(Hkv):
                    q = s["q"][b * qlen + i, h * G:(h + 1) * G].to(torch.float64)
                    k, v = K[first:last + 1, h], V[first:last + 1, h]
                    maps = [torch.softmax(q[:, m * half:(m + 1) * half] @ k[:, m * half:(m + 1) * half].T * s["attn_scale"], -1)
                            for m in (0, 1)]
                    lam = s["lam"][h * G:(h + 1) * G, None].to(torch.float64)
                    out[b * qlen + i, h * G:(h + 1) * G] = (maps[0] - lam * maps[1]) @ v
        if s["weight"] is not None:
            size = (out.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt()
            out = out / size * s["weight"].to(torch.float64) * s["gain"]
        return out
    chunks = []
    rows, N, step = case["rows"], case["N"], max(1, (1 << 25) // case["N"])
    for r in range(0, rows, step):
        h = s["x"][r:r + step].to(torch.float64)
        if s["added"] is not None:
            h = h + s["added"][r:r + step].to(torch.float64)
        size = (h.reshape(-1, N // case["norm"], case["norm"]).square().sum(-1, keepdim=True) / case["norm"] + s["eps"]).sqrt()
        y = h.reshape(-1, N // case["norm"], case["norm"]) / size * s["weight"].to(torch.float64)
        got = []
        if case["scale"]:
            z = y.reshape(-1, N // case["scale"], case["scale"])
            amax = z.abs().max(-1, keepdim=True).values / 448
            got = [(z / amax).reshape(-1, N), amax[..., 0]]
        else:
            got = [y.reshape(-1, N)]
        chunks.append(got + ([h] if s["added"] is not None else []))
    return [torch.cat(c) for c in zip(*chunks)]
