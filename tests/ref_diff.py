"""Differential decode in 64 bits from the fp64 oracle: each softmax map is the
oracle run on q with the other half of every row zeroed (a zero half adds
nothing to a score), so out = map 1 - lambda map 2, then the heads' norm.

Error bound of the GPU kernel, per element. u is half a step of the operands'
type (fp16 2^-11, bfloat16 2^-8; byte caches compute in fp16): each softmax
weight is rounded to it before P.V, so map m is off by at most u A_m, A_m =
sum_j w_j |v_j| (the oracle run on |V|). The fp32 parts: a score sums D / 2
products, off by at most (D / 2) 2^-24 sum |q_d k_d| scale < 2^-13 for the
N(0, 1) rows drawn here, which moves a weight by that relative amount, and
exponentials, rescalings and sums stay below it: 2^-12 A_m together. With e4m3
caches and several query rows per head, q enters as e4m3 terms that leave at
most 2^-17 max|q| of elements below 2^-6 max|q| (N(0, 1): fewer than a quarter
of a half row's 64 or 128); a score then moves by less than 2^-17 5.5 32 0.8
128^-1/2 < 2^-13 more, so 2^-11 stands for all of it there (f). So

    d = (u + f) (A_1 + |lambda| A_2),   |gpu - ref| <= d + u_out |ref|

with f = 2^-12, or 2^-11 for e4m3, and u_out the half step of the output type. The norm gives y = o f w, f = gain
/ sqrt(mean o^2 + eps); with e = rms(d) over the row, the computed row's rms
is within e of o's, so f lies between f_lo and f_hi, its values at rms(o) + e
and max(rms(o) - e, 0), and

    |y' - y| <= |w| (d f_hi + |o| max(f_hi - f, f - f_lo)).
"""
import numpy as np
import torch

import oracle

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def as_np(t):
    return t.view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.numpy()


def _oracle(w, q, v):
    kw = dict(k_scale=w.k_scale, v_scale=w.v_scale, kv_fp8=w.kv_fp8, kv_int8=w.kv_int8, bf16=w.bf16)
    k, bt, sl = as_np(w.k_cache), w.block_table.numpy(), w.seq_lens.numpy()
    if w.q_start is not None:
        return oracle.decode_paged_varlen(q, k, v, bt, sl, w.q_start.numpy(), w.scale, w.window, **kw)
    return oracle.decode_paged(q, k, v, bt, sl, w.scale, w.window, w.qlen, **kw)


def _abs_codes(w):
    v = as_np(w.v_cache).copy()
    if w.kv_int8:
        return np.abs(v.view(np.int8).astype(np.int16)).astype(np.uint8)
    if w.kv_fp8:
        return v & np.uint8(0x7F)
    return v.view(np.uint16) & np.uint16(0x7FFF)


def _bits(a):
    return a.view(np.uint16) if a.dtype == np.float16 else a


def reference(w, lam, norm_weight=None, eps=1e-5, gain=1.0):
    """(out, bound) in 64 bits for workload w; lam [Hq] as fp64."""
    half = w.D // 2
    q = _bits(as_np(w.q))
    out = bound = 0.0
    u = 2.0 ** -11 if (w.kv_fp8 or w.kv_int8) else HALF_STEP[w.q.dtype]
    for m in (0, 1):
        qm = q.copy()
        qm[..., half:] = qm[..., half:] if m else 0
        if m:
            qm[..., :half] = 0
        if not w.bf16:
            qm = qm.view(np.float16)
        c = (-1.0 if m else 1.0) * (lam[:, None] if m else 1.0)
        out = out + c * _oracle(w, qm, as_np(w.v_cache))
        va = _abs_codes(w)
        bound = bound + np.abs(c) * _oracle(w, qm, va.view(np.float16) if va.dtype == np.uint16 and not w.bf16 else va)
    bound = (u + 2.0 ** (-11 if w.kv_fp8 else -12)) * bound
    if norm_weight is not None:
        rms = np.sqrt(np.mean(out ** 2, axis=-1, keepdims=True))
        e = np.sqrt(np.mean(bound ** 2, axis=-1, keepdims=True))
        f, lo, hi = (gain / np.sqrt(x ** 2 + eps) for x in (rms, rms + e, np.maximum(rms - e, 0.0)))
        bound = np.abs(norm_weight) * (bound * hi + np.abs(out) * np.maximum(hi - f, f - lo))
        out = out * f * norm_weight
    return out, bound + HALF_STEP[w.q.dtype] * np.abs(out) + 2.0 ** -24
