"""Paged NVFP4 key/value cache: append with rotation, gather, attention.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Buffers are numpy uint8 arrays shaped as the library's header says: codes
[pages, heads, page, D/2], the keys' scales [pages, heads, page, D/16], the
values' scales [pages, heads, D/16, page].  Quantization is ``oracle.quantize``
(NVFP4); the rotation is fp32 with each product and sum rounded once; attention
is computed in fp64 from the cache's bytes.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from .add_rmsnorm_quant import quantize
from .formats import e2m1_decode, e4m3_decode

F32 = np.float32


def rotate(x, positions, cos_sin, interleaved: bool) -> np.ndarray:
    """x [T, H, D] fp32 with the pairs of its first cos_sin.shape[1] channels turned."""
    x = np.asarray(x, F32).copy()
    rot = cos_sin.shape[1]
    half = rot // 2
    row = np.asarray(cos_sin, F32)[positions]
    cos, sin = row[:, None, :half], row[:, None, half:]
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
        (slice(0, half), slice(half, rot))
    a, b = x[..., first].copy(), x[..., second].copy()
    x[..., first] = a * cos - b * sin          # numpy rounds each of the three operations
    x[..., second] = b * cos + a * sin
    return x


def append(cache, k, v, slots, positions=None, cos_sin=None, interleaved=False,
           k_gs=1.0, v_gs=1.0, q=None):
    """Writes k, v [T, heads, D] (fp32) into the four buffers in place; returns the
    rotated q (fp32, not rounded to 16 bits) and the mask of tokens that take part."""
    kp, ks, vp, vs = cache
    pages, heads, page, half = kp.shape
    D = 2 * half
    T = k.shape[0]
    here = np.ones(T, bool)
    if cos_sin is not None:
        here = (positions >= 0) & (positions < cos_sin.shape[0])
        safe = np.where(here, positions, 0)
        k = rotate(k, safe, cos_sin, interleaved)
        q = None if q is None else rotate(q, safe, cos_sin, interleaved)

    def blocks(x, gs):
        o = quantize(np.ascontiguousarray(x, F32).reshape(T * heads, D), "nvfp4", "rowmajor",
                     global_scale=gs)
        return (o.packed.reshape(T, heads, half), o.sf_rowmajor.reshape(T, heads, D // 16))
    kc, ksf = blocks(k, k_gs)
    vc, vsf = blocks(v, v_gs)
    for t in range(T):
        if not here[t] or not 0 <= slots[t] < pages * page:
            continue
        pg, at = divmod(int(slots[t]), page)
        kp[pg, :, at], ks[pg, :, at] = kc[t], ksf[t]
        vp[pg, :, at], vs[pg, :, :, at] = vc[t], vsf[t]
    return q, here


def _decode(codes, sf):
    """fp64 values of codes [..., D/2] and scale bytes [..., D/16]."""
    n = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]), np.uint8)
    n[..., 0::2], n[..., 1::2] = codes & 15, codes >> 4
    return e2m1_decode(n).astype(np.float64) * np.repeat(e4m3_decode(sf).astype(np.float64), 16, -1)


def gather(cache, slots, k_gs=1.0, v_gs=1.0):
    """fp64 (k, v) [T, heads, D] of valid slots."""
    kp, ks, vp, vs = cache
    pg, at = np.divmod(np.asarray(slots, np.int64), kp.shape[2])
    return _decode(kp[pg, :, at], ks[pg, :, at]) / k_gs, _decode(vp[pg, :, at], vs[pg, :, :, at]) / v_gs


@dataclass
class AttentionResult:
    out: np.ndarray        # [T, Hq, D] fp64; rows of no sequence are NaN
    lse: np.ndarray        # [T, Hq] fp64
    weight: np.ndarray     # [T, Hq, D] sum of p |v|: what errors of p and of the sum scale with
    logit: np.ndarray      # [T, Hq] largest sum of |scale q k| over the row's keys
    keys: np.ndarray       # [T] keys the row sees
    rows: np.ndarray       # [T] bool: rows of a sequence
    bias: np.ndarray       # [T, Hq] sum of p |bias|, and
    bias_weight: np.ndarray  # [T, Hq, D] sum of p |bias| |v|: what errors relative to a bias scale with
    largest: np.ndarray    # [T, Hq, D] largest |v| that the row sees


def attention(q, cache, tables, seq_lens, cu=None, causal=True, sm_scale=1.0, k_gs=1.0, v_gs=1.0,
              softcap=0.0, slopes=None, window=0, prefix=None):
    """Row i of a sequence's n_q stands at place len - n_q + i.  softcap: logits x become
    softcap * tanh(x / softcap); slopes [Hq]: slope * distance is taken off; window, prefix [B]:
    with causal, the latest `window` keys up to the row's place, and the first prefix[b]."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    pages, heads, page, _ = cache[0].shape
    B = len(seq_lens)
    cu = np.arange(B + 1) if cu is None else np.asarray(cu)
    res = AttentionResult(np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan), np.zeros((T, Hq, D)),
                          np.zeros((T, Hq)), np.zeros(T, np.int64), np.zeros(T, bool), np.zeros((T, Hq)),
                          np.zeros((T, Hq, D)), np.zeros((T, Hq, D)))
    for b in range(B):
        n_q = int(cu[b + 1] - cu[b])
        n = int(min(max(seq_lens[b], 0), tables.shape[1] * page))
        if n_q <= 0:
            continue
        j = np.arange(n)
        pg = np.asarray(tables[b], np.int64)[j // page]
        ok = (pg >= 0) & (pg < pages)
        safe = np.where(ok, pg, 0) * page + j % page
        k, v = gather(cache, safe, k_gs, v_gs)
        k[~ok], v[~ok] = 0.0, 0.0
        for i in range(n_q):
            t = int(cu[b]) + i
            place = n - n_q + i
            seen = j <= (place if causal else n - 1)
            if prefix is not None:
                seen |= j < prefix[b]
            if window:
                seen &= j > place - window
            seen &= ok
            res.rows[t], res.keys[t] = True, seen.sum()
            for h in range(Hq):
                kk, vv = k[seen, h // (Hq // heads)], v[seen, h // (Hq // heads)]
                if not len(kk):
                    res.out[t, h], res.lse[t, h] = 0.0, -np.inf
                    continue
                s = sm_scale * (kk @ q[t, h])
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                bias = np.zeros(len(s)) if slopes is None else float(slopes[h]) * np.abs(place - j[seen])
                s = s - bias
                top = s.max()
                p = np.exp(s - top)
                res.lse[t, h] = top + np.log(p.sum())
                p /= p.sum()
                res.out[t, h], res.weight[t, h] = p @ vv, p @ np.abs(vv)
                res.bias[t, h], res.bias_weight[t, h] = p @ bias, (p * bias) @ np.abs(vv)
                res.largest[t, h] = np.abs(vv).max(0)
                res.logit[t, h] = sm_scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return res
