"""Helpers of the paged cache's tests: caches built on the host, the 64-bit attention over them and the bounds that
the kernels' arithmetic allows."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle
from oracle import kv4

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # of a rounding, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}     # ... of a subnormal result


def block_table(lens, page_size, seed, spare=3, width=None):
    """A table of shuffled pages [b, width] and the pages there are; entries that no key reaches are out of range."""
    per = [math.ceil(n / page_size) for n in lens]
    count = sum(per) + spare
    order = np.random.default_rng(seed).permutation(count)
    width = max(1, max(per)) if width is None else width
    table = np.full((len(lens), width), 1 << 29, dtype=np.int32)
    at = 0
    for i, p in enumerate(per):
        table[i, :p] = order[at:at + p]
        at += p
    return table, count


def rope_table(positions, rot):
    half = rot // 2
    a = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def place(table, page_size, seq, pos):
    return int(table[seq, pos // page_size]), pos % page_size


def build_cache4(ks, vs, table, count, page_size, group, fill=0xFF):
    """A 4-bit cache of per-sequence rows ks[i], vs[i] [n, hkv, d] (16-bit); every other byte is `fill` (0xFF: NaN
    pairs).  Returns the bytes [count, hkv, page bytes] and the held values per sequence."""
    d, hkv = ks[0].shape[2], ks[0].shape[1]
    ub = kv4.unit_bytes(d, group)
    cache = np.full((count, hkv, page_size // 32 * ub), fill, dtype=np.uint8)
    held = []
    for i, (k, v) in enumerate(zip(ks, vs)):
        kc, kp = kv4.quantise(k, group)
        vc, vp = kv4.quantise(v, group)
        held.append(((kc, kp), (vc, vp)))
        for first in range(0, k.shape[0], page_size):
            page = int(table[i, first // page_size])
            end = min(k.shape[0], first + page_size)
            for h in range(hkv):
                kv4.write(cache[page, h], 0, ((kc[first:end, h], kp[first:end, h]), (vc[first:end, h], vp[first:end, h])),
                          group)
    return cache, held


def attend64(q, held, group, scale, window=-1, softcap=0.0):
    """O, LSE and bounds of |O - ref|, |LSE - ref| for q [b, sq, hq, d] over held values (see build_cache4).

    Score error: q K^T is a sum of d / group terms scale * (sum q c) + min * (sum q) of exact products in fp32, at
    most (d + 16) roundings of 2^-24 of the sum of their magnitudes |q| (15 scale + |min|); the cap adds 2^-21 of
    its width.  A probability is off by that times itself, plus 2^-21 of hardware exp2, plus one fp16 rounding of
    probability * V scale (2^-11), which multiplies V's centred part scale * (code - 8); then O is rounded once."""
    b, sq, hq, d = q.shape
    dt = q.dtype
    o, lse = np.zeros((b, sq, hq, d)), np.full((b, hq, sq), -np.inf)
    o_tol, l_tol = np.zeros((b, sq, hq, d)), np.zeros((b, hq, sq))
    hkv = held[0][0][0].shape[1]
    g = hq // hkv
    qd = q.double().numpy()
    for i, ((kc, kp), (vc, vp)) in enumerate(held):
        n = kc.shape[0]
        k, v = kv4.values(kc, kp, group), kv4.values(vc, vp, group)
        vs = np.repeat(vp[..., 0].double().numpy(), group, -1)
        mid = abs(vs * (vc.astype(np.float64) - 8))
        kmag = np.repeat((15 * kp[..., 0].double() + kp[..., 1].double().abs()).numpy(), group, -1)
        for t in range(sq):
            last = n - sq + t
            first = max(0, last - window) if window >= 0 else 0
            if last < 0:
                continue
            keys = slice(first, last + 1)
            for h in range(hq):
                kh, vh = k[keys, h // g], v[keys, h // g]
                x = scale * (kh @ qd[i, t, h])
                ds = scale * (d + 16) * 2.0 ** -24 * (kmag[keys, h // g] @ abs(qd[i, t, h])) + 2.0 ** -22 * abs(x)
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                    ds = ds + softcap * 2.0 ** -21
                m = x.max()
                p = np.exp(x - m)
                l = p.sum()
                p /= l
                o[i, t, h] = p @ vh
                lse[i, h, t] = m + math.log(l)
                e = ds + ds.max() + 2.0 ** -20
                o_tol[i, t, h] = (HALF_STEP[dt] * abs(o[i, t, h]) + TINY[dt] + 2.0 ** -11 * (p @ mid[keys, h // g])
                                  + 1.01 * ((p * e) @ abs(vh) + (p @ e) * abs(o[i, t, h]))
                                  + 2.0 ** -20 * (p @ (abs(vh) + mid[keys, h // g])))
                l_tol[i, h, t] = (p @ e) + 2.0 ** -21 * (1 + abs(lse[i, h, t]))
    return o, lse, o_tol, l_tol


def check_attention(got_o, got_lse, ref, what):
    o, lse, o_tol, l_tol = ref
    go = got_o.double().cpu().numpy().reshape(o.shape)
    gl = got_lse.double().cpu().numpy().reshape(lse.shape)
    none = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), none), f"{what}: rows without keys"
    assert np.all(go[np.moveaxis(none, 1, 2)] == 0), f"{what}: rows without keys must be 0"
    assert np.isfinite(go).all(), f"{what}: O not finite"
    bad = abs(go - o) > o_tol
    assert not bad.any(), f"{what}: O off by {abs(go - o)[bad].max():.3e}, allowed {o_tol[bad].min():.3e}"
    dl = abs(gl[~none] - lse[~none])
    bad = dl > l_tol[~none]
    assert not bad.any(), f"{what}: LSE off by {dl[bad].max():.3e}, allowed {l_tol[~none][bad].min():.3e}"


__all__ = ["DT", "HALF_STEP", "TINY", "attend64", "block_table", "build_cache4", "check_attention", "kv4", "oracle",
           "place", "rope_table"]
