"""The serving cache's operators, measured: appending keys and values to a paged cache (16-bit, and 4-bit with group
scales) with the rotary position rotation on the way, and attention of a few query tokens over the 4-bit cache.

With `own` false, `run` computes each operator from elementary torch operations; with `own` true it makes the calls
a user makes of the framework.

The 4-bit cache is a uint8 tensor [num_pages, hkv, page_size / 32 * U]: units of 32 keys, U = 32 (d + 8 d / group)
bytes each: K codes, V codes, K parameters, V parameters (see `unpack_units`).  A value is min + scale * code, with one
(scale, min) pair per key, head and group of `group` dims.
"""
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _append(name, kind, b, tokens, context, hq, hkv, d, dtype, page, rot, interleaved, group=0, ragged=0):
    """tokens: new tokens of each sequence (ragged: at most); context: keys that a sequence holds before them."""
    return {"name": name, "kind": kind, "b": b, "tokens": tokens, "context": context, "hq": hq, "hkv": hkv, "d": d,
            "dtype": dtype, "page": page, "rot": rot, "interleaved": interleaved, "group": group, "ragged": ragged}


def _attend(name, b, keys, hq, hkv, d, dtype, page, group, sq=1, window=-1, softcap=0.0, ragged=0):
    """keys: keys of each sequence (ragged: at most); sq: query tokens of each sequence."""
    return {"name": name, "kind": "attend4", "b": b, "keys": keys, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype,
            "page": page, "group": group, "sq": sq, "window": window, "softcap": softcap, "ragged": ragged}


def listed():
    return [
        # a decode step of the framework's decode configuration: one token for each of eight sequences
        _append("append step b8", "append", 8, 1, 4000, 32, 8, 128, "bf16", 256, 128, False),
        # a decode step of a large batch, one KV head per query head, narrow heads
        _append("append step b200 d64", "append", 200, 1, 600, 16, 16, 64, "fp16", 64, 64, False),
        # four prompts of the causal prefill configuration's length
        _append("append prompts 4x4096", "append", 4, 4096, 0, 32, 8, 128, "bf16", 256, 128, False),
        # prompt chunks of uneven length behind a cached prefix, wide heads, a quarter of each rotated in pairs
        _append("append chunks ragged d256", "append", 9, 1100, 333, 16, 2, 256, "fp16", 64, 64, True, ragged=5),
        # the same decode step into the 4-bit cache
        _append("append4 step b8", "append4", 8, 1, 4000, 32, 8, 128, "bf16", 256, 128, False, group=128),
        # the same prompts into the 4-bit cache
        _append("append4 prompts 4x4096", "append4", 4, 4096, 0, 32, 8, 128, "bf16", 256, 128, False, group=64),
        # uneven chunks, narrow heads, the finest groups
        _append("append4 chunks ragged d64", "append4", 13, 1500, 100, 16, 16, 64, "fp16", 64, 32, True, group=32,
                ragged=3),
        # one conversation with a short history: the latency of a call
        _attend("attend4 b1 777", 1, 777, 32, 8, 128, "bf16", 64, 128),
        # the framework's split-KV decode configuration
        _attend("attend4 b8 32768", 8, 32768, 32, 8, 128, "bf16", 256, 128),
        # a serving batch of very different lengths, fine groups
        _attend("attend4 b48 ragged g32", 48, 9000, 32, 4, 128, "fp16", 64, 32, ragged=7),
        # four drafted tokens verified at once, narrow heads
        _attend("attend4 b16 sq4 d64", 16, 5001, 16, 8, 64, "bf16", 128, 64, sq=4, ragged=2),
        # wide heads, sliding window, capped scores
        _attend("attend4 b6 d256 window", 6, 20000, 16, 4, 256, "bf16", 64, 64, window=4096, softcap=30.0, ragged=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["append", "append4", "attend4", "attend4"])
    d = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    page = rng.choice([64, 128, 192, 256])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    b = _log(rng, 1, 64)
    ragged = rng.randrange(1, 1000)
    if kind == "attend4":
        g, sq = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 1, 1, 2, 3, 8])
        most = 8 * 32768 * 8 * 128 // (b * hkv * d * (1 if g * sq <= 8 else 4))
        return {"kind": kind, "b": b, "keys": _log(rng, 1, min(32768, most)), "hq": g * hkv, "hkv": hkv, "d": d,
                "dtype": dtype, "page": page, "group": group, "sq": sq,
                "window": rng.choice([-1, -1, _log(rng, 1, 8192)]), "softcap": rng.choice([0.0, 0.0, 20.0]),
                "ragged": ragged}
    g = rng.choice([1, 2, 4, 8])
    tokens = rng.choice([1, _log(rng, 1, min(4096, 4 * 4096 * 8 * 128 // (b * hkv * d)))])
    interleaved = rng.random() < 0.5
    rot = rng.choice([0, d // 4, d // 2, d, d])
    return {"kind": kind, "b": b, "tokens": tokens, "context": rng.randrange(0, 700), "hq": g * hkv, "hkv": hkv, "d": d,
            "dtype": dtype, "page": page, "rot": rot, "interleaved": interleaved,
            "group": group if kind == "append4" else 0, "ragged": ragged}


def _counts(case):
    """(new tokens, keys after the call) of each sequence."""
    b, mix = case["b"], random.Random(case["ragged"])
    if case["kind"] == "attend4":
        most = case["keys"]
        keys = [most if not case["ragged"] or i == 0 else mix.randint(max(1, most // 8), most) for i in range(b)]
        return [case["sq"]] * b, keys
    most = case["tokens"]
    new = [most if not case["ragged"] or i == 0 else mix.randint(max(1, most // 8), most) for i in range(b)]
    return new, [n + (mix.randint(0, case["context"]) if case["ragged"] else case["context"]) for n in new]


def work(case):
    new, keys = _counts(case)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["kind"] == "attend4":
        per_key = hkv * (d + 8 * (d // case["group"]))
        read = seen = 0
        for n in keys:
            w, s = case["window"], case["sq"]
            first = max(0, n - s - w) if w >= 0 else 0
            read += n - first
            for i in range(s):
                at = n - s + i
                seen += max(0, at + 1 - (max(0, at - w) if w >= 0 else 0))
        rows = case["b"] * case["sq"] * hq
        return {"bytes": read * per_key + rows * (4 * d + 4), "flops": 4 * d * hq * seen}
    total = sum(new)
    rows = total * (hq + 2 * hkv) * d * 2
    table = total * case["rot"] * 4
    if case["kind"] == "append":
        return {"bytes": 2 * rows + table, "flops": 3 * total * (hq + hkv) * case["rot"]}
    held = total * hkv * (d + 8 * (d // case["group"]))
    back = total * hkv * d * 4
    return {"bytes": rows + total * hq * d * 2 + table + 2 * held + back,
            "flops": 3 * total * (hq + hkv) * case["rot"] + 12 * total * hkv * d}


# ---------------------------------------------------------------------------------------------------------------
# the 4-bit cache's layout, with elementary operations
# ---------------------------------------------------------------------------------------------------------------
def _shape(d):
    """Words of 32 dims per run (J) and runs (C) of a head."""
    j = min(d // 32, 4)
    return j, d // 32 // j


def _words(codes):
    """Eight codes along the last axis to one 32-bit word, the first in the lowest bits."""
    shift = torch.arange(0, 32, 4, device=codes.device)
    w = (codes.to(torch.int64) << shift).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def pack_units(kc, vc, kp, vp):
    """Codes [n, 32, d] (values 0..15) and parameters [n, 32, groups, 2] of n units to bytes [n, U]."""
    n, _, d = kc.shape
    j, c = _shape(d)
    # K: a word holds dims 32 (J c + j) + 8 t .. + 7 of one key, at [c][key][t][j]
    kw = _words(kc.view(n, 32, c, j, 4, 8).permute(0, 2, 1, 4, 3, 5))
    # V: a word holds dims 32 (J c + j) + 4 g .. + 3 of keys 16 a + 8 h + 2 t and + 1, at [a][h][c][g][t][j]
    vw = _words(vc.view(n, 2, 2, 4, 2, c, j, 8, 4).permute(0, 1, 2, 5, 7, 3, 6, 4, 8).reshape(n, 2, 2, c, 8, 4, j, 8))
    parts = [kw.reshape(n, -1).view(torch.uint8), vw.reshape(n, -1).view(torch.uint8),
             kp.reshape(n, -1).view(torch.uint8), vp.reshape(n, -1).view(torch.uint8)]
    return torch.cat(parts, 1)


def unpack_units(units, d, group, dtype):
    """Bytes [n, U] to the values [n, 32, d] of K and V in fp32."""
    n, ng = units.shape[0], d // group
    j, c = _shape(d)
    shift = torch.arange(0, 32, 4, device=units.device, dtype=torch.int32)
    kw = units[:, :16 * d].contiguous().view(torch.int32).view(n, c, 32, 4, j, 1)
    kc = ((kw >> shift) & 15).permute(0, 2, 1, 4, 3, 5).reshape(n, 32, ng, group).float()
    vw = units[:, 16 * d:32 * d].contiguous().view(torch.int32).view(n, 2, 2, c, 8, 4, j, 1)
    vc = ((vw >> shift) & 15).view(n, 2, 2, c, 8, 4, j, 2, 4)
    vc = vc.permute(0, 1, 2, 5, 7, 3, 6, 4, 8).reshape(n, 32, ng, group).float()
    par = units[:, 32 * d:].contiguous().view(dtype).view(n, 2, 32, ng, 2).float()
    k = par[:, 0, :, :, 1:] + par[:, 0, :, :, :1] * kc
    v = par[:, 1, :, :, 1:] + par[:, 1, :, :, :1] * vc
    return k.view(n, 32, d), v.view(n, 32, d)


def quantise(x, group):
    """16-bit rows [..., d] to codes and (scale, min) pairs [..., d / group, 2] of the same type."""
    dtype = x.dtype
    x = x.float().unflatten(-1, (-1, group))
    mn, mx = x.amin(-1, True), x.amax(-1, True)
    s = ((mx * 0.5 - mn * 0.5) / 7.5).to(dtype).float()
    s = torch.where(s < 2.0 ** -100, torch.zeros_like(s), s)
    # (a quotient, not a product with 1 / s: many values lie exactly between two codes)
    code = torch.where(s > 0, torch.round((x - mn) / s), torch.zeros_like(x)).clamp(max=15.0)
    return code.flatten(-2).to(torch.uint8), torch.cat([s, mn], -1).to(dtype)


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _table(gen, keys, page):
    """Shuffled pages for sequences of these lengths, with a few pages that nobody owns."""
    per = [(n + page - 1) // page for n in keys]
    count = sum(per) + 3
    order = torch.randperm(count, generator=gen, device=DEV).to(torch.int32)
    width = max(max(per), 1)
    rows, at = [], 0
    for p in per:
        row = torch.zeros(width, dtype=torch.int32, device=DEV)
        row[:p] = order[at:at + p]
        rows.append(row)
        at += p
    return count, torch.stack(rows)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    new, keys = _counts(case)
    dtype, d, hkv, page = TYPES[case["dtype"]], case["d"], case["hkv"], case["page"]
    count, table = _table(gen, keys, page)
    s = {"case": case, "dtype": dtype, "table": table, "lens": _ints(keys)}
    if case["kind"] == "attend4":
        # keys with a few strong channels and values without, as trained models leave them
        units = []
        strong = 1.0 + 3.0 * (torch.rand(d, generator=gen, device=DEV) < 0.05)
        for first in range(0, count * hkv * page // 32, 1 << 16):
            n = min(1 << 16, count * hkv * page // 32 - first)
            kc, kp = quantise((_normal(gen, (n, 32, d), torch.float32) * strong).to(dtype), case["group"])
            vc, vp = quantise(_normal(gen, (n, 32, d), dtype), case["group"])
            units.append(pack_units(kc, vc, kp, vp))
        s["cache"] = torch.cat(units).view(count, hkv, -1)
        s["q"] = _normal(gen, (case["b"], case["sq"], case["hq"], d), dtype)
        # the buffers that a serving loop keeps from step to step
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["b"], case["hq"], case["sq"], dtype=torch.float32, device=DEV)
        s["work"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        return s
    total = sum(new)
    for name, h in (("q", case["hq"]), ("k", hkv), ("v", hkv)):
        s[name] = _normal(gen, (total, h, d), dtype)
    s["cu"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
    s["q_out"] = torch.empty_like(s["q"])
    if case["rot"]:
        at = torch.arange(max(keys), device=DEV, dtype=torch.float64)[:, None]
        half = case["rot"] // 2
        angle = at * 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    else:
        s["cos_sin"] = None
    if case["kind"] == "append":
        s["k_cache"] = _normal(gen, (count, page, hkv, d), dtype)
        s["v_cache"] = _normal(gen, (count, page, hkv, d), dtype)
    else:
        s["k_back"], s["v_back"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        size = page * (d + 8 * (d // case["group"]))
        s["cache"] = torch.zeros((count, hkv, size), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return _attend_plain(s, case) if case["kind"] == "attend4" else _append_plain(s, case)


def _own(s, case):
    import tiled_exact_attention_gb300 as fa

    if case["kind"] == "attend4":
        return fa.fa_fwd_kvcache_int4(s["q"], s["cache"], group=case["group"], block_table=s["table"],
                                      seqlens_k=s["lens"], window_left=case["window"] if case["window"] >= 0 else None,
                                      softcap=case["softcap"], out=s["out"], lse=s["lse"], workspace=s["work"])
    if case["kind"] == "append":
        q = fa.fa_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], block_table=s["table"], seqlens_k=s["lens"],
                            cu_seqlens=s["cu"], q=s["q"], q_out=s["q_out"], cos_sin=s["cos_sin"],
                            interleaved=case["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    q = fa.fa_kv_append_int4(s["k"], s["v"], s["cache"], group=case["group"], block_table=s["table"],
                             seqlens_k=s["lens"], cu_seqlens=s["cu"], q=s["q"], q_out=s["q_out"],
                             cos_sin=s["cos_sin"], interleaved=case["interleaved"])
    k, v = fa.fa_kv_gather_int4(s["cache"], group=case["group"], block_table=s["table"], seqlens_k=s["lens"],
                                cu_seqlens=s["cu"], k_out=s["k_back"], v_out=s["v_back"])
    return q, k, v


def _rotate(x, cos_sin, pos, interleaved):
    if cos_sin is None:
        return x
    rot = cos_sin.shape[1]
    cs = cos_sin[pos][:, None, :]
    c, sn = cs[..., :rot // 2], cs[..., rot // 2:]
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _append_plain(s, case):
    cu, lens, page = s["cu"].long(), s["lens"].long(), case["page"]
    row = torch.arange(s["k"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    pos = lens[seq] - cu[seq + 1] + row
    where, slot = s["table"].long()[seq, pos // page], pos % page
    q = _rotate(s["q"], s["cos_sin"], pos, case["interleaved"])
    k = _rotate(s["k"], s["cos_sin"], pos, case["interleaved"])
    if case["kind"] == "append":
        s["k_cache"][where, slot] = k
        s["v_cache"][where, slot] = s["v"]
        return q, s["k_cache"], s["v_cache"]
    back = []
    for x in (k, s["v"]):
        code, par = quantise(x, case["group"])
        par = par.float()
        y = par[..., 1:] + par[..., :1] * code.float().unflatten(-1, (-1, case["group"]))
        back.append(y.flatten(-2).to(s["dtype"]))
    return q, back[0], back[1]


def _attend_plain(s, case):
    d, hkv, hq, b, sq, page = (case[n] for n in ("d", "hkv", "hq", "b", "sq", "page"))
    pages = s["table"].long()
    unit = 32 * (d + 8 * (d // case["group"]))
    units = s["cache"][pages].view(-1, unit)                         # [b, pages, hkv, units of a page]
    k, v = unpack_units(units, d, case["group"], s["dtype"])
    k = k.view(b, -1, hkv, page, d).transpose(1, 2).reshape(b, hkv, -1, d)
    v = v.view(b, -1, hkv, page, d).transpose(1, 2).reshape(b, hkv, -1, d)
    q = s["q"].float().view(b, sq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    x = (q @ k.transpose(2, 3)) * d ** -0.5                          # [b, hkv, g sq, keys]
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    at = s["lens"].long()[:, None] - sq + torch.arange(sq, device=DEV)
    at = at[:, None, None, :, None]                                  # [b, 1, 1, sq, 1]
    key = torch.arange(k.shape[2], device=DEV)
    seen = key <= at
    if case["window"] >= 0:
        seen = seen & (key >= at - case["window"])
    x = x.view(b, hkv, -1, sq, x.shape[-1]).masked_fill(~seen, float("-inf"))
    m = x.amax(-1, True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(-1, True)
    o = (p.flatten(2, 3) @ v).view(b, hkv, -1, sq, d) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).view(b, hq, sq)
    return o.permute(0, 3, 1, 2, 4).reshape(b, sq, hq, d).to(s["dtype"]), lse


# ---------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _turn64(x, angles, at, interleaved):
    """Rows of one sequence [n, h, d] turned as complex numbers by the table's entries at positions `at`."""
    x = x.double()
    if angles is None:
        return x
    rot = angles.shape[1]
    w = torch.complex(angles[at, :rot // 2].double(), angles[at, rot // 2:].double())[:, None, :]
    first, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        z = torch.view_as_complex(first.unflatten(-1, (rot // 2, 2)).contiguous()) * w
        first = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(first[..., :rot // 2].contiguous(), first[..., rot // 2:].contiguous()) * w
        first = torch.cat([z.real, z.imag], -1)
    return torch.cat([first, rest], -1)


def _held64(x, group, dtype):
    """What the 4-bit cache holds for rows x: the rows rounded to the cache's type, then to the nearest of 16 levels."""
    x = x.to(dtype).double()
    out = torch.empty_like(x)
    for g in range(0, x.shape[-1], group):
        y = x[..., g:g + group]
        low = y.min(-1, keepdim=True).values
        step = ((y.max(-1, keepdim=True).values - low) / 15).to(dtype).double()
        level = torch.where(step > 0, (y - low) / step, torch.zeros_like(y)).round().clamp(0, 15)
        out[..., g:g + group] = low + step * level
    return out


def _dense64(s, case, i, n):
    """K and V of sequence i, [n, hkv, d], each element looked up in the cache's bytes."""
    d, page, group = case["d"], case["page"], case["group"]
    j, c = _shape(d)
    ng = d // group
    unit = 32 * (d + 8 * ng)
    key = torch.arange(n, device=DEV)
    r, dim = (key % 32)[:, None], torch.arange(d, device=DEV)[None, :]
    block = dim // 32
    k_word = (((block // j) * 32 + r) * 4 + (dim % 32) // 8) * j + block % j
    k_at, k_shift = 4 * k_word + (dim % 8) // 2, 4 * (dim % 2)
    r16 = r % 16
    v_word = ((((r // 16 * 2 + r16 // 8) * c + block // j) * 8 + (dim % 32) // 4) * 4 + (r16 % 8) // 2) * j + block % j
    v_at, v_shift = 16 * d + 4 * v_word + 2 * (r % 2) + (dim % 4) // 2, 4 * (dim % 2)
    par_at = 32 * d + (r * ng + torch.arange(ng, device=DEV)) * 4
    where = s["table"][i].long()[key // page]
    base = (key % page // 32 * unit)[:, None]
    out = []
    for at, shift, par in ((k_at, k_shift, par_at), (v_at, v_shift, par_at + 128 * ng)):
        heads = []
        for h in range(case["hkv"]):
            rows = s["cache"][:, h]
            code = ((rows[where[:, None], base + at] >> shift.to(torch.uint8)) & 15).double()
            pair = rows[where[:, None, None], (base + par)[..., None] + torch.arange(4, device=DEV)]
            pair = pair.contiguous().view(s["dtype"]).double().repeat_interleave(group, 1)
            heads.append(pair[..., 1] + pair[..., 0] * code)
        out.append(torch.stack(heads, 1))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    new, keys = _counts(case)
    if case["kind"] == "attend4":
        b, sq, hq, hkv, d = (case[n] for n in ("b", "sq", "hq", "hkv", "d"))
        o = torch.zeros(b, sq, hq, d, dtype=torch.float64, device=DEV)
        lse = torch.full((b, hq, sq), -float("inf"), dtype=torch.float64, device=DEV)
        for i, n in enumerate(keys):
            k, v = _dense64(s, case, i, n)
            for t in range(sq):
                last = n - sq + t
                first = max(0, last - case["window"]) if case["window"] >= 0 else 0
                if last < first:
                    continue
                kk, vv = k[first:last + 1], v[first:last + 1]
                q = s["q"][i, t].double().view(hkv, hq // hkv, d)
                x = torch.einsum("hgd,nhd->hgn", q, kk) / d ** 0.5
                if case["softcap"]:
                    x = torch.tanh(x / case["softcap"]) * case["softcap"]
                lse[i, :, t] = torch.logsumexp(x, -1).reshape(-1)
                o[i, t] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), vv).reshape(hq, d)
        return o, lse
    q, k, v = (torch.empty(s[n].shape, dtype=torch.float64, device=DEV) for n in ("q", "k", "v"))
    if case["kind"] == "append":
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    begin = 0
    for i, n in enumerate(new):
        at = torch.arange(keys[i] - n, keys[i], device=DEV)
        rows = slice(begin, begin + n)
        q[rows] = _turn64(s["q"][rows], s["cos_sin"], at, case["interleaved"])
        k[rows] = _turn64(s["k"][rows], s["cos_sin"], at, case["interleaved"])
        v[rows] = s["v"][rows].double()
        if case["kind"] == "append":
            for t in range(n):
                p = int(keys[i] - n + t)
                if t and p % case["page"]:
                    continue
                end = min(n, t + case["page"] - p % case["page"])
                page = int(s["table"][i, p // case["page"]])
                slots = slice(p % case["page"], p % case["page"] + end - t)
                k_cache[page, slots] = k[begin + t:begin + end]
                v_cache[page, slots] = v[begin + t:begin + end]
        begin += n
    if case["kind"] == "append":
        return q, k_cache, v_cache
    return q, _held64(k, case["group"], s["dtype"]), _held64(v, case["group"], s["dtype"])
